"""gf_rope on the GPU: an angle is reduced to its nearest quarter turn before it is rounded to 32 bits, so that
cosine and sine have their own relative precision wherever an integer position's angle comes near a multiple of
a quarter turn."""

import numpy as np
import pytest

import attend_util as au
from oracle import attend as oatt
from test_gpu_rope import run, table_of

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.fixture(scope="module")
def G(lib):
    yield lib
    assert lib.device_status() == 0


# What is left of the angle, an eighth of a turn at most, rounded to 32 bits: one unit of the cosine or sine that is
# small with it, and pi / 4 units where it is not small; cosine and sine themselves two units of their last place,
# which is up to two of 2^-24.
REL = 5 * au.U
# The frequency's own error (2^-49 of the angle) and the table's last bit (2^-65 turns a position).
FREQ = 2.0 ** -49


@pytest.mark.parametrize("layout", ["halves", "pairs"])
def test_near_quarter_turns(G, layout):
    """The first pair turns by its position in radians; 11, 22, 355 and their like lie next to multiples of pi / 2."""
    pos = np.concatenate((np.arange(0, 4096), -np.arange(1, 4096)))
    n = 64
    x = np.zeros((len(pos), 1, n))
    x[:, 0, 0] = 1.0  # (cos, sin) of the first pair
    got, _ = run(G, x, pos, n, layout, table_of(G, n))
    c, s = got[:, 0, 0], got[:, 0, n // 2 if layout == "halves" else 1]
    p = pos.astype(np.float64)
    tol = np.abs(p) * FREQ
    assert np.all(np.abs(c - np.cos(p)) <= REL * np.abs(np.cos(p)) + tol)
    assert np.all(np.abs(s - np.sin(p)) <= REL * np.abs(np.sin(p)) + tol)


def test_every_pair(G):
    """Absolute errors: pi / 4 units of the angle, two of cosine and sine, and the frequency's."""
    pos = np.concatenate(([0, 1, 2, 3, 65535], np.random.default_rng(1).integers(0, 1 << 16, 500)))
    n = 128
    x = np.zeros((len(pos), 1, n))
    x[:, 0, :n // 2] = 1.0
    got, _ = run(G, x, pos, n, "halves", table_of(G, n))
    want = oatt.rope(x, pos, oatt.freqs(n))
    assert np.all(np.abs(got - want) <= (2 + np.pi / 4) * au.U + 2 * pos[:, None, None] * FREQ)  # (the oracle's angle, too)


def test_axes_are_exact(G):
    """Divisors of pi and a position of whole quarter turns: as near as the divisor's 32 bits are."""
    d = torch.full((32,), 2.0 / np.pi, device="cuda")  # the first pair's frequency becomes pi / 2 to 2^-25
    pos = np.arange(-8, 9)
    x = np.zeros((len(pos), 1, 64))
    x[:, 0, 0] = 1.0
    got, _ = run(G, x, pos, 64, "halves", table_of(G, 64, divisors=d))
    f = 1.0 / float(np.float32(2.0 / np.pi))
    for t, p in enumerate(pos):
        assert abs(got[t, 0, 0] - np.cos(p * f)) <= REL * abs(np.cos(p * f)) + 8 * FREQ
        assert abs(got[t, 0, 32] - np.sin(p * f)) <= REL * abs(np.sin(p * f)) + 8 * FREQ

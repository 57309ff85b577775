"""Sizes of a cache that no cache has: refused, and at once (on the CPU; pointers are fake, well-separated addresses)."""

import threading

import pytest

import test_attend_host as host

SIZES = [(1 << 62) + 1, 1 << 62, (1 << 63) - 1, (1 << 63) - 2, 1 << 31, (1 << 40) + 3, -(1 << 63), -1, -(1 << 62) - 1]


def in_time(call, seconds=20):
    """What `call` returns; a call that does not come back stays behind in a thread that ends with the process."""
    out = []
    t = threading.Thread(target=lambda: out.append(call()), daemon=True)
    t.start()
    t.join(seconds)
    assert out, "still running after %d s" % seconds
    return out[0]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("name", ["page", "block"])
@pytest.mark.parametrize("entry", ["store", "load", "att"])
def test_page_and_block(lib, entry, name, size):
    want = lib.ERR_INVALID if size < 1 or size & (size - 1) or name == "block" else lib.ERR_UNSUPPORTED
    assert in_time(lambda: getattr(host, entry)(lib, c={name: size})) == want


def test_both(lib):
    for page, block in (((1 << 63) - 1, (1 << 63) - 1), (1 << 62, 1 << 62), (1 << 62, 16), (1 << 20, 1 << 20)):
        e = in_time(lambda: host.store(lib, c=dict(page=page, block=block)))
        assert e == (lib.ERR_INVALID if page & (page - 1) else lib.ERR_UNSUPPORTED)

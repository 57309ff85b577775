"""The attention block of one layer's decode step for a batch of requests, as one graph:

    n       = x / rms(x) * gamma
    q, k, v = Wq n, Wk n, Wv n                      one pass over the three matrices
    q, k    rotated by each token's position; k, v quantised into the requests' 8-bit caches
    o       = attention of q over the cache
    y       = x + Wo o

    python -m decode_gemv_epilogue_gb300.attn_step

runs steps of 16 requests at contexts around 4000 tokens and prints their time."""

import numpy as np
import torch

from . import gemvfuse as gf
from . import synth


class AttnStep:
    """The buffers and the graph of one layer's step.  `x` [T, d] is read, `y` [T, d] written by launch();
    token t is position pos[t] of request seq[t] (-1: padding), both int32 [T] and free to change
    between launches; request r's pages are row r of `table`.  `run`: tokens of a request next to each
    other (1 for plain decoding)."""

    def __init__(self, T, d, heads, kv_heads, dim, n_seqs, context, wtype=synth.Q4_0, fmt=gf.CACHE_I8, page=64, block=16, run=1,
                 base=10000.0, eps=1e-6, seed=0, device="cuda"):
        self.T, self.d, self.heads, self.kv_heads, self.dim, self.eps, self.wtype = T, d, heads, kv_heads, dim, eps, wtype
        dist = {synth.Q4_0: (0.001, 0.008), synth.Q8_0: (0.0002, 0.0006)}.get(wtype)
        shapes = dict(wq=(heads * dim, d), wk=(kv_heads * dim, d), wv=(kv_heads * dim, d), wo=(d, heads * dim))
        self.host = {k: synth.weights(wtype, *s, seed=seed + i, dist=dist) for i, (k, s) in enumerate(shapes.items())}
        self.host["gamma"] = (1.0 + 0.1 * synth.normal(d, seed + 10)).astype(np.float32)
        w = self.dev = {k: torch.from_numpy(v).to(device) for k, v in self.host.items()}

        def buf(*shape, dtype=torch.float32):
            return torch.zeros(*shape, dtype=dtype, device=device)

        per = -(-context // page)
        pages = n_seqs * per
        self.k, self.v = (buf(pages, kv_heads, page, dim, dtype=torch.uint8) for _ in range(2))
        self.k_scale, self.v_scale = (buf(pages, kv_heads, page // block) for _ in range(2))
        self.table = torch.arange(pages, dtype=torch.int32, device=device).view(n_seqs, per).contiguous()
        self.cache = gf.Cache(self.k, self.v, self.k_scale, self.v_scale, fmt, pages, kv_heads, page, dim, block, self.table,
                              n_seqs, per)
        self.rope = buf(gf.rope_table_bytes(dim), dtype=torch.uint8)
        gf.rope_table(self.rope, dim, base=base)
        self.x, self.y = buf(T, d), buf(T, d)
        self.q, self.o = buf(T, heads, dim), buf(T, heads, dim)
        self.new_k, self.new_v = buf(T, kv_heads, dim), buf(T, kv_heads, dim)
        self.seq, self.pos = buf(T, dtype=torch.int32), buf(T, dtype=torch.int32)
        self.ws = buf(gf.attend_workspace(T, heads, kv_heads, dim, run), dtype=torch.uint8)
        none = gf.EPI_NONE
        self.calls = [
            gf.prepare_multi([(w["wq"], heads * dim, none, None, self.q), (w["wk"], kv_heads * dim, none, None, self.new_k),
                              (w["wv"], kv_heads * dim, none, None, self.new_v)], wtype, self.x, d, ncols=T,
                             rms_norm_weight=w["gamma"], rms_norm_eps=eps),
            gf.prepare_cache_store(self.cache, self.new_k, self.new_v, T, self.seq, self.pos, rope=self.rope, q=self.q,
                                   q_heads=heads, q_dst=self.q, pdl=True),
            gf.prepare_attend(self.cache, self.q, T, heads, self.seq, self.pos, self.o, self.ws, run=run, pdl=True),
            gf.prepare(w["wo"], wtype, self.o, d, heads * dim, gf.EPI_ADD, self.x, self.y, ncols=T, pdl=True),
        ]
        self.graph = gf.Graph(self.calls)

    def launch(self, stream=None):
        self.graph.launch(stream=stream)


def main():
    T, context = 16, 4096
    step = AttnStep(T, d=4096, heads=32, kv_heads=8, dim=128, n_seqs=T, context=context)
    step.x.normal_()
    step.seq.copy_(torch.arange(T, dtype=torch.int32))
    # caches as if they had been filled
    step.k.random_(0, 256)
    step.v.random_(0, 256)
    step.k_scale.fill_(1.0 / 64)
    step.v_scale.fill_(1.0 / 64)
    first = context - 64 - 37 * torch.arange(T, dtype=torch.int32)
    for s in range(10):
        step.pos.copy_(first + s)
        step.launch()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(50):
        step.launch()
    b.record()
    torch.cuda.synchronize()
    status = gf.device_status()
    print("16 requests, 4096 wide, 32 heads of 128 over 8, contexts of 3500 to 4000 in 8 bits, Q4_0: %.1f us a step (status %d)"
          % (a.elapsed_time(b) * 20, status))
    return 0 if status == 0 and bool(torch.isfinite(step.y).all()) else 1


if __name__ == "__main__":
    raise SystemExit(main())

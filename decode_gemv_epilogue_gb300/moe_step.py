"""A decode step of one mixture-of-experts layer for a batch of requests, as one graph:

    h   = x + (Wo x + scale_a B_a (A_a x))          output projection, an adapter per request
    l   = Wr (h / rms(h) * gamma)                   router logits
    ids, w = the top_k experts of l
    y   = h + sum_j w_j Wd_e (silu(Wg_e n) * (Wu_e n)),  n = h / rms(h) * gamma

(x stands for the attention block's output; attn_step is a step of that block).

    python -m decode_gemv_epilogue_gb300.moe_step

runs a step of 8 requests and prints its time."""

import numpy as np
import torch

from . import gemvfuse as gf
from . import synth


class MoeStep:
    """The buffers and the graph of one layer's step.  `x` [T, d] is read, `y` [T, d] written by
    launch(); `adapters` [T] (int32, -1: none) chooses each request's adapter and may change
    between launches, as may every other buffer's contents."""

    def __init__(self, T, d, ffn, E, top_k, n_adapters, rank, wtype=synth.Q4_0, eps=1e-6, seed=0, device="cuda"):
        self.T, self.d, self.ffn, self.E, self.top_k, self.eps = T, d, ffn, E, top_k, eps
        self.wtype, self.n_adapters, self.rank = wtype, n_adapters, rank
        dist = {synth.Q4_0: (0.001, 0.008), synth.Q8_0: (0.0002, 0.0006)}.get(wtype)
        shapes = dict(wo=(d, d), gate=(E * ffn, d), up=(E * ffn, d), down=(E * d, ffn))
        self.host = {k: synth.weights(wtype, *s, seed=seed + i, dist=dist) for i, (k, s) in enumerate(shapes.items())}
        self.host["router"] = synth.weights(synth.F16, E, d, seed=seed + 10)
        self.host["A"] = (synth.normal(n_adapters * rank * d, seed + 11) * d ** -0.5).astype(np.float16)
        self.host["B"] = (synth.normal(n_adapters * d * rank, seed + 12) * rank ** -0.5).astype(np.float16)
        self.host["scales"] = np.full(n_adapters, 0.5, dtype=np.float32)
        self.host["gamma"] = (1.0 + 0.1 * synth.normal(d, seed + 13)).astype(np.float32)
        w = self.dev = {k: torch.from_numpy(v).to(device) for k, v in self.host.items()}

        def buf(*shape, dtype=torch.float32):
            return torch.zeros(*shape, dtype=dtype, device=device)

        self.x, self.h, self.y = buf(T, d), buf(T, d), buf(T, d)
        self.logits, self.weights = buf(T, E), buf(T, top_k)
        self.ids, self.adapters = buf(T, top_k, dtype=torch.int32), buf(T, dtype=torch.int32)
        self.ws_lora = buf(gf.lora_workspace(T, d, d, rank, n_adapters), dtype=torch.uint8)
        self.ws_experts = buf(gf.experts_workspace(E, T, top_k, ffn, d), dtype=torch.uint8)
        norm = dict(rms_norm_weight=w["gamma"], rms_norm_eps=eps)
        self.calls = [
            gf.prepare_lora(w["wo"], wtype, self.x, d, d, gf.EPI_ADD, self.x, self.h, w["A"],
                            w["B"], gf.F16, n_adapters, rank, self.adapters, w["scales"], self.ws_lora, ncols=T),
            gf.prepare(w["router"], gf.F16, self.h, E, d, gf.EPI_NONE, None, self.logits, ncols=T, pdl=True, **norm),
            gf.prepare_route(self.logits, T, E, top_k, self.ids, self.weights, pdl=True),
            gf.prepare_experts(w["gate"], w["up"], wtype, w["down"], wtype, E, self.h, ffn, d, self.ids, self.weights, T,
                               top_k, self.h, self.y, self.ws_experts, pdl=True, **norm),
        ]
        self.graph = gf.Graph(self.calls)

    def launch(self, stream=None):
        self.graph.launch(stream=stream)


def main():
    step = MoeStep(T=8, d=2048, ffn=768, E=64, top_k=8, n_adapters=4, rank=16)
    step.x.normal_()
    step.adapters.copy_(torch.arange(8, dtype=torch.int32) % 5 - 1)
    for _ in range(10):
        step.launch()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(100):
        step.launch()
    b.record()
    torch.cuda.synchronize()
    status = gf.device_status()
    print("8 requests, 2048 wide, 64 experts of 768, 8 each, Q4_0, adapters of rank 16: %.1f us a step (status %d)"
          % (a.elapsed_time(b) * 10, status))
    return 0 if status == 0 and bool(torch.isfinite(step.y).all()) else 1


if __name__ == "__main__":
    raise SystemExit(main())

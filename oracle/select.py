"""Oracle of the operators whose weights are chosen per token (fp64).  Test infrastructure
only.  The formulas are the ones in include/gemvfuse.h (gf_route, gemv_experts,
gemv_lora); the pages have no counterpart.  Written out token by token.
"""

import numpy as np

from . import gemv, quant


def route(logits, top_k, score="softmax", bias=None, n_group=1, topk_group=1, group_top=2, norm=True, scale=1.0):
    """ids int32 [T, top_k], weights float64 [T, top_k]."""
    L = np.asarray(logits, dtype=np.float64)
    T, E = L.shape
    ids = np.full((T, top_k), -1, dtype=np.int32)
    w = np.zeros((T, top_k))
    big = float(np.finfo(np.float32).max)
    for t in range(T):
        live = ~np.isnan(L[t]) & (L[t] > -np.inf)
        l = np.where(live, np.minimum(L[t], big), 0.0)
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                s = 1.0 / (1.0 + np.exp(-l))
            logs = -np.logaddexp(0.0, -l)
        else:
            m = l[live].max() if live.any() else 0.0
            logs = l - m - (np.log(np.exp(l[live] - m).sum()) if live.any() else 0.0)
            s = np.exp(logs)
        key = s.copy() if bias is None else s + np.asarray(bias, dtype=np.float64)
        order_by = l if bias is None else key
        live = live & ~np.isnan(key) & (key > -np.inf)
        if n_group > 1:
            per = E // n_group
            sc = []
            for g in range(n_group):
                ks = sorted((key[e] for e in range(g * per, (g + 1) * per) if live[e]), reverse=True)
                sc.append(sum(ks[:group_top]) if ks else -np.inf)
            keep = sorted(range(n_group), key=lambda g: (-sc[g], g))[:topk_group]
            live = live & np.isin(np.arange(E) // per, keep)
        order = sorted((e for e in range(E) if live[e]), key=lambda e: (-order_by[e], e))[:top_k]
        ids[t, :len(order)] = order
        if order:
            if norm:  # relative to the largest: the ratio survives where the scores underflow
                r = np.exp(logs[order] - logs[order].max())
                w[t, :len(order)] = r / r.sum()
            else:
                w[t, :len(order)] = s[order]
    return ids, w * scale


def experts(raw_gate, raw_up, wtype, raw_down, wtype_down, E, x, M, K, ids, weights, aux=None):
    """dst float64 [T, K], and the tolerance scale of each element: (dst, bound), with the
    bound of the literal parity tolerance of each product (2e-5 of the absolute sum),
    carried through silu(g) * u (slope <= 1.1) and the down product."""
    X = np.asarray(x, dtype=np.float64).reshape(-1, K)
    T = X.shape[0]
    ids = np.asarray(ids).reshape(T, -1)
    wts = np.asarray(weights, dtype=np.float64).reshape(T, -1)
    y = np.zeros((T, K)) if aux is None else np.asarray(aux, dtype=np.float64).reshape(T, K).copy()
    b = np.full((T, K), 1e-6) + 1e-6 * np.abs(y)
    rg, rd = quant_rows(raw_gate, E), quant_rows(raw_down, E)
    ru = quant_rows(raw_up, E)
    for e in range(E):
        ts, js = np.nonzero(ids == e)
        if ts.size == 0:
            continue
        xe = X[ts]
        g, u = gemv.gemv(rg[e], wtype, xe, M, K), gemv.gemv(ru[e], wtype, xe, M, K)
        bg = 2e-5 * gemv.abs_dot(rg[e], wtype, xe, M, K) + 1e-6
        bu = 2e-5 * gemv.abs_dot(ru[e], wtype, xe, M, K) + 1e-6
        h = gemv.silu(g) * u
        bh = 1.1 * bg * (np.abs(u) + bu) + np.abs(gemv.silu(g)) * bu + 1e-6 * np.abs(h)
        ye = gemv.gemv(rd[e], wtype_down, h, K, M)
        be = 2e-5 * gemv.abs_dot(rd[e], wtype_down, h, K, M) + gemv.abs_w_dot(rd[e], wtype_down, bh, K, M) + 1e-6
        for i in range(ts.size):
            c = wts[ts[i], js[i]]
            y[ts[i]] += c * ye[i]
            b[ts[i]] += np.abs(c) * be[i]
    return y, b


def quant_rows(raw, E):
    """The E matrices of a packed stack, each as raw bytes."""
    return np.asarray(raw).reshape(-1).view(np.uint8).reshape(E, -1)


def lora(raw, wtype, x, M, K, epilogue, aux, A, B, ids, scales):
    """dst float64 [ncols, M] and its bound; A [n, r, K], B [n, M, r] (any float type)."""
    X = np.asarray(x, dtype=np.float64).reshape(-1, K)
    y = gemv.gemv(raw, wtype, X, M, K)
    b = 2e-5 * gemv.abs_dot(raw, wtype, X, M, K) + 1e-6
    n = A.shape[0]
    for c, a in enumerate(np.asarray(ids).tolist()):
        if 0 <= a < n:
            s = 1.0 if scales is None else float(scales[a])
            Ad, Bd = A[a].astype(np.float64), B[a].astype(np.float64)
            v = s * (Ad @ X[c])
            bv = 2e-5 * abs(s) * (np.abs(Ad) @ np.abs(X[c]))
            y[c] += Bd @ v
            b[c] += np.abs(Bd) @ (bv + 2e-5 * np.abs(v))
    out = gemv.apply_epilogue(y, epilogue, None if aux is None else np.asarray(aux).reshape(y.shape))
    slope = {gemv.EPI_SIGMOID: 0.25, gemv.EPI_SILU: 1.1, gemv.EPI_SILU_MUL: 1.1}.get(epilogue, 1.0)
    if epilogue == gemv.EPI_SILU_MUL:
        slope = slope * np.abs(np.asarray(aux, dtype=np.float64).reshape(y.shape))
    return out, slope * b + 1e-6 * np.abs(out) + 1e-6

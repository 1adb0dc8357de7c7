"""Plain 64-bit forms of the dense side's operators (numpy, CPU), for the tests only."""
import numpy as np


def route(logits, topk, *, score="softmax", bias=None, groups=0, topk_groups=0, group_score="max", renorm=True,
          scale=1.0):
    """One token at a time, by sorting (choice, -index) pairs."""
    logits = np.asarray(logits, np.float64)
    B, E = logits.shape
    ids, weights = np.zeros((B, topk), np.int32), np.zeros((B, topk))
    with np.errstate(all="ignore"):
        for t in range(B):
            l = np.where(np.isnan(logits[t]), -np.inf, logits[t])
            if score == "softmax":
                m = l.max()
                s = np.where(l == -np.inf, 0.0, np.where(l == m, 1.0, np.exp(l - m)))
                s = s / s.sum() if s.sum() > 0 else s
            else:
                s = np.where(l == -np.inf, 0.0, 1.0 / (1.0 + np.exp(-l)))
            c = l.copy() if bias is None else s + np.asarray(bias, np.float64)
            c[(l == -np.inf) | np.isnan(c)] = -np.inf
            cand = list(range(E))
            if groups:
                size, ranks = E // groups, []
                for g in range(groups):
                    members = [e for e in range(g * size, (g + 1) * size) if c[e] > -np.inf]
                    vals = sorted(((s[e] if bias is None and group_score == "top2" else c[e]) for e in members),
                                  reverse=True)
                    vals = vals[:2] if group_score == "top2" else vals[:1]
                    ranks.append((-sum(vals) if vals else np.inf, g))
                kept = {g for _, g in sorted(ranks)[:topk_groups]}
                cand = [e for e in cand if e // size in kept]
            sel = sorted(cand, key=lambda e: (-c[e], e))[:topk]
            w = s[sel]
            if renorm:
                w = w / w.sum() if w.sum() > 0 else np.zeros_like(w)
            ids[t], weights[t] = sel, w * scale
    return ids, weights


def quant(x):
    """x float64 [M, K] (values of the input's type) -> codes, FP32 scales."""
    amax = np.abs(x).max(axis=1)
    bad = ~np.isfinite(x).all(axis=1)
    safe = np.where((amax > 0) & ~bad, amax, 1.0)
    q = np.rint(np.where(bad[:, None], 0.0, x) * 127.0 / safe[:, None])
    scales = (np.where(bad, 1.0, amax).astype(np.float32) / np.float32(127.0)).astype(np.float32)
    scales[bad] = np.nan
    return q.astype(np.int8), scales


def linear(a, sa, w, sw, *, act="none", bias=None, add=None):
    """-> (y, slack): y in FP64, and the FP32 evaluation's error bound for each element.

    acc converts to FP32 (half a step, u = 2^-24), two products and one sum follow (u each): within
    4.01 u (|acc sa sw| + |bias|).  silu(g) = g / (1 + exp(-g)): the exponent's argument g log2(e)
    and its constant are off by 2 u |g| relative in exp, the hardware exp2, sum, reciprocal and
    products by a few u, so a relative (16 + 2 |g|) u on top of the inputs' own errors (silu' <=
    1.1); below -87 exp(-g) overflows to infinity and silu to 0, off by at most 88 * 2^-125."""
    u = 2.0 ** -24
    p = (a.astype(np.float64) @ w.astype(np.float64).T) * sa.astype(np.float64)[:, None] * sw.astype(np.float64)
    b = np.zeros(w.shape[0]) if bias is None else bias.astype(np.float64)
    y, e = p + b, 4.01 * u * (np.abs(p) + np.abs(b))
    if act == "swiglu":
        h = w.shape[0] // 2
        g, up, eg, eu = y[:, :h], y[:, h:], e[:, :h], e[:, h:]
        with np.errstate(over="ignore"):
            s = g / (1.0 + np.exp(-g))
        es = 1.1 * eg + (16 + 2 * np.abs(g)) * u * np.abs(s) + 88 * 2.0 ** -125
        y, e = s * up, es * np.abs(up) + np.abs(s) * eu + es * eu + 2 * u * np.abs(s * up)
    if add is not None:
        y = y + add
        e = e + u * np.abs(y) * 1.01
    return y, e

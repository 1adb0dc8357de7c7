"""Plain 64-bit forms of the block-scaled FP8 operators (numpy, CPU), for the tests only."""
import numpy as np

from helpers import E4M3

U = 2.0 ** -24  # half a step of FP32
_FINITE = np.sort(E4M3[np.isfinite(E4M3) & (E4M3 >= 0)])[1:]  # 0, then every positive value (one zero)


def kb(K):
    return (K + 127) // 128


def e4m3(v):
    """Nearest e4m3 values of 64-bit numbers of at most 448 in magnitude, half to even, by search."""
    a = np.abs(v)
    hi = np.searchsorted(_FINITE, a).clip(0, len(_FINITE) - 1)
    lo = (hi - 1).clip(0)
    below, above = a - _FINITE[lo], _FINITE[hi] - a
    up = (above < below) | ((above == below) & (hi % 2 == 0))   # the table's index is the code
    return np.copysign(np.where(up, _FINITE[hi], _FINITE[lo]), v)


def quant(x):
    """x float64 [M, K] -> code values, scales (float64)."""
    M, K = x.shape
    codes, scales = np.zeros((M, K)), np.zeros((M, kb(K)))
    for b in range(kb(K)):
        part = x[:, 128 * b:128 * b + 128]
        with np.errstate(invalid="ignore"):
            amax = np.abs(part).max(axis=1)
        fine, e = np.isfinite(amax), np.full(M, -126)
        while (over := fine & (amax * np.ldexp(1.0, -e) > 448)).any():
            e += over
        scales[:, b] = np.where(fine, np.where(amax > 0, np.ldexp(1.0, e), 0.0), np.nan)
        codes[:, 128 * b:128 * b + 128] = e4m3(np.where(fine[:, None], part, 0.0) * np.ldexp(1.0, -e)[:, None])
    return codes, scales


def norm(x, weight, residual, eps, round_to):
    """-> h, y (FP32 values) as float64; round_to: rounds float64 to x's type, once."""
    h = x if residual is None else round_to((x.astype(np.float32) + residual.astype(np.float32)).astype(np.float64))
    with np.errstate(all="ignore"):
        mean = (h.astype(np.longdouble) ** 2).sum(axis=1) / x.shape[1]
        r = (1 / np.sqrt(mean.astype(np.float64) + eps)).astype(np.float32)
        y = (h.astype(np.float32) * r[:, None]) * weight.astype(np.float32)
    return h, y.astype(np.float64)


def row_blocks(N, halves):
    """The scale block of each weight row."""
    if not halves:
        return np.arange(N) // 128
    r = np.arange(N // 2) // 128
    return np.concatenate([r, r + kb(N // 2)])


def linear(a, sa, w, sw, *, act="none", bias=None, add=None, cut=True):
    """a, w: code values -> (y, bound of the FP32 evaluation's error), both float64.

    Products of codes are exact.  Within a block at most 128 of them are added, by whatever tree the matrix cores have,
    each addition within two half steps of the magnitudes' sum: 2 * 128 U.  The factor sa * sw, its product with
    the block's sum and that's addition: U each; so is each of the kb(K) blocks' additions and of up to 16
    partial sums'.  So (2 * 128 + kb(K) + 20) U of sum |sa sw a w|, and U each for bias and add.  silu as in dense_ref.linear.
    cut (outputs in 16 bits): of each eight products of neighbours, all but the largest lose less than 2^-13 of that:
    16 * 7 * 2^-13 of the block's largest |a| times its largest |w|."""
    K = a.shape[1]
    wide = np.repeat(sw[row_blocks(w.shape[0], act == "swiglu")], 128, axis=1)[:, :K] * w
    aw = np.repeat(sa, 128, axis=1)[:, :K] * a
    with np.errstate(invalid="ignore"):
        y, e = aw @ wide.T, (256 + kb(K) + 20) * U * (np.abs(aw) @ np.abs(wide).T)
    if cut:
        pa, pw = (np.pad(np.abs(v), ((0, 0), (0, -K % 128))).reshape(len(v), -1, 128).max(axis=2) for v in (aw, wide))
        e = e + 112 * 2.0 ** -13 * (pa @ pw.T)
    if bias is not None:
        y = y + bias
        e = e + U * 1.01 * np.abs(y)
    if act == "swiglu":
        h = w.shape[0] // 2
        g, up, eg, eu = y[:, :h], y[:, h:], e[:, :h], e[:, h:]
        with np.errstate(over="ignore"):
            s = g / (1.0 + np.exp(-g))
        es = 1.1 * eg + (16 + 2 * np.abs(g)) * U * np.abs(s) + 88 * 2.0 ** -125
        y, e = s * up, es * np.abs(up) + np.abs(s) * eu + es * eu + 2 * U * np.abs(s * up)
    if add is not None:
        y = y + add
        e = e + 1.01 * U * np.abs(y)
    return y, e


def lists(ids, E):
    flat = ids.reshape(-1).astype(np.int64)
    pairs = np.full(flat.size, -1, np.int32)
    offsets, n = np.zeros(E + 1, np.int32), 0
    for e in range(E):
        mine = np.flatnonzero(flat == e)
        pairs[n:n + mine.size] = mine
        n += mine.size
        offsets[e + 1] = n
    return offsets, pairs

"""The block-scaled FP8 operators and the norm on the GPU against plain 64-bit forms (f8_ref, dense_ref): norm with
codes in 8 bits, quantization into blocks, product, route lists, products grouped by expert; then the layer made
of them."""
import numpy as np
import pytest
import torch

import dense_ref
import f8_ref as ref
from helpers import log

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F16, F32, F8, I32 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn, torch.int32
HALF_STEP = {BF: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}   # largest rounding, relative
TINY = {BF: 2.0 ** -134, F16: 2.0 ** -25, F32: 2.0 ** -150}     # and among subnormals
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_routed_expert_mx_amd as pkg
    return pkg


def _gen(seed):
    return torch.Generator("cpu").manual_seed(seed)


def _np(t):
    return t.cpu().double().numpy()


def _padded(t, pad, fill=0.0):
    """The same matrix on the GPU, its rows `pad` elements further apart."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), fill, device=DEV).to(t.dtype)
    wide[:, :t.shape[1]] = t.to(DEV)
    return wide[:, :t.shape[1]]


def _same(got, want):
    """Equal values, NaN where NaN."""
    return np.array_equal(got, want, equal_nan=True)


# --------------------------------------------------------------------- quant
def _quant(m, x, pad=0, stream=None):
    M, K = x.shape
    codes = torch.full((M + 1, K + pad), 0x33, dtype=torch.uint8, device=DEV).view(F8)
    scales = torch.full((M + 1, ref.kb(K) + (1 if pad else 0)), -7.0, device=DEV)
    c, s = codes[:M, :K], scales[:M, :ref.kb(K)]
    m.moe_quant_f8(x, c, s, stream=stream)
    torch.cuda.synchronize()
    raw = codes.view(torch.uint8)
    assert (raw[M] == 0x33).all() and (raw[:, K:] == 0x33).all()          # nothing behind rows and tokens
    assert (scales[M] == -7).all() and (scales[:, ref.kb(K):] == -7).all()
    return c, s


@pytest.mark.parametrize("M,K", [(1, 1), (1, 128), (2, 129), (3, 127), (5, 16), (1, 3584), (7, 511), (9, 513), (33, 1000),
                                 (300, 640), (1, 16384), (2, 20011), (70000, 24), (40000, 1030)])
@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_quant_sizes(m, M, K, dtype):
    log(f"quant_f8 {M}x{K} {dtype}")
    g = _gen(M + K)
    x = (torch.randn(M, K, generator=g) * torch.exp2(torch.randint(-6, 6, (M, 1), generator=g).float())).to(dtype)
    pad = (0, 3, 8)[(M + K) % 3]
    c, s = _quant(m, _padded(x, pad, NAN), pad)
    if M * K > 1 << 23:                       # some rows
        rows = torch.randint(0, M, (40,), generator=g)
        rows[0], rows[1] = 0, M - 1
    else:
        rows = torch.arange(M)
    rc, rs = ref.quant(_np(x[rows]))
    rows = rows.numpy()
    assert np.array_equal(_np(c.float())[rows], rc) and np.array_equal(_np(s)[rows], rs)


@pytest.mark.parametrize("dtype", [BF, F16])
def test_quant_every_pattern(m, dtype):
    """Every value of the type, in blocks with different neighbours: rounding, subnormals, infinity and NaN."""
    bits = torch.arange(65536, dtype=torch.int32)
    for order in (bits, bits.view(256, 256).t().reshape(-1)):
        x = order.to(torch.int16).view(dtype).view(128, 512)
        c, s = _quant(m, x.to(DEV))
        rc, rs = ref.quant(_np(x))
        assert _same(_np(s), rs) and np.array_equal(_np(c.float()), rc)


def test_quant_special_blocks(m):
    """Zeros of both signs, one huge or tiny value, infinity and NaN in a block, halves between codes, the border of a
    scale."""
    x = torch.randn(24, 300, generator=_gen(3))
    x[0] = 0.0
    x[1] = -0.0
    x[2, 130] = INF
    x[3, 5] = NAN
    x[4, 299] = -INF
    x[5] = 1e-40                                   # subnormal
    x[6], x[6, 7] = 1e-30, 3e38
    x[7] = torch.finfo(F32).max
    x[8, :128], x[8, 0] = torch.arange(128) / 16, 448.0
    x[9, :128], x[9, 0] = torch.arange(128) / 16, 449.0
    x[10] = 2.0 ** -149
    x[11] = 448.0 * 2.0 ** -126
    x[12] = 449.0 * 2.0 ** -126
    x[13, :128], x[13, 0] = torch.arange(128) * 2.0 ** -11, 448.0     # among e4m3's subnormals
    c, s = _quant(m, x.to(DEV))
    rc, rs = ref.quant(_np(x))
    assert _same(_np(s), rs) and np.array_equal(_np(c.float()), rc)


# ---------------------------------------------------------------------- norm
def _norm_case(m, x, weight, residual=None, codes=None, eps=1e-6, pad=0, inplace=False, stream=None):
    M, K = x.shape
    dtype = x.dtype
    xd = _padded(x, pad, NAN)
    rd = None if residual is None else _padded(residual, pad, NAN)
    out = xd if inplace else _padded(torch.full_like(x, 7.0), pad, 7.0)
    total = None if residual is None else rd if inplace else _padded(torch.full_like(x, 7.0), pad, 7.0)
    q = s = None
    if codes is not None:
        q = torch.full((M + 1, K + pad), 0x33, dtype=torch.uint8, device=DEV).view(codes)
        s = torch.full((M + 1,) if codes == torch.int8 else (M + 1, ref.kb(K)), -7.0, device=DEV)
    m.moe_rms_norm(xd, weight.to(DEV), out=out, residual=rd, total=total, codes=None if q is None else q[:M, :K],
                   scales=None if s is None else s[:M], eps=eps, stream=stream)
    torch.cuda.synchronize()
    if q is not None:
        raw = q.view(torch.uint8)
        assert (raw[M] == 0x33).all() and (raw[:, K:] == 0x33).all() and (s[M:] == -7).all()
    round_to = (lambda v: v) if dtype == F32 else (lambda v: torch.from_numpy(v).to(dtype).double().numpy())
    h, y = ref.norm(_np(x), _np(weight), None if residual is None else _np(residual), eps, round_to)
    with np.errstate(over="ignore"):
        want = torch.from_numpy(y).float().to(dtype).double().numpy()
    assert _same(_np(out), want)
    if total is not None:
        assert _same(_np(total), h)
    if codes == torch.int8:
        rq, rs = dense_ref.quant(y)
        assert _same(_np(s[:M]), rs.astype(np.float64))
        assert np.array_equal(q[:M, :K].cpu().numpy(), rq)
    elif codes == F8:
        rq, rs = ref.quant(y)
        assert _same(_np(s[:M]), rs) and np.array_equal(_np(q[:M, :K].float()), rq)


# Codes and outputs are compared for equality: the definition rounds r once from a 64-bit value (whose own sum is some
# 2^-50 off: in one row of 2^26 or so r could round the other way), and everything after it is FP32 arithmetic in
# the order stated.
@pytest.mark.parametrize("M,K", [(1, 1), (1, 3584), (3, 7), (2, 128), (5, 130), (8, 3584), (17, 1000), (1030, 512),
                                 (1025, 1023), (1100, 1900), (1024, 4096), (6, 4097), (1027, 4100), (2, 16384), (3, 16383)])
@pytest.mark.parametrize("codes", [None, torch.int8, F8])
def test_norm_sizes(m, M, K, codes):
    g = _gen(M * 7 + K)
    dtype = (BF, F16, F32)[(M + K) % 3]
    wtype = (F32, dtype)[(M + K // 2) % 2]
    log(f"norm {M}x{K} {dtype} weight {wtype} codes {codes}")
    x = (torch.randn(M, K, generator=g) * 3).to(dtype)
    residual = torch.randn(M, K, generator=g).to(dtype) if (M + K) % 4 else None
    weight = (1 + 0.3 * torch.randn(K, generator=g)).to(wtype)
    pad = (0, 5, 8)[(M + 2 * K) % 3]
    _norm_case(m, x, weight, residual, codes, pad=pad)


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("codes", [None, torch.int8, F8])
def test_norm_special_rows(m, dtype, wide, codes):
    """Rows of zeros, infinities, NaN, the type's extremes, sums beyond its range; eps of 0; in place."""
    log(f"norm special rows {dtype} {codes}")
    fi = torch.finfo(dtype)
    x = torch.randn(1100 if wide else 16, 200, generator=_gen(9))
    r = torch.randn(x.shape, generator=_gen(10))
    x, r = x.to(dtype), r.to(dtype)
    x[0], r[0] = 0, 0
    x[1], r[1] = -0.0, 0
    x[2, 150] = INF
    x[3, 3] = NAN
    x[4], r[4] = fi.max, fi.max                    # the sum overflows to infinity
    x[5], r[5] = fi.max, -fi.max
    x[6], r[6] = fi.tiny, fi.tiny
    x[7], r[7] = fi.smallest_normal / 4, 0
    x[8, 0] = fi.max
    x[9], r[9] = 0, 0
    x[9, 199] = 1
    for eps in (1e-6, 0.0, 1.0):
        _norm_case(m, x, torch.ones(200), r, codes, eps=eps)
        _norm_case(m, x, torch.randn(200, generator=_gen(11)), r, codes, eps=eps, inplace=True, pad=3)


def test_norm_codes_alone_and_without_residual(m):
    """Outputs that are not asked for are not written; codes without out."""
    x, w = torch.randn(5, 384, generator=_gen(1)).to(BF).to(DEV), torch.ones(384, device=DEV)
    out, q1, s1 = torch.empty_like(x), torch.empty(5, 384, dtype=F8, device=DEV), torch.empty(5, 3, device=DEV)
    q2, s2 = torch.empty_like(q1), torch.empty_like(s1)
    m.moe_rms_norm(x, w, out=out, codes=q1, scales=s1)
    m.moe_rms_norm(x, w, codes=q2, scales=s2)
    r = torch.zeros_like(x)
    q3, s3 = torch.empty_like(q1), torch.empty_like(s1)
    m.moe_rms_norm(x, w, codes=q3, scales=s3, residual=r)                 # added, not kept
    torch.cuda.synchronize()
    assert torch.equal(q1.view(torch.uint8), q2.view(torch.uint8)) and torch.equal(s1, s2) and (r == 0).all()
    assert torch.equal(q1.view(torch.uint8), q3.view(torch.uint8))


# ------------------------------------------------------------------- product
def _codes(shape, g, spread=1.0):
    return (torch.randn(shape, generator=g) * spread).to(F8)


def _scales(shape, g):
    """Scales as weights have them (any FP32) or as quantization leaves them (powers of two)."""
    s = torch.rand(shape, generator=g) + 0.5
    return torch.exp2(torch.randint(-6, 3, shape, generator=g).float()) if len(shape) == 2 and shape[0] % 2 else s * 0.03


def _check(got, y, e, dtype, what=""):
    """got is y, off by e and one rounding."""
    bound = e + HALF_STEP[dtype] * (np.abs(y) + e) * 1.001 + TINY[dtype]
    bad = ~(np.abs(got - y) <= bound)
    assert not bad.any(), (what, np.argwhere(bad)[:4], got[bad][:4], y[bad][:4], bound[bad][:4])


def _linear(m, M, N, K, *, dtype=BF, act="none", bias=False, add=False, pad=0, seed=0, stream=None, inplace=False):
    g = _gen(seed * 1009 + M * 31 + N * 7 + K)
    cols = N // 2 if act == "swiglu" else N
    nb = 2 * ref.kb(cols) if act == "swiglu" else ref.kb(N)
    a, w = _codes((M, K), g, 4), _codes((N, K), g, 4)
    sa, sw = _scales((M, ref.kb(K)), g), _scales((nb, ref.kb(K)), g) / K ** 0.5
    b = torch.randn(N, generator=g) if bias else None
    d = torch.randn(M, cols, generator=g).to(dtype) if add else None
    out = torch.full((M + 1, cols + 5), 7.0, device=DEV).to(dtype)
    o = out[:M, :cols]
    if inplace:
        o.copy_(d)
    dd = o if inplace else None if d is None else _padded(d, pad // 16)
    m.moe_linear_f8(_padded(a, pad), _padded(sa, 1 if pad else 0), _padded(w, pad), sw.to(DEV), o, act=act,
                    bias=None if b is None else b.to(DEV), add=dd, stream=stream)
    torch.cuda.synchronize()
    assert (out[M] == 7).all() and (out[:, cols:] == 7).all()
    y, e = ref.linear(_np(a.float()), _np(sa), _np(w.float()), _np(sw), act=act, bias=None if b is None else _np(b),
                      add=None if d is None else _np(d), cut=dtype != F32)
    _check(_np(o), y, e, dtype, (M, N, K, act))
    return o


LINEAR_SIZES = [(1, 1, 16), (1, 16, 128), (2, 17, 144), (1, 768, 3584), (8, 3584, 384), (16, 100, 1040), (17, 64, 256),
                (31, 130, 112), (33, 256, 128), (64, 512, 1024), (65, 300, 640), (64, 8190, 272), (100, 129, 2064),
                (128, 128, 128), (129, 257, 400), (200, 640, 512), (300, 1000, 1536), (513, 258, 16), (700, 2050, 784),
                (1000, 520, 2048), (2500, 384, 384), (1, 100000, 32), (5000, 33, 96), (260, 6000, 640)]


@pytest.mark.parametrize("M,N,K", LINEAR_SIZES)
def test_linear_sizes(m, M, N, K):
    log(f"linear_f8 {M}x{N}x{K}")
    i = LINEAR_SIZES.index((M, N, K))
    _linear(m, M, N, K, dtype=(BF, F16, F32)[i % 3], bias=i % 2 == 0, add=i % 4 > 1, pad=(0, 16, 48)[i % 3])
    _linear(m, M, N, K, dtype=F32, seed=1)
    n = N + N % 2
    _linear(m, M, n, K, dtype=(F32, BF, F16)[i % 3], act="swiglu", bias=i % 3 == 0, add=i % 2 == 0, pad=(16, 0, 0)[i % 3])


@pytest.mark.parametrize("M", [1, 15, 16, 40, 70, 140, 300, 1100])
@pytest.mark.parametrize("K", [128, 16, 1152])
def test_linear_rows_and_types(m, M, K):
    """Tiles with a last row alone, each output type, with and without SwiGLU."""
    log(f"linear_f8 {M} rows, K = {K}")
    for dtype in (BF, F16, F32):
        _linear(m, M + 1, 270, K, dtype=dtype, act="swiglu", seed=3)
        _linear(m, M, 300, K, dtype=dtype, bias=True, add=True, inplace=True, seed=4)


@pytest.mark.parametrize("M", [3, 200, 600])
def test_linear_special_values(m, M):
    """NaN codes and scales stay in their rows and columns; scales of 0; the largest codes; all 256 codes."""
    log(f"linear_f8 special values {M}")
    g = _gen(M)
    N, K = 300, 400
    a, w = _codes((M, K), g), _codes((N, K), g)
    a[0] = torch.arange(400).remainder(127).to(torch.uint8).view(F8)
    w[0] = torch.full((K,), 0x7e, dtype=torch.uint8).view(F8)          # 448
    a[1] = torch.full((K,), 0xfe, dtype=torch.uint8).view(F8)
    sa, sw = torch.ones(M, 4), torch.ones(3, 4)
    a.view(torch.uint8)[2, 399] = 0x7f                                  # NaN in the last, short block
    w.view(torch.uint8)[7, 0] = 0xff
    sw[1, 2] = 0.0
    sa[1, 3] = 0.0
    if M > 100:
        sa[150, 1] = NAN
        sa[151, 0] = INF
    out = torch.empty(M, N, device=DEV)
    m.moe_linear_f8(a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), out)
    torch.cuda.synchronize()
    got = _np(out)
    with np.errstate(invalid="ignore"):
        y, e = ref.linear(_np(a.float()), _np(sa), _np(w.float()), _np(sw), cut=False)
    fine = np.isfinite(y)
    assert not fine[2].any() and not fine[:, 7].any() and fine[0, 0] and (M < 100 or not fine[150:152].any())
    assert np.array_equal(np.isfinite(got), fine)
    assert np.all(np.abs(got - y)[fine] <= (e + U32(y))[fine])


def U32(y):
    return HALF_STEP[F32] * np.abs(y) * 1.001 + TINY[F32]


def test_linear_beyond_32_bits(m):
    """Rows of a and of out whose offsets pass 2^32 bytes."""
    g = _gen(5)
    M, N, K = 1100, 130, 256
    if torch.cuda.get_device_properties(0).total_memory < 64 << 30:
        pytest.skip("needs 20 GiB")
    lda = (1 << 22) - 16
    big = torch.zeros(M * lda, dtype=torch.uint8, device=DEV)
    a = torch.as_strided(big, (M, K), (lda, 1)).view(F8)
    av, w = _codes((M, K), g), _codes((N, K), g)
    a.view(torch.uint8).copy_(av.view(torch.uint8))
    sa, sw = torch.rand(M, 2, generator=g), torch.rand(2, 2, generator=g)
    ldo = (1 << 22) + 8
    wide = torch.empty(M * ldo, dtype=BF, device=DEV)
    out = torch.as_strided(wide, (M, N), (ldo, 1))
    m.moe_linear_f8(a, sa.to(DEV), w.to(DEV), sw.to(DEV), out)
    torch.cuda.synchronize()
    y, e = ref.linear(_np(av.float()), _np(sa), _np(w.float()), _np(sw))
    _check(_np(out), y, e, BF)


# --------------------------------------------------------------------- lists
def _lists(m, ids, E, stream=None):
    R = ids.numel()
    offsets = torch.full((E + 2,), -9, dtype=I32, device=DEV)
    pairs = torch.full((R + 1,), -9, dtype=I32, device=DEV)
    ws = torch.full((m.moe_lists_ws_bytes(R, E),), 0x5a, dtype=torch.uint8, device=DEV)
    m.moe_lists(ids.to(DEV), offsets[:E + 1], pairs[:R], ws=ws, stream=stream)
    torch.cuda.synchronize()
    assert offsets[E + 1] == -9 and pairs[R] == -9
    return offsets[:E + 1].cpu().numpy(), pairs[:R].cpu().numpy()


@pytest.mark.parametrize("B,K,E", [(1, 1, 1), (1, 16, 160), (3, 4, 16), (64, 16, 160), (65, 1, 1024), (512, 16, 7),
                                   (513, 16, 160), (1000, 64, 1023), (1, 64, 64), (8192, 1, 2), (8193, 1, 2), (3001, 5, 63),
                                   (16384, 16, 160), (70001, 16, 256)])
@pytest.mark.parametrize("kind", ["uniform", "skewed", "foreign"])
def test_lists(m, B, K, E, kind):
    log(f"lists {B}x{K} of {E} {kind}")
    g = _gen(B + K + E)
    ids = torch.randint(0, E, (B, K), generator=g, dtype=I32)
    if kind == "skewed":
        ids = torch.where(torch.rand(B, K, generator=g) < 0.9, torch.full_like(ids, E // 2), ids)
    if kind == "foreign":
        ids = torch.randint(-2 * E, 2 * E, (B, K), generator=g, dtype=I32)
        ids[0, 0] = -2 ** 31
        ids[-1, -1] = 2 ** 31 - 1
    o, p = _lists(m, ids, E)
    ro, rp = ref.lists(ids.numpy(), E)
    assert np.array_equal(o, ro) and np.array_equal(p, rp)


def test_lists_of_nothing_and_of_one(m):
    for R in (1, 64, 8192, 30000):
        o, p = _lists(m, torch.full((R, 1), -1, dtype=I32), 5)
        assert (o == 0).all() and (p == -1).all()
        o, p = _lists(m, torch.full((R, 1), 4, dtype=I32), 5)
        assert (o[:5] == 0).all() and o[5] == R and np.array_equal(p, np.arange(R))


# ------------------------------------------------------------------- grouped
def _grouped(m, ids, E, N, K, *, dtype=BF, act="none", gather=True, scatter=True, seed=0, pad=0, expert_pad=0, stream=None):
    """ids [B, topk]; without gather a has a row for each place of the lists."""
    g = _gen(seed + N + K + E)
    B, topk = ids.shape
    R, cols = B * topk, N // 2 if act == "swiglu" else N
    nb = 2 * ref.kb(cols) if act == "swiglu" else ref.kb(N)
    rows = B if gather else R
    a, w = _codes((rows, K), g, 4), _codes((E, N, K), g, 4)
    sa, sw = _scales((rows, ref.kb(K)), g), torch.rand(E, nb, ref.kb(K), generator=g) / K ** 0.5
    offsets, pairs = torch.empty(E + 1, dtype=I32, device=DEV), torch.empty(R, dtype=I32, device=DEV)
    m.moe_lists(ids.to(DEV), offsets, pairs, ws=torch.empty(m.moe_lists_ws_bytes(R, E), dtype=torch.uint8, device=DEV),
                stream=stream)
    out = torch.full((R + 1, cols + 3), 7.0, device=DEV).to(dtype)
    o = out[:R, :cols]
    wd = torch.zeros(E, N + expert_pad, K + pad, dtype=torch.uint8, device=DEV).view(F8)
    wd.view(torch.uint8)[:, :N, :K] = w.view(torch.uint8).to(DEV)
    m.moe_grouped_f8(_padded(a, pad), _padded(sa, 1 if pad else 0), wd[:, :N, :K], sw.to(DEV), offsets, o, act=act,
                     pairs=pairs if gather or scatter else None, gather=topk if gather else 0, scatter=scatter,
                     stream=stream)
    torch.cuda.synchronize()
    assert (out[R] == 7).all() and (out[:, cols:] == 7).all()
    ro, rp = ref.lists(ids.numpy(), E)
    got, av, sav = _np(o), _np(a.float()), _np(sa)
    left = np.ones(R, bool)
    for e in range(E):
        i = np.arange(ro[e], ro[e + 1])
        if not i.size:
            continue
        src, dst = rp[i] // topk if gather else i, rp[i] if scatter else i
        y, err = ref.linear(av[src], sav[src], _np(w[e].float()), _np(sw[e]), act=act, cut=dtype != F32)
        _check(got[dst], y, err, dtype, (e, i.size))
        left[dst] = False
    assert (got[left] == 7).all()                       # rows of no expert are left as they were
    return o


def _ids(B, topk, E, kind, seed=0):
    g = _gen(seed + B + E)
    if kind == "zipf":
        score = -1.3 * torch.log1p(torch.arange(E)) - torch.log(-torch.log(torch.rand(B, E, generator=g).clamp(1e-6, 1 - 1e-6)))
    else:
        score = torch.rand(B, E, generator=g)
    ids = score.argsort(dim=1, descending=True)[:, :topk].to(I32).contiguous()
    if kind == "foreign":
        ids = torch.where(ids % 3 == 0, -1 - ids, ids)
    return ids


GROUPED = [(1, 1, 1, 16, 16), (1, 4, 16, 64, 128), (1, 16, 160, 48, 272), (5, 3, 8, 130, 400), (64, 4, 9, 96, 256),
           (40, 8, 300, 32, 144), (130, 2, 5, 256, 512), (257, 6, 24, 200, 384), (700, 2, 3, 384, 640), (1200, 4, 8, 270, 256),
           (33, 1, 1024, 16, 32), (2000, 3, 4, 512, 128)]


@pytest.mark.parametrize("B,topk,E,N,K", GROUPED)
@pytest.mark.parametrize("kind", ["uniform", "zipf", "foreign"])
def test_grouped_sizes(m, B, topk, E, N, K, kind):
    log(f"grouped {B}x{topk} of {E}, {N}x{K}, {kind}")
    i = GROUPED.index((B, topk, E, N, K))
    ids = _ids(B, topk, E, kind)
    dtype = (BF, F16, F32)[i % 3]
    _grouped(m, ids, E, N, K, dtype=dtype, pad=(0, 16)[i % 2], expert_pad=i % 3)
    _grouped(m, ids, E, N, K, dtype=F32, act="swiglu", scatter=False)
    _grouped(m, ids, E, N, K, dtype=BF, gather=False)
    _grouped(m, ids, E, N, K, dtype=(F32, BF, F16)[i % 3], act="swiglu", gather=False, scatter=False)


def test_grouped_all_foreign(m):
    """No route has an expert here: nothing is read or written."""
    for B in (1, 300):
        _grouped(m, torch.full((B, 4), -1, dtype=I32), 8, 64, 128)


@pytest.mark.parametrize("B", [4, 600])
def test_grouped_bad_lists(m, B):
    """Lists that no moe_lists made: offsets that fall or pass R, pairs that name no row.  Rows of a valid pair come out,
    the others are left, nothing outside is touched."""
    log(f"grouped bad lists {B}")
    g = _gen(B)
    E, N, K, topk = 4, 64, 128, 2
    R = B * topk
    a, w = _codes((B, K), g), _codes((E, N, K), g)
    sa, sw = torch.ones(B, 1, device=DEV), torch.ones(E, 1, 1, device=DEV)
    pairs = torch.arange(R, dtype=I32)
    pairs[1], pairs[2], pairs[R - 1] = -1, R + 5, 2 ** 31 - 1
    offsets = torch.tensor([-5, R // 2, R // 4, R + 100, R + 7], dtype=I32, device=DEV)
    out = torch.full((R + 1, N), 7.0, device=DEV)
    m.moe_grouped_f8(a.to(DEV), sa, w.to(DEV), sw, offsets, out[:R], pairs=pairs.to(DEV), gather=topk, scatter=True)
    torch.cuda.synchronize()
    got = _np(out)
    assert (got[R] == 7).all() and (got[[1, 2, R - 1]] == 7).all()
    for i in range(R // 2):                             # expert 0 has 0 .. R/2 - 1; expert 2 again R/4 .. R - 1
        if i < R // 4 and i not in (1, 2):
            y, e = ref.linear(_np(a[i // topk:i // topk + 1].float()), np.ones((1, 1)), _np(w[0].float()), np.ones((1, 1)), cut=False)
            _check(got[i:i + 1], y, e, F32)


# ------------------------------------------------------------- streams, graphs
def _operands(g, B=40, E=8, topk=2, D=512, I=96):
    x = torch.randn(B, D, generator=g).to(BF).to(DEV)
    return x, _ids(B, topk, E, "uniform").to(DEV)


def test_without_the_native_binding(m, monkeypatch):
    """Where the binding is not built, the same calls go through ctypes and give the same."""
    g = _gen(77)
    x, w = torch.randn(6, 256, generator=g).to(BF).to(DEV), torch.randn(256, generator=g).to(DEV)
    wq, ws = _codes((64, 256), g).to(DEV), torch.rand(2, 2, generator=g).to(DEV)
    we, se = _codes((3, 64, 256), g).to(DEV), torch.rand(3, 2, 2, generator=g).to(DEV)
    ids = _ids(6, 2, 3, "uniform").to(DEV)
    res = []
    for binding in (m._lib._dense, m._lib._NoBinding):
        monkeypatch.setattr(m._lib, "_dense", binding)
        n, t = torch.empty_like(x), torch.empty_like(x)
        q, s = torch.empty(6, 256, dtype=F8, device=DEV), torch.empty(6, 2, device=DEV)
        q8, s8 = torch.empty(6, 256, dtype=torch.int8, device=DEV), torch.empty(6, device=DEV)
        y, o, p = torch.empty(6, 32, device=DEV), torch.empty(4, dtype=I32, device=DEV), torch.empty(12, dtype=I32, device=DEV)
        z, u = torch.empty(12, 32, dtype=F16, device=DEV), torch.empty(6, 256, dtype=F8, device=DEV)
        m.moe_rms_norm(x, w, out=n, residual=x, total=t, codes=q, scales=s)
        m.moe_rms_norm(x, w, codes=q8, scales=s8)
        m.moe_quant_f8(x, u, s)
        m.moe_linear_f8(u, s, wq, ws, y, act="swiglu", add=torch.ones_like(y), bias=torch.ones(64, device=DEV))
        m.moe_lists(ids, o, p)
        m.moe_grouped_f8(u, s, we, se, o, z, act="swiglu", pairs=p, gather=2, scatter=True)
        torch.cuda.synchronize()
        res.append((n, t, q.view(torch.uint8), s, q8, s8, u.view(torch.uint8), y, o, p, z))
    assert all(torch.equal(a, b) for a, b in zip(*res))


@pytest.mark.parametrize("binding", [True, False])
def test_side_stream_by_name(m, monkeypatch, binding):
    """A named stream that lags behind: the calls wait for what it holds, not for the current one."""
    g = _gen(78)
    x = torch.randn(300, 256, generator=g).to(BF)
    want = ref.quant(_np(x))
    s = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device=DEV)
    late, codes, scales = torch.zeros(300, 256, dtype=BF, device=DEV), torch.empty(300, 256, dtype=F8, device=DEV), \
        torch.empty(300, 2, device=DEV)
    xd = x.to(DEV)
    if not binding:
        monkeypatch.setattr(m._lib, "_dense", m._lib._NoBinding)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(4):
            torch.mm(big, big)
        late.copy_(xd)
    m.moe_quant_f8(late, codes, scales, stream=s if binding else s.cuda_stream)
    s.synchronize()
    assert np.array_equal(_np(codes.float()), want[0]) and np.array_equal(_np(scales), want[1])


@pytest.mark.parametrize("B", [1, 3, 700])
def test_experts_against_the_plain_form(m, B):
    """ExpertsF8 stage by stage on the values that the GPU handed on, ids of another rank among them."""
    from moe_routed_expert_mx_amd.block import ExpertsF8, f8_weight_blocks
    log(f"experts B={B}")
    g = _gen(B)
    E, topk, D, I = 12, 3, 320, 144
    w13, s13 = f8_weight_blocks(torch.randn(E, 2 * I, D, generator=g) / 18, halves=True)
    w2, s2 = f8_weight_blocks(torch.randn(E, D, I, generator=g) / 12)
    ex = ExpertsF8(w13, s13, w2, s2, topk=topk, B_max=800)
    x, ids = torch.randn(B, D, generator=g).to(BF), _ids(B, topk, E, "foreign" if B > 1 else "uniform")
    rows = torch.full((B * topk, D), 7.0, dtype=BF, device=DEV)
    assert ex.forward(x.to(DEV), ids.to(DEV), rows) is rows
    torch.cuda.synchronize()
    ro, rp = ref.lists(ids.numpy(), E)
    assert np.array_equal(ex.offsets.cpu().numpy(), ro) and np.array_equal(ex.pairs[:B * topk].cpu().numpy(), rp)
    q, s = ref.quant(_np(x))
    n = ro[E]
    hidden = _np(ex.hidden[:n])
    hq, hs = ref.quant(hidden)
    got, left = _np(rows), np.ones(B * topk, bool)
    for e in range(E):
        i = np.arange(ro[e], ro[e + 1])
        if not i.size:
            continue
        t = rp[i] // topk
        y, err = ref.linear(q[t], s[t], _np(w13[e].float()), _np(s13[e]), act="swiglu")
        _check(hidden[i], y, err, BF)
        y, err = ref.linear(hq[i], hs[i], _np(w2[e].float()), _np(s2[e]))
        _check(got[rp[i]], y, err, BF)
        left[rp[i]] = False
    assert (got[left] == 7).all()
    with pytest.raises(ValueError):
        ex.forward(x.to(DEV), ids[:, :2].to(DEV))
    with pytest.raises(ValueError):
        ex.forward(torch.zeros(801, D, dtype=BF, device=DEV), torch.zeros(801, topk, dtype=I32, device=DEV))


def _block(g, D=512, E=24, topk=4, I=64, B_max=300, f8=(True, True)):
    import workloads
    from moe_routed_expert_mx_amd.block import ExpertsF8, MoeBlock, Norm, Router, SharedExpertF8, SharedExpertI8, f8_weight_blocks
    from moe_routed_expert_mx_amd.layer import MoeLayer
    router = Router(torch.randn(E, D, generator=g) / 22, topk=topk, B_max=B_max)
    w13, w2 = torch.randn(2 * 96, D, generator=g) / 22, torch.randn(D, 96, generator=g) / 10
    if f8[0]:
        layer = ExpertsF8(*f8_weight_blocks(torch.randn(E, 2 * I, D, generator=g) / 22, halves=True),
                          *f8_weight_blocks(torch.randn(E, D, I, generator=g) / 8), topk=topk, B_max=B_max)
    else:
        d = workloads.generate(workloads.custom(B=1, E=E, K=topk, D=D, I=I, seed=3))
        layer = MoeLayer(d["w13"], d["s13"], d["w2"], d["s2"], B_max=B_max, topk=topk, device=DEV)
    if f8[1]:
        shared = SharedExpertF8(*f8_weight_blocks(w13, halves=True), *f8_weight_blocks(w2), B_max=B_max)
    else:
        shared = SharedExpertI8.quantize(w13, w2, B_max=B_max)
    return MoeBlock(router, layer, shared, Norm(1 + 0.1 * torch.randn(D, generator=g)))


@pytest.mark.parametrize("B", [1, 8, 300])
@pytest.mark.parametrize("f8", [(True, True), (True, False), (False, True)])
def test_block_with_norm(m, B, f8):
    """Norm, router, experts, combine, shared expert in one call are the parts called one by one; the residual stream
    holds the sum."""
    log(f"block with norm B={B} {f8}")
    g = _gen(B)
    block = _block(g, f8=f8)
    x, r = torch.randn(B, 512, generator=g).to(BF).to(DEV), torch.randn(B, 512, generator=g).to(BF).to(DEV)
    r1, r2 = r.clone(), r.clone()
    y = block.forward(x, residual=r1)
    n = block.norm.forward(x, r2)
    assert torch.equal(r1, (x.float() + r.float()).to(BF)) and torch.equal(r1, r2)
    n2, q, s = block.norm.forward(r1, codes=F8)          # (the sum is the stream by now)
    assert torch.equal(n, n2)
    ids, wts = block.router.forward(n)
    rows = block.layer.forward((q, s) if f8[0] else n, ids)
    want = block.layer.combine(rows, wts)
    block.shared.forward((q, s) if f8[1] else n, add=want, out=want)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    # against the float layer's order of magnitude: codes of y itself, from FP32, not of its BF16 rounding
    assert torch.isfinite(y.float()).all() and y.float().norm() > 0
    with pytest.raises(ValueError, match="residual"):
        type(block)(block.router, block.layer).forward(x, residual=r)


@pytest.mark.parametrize("B", [3, 200])
def test_block_captured_and_replayed(m, B):
    """The layer in a graph; replays with new inputs, eager calls of the same objects between them."""
    log(f"f8 block captured B={B}")
    g = _gen(B + 1)
    block = _block(g)
    x, r = torch.randn(B, 512, generator=g).to(BF).to(DEV), torch.zeros(B, 512, dtype=BF, device=DEV)
    block.forward(x, residual=r)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y1 = block.forward(x, residual=r)
        y2 = block.forward(x, stream=torch.cuda.current_stream())
    for _ in range(4):
        x.copy_(torch.randn(B, 512, generator=g).to(BF))
        r0 = torch.randn(B, 512, generator=g).to(BF).to(DEV)
        want_r = r0.clone()
        want1, want2 = block.forward(x, residual=want_r), block.forward(x)
        r.copy_(r0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y1, want1) and torch.equal(y2, want2) and torch.equal(r, want_r)


@pytest.mark.parametrize("raw", [False, True])
def test_objects_on_a_side_stream(m, raw):
    """Calls on a stream that lags behind: what the current stream allocates right after them is not what they use."""
    log(f"f8 objects on a side stream raw={raw}")
    g, B = _gen(12), 40
    block = _block(g)
    x = torch.randn(B, 512, generator=g).to(BF).to(DEV)
    ids = block.router.forward(x)[0]
    calls = [block.forward, block.shared.forward, lambda x, stream=None: block.layer.forward(x, ids, stream=stream),
             lambda x, stream=None: block.norm.forward(x, codes=F8, stream=stream)[2]]
    want = [c(x).clone() for c in calls]
    big = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for call, w in zip(calls, want):
        with torch.cuda.stream(s):
            for _ in range(8):
                torch.mm(big, big)
        y = call(x, stream=s.cuda_stream if raw else s)
        junk = [torch.zeros(B, 4, dtype=I32, device=DEV), torch.zeros(B, 4, device=DEV), torch.zeros(B * 4, 512, dtype=BF, device=DEV),
                torch.zeros(B, 512, dtype=BF, device=DEV), torch.zeros(B, 512, dtype=torch.uint8, device=DEV)]
        torch.cuda.current_stream().wait_stream(s)
        got = y.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, w)
        assert not any(j.any() for j in junk)


def test_repeated_calls_are_identical(m):
    """Sums run in an order that the sizes decide: the same bits each time."""
    g = _gen(21)
    block = _block(g)
    for B in (1, 64, 300):
        x = torch.randn(B, 512, generator=g).to(BF).to(DEV)
        first = block.forward(x).clone()
        for _ in range(5):
            assert torch.equal(block.forward(x), first)


@pytest.mark.parametrize("through", ["binding", "ctypes"])
def test_an_earlier_error_is_not_this_calls(m, through):
    """An error that another call left on the thread (no such device: the runtime refuses that) fails no call here."""
    st = None if through == "binding" else torch.cuda.current_stream()
    hip = m._lib.lib
    x, w = torch.ones(3, 128, dtype=BF, device=DEV), torch.ones(128, device=DEV)
    q, s, out = torch.zeros(3, 128, dtype=F8, device=DEV), torch.zeros(3, 1, device=DEV), torch.zeros(3, 128, dtype=BF, device=DEV)
    one = torch.ones(1, 1, device=DEV)
    ids, o, p = torch.zeros(3, 1, dtype=I32, device=DEV), torch.zeros(2, dtype=I32, device=DEV), torch.zeros(3, dtype=I32, device=DEV)
    y, z = torch.zeros(3, 3, device=DEV), torch.zeros(3, 3, device=DEV)
    torch.cuda.synchronize()
    try:
        for call in (lambda: m.moe_rms_norm(x, w, out=out, stream=st), lambda: m.moe_quant_f8(x, q, s, stream=st),
                     lambda: m.moe_linear_f8(q, s, q, one, y, add=y, stream=st), lambda: m.moe_lists(ids, o, p, stream=st),
                     lambda: m.moe_grouped_f8(q, s, q[None], one[None], o, z, stream=st)):
            assert hip.hipSetDevice(100000) != 0
            call()
    finally:
        hip.hipGetLastError()
    torch.cuda.synchronize()
    # the block's largest value is 1: scale 2^-8, code 256
    assert (s == 2.0 ** -8).all() and (q.float() == 256).all()
    assert torch.equal(y, torch.full_like(y, 128.0 * 256 * 256 * 2.0 ** -8)) and torch.equal(y, z) and o.tolist() == [0, 3]


# --------------------------------------------------------------- every tile
def _whole(m, M, N, K, dtype, act, seed, plain=True):
    """A product whose out (and add) is contiguous, its rows 16-byte aligned where N allows."""
    g = _gen(seed)
    cols = N // 2 if act == "swiglu" else N
    nb = 2 * ref.kb(cols) if act == "swiglu" else ref.kb(N)
    a, w = _codes((M, K), g, 4), _codes((N, K), g, 4)
    sa, sw, b = torch.rand(M, ref.kb(K), generator=g), torch.rand(nb, ref.kb(K), generator=g) / K ** 0.5, torch.randn(N, generator=g)
    d = None if plain else torch.randn(M, cols, generator=g).to(dtype)
    out = torch.empty(M, cols, dtype=dtype, device=DEV)
    m.moe_linear_f8(a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), out, act=act, bias=None if plain else b.to(DEV),
                    add=None if plain else d.to(DEV))
    torch.cuda.synchronize()
    y, e = ref.linear(_np(a.float()), _np(sa), _np(w.float()), _np(sw), act=act, bias=None if plain else _np(b),
                      add=None if plain else _np(d), cut=dtype != F32)
    _check(_np(out), y, e, dtype, (M, N, K, act))


# sizes for which each of the tiles (64 and 128 x 128 two and four deep, 128 and 256 x 256) is chosen, with rows and
# columns over
@pytest.mark.parametrize("M,N", [(100, 4096), (800, 9000), (230, 2048), (990, 3600), (1990, 4000), (1985, 3990), (4090, 4064),
                                 (4081, 4070), (700, 32768)])
@pytest.mark.parametrize("dtype,act,plain", [(BF, "none", True), (F16, "swiglu", False), (BF, "swiglu", True), (F16, "none", False),
                                             (F32, "none", False), (F32, "swiglu", True)])
def test_linear_tiles(m, M, N, dtype, act, plain):
    K = (144, 272, 400)[(M + N) % 3]
    log(f"linear_f8 tiles {M}x{N}x{K} {dtype} {act}")
    _whole(m, M, N, K, dtype, act, M + N, plain)


@pytest.mark.parametrize("K", [16, 128, 256, 384, 1024, 1040, 2048, 8320])
def test_linear_depths(m, K):
    """K of fewer blocks than stages, and of many, in each tile."""
    log(f"linear_f8 K = {K}")
    for M, N in ((70, 33000), (200, 1024), (1000, 3584)):
        if M * N * K < 1 << 35:
            _whole(m, M, N, K, BF, "none", K)
            _whole(m, M, N, K, F32, "swiglu", K)
    _whole(m, 5, 96, 65536 if K == 8320 else K, BF, "none", K)


@pytest.mark.parametrize("B,topk,E,N", [(1000, 2, 8, 4000), (2040, 2, 8, 4064), (300, 2, 30, 1030), (50, 16, 160, 272), (8, 16, 160, 768),
                                        (700, 1, 16, 2048), (1, 16, 160, 3584), (6, 16, 1024, 160)])
@pytest.mark.parametrize("kind", ["uniform", "zipf"])
def test_grouped_tiles(m, B, topk, E, N, kind):
    K = (144, 1168)[E % 16 == 0]
    log(f"grouped tiles {B}x{topk} of {E}, {N}x{K} {kind}")
    ids = _ids(B, topk, E, kind)
    _grouped(m, ids, E, N, K, dtype=BF, act="swiglu", scatter=False)
    _grouped(m, ids, E, N, K, dtype=F16)
    if B <= 300:
        _grouped(m, ids, E, N, K, dtype=F32, gather=False)


def test_grouped_two_streams_share_inputs(m):
    """Two calls at once on the same weights and lists, each with its own rows."""
    g = _gen(91)
    E, N, K, B, topk = 6, 512, 512, 300, 2
    ids = _ids(B, topk, E, "uniform").to(DEV)
    o, p = torch.empty(E + 1, dtype=I32, device=DEV), torch.empty(B * topk, dtype=I32, device=DEV)
    m.moe_lists(ids, o, p)
    w, sw = _codes((E, N, K), g).to(DEV), torch.rand(E, 4, 4, generator=g).to(DEV)
    xs = [(_codes((B, K), g).to(DEV), torch.rand(B, 4, generator=g).to(DEV)) for _ in range(2)]
    want = []
    for a, sa in xs:
        out = torch.empty(B * topk, N, device=DEV, dtype=BF)
        m.moe_grouped_f8(a, sa, w, sw, o, out, pairs=p, gather=topk, scatter=True)
        want.append(out)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in xs], [torch.zeros_like(t) for t in want]
    torch.cuda.synchronize()
    for _ in range(20):
        for (a, sa), s, out in zip(xs, streams, outs):
            m.moe_grouped_f8(a, sa, w, sw, o, out, pairs=p, gather=topk, scatter=True, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_lists_captured(m):
    """Both launches in a graph, replayed with other ids; eager calls with a workspace of their own between."""
    R, E = 20000, 40
    ids = torch.zeros(R, 1, dtype=I32, device=DEV)
    o, p = torch.empty(E + 1, dtype=I32, device=DEV), torch.empty(R, dtype=I32, device=DEV)
    ws = torch.empty(m.moe_lists_ws_bytes(R, E), dtype=torch.uint8, device=DEV)
    m.moe_lists(ids, o, p, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.moe_lists(ids, o, p, ws=ws)
    for seed in range(4):
        new = torch.randint(-1, E, (R, 1), generator=_gen(seed), dtype=I32)
        ids.copy_(new)
        graph.replay()
        want = _lists(m, new, E)
        torch.cuda.synchronize()
        assert np.array_equal(o.cpu().numpy(), want[0]) and np.array_equal(p.cpu().numpy(), want[1])
        ro, rp = ref.lists(new.numpy(), E)
        assert np.array_equal(want[0], ro) and np.array_equal(want[1], rp)


@pytest.mark.parametrize("dtype", [BF, F16])
@pytest.mark.parametrize("M", [4, 100, 2000])
def test_linear_special_codes_in_16_bits(m, M, dtype):
    """NaN codes and scales through the FP8 cores: they stay in their rows and columns, also in the last block and in
    padded rows of a tile."""
    g = _gen(M)
    N, K = 4000 if M == 2000 else 300, 272
    a, w = _codes((M, K), g), _codes((N, K), g)
    a.view(torch.uint8)[1, 271] = 0x7f
    w.view(torch.uint8)[N - 1, 0] = 0xff
    sa, sw = torch.ones(M, 3), torch.ones(ref.kb(N), 3)
    sa[M - 1, 2] = NAN
    sw[0, 1] = 0.0
    out = torch.empty(M, N, dtype=dtype, device=DEV)
    m.moe_linear_f8(a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), out)
    torch.cuda.synchronize()
    got = _np(out)
    with np.errstate(invalid="ignore"):
        y, e = ref.linear(_np(a.float()), _np(sa), _np(w.float()), _np(sw))
    fine = np.isfinite(y)
    assert not fine[[1, M - 1]].any() and not fine[:, N - 1].any() and fine[0, 0]
    assert np.array_equal(np.isfinite(got), fine)
    _check(got[fine], y[fine], np.nan_to_num(e[fine]), dtype)


@pytest.mark.parametrize("B", [1, 40])
def test_block_with_norm_and_int8_shared_expert(m, B):
    """FP4 experts and an int8 shared expert behind a norm: that one's int8 codes; without a shared expert none."""
    log(f"block with norm, int8 B={B}")
    g = _gen(B + 3)
    block = _block(g, f8=(False, False))
    x, r = torch.randn(B, 512, generator=g).to(BF).to(DEV), torch.randn(B, 512, generator=g).to(BF).to(DEV)
    r1 = r.clone()
    y = block.forward(x, residual=r1)
    n, q, s = block.norm.forward(r1, codes=torch.int8)
    ids, wts = block.router.forward(n)
    comb = block.layer.combine(block.layer.forward(n, ids), wts)
    want = block.shared.forward((q, s), add=comb)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(r1, (x.float() + r.float()).to(BF))
    h, eh = dense_ref.linear(q.cpu().numpy(), s.cpu().numpy(), block.shared.w13.cpu().numpy(), block.shared.s13.cpu().numpy(), act="swiglu")
    block.shared.forward((q, s))
    torch.cuda.synchronize()
    assert np.all(np.abs(_np(block.shared.hidden[:B]) - h) <= eh + 2.0 ** -8 * (np.abs(h) + eh))
    bare = type(block)(block.router, block.layer, None, block.norm)
    assert torch.equal(bare.forward(r1), comb)

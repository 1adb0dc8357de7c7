"""The dense side's operators on the GPU against plain 64-bit forms (dense_ref): the router's
product, the choice of experts, int8 quantization and the int8 product; then the whole
layer made of them."""
import numpy as np
import pytest
import torch

import dense_ref as ref
from helpers import log

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
HALF_STEP = {BF: 2.0 ** -8, F16: 2.0 ** -11, F32: 2.0 ** -24}   # largest rounding, relative
TINY = {BF: 2.0 ** -134, F16: 2.0 ** -25, F32: 2.0 ** -150}     # and among subnormals


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import moe_routed_expert_mx_amd as pkg
    return pkg


def _gen(seed):
    return torch.Generator("cpu").manual_seed(seed)


# --------------------------------------------------------------------- route
def _route(m, logits, topk, stream=None, **o):
    lg = logits.to(DEV) if logits.device.type == "cpu" else logits
    B = lg.shape[0]
    ids = torch.full((B + 1, topk), -7, dtype=torch.int32, device=DEV)
    w = torch.full((B + 1, topk), -7.0, device=DEV)
    bias = o.pop("bias", None)
    m.moe_route(lg, ids[:B], w[:B], bias=None if bias is None else bias.to(DEV), stream=stream, **o)
    torch.cuda.synchronize()
    assert (ids[B] == -7).all() and (w[B] == -7).all()          # nothing behind the last token
    return ids[:B].cpu().numpy(), w[:B].cpu().numpy()


def _check_route(m, logits, topk, **o):
    ids, w = _route(m, logits, topk, **dict(o))
    bias = o.pop("bias", None)
    rid, rw = ref.route(logits.double().numpy(), topk, bias=None if bias is None else bias.double().numpy(), **o)
    assert np.array_equal(ids, rid)
    # FP64 weights, some 2^-50 off, rounded to FP32 once
    assert np.all(np.abs(w - rw) <= np.abs(rw) * (2.0 ** -24 * 1.001) + TINY[F32])


MODES = [dict(), dict(renorm=False), dict(score="sigmoid", scale=2.5), dict(bias=True),
         dict(score="sigmoid", bias=True), dict(score="sigmoid", bias=True, renorm=False, scale=0.5)]


@pytest.mark.parametrize("B,E,K", [(1, 1, 1), (1, 160, 16), (3, 16, 4), (7, 63, 8), (33, 64, 1), (5, 65, 64),
                                   (257, 160, 16), (9, 257, 5), (6, 1024, 64), (2, 64, 64), (1000, 8, 2)])
@pytest.mark.parametrize("mode", range(len(MODES)))
def test_route_sizes(m, B, E, K, mode):
    log(f"route {B}x{E} top {K} {MODES[mode]}")
    g = _gen(B * 31 + E + mode)
    o = dict(MODES[mode])
    if o.pop("bias", False):
        o["bias"] = torch.randn(E, generator=g) * 0.1
    dtype = (F32, BF, F16)[(B + E + mode) % 3]          # the narrow types bring ties
    _check_route(m, (torch.randn(B, E, generator=g) * 2).to(dtype), K, **o)


@pytest.mark.parametrize("E,groups,kept,K", [(160, 10, 5, 16), (256, 8, 4, 8), (64, 64, 7, 7), (12, 2, 1, 6),
                                             (16, 1, 1, 3), (1024, 64, 3, 48), (35, 7, 7, 35), (96, 3, 2, 64),
                                             (160, 20, 1, 8), (1020, 4, 2, 10)])
@pytest.mark.parametrize("score,bias,group_score", [("softmax", False, "max"), ("sigmoid", True, "top2"),
                                                    ("softmax", False, "top2"), ("softmax", True, "max")])
def test_route_groups(m, E, groups, kept, K, score, bias, group_score):
    log(f"route groups E={E} {groups}/{kept} K={K} {score} {bias} {group_score}")
    g = _gen(E + groups)
    o = dict(score=score, groups=groups, topk_groups=kept, group_score=group_score)
    if bias:
        o["bias"] = torch.randn(E, generator=g) * 0.2
    dtype = (F32, BF)[(E + groups) % 2]
    _check_route(m, torch.randn(37, E, generator=g).to(dtype), K, **o)


@pytest.mark.parametrize("o", [dict(), dict(renorm=False), dict(score="sigmoid"),
                               dict(bias=True), dict(score="sigmoid", bias=True),
                               dict(groups=4, topk_groups=2), dict(groups=4, topk_groups=2, group_score="top2"),
                               dict(score="sigmoid", bias=True, groups=4, topk_groups=2, group_score="top2")])
def test_route_masked_infinite_and_tied(m, o):
    """Rows that are masked in part or whole, by -inf, NaN or the type's lowest value; +inf;
    equal logits; equal after the score saturates."""
    log(f"route special values {o}")
    o, E, inf, nan, low = dict(o), 32, float("inf"), float("nan"), torch.finfo(F32).min
    x = torch.randn(24, E, generator=_gen(5))
    x[0] = -inf
    x[1] = nan
    x[2] = low
    x[3], x[3, 5] = -inf, 1.0
    x[4], x[4, 31] = nan, -1000.0
    x[5, ::2] = -inf
    x[6, 3] = inf
    x[7, 3:9] = inf
    x[8] = inf
    x[9] = 0.0
    x[10], x[10, 7:] = 1.0, 2.0
    x[11] = 100.0 + torch.arange(E)                    # sigmoid is 1 for all: the logits differ still
    x[12] = -1000.0 - torch.arange(E)                  # sigmoid underflows
    x[13, 4], x[13, 5] = inf, nan
    x[14, :] = low
    x[14, 9] = -low
    x[15, 8:16] = -inf                                  # a whole group
    x[16, 8:] = -inf                                    # all groups but one
    x[17, :24] = nan
    x[18] = torch.where(torch.arange(E) % 8 == 3, 0.5, -inf)     # one open expert a group
    x[19, 0] = -0.0
    x[20] *= 1e-30                                      # a choice closer than a score can tell
    if o.pop("bias", False):
        b = torch.randn(E, generator=_gen(6)) * 0.1
        b[2], b[11], b[20] = -inf, nan, 3.0
        o["bias"] = b
    _check_route(m, x, 9, **o)


def test_route_signed_zeros_are_equal(m):
    x = torch.zeros(4200, 40)
    x[:, ::3] = -0.0
    _check_route(m, x[:5], 7)
    _check_route(m, x, 7)                               # many tokens: another division of the lanes
    _check_route(m, x[:5].to(BF), 7, bias=torch.zeros(40))


@pytest.mark.parametrize("E,K,o", [(160, 16, dict(score="sigmoid", bias=True, groups=10, topk_groups=5,
                                                  group_score="top2")), (64, 6, dict()), (200, 33, dict(renorm=False)),
                                   (256, 8, dict(groups=16, topk_groups=3)), (17, 17, dict(bias=True))])
def test_route_many_tokens(m, E, K, o):
    log(f"route 5000x{E} {o}")
    o, g = dict(o), _gen(E)
    if o.pop("bias", False):
        o["bias"] = torch.randn(E, generator=g) * 0.1
    x = (torch.randn(5001, E, generator=g) * 2).to(F32 if E != 64 else F16)
    x[::7, ::2] = -float("inf")
    x[3] = float("nan")
    _check_route(m, x, K, **o)


@pytest.mark.parametrize("E,K,o", [(48, 8, dict(groups=6, topk_groups=2)), (160, 16, dict(bias=True)), (250, 64, dict()),
                                   (170, 5, dict(groups=17, topk_groups=3, bias=True)), (300, 7, dict(score="sigmoid")),
                                   (1023, 20, dict(groups=33, topk_groups=4, group_score="top2"))])
@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_route_many_tokens_each_type(m, E, K, o, dtype):
    """Beyond 4096 tokens: 16 lanes a token in their three sizes, and 64 for more experts or groups than those take."""
    log(f"route 4111x{E} {o} {dtype}")
    o, g = dict(o), _gen(E)
    if o.pop("bias", False):
        o["bias"] = torch.randn(E, generator=g) * 0.1
    x = (torch.randn(4111, E, generator=g) * 2).to(dtype)
    x[::9, ::2] = -float("inf")
    _check_route(m, x, K, **o)


def test_route_infinite_bias(m):
    b = torch.zeros(20)
    b[7], b[3] = float("inf"), float("inf")
    _check_route(m, torch.randn(5, 20, generator=_gen(1)), 4, bias=b)
    _check_route(m, torch.randn(5, 20, generator=_gen(1)), 4, bias=b, groups=5, topk_groups=2, group_score="top2")


@pytest.mark.parametrize("B", [5, 4500])
@pytest.mark.parametrize("o", [dict(), dict(renorm=False), dict(score="sigmoid"),
                               dict(score="sigmoid", groups=4, topk_groups=4, group_score="top2"),
                               dict(groups=4, topk_groups=3)])
def test_route_selects_experts_whose_bias_is_not_finite(m, B, o):
    """Experts with a bias of NaN or -inf come last, among them the masked ones, by index; selected, they keep the weight
    that their score gives them."""
    log(f"route nan bias B={B} {o}")
    E = 16
    g = _gen(B)
    b = torch.randn(E, generator=g) * 0.1
    b[1], b[6], b[15] = float("nan"), -float("inf"), float("nan")
    x = torch.randn(B, E, generator=g)
    x[1, 3], x[2, 6], x[3, ::2] = -float("inf"), float("nan"), -float("inf")
    _check_route(m, x, 12 if o.get("topk_groups") == 3 else E, bias=b, **o)


@pytest.mark.parametrize("through", ["binding", "ctypes"])
def test_route_scales_near_the_ends_of_fp32(m, through):
    st = None if through == "binding" else torch.cuda.current_stream()
    x = torch.zeros(3, 16)
    for scale in (2.0 ** -149, -2.0 ** -126, 2.0 ** 127, 1e-45, True):
        _, w = _route(m, x, 4, stream=st, scale=scale)
        assert np.array_equal(w, np.full((3, 4), float(np.float32(np.float64(np.float32(scale)) / 4)), np.float32))
    for scale in (1e-46, 0.0, float("inf"), 1e39):
        with pytest.raises(ValueError, match="scale"):
            _route(m, x, 4, stream=st, scale=scale)


def test_route_strided_rows_and_streams(m):
    big = torch.randn(50, 200, generator=_gen(9)).to(DEV)
    view = big[:, 13:13 + 96]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ids, w = _route(m, view, 6, stream=s)
    rid, rw = ref.route(view.cpu().double().numpy(), 6)
    assert np.array_equal(ids, rid) and np.allclose(w, rw, rtol=1e-6)
    with torch.cuda.stream(s):                          # the tensors' current stream
        ids2, _ = _route(m, view, 6)
    assert np.array_equal(ids2, rid)


def test_route_near_choices(m):
    """Choices that differ by less than an FP32 step: FP64 decides, as in the plain form."""
    g = _gen(77)
    x = torch.randn(300, 64, generator=g)
    x[:, 1::2] = x[:, ::2] + torch.randn(300, 32, generator=g) * 1e-7
    _check_route(m, x, 16, score="sigmoid", bias=torch.zeros(64))
    _check_route(m, x, 16, bias=torch.full((64,), 3.0))
    _check_route(m, x, 16, score="sigmoid", bias=torch.full((64,), 1000.0), groups=8, topk_groups=4,
                 group_score="top2")


# ---------------------------------------------------------------------- gate
def _gate(m, x, w, ld=None, out_ld=None):
    E, D = w.shape
    packed = torch.empty(m.moe_gate_packed_bytes(E, D, w.dtype), dtype=torch.uint8, device=DEV)
    h = m.moe_gate_pack(w.to(DEV), packed)
    B = x.shape[0]
    xd = torch.zeros(B, ld or D, dtype=BF, device=DEV)[:, :D]
    xd.copy_(x)
    out = torch.full((B + 1, out_ld or E), -7.0, device=DEV)
    m.moe_gate(h, xd, out[:B, :E])
    torch.cuda.synchronize()
    assert (out[B] == -7).all() and (out[:, E:] == -7).all()
    return out[:B, :E].cpu().double()


@pytest.mark.parametrize("B,E,D", [(1, 160, 3584), (8, 160, 3584), (1, 1, 512), (17, 16, 512), (64, 81, 1024),
                                   (65, 200, 512), (129, 15, 1536), (300, 1024, 512), (256, 160, 3584), (31, 96, 512),
                                   (2, 256, 16384),
                                   # one for each further tile: 32 x 16, 32 x 32, 64 x 32, 64 x 48, 64 x 80
                                   (600, 160, 512), (1300, 161, 512), (2601, 160, 512), (5000, 100, 512),
                                   (8191, 159, 512), (9000, 250, 512)])
@pytest.mark.parametrize("wtype", [BF, F32])
def test_gate_whole_numbers_are_exact(m, B, E, D, wtype):
    """Whole numbers whose sums stay below 2^24: every order of summation gives the same."""
    log(f"gate exact {B}x{E}x{D} {wtype}")
    g = _gen(B + E + D)
    x = torch.randint(-8, 9, (B, D), generator=g).to(BF)
    w = torch.randint(-100, 101, (E, D), generator=g).to(wtype)
    want = x.double() @ w.double().T
    assert torch.equal(_gate(m, x, w, ld=D + 64, out_ld=E + 3), want)


@pytest.mark.parametrize("B,E", [(600, 160), (1300, 161), (2601, 160), (5000, 100), (8191, 159)])
@pytest.mark.parametrize("D", [1536, 3584])
@pytest.mark.parametrize("wtype", [BF, F32])
def test_gate_tiles_with_long_rows(m, B, E, D, wtype):
    """Each larger tile with more features to a wave than it has in flight, and with unequal shares."""
    log(f"gate long rows {B}x{E}x{D} {wtype}")
    g = _gen(B + E + D)
    x = torch.randint(-8, 9, (B, D), generator=g).to(BF)
    w = torch.randint(-100, 101, (E, D), generator=g).to(wtype)
    assert torch.equal(_gate(m, x, w, out_ld=E + 1), x.double() @ w.double().T)


def test_gate_fp32_weight_keeps_all_its_bits(m):
    """One feature a token: the logits are the FP32 weights themselves times a power of two."""
    g = _gen(3)
    w = (torch.randn(48, 512, generator=g) * torch.exp2(torch.randint(-40, 40, (48, 512), generator=g).float()))
    x = torch.zeros(512, 512)
    x[torch.arange(512), torch.randperm(512, generator=g)] = torch.exp2(torch.randint(-8, 9, (512,), generator=g).float())
    got = _gate(m, x.to(BF), w)
    assert torch.equal(got, x.double() @ w.double().T)


@pytest.mark.parametrize("B,E,D", [(8, 160, 3584), (200, 100, 1024), (1030, 160, 512)])
@pytest.mark.parametrize("wtype", [BF, F32])
def test_gate_normal_values(m, B, E, D, wtype):
    """FP32 sums of D (three planes: 3 D) exact products: each addition is off by at most a step
    2^-23 of the partial sum (the matrix unit need not round to nearest), the partial sums at
    most sum |x w| (planes of one sign: the same)."""
    log(f"gate normal {B}x{E}x{D} {wtype}")
    g = _gen(D)
    x, w = torch.randn(B, D, generator=g).to(BF), (torch.randn(E, D, generator=g) / D ** 0.5).to(wtype)
    got = _gate(m, x, w)
    err = (got - x.double() @ w.double().T).abs()
    bound = (3 * D if wtype == F32 else D) * 2.0 ** -23 * (x.double().abs() @ w.double().abs().T)
    assert (err <= bound).all()


def test_gate_rows_do_not_meet(m):
    """A token with a non-finite feature has non-finite logits and leaves the others alone."""
    g = _gen(4)
    x, w = torch.randint(-8, 9, (40, 512), generator=g).to(BF), torch.randint(1, 9, (20, 512), generator=g).to(F32)
    want = x.double() @ w.double().T
    x[7, 100], x[33, 0] = float("inf"), float("nan")
    got = _gate(m, x, w)
    bad = torch.zeros(40, dtype=torch.bool)
    bad[[7, 33]] = True
    assert not got[bad].isfinite().any() and torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("through", ["binding", "ctypes"])
def test_gate_weight_elsewhere_is_refused(m, through):
    """The packed weight is held to the GPU of x, on both ways into the library."""
    import ctypes
    st = None if through == "binding" else torch.cuda.current_stream()
    h = m.moe_gate_pack(torch.ones(16, 512, device=DEV),
                        torch.empty(m.moe_gate_packed_bytes(16, 512, F32), dtype=torch.uint8, device=DEV))
    x, lg = torch.ones(4, 512, dtype=BF, device=DEV), torch.zeros(4, 16, device=DEV)
    m.moe_gate(h, x, lg, stream=st)
    assert (lg == 512).all()
    lg.zero_()
    packed, h.tensor = h.tensor, h.tensor.cpu()
    assert m._lib._dense.gate(ctypes.addressof(h), 512, 16, x, lg, h.tensor) == -100
    with pytest.raises(ValueError, match="one GPU"):
        m.moe_gate(h, x, lg, stream=st)
    assert not lg.any()
    h.tensor = packed
    assert m._lib._dense.gate(ctypes.addressof(h), 512, 16, x, lg, packed) == 0
    assert (lg == 512).all()


# --------------------------------------------------------------------- quant
def _check_quant(m, x, ldx=0, ldc=0):
    M, K = x.shape
    xd = torch.zeros(M, K + ldx, dtype=x.dtype, device=DEV)[:, :K]
    xd.copy_(x)
    q = torch.full((M + 1, K + ldc), 99, dtype=torch.int8, device=DEV)
    s = torch.full((M + 1,), -7.0, device=DEV)
    m.moe_quant_i8(xd, q[:M, :K], s[:M])
    torch.cuda.synchronize()
    assert (q[M] == 99).all() and (q[:, K:] == 99).all() and s[M] == -7
    rq, rs = ref.quant(x.double().numpy())
    assert np.array_equal(q[:M, :K].cpu().numpy(), rq)
    assert np.array_equal(s[:M].cpu().numpy(), rs, equal_nan=True)


@pytest.mark.parametrize("M,K,ldx,ldc", [(1, 1, 0, 0), (8, 3584, 0, 0), (3, 384, 0, 0), (5, 17, 0, 0), (4, 64, 3, 5),
                                         (2, 4096, 8, 16), (9, 1000, 0, 0), (1, 131072, 0, 0), (300, 129, 0, 0),
                                         (2, 8191, 1, 0), (3, 20000, 0, 0), (1031, 512, 0, 0), (2, 16392, 0, 0)])
@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_quant_sizes(m, M, K, ldx, ldc, dtype):
    log(f"quant {M}x{K}+{ldx} {dtype}")
    g = _gen(M + K)
    _check_quant(m, (torch.randn(M, K, generator=g) * torch.exp2(torch.randint(-6, 7, (M, 1), generator=g))).to(dtype),
                 ldx, ldc)


@pytest.mark.parametrize("K,ldx,ldc", [(250, 0, 0), (257, 0, 3), (1021, 3, 0), (1032, 0, 0), (2040, 8, 8), (2050, 0, 0),
                                       (4090, 0, 0), (4097, 1, 1)])
@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_quant_many_tokens(m, K, ldx, ldc, dtype):
    """A wave a token, 1 to 8 pieces a lane, and rows too long for that."""
    log(f"quant 1027x{K}+{ldx} {dtype}")
    _check_quant(m, torch.randn(1027, K, generator=_gen(K)).to(dtype), ldx, ldc)


@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_quant_halves_and_extremes(m, dtype):
    """Quotients at exactly a half (even wins) and one step beside it, zeros, subnormals, the
    type's largest values, infinities and NaN."""
    fi = torch.finfo(dtype)
    K = 254
    x = torch.zeros(14, K)
    x[0] = torch.arange(K) / 2 - 63.5                 # amax 63.5: x * 127 / amax = 2 x
    x[1] = (torch.arange(K) - 127) * 1.0              # amax 127
    x[1, 0] = 254.0                                    # amax 254: halves of whole numbers
    x[2] = 0.0
    x[3] = -0.0
    x[4, 3], x[4, 4] = fi.max, -fi.max / 2
    x[5] = fi.tiny * (torch.arange(K) / K)            # subnormal or just above
    x[6, 0] = fi.smallest_normal
    x[7, 9] = float("inf")
    x[8, 9] = float("-inf")
    x[9, 0] = float("nan")
    x[10] = torch.randn(K, generator=_gen(1))
    x[10, 200], x[10, 3] = float("nan"), float("inf")
    x[11, 100] = -3.0
    x = x.to(dtype)
    # amax with halves in reach, each neighboured by the next value of the type up and down
    up = (x[1].view(torch.int32 if dtype == F32 else torch.int16) + 1).view(dtype)
    dn = (x[1].view(torch.int32 if dtype == F32 else torch.int16) - 1).view(dtype)
    x[12], x[13] = torch.where(x[1].abs() < 127, up, x[1]), torch.where(x[1].abs() < 127, dn, x[1])
    x[12, 127] = x[13, 127] = 0                        # 0 has no neighbour below
    x[12, 0] = x[13, 0] = 254.0
    _check_quant(m, x)


@pytest.mark.parametrize("dtype", [BF, F16])
def test_quant_every_mantissa(m, dtype):
    """Every pair of significands of amax and x over a range of exponents."""
    bits = 7 if dtype == BF else 10
    top = 1 + torch.arange(2 ** bits)[:: 1 if dtype == BF else 7] / 2 ** bits
    row = torch.cat([(1 + torch.arange(2 ** bits) / 2 ** bits) * 2.0 ** -e for e in range(1, 9)])
    x = torch.cat([top[:, None], -row.expand(len(top), -1)], dim=1).to(dtype)
    _check_quant(m, x)


@pytest.mark.parametrize("dtype", [BF, F16])
def test_quant_every_pair_of_significands(m, dtype):
    """amax of every significand, x of every one up to it and in the binade below: among them the quotient nearest
    to a half, FP16's 2025 * 127 / 2033, off it by 2^-18.97 of itself."""
    n = 2 ** (7 if dtype == BF else 10)
    sig = torch.arange(n, 2 * n)
    same = torch.where(sig[None, :] <= sig[:, None], sig[None, :], 0)
    x = torch.cat([sig[:, None], same, -(sig / 2).expand(n, -1)], dim=1)
    assert dtype == BF or x[2033 - n, 1 + 2025 - n] == 2025
    _check_quant(m, x.to(dtype))
    _check_quant(m, (x / n).to(dtype)[:1000])          # few tokens: four waves each


# -------------------------------------------------------------------- linear
def _codes(shape, g):
    return torch.randint(-128, 128, shape, generator=g).to(torch.int8)


def _place(t, ld, offset=0):
    """A copy of t [rows, cols] on the GPU with row distance ld, `offset` elements into its
    storage, and nothing behind its last element."""
    r, c = t.shape
    flat = torch.zeros(offset + (r - 1) * ld + c, dtype=t.dtype, device=DEV)
    v = torch.as_strided(flat, (r, c), (ld, 1), offset)
    v.copy_(t)
    return v


def _check_linear(m, M, N, K, *, out=BF, act="none", bias=False, add=False, inplace=False, lda=0, ldw=0, ldo=0,
                  offset=0, seed=0, codes=None):
    log(f"linear {M}x{N}x{K} {out} {act} bias={bias} add={add} ld+={lda},{ldw},{ldo} @{offset}")
    g = _gen(seed + M * 7 + N * 3 + K)
    cols = N // 2 if act == "swiglu" else N
    a, w = codes if codes is not None else (_codes((M, K), g), _codes((N, K), g))
    sa, sw = (0.5 + torch.rand(M, generator=g)) * 0.02, (0.5 + torch.rand(N, generator=g)) * 0.02 / K ** 0.5
    b = torch.randn(N, generator=g) if bias else None
    d = torch.randn(M, cols, generator=g).to(out) if add else None
    buf = torch.full((M + 1, cols + ldo), -7.0, dtype=out, device=DEV)
    o = buf[:M, :cols]
    if inplace:
        o.copy_(d)
    ad, wd = _place(a, K + lda, offset), _place(w, K + ldw, offset)
    m.moe_linear_i8(ad, sa.to(DEV), wd, sw.to(DEV), o, act=act, bias=None if b is None else b.to(DEV),
                    add=None if d is None else o if inplace else d.to(DEV))
    torch.cuda.synchronize()
    assert (buf[M] == -7).all() and (buf[:, cols:] == -7).all()
    y, slack = ref.linear(a.numpy(), sa.numpy(), w.numpy(), sw.numpy(), act=act,
                          bias=None if b is None else b.numpy(), add=None if d is None else d.double().numpy())
    err = np.abs(o.cpu().double().numpy() - y)
    tol = slack + HALF_STEP[out] * (np.abs(y) + slack) + TINY[out]
    assert np.all(err <= tol), (err / tol).max()


SIZES = [(1, 1, 1), (1, 768, 3584), (8, 3584, 384), (2, 16, 64), (3, 18, 65), (16, 32, 128), (17, 34, 100),
         (31, 66, 17), (64, 64, 256), (65, 130, 1000), (64, 512, 4096), (100, 200, 48), (127, 126, 129),
         (128, 256, 512), (129, 258, 640), (200, 1024, 384), (255, 512, 1023), (256, 768, 3584), (300, 520, 2048),
         (1000, 384, 272), (513, 770, 144), (1, 2, 131071)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_linear_sizes(m, M, N, K, act):
    if act == "swiglu" and N % 2:
        N += 1
    i = M + N + K
    _check_linear(m, M, N, K, act=act, out=(BF, F16, F32)[i % 3] if act == "none" else (BF, F32)[i % 2],
                  bias=i % 2 == 0, add=i % 4 < 2)


# sizes that take each of the tiles (64 x 64, 64 x 128, 128 x 128, 128 x 256, 256 x 256) and the kernel for unaligned
# rows
TILES = [(300, 2050, 272), (500, 3000, 272), (1000, 3000, 144), (2000, 4000, 80), (4090, 4090, 80), (520, 2050, 273), (700, 2500, 130)]


@pytest.mark.parametrize("M,N,K", TILES)
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_linear_tiles(m, M, N, K, act):
    _check_linear(m, M, N, K, act=act, out=BF, bias=True, add=True, seed=1)
    pad = 16 if K % 16 == 0 else 1
    _check_linear(m, M, N, K, act=act, out=F32 if M < 2000 else F16, lda=pad, ldw=2 * pad, ldo=3, offset=pad, seed=2)


# The streaming kernel's variants by the launch rule: 16, 32 and 64 tokens a block; one row tile (up to 256 blocks,
# the first size of a pair) and two; aligned and unaligned rows (K or K + 1), with more than 64 tokens too.  M, N and
# K leave a remainder in each; K = 9008 gives each wave more pieces than it has in flight, 272 leaves most waves none.
STREAM = [(11, 100), (11, 4114), (24, 100), (24, 4114), (50, 100), (50, 4130), (70, 258), (500, 770), (130, 2070)]


@pytest.mark.parametrize("M,N", STREAM)
@pytest.mark.parametrize("K", [272, 273, 9008, 9009])
@pytest.mark.parametrize("act", ["none", "swiglu"])
def test_linear_streaming_variants(m, M, N, K, act):
    if M > 100 and K > 1000:
        K -= 7008
    _check_linear(m, M, N, K, act=act, out=(BF, F32)[K % 2], bias=K % 2 == 0, add=True, seed=5)
    _check_linear(m, M, N, K, act=act, out=F16, bias=K % 2 == 1, lda=16, ldw=32, offset=16, ldo=1, seed=6)


# a single row in the last tile of each size, plain (64 x 64, 64 x 128, 128 x 128, 128 x 256, 256 x 256) and SwiGLU
@pytest.mark.parametrize("M,N,act", [(257, 1793, "none"), (257, 3329, "none"), (513, 3585, "none"), (3585, 1025, "none"),
                                     (3073, 3841, "none"), (513, 1026, "swiglu"), (257, 6658, "swiglu"),
                                     (513, 7170, "swiglu"), (2305, 5122, "swiglu")])
def test_linear_last_tile_of_one_row(m, M, N, act):
    """Its extent is one row of K bytes, and the stages issued ahead lie behind that."""
    _check_linear(m, M, N, 16, act=act, out=F32, seed=3)
    _check_linear(m, M, N, 144, act=act, bias=True, lda=16, ldw=32, seed=4)


@pytest.mark.parametrize("M,N", [(300, 2050), (1000, 3000)])
def test_linear_tiles_longest_rows(m, M, N):
    K = 131056
    a = torch.full((M, K), -128, dtype=torch.int8, device=DEV)
    w = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
    w[N - 1] = 127
    out = torch.empty(M, N, device=DEV)
    m.moe_linear_i8(a, torch.ones(M, device=DEV), w, torch.ones(N, device=DEV), out)
    assert (out[:, :N - 1] == float(16384 * K)).all()
    assert (out[:, N - 1] == float(np.float32(-128 * 127 * K))).all()


@pytest.mark.parametrize("out", [BF, F16, F32])
@pytest.mark.parametrize("M", [1, 5, 24, 40, 70, 300])
def test_linear_epilogues(m, out, M):
    for act in ("none", "swiglu"):
        for bias in (False, True):
            for add in (False, True):
                _check_linear(m, M, 96, 256, out=out, act=act, bias=bias, add=add, ldo=5 if add else 0)
    _check_linear(m, M, 96, 256, out=out, add=True, inplace=True)


@pytest.mark.parametrize("M", [1, 20, 64, 150, 600])
@pytest.mark.parametrize("lda,ldw,offset,K", [(16, 0, 0, 256), (0, 32, 16, 256), (1, 0, 0, 256), (0, 3, 0, 256),
                                              (0, 0, 5, 256), (7, 9, 3, 250), (6, 6, 0, 250), (1000, 2000, 0, 320)])
def test_linear_strides(m, M, lda, ldw, offset, K):
    _check_linear(m, M, 130, K, lda=lda, ldw=ldw, ldo=3, offset=offset)
    _check_linear(m, M, 130, K, lda=lda, ldw=ldw, offset=offset, act="swiglu", out=F32)


@pytest.mark.parametrize("M,N,K", [(2, 32, 131071), (40, 64, 131056), (300, 320, 20000)])
def test_linear_extreme_codes(m, M, N, K):
    """-128 times -128 over the longest rows: the sum's largest value, 2^31 - 2^14."""
    a, w = torch.full((M, K), -128, dtype=torch.int8), torch.full((N, K), -128, dtype=torch.int8)
    w[1] = 127
    _check_linear(m, M, N, K, out=F32, codes=(a, w))


def test_linear_non_finite_scales(m):
    """A NaN scale makes its row or column NaN and no other; so the quantization of a row with an
    infinity reaches the result."""
    g = _gen(8)
    x = torch.randn(40, 64, generator=g).to(BF)
    x[11, 5] = float("inf")
    q, s = torch.empty(40, 64, dtype=torch.int8, device=DEV), torch.empty(40, device=DEV)
    m.moe_quant_i8(x.to(DEV), q, s)
    w, sw = _codes((48, 64), g).to(DEV), torch.rand(48, generator=g).to(DEV)
    sw[7] = float("nan")
    out = torch.empty(40, 48, dtype=BF, device=DEV)
    m.moe_linear_i8(q, s, w, sw, out)
    bad = out.cpu().isnan()
    want = torch.zeros(40, 48, dtype=torch.bool)
    want[11], want[:, 7] = True, True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("N,K", [(32, 64), (2050, 64), (2050, 65)])
def test_linear_rows_past_32_bit_offsets(m, N, K):
    """A row distance that puts the last rows of a and out beyond 2^32 bytes."""
    M, ld = 1100, (1 << 22) - 16
    store = torch.zeros((M - 1) * ld + K, dtype=torch.int8, device=DEV)
    a = torch.as_strided(store, (M, K), (ld, 1))
    g = _gen(2)
    codes, w = _codes((M, K), g), _codes((N, K), g)
    a.copy_(codes)
    sa, sw = torch.ones(M), torch.ones(N)
    ostore = torch.zeros((M - 1) * ld + N, dtype=F32, device=DEV)
    o = torch.as_strided(ostore, (M, N), (ld, 1))
    m.moe_linear_i8(a, sa.to(DEV), w.to(DEV), sw.to(DEV), o)
    want = codes.double() @ w.double().T
    assert torch.equal(o.cpu().double(), want)


# ----------------------------------------------------------- graphs and chains
def test_captured_and_replayed(m):
    """All operators in one graph, replayed with eager work and new inputs between."""
    g = _gen(21)
    B, D, E, K, I = 24, 512, 40, 6, 96
    w = torch.randn(E, D, generator=g).to(DEV)
    packed = torch.empty(m.moe_gate_packed_bytes(E, D, F32), dtype=torch.uint8, device=DEV)
    h = m.moe_gate_pack(w, packed)
    wq, ws = _codes((2 * I, D), g).to(DEV), torch.rand(2 * I, generator=g).to(DEV) * 1e-3
    x = torch.randn(B, D, generator=g).to(BF).to(DEV)

    def buffers():
        return dict(lg=torch.empty(B, E, device=DEV), ids=torch.empty(B, K, dtype=torch.int32, device=DEV),
                    w=torch.empty(B, K, device=DEV), q=torch.empty(B, D, dtype=torch.int8, device=DEV),
                    s=torch.empty(B, device=DEV), y=torch.empty(B, I, dtype=BF, device=DEV))

    def step(b):
        m.moe_gate(h, x, b["lg"])
        m.moe_route(b["lg"], b["ids"], b["w"], score="sigmoid", groups=4, topk_groups=2)
        m.moe_quant_i8(x, b["q"], b["s"])
        m.moe_linear_i8(b["q"], b["s"], wq, ws, b["y"], act="swiglu")

    cap, eager = buffers(), buffers()
    step(cap)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cap)
    for i in range(4):
        x.copy_(torch.randn(B, D, generator=g).to(BF))
        step(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k in cap:
            assert torch.equal(cap[k], eager[k]), (i, k)


def test_two_streams_at_once(m):
    """Calls that overlap on two streams give what they give alone (no shared state)."""
    g = _gen(23)
    sets = []
    for i in range(2):
        a, w = _codes((300, 1024), g).to(DEV), _codes((512, 1024), g).to(DEV)
        sets.append((a, torch.rand(300, generator=g).to(DEV), w, torch.rand(512, generator=g).to(DEV),
                     torch.empty(300, 512, dtype=F32, device=DEV)))
    alone = []
    for s in sets:
        m.moe_linear_i8(*s)
        torch.cuda.synchronize()
        alone.append(s[4].clone())
        s[4].zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        for st, s in zip(streams, sets):
            m.moe_linear_i8(*s, stream=st)
    torch.cuda.synchronize()
    for s, want in zip(sets, alone):
        assert torch.equal(s[4], want)


def test_host_threads(m):
    """Threads that call at once, each on a stream of its own."""
    import threading
    g = _gen(25)
    a, w = _codes((300, 512), g).to(DEV), _codes((2050, 512), g).to(DEV)
    sa, sw = torch.rand(300, generator=g).to(DEV), torch.rand(2050, generator=g).to(DEV)
    want = torch.empty(300, 2050, device=DEV)
    m.moe_linear_i8(a, sa, w, sw, want)
    outs = [torch.zeros_like(want) for _ in range(4)]
    torch.cuda.synchronize()

    def work(out):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                m.moe_linear_i8(a, sa, w, sw, out)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(o,)) for o in outs]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert all(torch.equal(want, o) for o in outs)


def test_native_binding_and_ctypes_agree(m):
    """A call without a stream goes through the native binding, one with a stream through ctypes: the same
    results, and the native binding does take what is right."""
    g, d, st = _gen(41), m._lib._dense, torch.cuda.current_stream()
    x = torch.randn(6, 512, generator=g).to(BF).to(DEV)
    w = torch.randn(40, 512, generator=g).to(DEV)
    h = m.moe_gate_pack(w, torch.empty(m.moe_gate_packed_bytes(40, 512, F32), dtype=torch.uint8, device=DEV))
    bias = torch.randn(40, generator=g).to(DEV)
    wq, ws = _codes((64, 512), g).to(DEV), torch.rand(64, generator=g).to(DEV)
    b, add = torch.randn(64, generator=g).to(DEV), torch.randn(6, 32, generator=g).to(BF).to(DEV)
    res = []
    for s in (None, st):
        lg, ids, wt = torch.empty(6, 40, device=DEV), torch.empty(6, 5, dtype=torch.int32, device=DEV), \
            torch.empty(6, 5, device=DEV)
        q, sc, y = torch.empty(6, 512, dtype=torch.int8, device=DEV), torch.empty(6, device=DEV), \
            torch.empty(6, 32, dtype=BF, device=DEV)
        m.moe_gate(h, x, lg, stream=s)
        m.moe_route(lg, ids, wt, score="sigmoid", bias=bias, groups=5, topk_groups=3, group_score="top2", scale=3,
                    stream=s)
        m.moe_quant_i8(x, q, sc, stream=s)
        m.moe_linear_i8(q, sc, wq, ws, y, act="swiglu", bias=b, add=add, stream=s)
        torch.cuda.synchronize()
        res.append((lg, ids, wt, q, sc, y))
    assert all(torch.equal(p, r) for p, r in zip(*res))
    lg, ids, wt, q, sc, y = res[0]
    import ctypes
    assert d.gate(ctypes.addressof(h), 512, 40, x, lg) == 0
    assert d.route(lg, ids, wt, 1, bias, 5, 3, 1, True, 3.0) == 0
    assert d.quant(x, q, sc) == 0
    assert d.linear(q, sc, wq, ws, y, 1, b, add) == 0
    assert d.linear(q, sc, wq, ws, y, 0, b, add) == -100        # out has half the columns
    assert d.quant(x, q.cpu(), sc) == -100
    with pytest.raises(ValueError, match="one GPU"):
        m.moe_quant_i8(x, q.cpu(), sc)
    with pytest.raises(m.MoeError):
        m.moe_route(lg, ids, wt, groups=7, topk_groups=1)       # 40 experts, 7 groups


def test_without_the_native_binding(m, monkeypatch):
    """Where the binding is not built, the same calls go through ctypes and give the same."""
    g = _gen(43)
    x, w = torch.randn(6, 512, generator=g).to(BF).to(DEV), torch.randn(40, 512, generator=g).to(DEV)
    h = m.moe_gate_pack(w, torch.empty(m.moe_gate_packed_bytes(40, 512, F32), dtype=torch.uint8, device=DEV))
    wq, ws = _codes((64, 512), g).to(DEV), torch.rand(64, generator=g).to(DEV)
    res = []
    for binding in (m._lib._dense, m._lib._NoBinding):
        monkeypatch.setattr(m._lib, "_dense", binding)
        lg, ids, wt = torch.empty(6, 40, device=DEV), torch.empty(6, 5, dtype=torch.int32, device=DEV), \
            torch.empty(6, 5, device=DEV)
        q, s, y = torch.empty(6, 512, dtype=torch.int8, device=DEV), torch.empty(6, device=DEV), \
            torch.empty(6, 32, dtype=BF, device=DEV)
        m.moe_gate(h, x, lg)
        m.moe_route(lg, ids, wt)
        m.moe_quant_i8(x, q, s)
        m.moe_linear_i8(q, s, wq, ws, y, act="swiglu")
        torch.cuda.synchronize()
        res.append((lg, ids, wt, q, s, y))
    assert all(torch.equal(p, r) for p, r in zip(*res))


def test_native_binding_calls_once_or_not_at_all(m):
    """The library's status comes back as it is, after one call; a stream that is no handle means no call.  (The
    library's function is a stand-in that launches nothing.)"""
    import ctypes
    calls, status = [], [0]

    @ctypes.CFUNCTYPE(ctypes.c_int, *[ctypes.c_void_p] * 14)
    def linear(*a):
        calls.append(a)
        return status[0]

    lib, d = m._lib, m._lib._dense
    names = ("moe_gate", "moe_route", "moe_quant_i8", "moe_linear_i8")
    own = [ctypes.cast(getattr(lib.lib, n), ctypes.c_void_p).value for n in names]
    stub = own[:3] + [ctypes.cast(linear, ctypes.c_void_p).value]
    q, s, out = torch.zeros(4, 16, dtype=torch.int8, device=DEV), torch.zeros(4, device=DEV), torch.zeros(4, 4, device=DEV)
    try:
        d.bind(*stub, lib._current_stream, lib._current_device)
        for status[0] in (0, lib.MOE_EHIP, lib.MOE_EINVAL):
            assert d.linear(q, s, q, s, out, 0, None, out) == status[0]
        assert len(calls) == 3
        for st in ("stream", None, 1 << 70):
            d.bind(*stub, lambda dev: st, lib._current_device)
            assert d.linear(q, s, q, s, out, 0, None, out) == -100
        d.bind(*stub, lib._current_stream, lambda: "device")
        assert d.linear(q, s, q, s, out, 0, None, out) == -100
        assert len(calls) == 3
    finally:
        d.bind(*own, lib._current_stream, lib._current_device)


@pytest.mark.parametrize("through", ["binding", "ctypes"])
def test_an_earlier_error_is_not_this_calls(m, through):
    """An error that another call left on the thread (no such device: the runtime refuses that) neither fails the
    calls here nor makes them run twice."""
    st = None if through == "binding" else torch.cuda.current_stream()
    g, hip = _gen(51), m._lib.lib
    a, w = _codes((3, 64), g).to(DEV), _codes((32, 64), g).to(DEV)
    sa, sw, out = torch.ones(3, device=DEV), torch.ones(32, device=DEV), torch.zeros(3, 32, device=DEV)
    x, gw = torch.ones(3, 512, dtype=BF, device=DEV), torch.ones(16, 512, dtype=BF, device=DEV)
    packed = torch.zeros(m.moe_gate_packed_bytes(16, 512, BF), dtype=torch.uint8, device=DEV)
    lg, ids, wt = torch.zeros(3, 16, device=DEV), torch.zeros(3, 2, dtype=torch.int32, device=DEV), torch.zeros(3, 2, device=DEV)
    q, s = torch.zeros(3, 512, dtype=torch.int8, device=DEV), torch.zeros(3, device=DEV)
    want = a.cpu().double() @ w.cpu().double().T
    torch.cuda.synchronize()
    gate = []
    try:
        for call in (lambda: m.moe_linear_i8(a, sa, w, sw, out, add=out, stream=st),
                     lambda: gate.append(m.moe_gate_pack(gw, packed, stream=st)),
                     lambda: m.moe_gate(gate[0], x, lg, stream=st), lambda: m.moe_route(lg, ids, wt, stream=st),
                     lambda: m.moe_quant_i8(x, q, s, stream=st)):
            assert hip.hipSetDevice(100000) != 0
            call()
    finally:
        hip.hipGetLastError()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu().double(), want)
    assert (lg == 512).all() and (ids == torch.tensor([0, 1], device=DEV)).all() and (wt == 0.5).all()
    assert (q == 127).all()


@pytest.mark.parametrize("B", [1, 8, 40])
def test_block_end_to_end(m, B):
    """The layer as it is used: router, routed experts, combine, shared expert.  Each stage is
    checked against the plain form of the stage on the values that the GPU handed it."""
    import workloads
    from moe_routed_expert_mx_amd.block import MoeBlock, Router, SharedExpertI8
    from moe_routed_expert_mx_amd.layer import MoeLayer
    log(f"block B={B}")
    d = workloads.generate(workloads.custom(B=B, E=24, K=4, D=512, I=64, seed=B))
    g = _gen(B)
    x = torch.from_numpy(d["x"]).view(BF).to(DEV)
    gw, bias = torch.randn(24, 512, generator=g) / 22, torch.randn(24, generator=g) * 0.05
    router = Router(gw, topk=4, B_max=48, bias=bias, score="sigmoid", groups=6, topk_groups=3, group_score="top2",
                    scale=2.0)
    layer = MoeLayer(d["w13"], d["s13"], d["w2"], d["s2"], B_max=48, topk=4, device=DEV)
    w13, w2 = torch.randn(2 * 96, 512, generator=g) / 22, torch.randn(512, 96, generator=g) / 10
    shared = SharedExpertI8.quantize(w13, w2, B_max=48)
    y = MoeBlock(router, layer, shared).forward(x)
    ids, wts = router.forward(x)
    rows = layer.forward(x, ids)
    comb = layer.combine(rows, wts)
    torch.cuda.synchronize()
    logits = router.logits[:B].cpu()
    rid, rw = ref.route(logits.double().numpy(), 4, score="sigmoid", bias=bias.numpy(), groups=6, topk_groups=3,
                        group_score="top2", scale=2.0)
    assert np.array_equal(ids.cpu().numpy(), rid)
    assert np.allclose(wts.cpu().numpy(), rw, rtol=2.0 ** -23)
    q, s = ref.quant(x.cpu().double().numpy())
    h, eh = ref.linear(q, s, shared.w13.cpu().numpy(), shared.s13.cpu().numpy(), act="swiglu")
    hid = shared.hidden[:B].cpu()
    assert np.all(np.abs(hid.double().numpy() - h) <= eh + 2.0 ** -8 * (np.abs(h) + eh))
    q2, s2 = ref.quant(hid.double().numpy())
    out, eo = ref.linear(q2, s2, shared.w2.cpu().numpy(), shared.s2.cpu().numpy(), add=comb.cpu().double().numpy())
    assert np.all(np.abs(y.cpu().double().numpy() - out) <= eo + 2.0 ** -8 * (np.abs(out) + eo))
    # the int8 shared expert stands for the float one: two quantizations of a hundredth each
    f = x.cpu().double() @ w13.double().T
    f = (torch.nn.functional.silu(f[:, :96]) * f[:, 96:]) @ w2.double().T + comb.cpu().double()
    assert (y.cpu().double() - f).norm() <= 0.05 * f.norm()
    # without the shared expert: the combined rows
    assert torch.equal(MoeBlock(router, layer).forward(x), comb)


def test_shared_expert_twice_with_other_batches(m):
    """One object, batches of different sizes in turn: nothing of an earlier call is left."""
    from moe_routed_expert_mx_amd.block import SharedExpertI8
    g = _gen(31)
    sh = SharedExpertI8.quantize(torch.randn(128, 512, generator=g), torch.randn(512, 64, generator=g), B_max=100)
    xs = [torch.randn(b, 512, generator=g).to(BF).to(DEV) for b in (100, 3, 64, 100, 1)]
    first = [sh.forward(x).clone() for x in xs]
    for x, want in list(zip(xs, first))[::-1]:
        assert torch.equal(sh.forward(x), want)
    with pytest.raises(ValueError):
        sh.forward(torch.zeros(101, 512, dtype=BF, device=DEV))


def test_objects_keep_the_gpu_they_were_made_on(m):
    """... by its index, so that a call allocates there whichever GPU is current by then."""
    from moe_routed_expert_mx_amd.block import Router, SharedExpertI8
    here = torch.device("cuda", torch.cuda.current_device())
    router = Router(torch.ones(16, 512), topk=2, B_max=4)
    shared = SharedExpertI8(torch.ones(64, 512, dtype=torch.int8), torch.ones(64), torch.ones(512, 32, dtype=torch.int8),
                            torch.ones(512), B_max=4)
    assert router.device == here and shared.device == here
    x = torch.zeros(4, 512, dtype=BF, device=DEV)
    assert [t.device for t in (*router.forward(x), shared.forward(x))] == [here] * 3


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("B", [3, 40])
def test_block_on_a_side_stream(m, B, raw):
    """The layer on a stream that lags behind: what the current stream allocates and fills right after the call
    must not be what the call still uses."""
    import workloads
    from moe_routed_expert_mx_amd.block import MoeBlock, Router, SharedExpertI8
    from moe_routed_expert_mx_amd.layer import MoeLayer
    log(f"block on a side stream B={B} raw={raw}")
    d = workloads.generate(workloads.custom(B=B, E=24, K=4, D=512, I=64, seed=B + 5))
    g = _gen(B)
    x = torch.from_numpy(d["x"]).view(BF).to(DEV)
    router = Router(torch.randn(24, 512, generator=g) / 22, topk=4, B_max=48)
    layer = MoeLayer(d["w13"], d["s13"], d["w2"], d["s2"], B_max=48, topk=4, device=DEV)
    shared = SharedExpertI8.quantize(torch.randn(2 * 96, 512, generator=g) / 22, torch.randn(512, 96, generator=g) / 10,
                                     B_max=48)
    block = MoeBlock(router, layer, shared)
    calls = [block.forward, shared.forward, lambda x, stream=None: router.forward(x, stream=stream)[1]]
    want = [c(x).clone() for c in calls]
    big = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for call, w in zip(calls, want):
        for _ in range(3):
            with torch.cuda.stream(s):
                for _ in range(8):
                    torch.mm(big, big)
            y = call(x, stream=s.cuda_stream if raw else s)
            junk = []
            for _ in range(4):
                junk += [torch.zeros(B, 4, dtype=torch.int32, device=DEV), torch.zeros(B, 4, device=DEV),
                         torch.zeros(B * 4, 512, dtype=BF, device=DEV), torch.zeros(B, 512, dtype=BF, device=DEV)]
            torch.cuda.current_stream().wait_stream(s)
            got = y.clone()
            torch.cuda.synchronize()
            assert torch.equal(got, w)
            assert not any(j.any() for j in junk)
    y = block.forward(x, stream=torch.cuda.default_stream().cuda_stream if raw else torch.cuda.default_stream())
    torch.cuda.synchronize()
    assert torch.equal(y, want[0])


@pytest.mark.parametrize("B", [3, 40])
def test_block_captured_and_replayed(m, B):
    """The whole layer in a graph, by the current stream and by the capturing stream's name; replays with new inputs
    and eager calls of the same object between them."""
    import workloads
    from moe_routed_expert_mx_amd.block import MoeBlock, Router, SharedExpertI8
    from moe_routed_expert_mx_amd.layer import MoeLayer
    log(f"block captured B={B}")
    d = workloads.generate(workloads.custom(B=B, E=24, K=4, D=512, I=64, seed=B + 9))
    g = _gen(B)
    router = Router(torch.randn(24, 512, generator=g) / 22, topk=4, B_max=48)
    layer = MoeLayer(d["w13"], d["s13"], d["w2"], d["s2"], B_max=48, topk=4, device=DEV)
    shared = SharedExpertI8.quantize(torch.randn(2 * 96, 512, generator=g) / 22, torch.randn(512, 96, generator=g) / 10,
                                     B_max=48)
    block = MoeBlock(router, layer, shared)
    x = torch.randn(B, 512, generator=g).to(BF).to(DEV)
    block.forward(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y1 = block.forward(x)
        y2 = block.forward(x, stream=torch.cuda.current_stream())
    for _ in range(4):
        x.copy_(torch.randn(B, 512, generator=g).to(BF))
        want = block.forward(x)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y1, want) and torch.equal(y2, want)

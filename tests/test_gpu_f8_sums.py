"""How exact the sums of the block-scaled FP8 products are, on the GPU: by inputs whose sums FP32 holds in any order, and
in the 2-norm, beside the worst-case bounds of test_gpu_f8.py; then the layer's parts from end to end."""
import numpy as np
import pytest
import torch

import f8_ref as ref
from helpers import log

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F16, F32, F8, I32 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e4m3fn, torch.int32


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


# In each eight neighbours along k two products of 2^16 that cancel, five of -3 .. 3, and one with k = 7 (0, or 1 in a gate row).
# Sums of a block's products, in any order, are whole numbers of at most 16 (2^16 + 18) < 2^24, and a block's own at most 288:
# FP32 holds every partial sum, so what adds in FP32 returns the sum itself.  Products cut at 2^-13 of the largest of their
# eight, at 8, leave nothing but the two that cancel.
def _cancelling(shape, g, *, weight, gate=0):
    *lead, n, K = shape
    v = torch.randint(-3, 4, shape, generator=g).float() if weight else torch.randint(0, 2, shape, generator=g).float() * 2 - 1
    v[..., 0::8] = 256.0
    v[..., 1::8] = -256.0 if weight else 256.0
    v[..., 7::8] = 0.0 if weight else 1.0
    if gate:                                   # the first rows: K / 8 for every row of a
        v[..., :gate, :] = 0.0
        v[..., :gate, 7::8] = 1.0
    return v


@pytest.mark.parametrize("B", [1, 3, 20, 100, 700])
def test_hidden_of_the_experts_is_exact(m, B):
    """What is quantized again between the products comes from sums in FP32: a code more or less there costs 2^-4 of a value."""
    from moe_routed_expert_mx_amd.block import ExpertsF8
    log(f"hidden of the experts B={B}")
    g = _gen(B)
    E, topk, D, I = 8, 2, 512, 160
    w13, w2 = _cancelling((E, 2 * I, D), g, weight=True, gate=I), torch.randn(E, D, I, generator=g)
    ex = ExpertsF8(w13.to(F8), torch.ones(E, 2 * ref.kb(I), 4), w2.to(F8), torch.ones(E, 4, ref.kb(I)), topk=topk, B_max=B)
    x = _cancelling((B, D), g, weight=False)
    ids = torch.rand(B, E, generator=g).argsort(1)[:, :topk].to(I32)
    ex.forward((x.to(F8).to(DEV), torch.ones(B, 4, device=DEV)), ids.contiguous().to(DEV))
    torch.cuda.synchronize()
    ro, rp = ref.lists(ids.numpy(), E)
    got = _np(ex.hidden[:B * topk])
    for e in range(E):
        i = np.arange(ro[e], ro[e + 1])
        want = D // 8 * (_np(x)[rp[i] // topk] @ _np(w13[e, I:]).T)       # silu(64) = 64 (1 - 2^-92)
        assert np.abs(want).max(initial=0) < 2 ** 16
        assert np.all(np.abs(got[i] - want) <= (2.0 ** -8 + 2.0 ** -15) * np.abs(want)), e


@pytest.mark.parametrize("B", [1, 20, 50, 100, 600, 2100])
def test_hidden_of_the_shared_expert_is_exact(m, B):
    from moe_routed_expert_mx_amd.block import SharedExpertF8
    log(f"hidden of the shared expert B={B}")
    g = _gen(B)
    D, I = 512, 1040
    w13, w2 = _cancelling((2 * I, D), g, weight=True, gate=I), torch.randn(D, I, generator=g)
    shared = SharedExpertF8(w13.to(F8), torch.ones(2 * ref.kb(I), 4), w2.to(F8), torch.ones(4, ref.kb(I)), B_max=B)
    x = _cancelling((B, D), g, weight=False)
    shared.forward((x.to(F8).to(DEV), torch.ones(B, 4, device=DEV)))
    torch.cuda.synchronize()
    want = D // 8 * (_np(x) @ _np(w13[I:]).T)
    assert np.all(np.abs(_np(shared.hidden[:B]) - want) <= (2.0 ** -8 + 2.0 ** -15) * np.abs(want))


EXACT = [(1, 96, 144), (1, 33000, 128), (3, 33000, 272), (9, 300, 1040), (20, 300, 400), (50, 640, 272), (64, 100, 2064), (100, 4096, 144),
         (230, 2048, 400), (800, 9000, 144), (990, 3600, 272), (1990, 4000, 144), (4081, 4070, 144), (700, 20000, 144)]


@pytest.mark.parametrize("M,N,K", EXACT)
def test_exact_linear(m, M, N, K):
    """FP32 outputs, and with `exact` all others, are the sum rounded once, in each form of the product."""
    log(f"exact linear_f8 {M}x{N}x{K}")
    g = _gen(M + N + K)
    a, w = _cancelling((M, K), g, weight=False), _cancelling((N, K), g, weight=True)
    sa, sw = torch.exp2(torch.randint(-3, 4, (M, 1), generator=g).float()).repeat(1, ref.kb(K)), torch.full((ref.kb(N), ref.kb(K)), 0.5)
    want = torch.from_numpy(_np(a) @ _np(w).T * (_np(sa[:, :1]) * 0.5))    # whole numbers of at most 2^13, times a power of two
    args = [t.to(DEV) for t in (a.to(F8), sa, w.to(F8), sw)]
    for dtype in (BF, F16, F32):
        out = torch.empty(M, N, dtype=dtype, device=DEV)
        m.moe_linear_f8(*args, out, exact=dtype != F32)
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want.to(dtype)), dtype


@pytest.mark.parametrize("B,topk,E,N,K", [(1, 4, 16, 64, 272), (1, 16, 160, 3584, 144), (5, 3, 8, 130, 400), (8, 16, 160, 768, 272),
                                          (40, 8, 30, 270, 1168), (50, 16, 160, 272, 400), (300, 2, 30, 1030, 144), (700, 1, 16, 2048, 272),
                                          (1000, 2, 8, 4000, 144)])
def test_exact_grouped(m, B, topk, E, N, K):
    log(f"exact grouped {B}x{topk} of {E}, {N}x{K}")
    g = _gen(B + E + K)
    ids = torch.rand(B, E, generator=g).argsort(1)[:, :topk].to(I32).contiguous()
    a, w = _cancelling((B, K), g, weight=False), _cancelling((E, N, K), g, weight=True)
    o, p = torch.empty(E + 1, dtype=I32, device=DEV), torch.empty(B * topk, dtype=I32, device=DEV)
    m.moe_lists(ids.to(DEV), o, p, ws=torch.empty(m.moe_lists_ws_bytes(B * topk, E), dtype=torch.uint8, device=DEV))
    want = torch.empty(B * topk, N, dtype=torch.float64)
    for e in range(E):
        r = torch.nonzero(ids.flatten() == e).flatten()
        want[r] = a[r // topk].double() @ w[e].double().T
    args = (a.to(F8).to(DEV), torch.ones(B, ref.kb(K), device=DEV), w.to(F8).to(DEV), torch.ones(E, ref.kb(N), ref.kb(K), device=DEV))
    for dtype in (BF, F16, F32):
        out = torch.empty(B * topk, N, dtype=dtype, device=DEV)
        m.moe_grouped_f8(*args, o, out, pairs=p, gather=topk, scatter=True, exact=dtype != F32)
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want.to(dtype)), dtype


@pytest.mark.parametrize("M,N,K", [(1, 4000, 3584), (5, 33000, 512), (20, 700, 1040), (50, 640, 3584), (100, 4096, 384), (990, 3600, 1024),
                                   (1990, 4000, 384), (4081, 4070, 512)])
@pytest.mark.parametrize("exact", [False, True])
def test_error_in_the_2_norm(m, M, N, K, exact):
    """Of up to 60 x 60 outputs, products of random codes.  Rounding: uniform within half a step, which is at most h |y|: h |y| /
    sqrt(3).  Sums in FP32: a block's partial sums are no larger in the mean than its sum, each addition is within two half
    steps of its own: (2 * 128 + blocks + 20) U |y| (f8_ref.linear, with the sum itself in place of the magnitudes').  A product
    cut at 2^-13 of the largest of its eight loses between nothing and that, of either sign: 2^-13 / sqrt(3) of it in the mean,
    and losses add as squares.  1.2 of it all: some 3600 samples scatter by less."""
    log(f"2-norm {M}x{N}x{K} exact={exact}")
    g = _gen(M + N + K + 1)
    a, w = (torch.randn(M, K, generator=g) * 4).to(F8), (torch.randn(N, K, generator=g) * 4).to(F8)
    sa, sw = torch.ones(M, ref.kb(K)), torch.ones(ref.kb(N), ref.kb(K))
    r, c = torch.randint(0, M, (60,), generator=g), torch.randint(0, N, (60 if M > 1 else 600,), generator=g)
    av, wv = _np(a[r[:1] if M == 1 else r].float()), _np(w[c].float())
    y = av @ wv.T
    lost = 0.0
    if not exact:
        top = np.stack([np.max(np.abs(row.reshape(1, K // 8, 8) * wv.reshape(len(wv), K // 8, 8)), axis=2) for row in av])
        lost = np.sqrt(8 * np.sum(np.square(top)) / 3) * 2.0 ** -13
    for dtype, h in ((BF, 2.0 ** -8), (F16, 2.0 ** -11), (F32, 2.0 ** -24)):
        if dtype == F32 and not exact:
            continue
        out = torch.empty(M, N, dtype=dtype, device=DEV)
        m.moe_linear_f8(a.to(DEV), sa.to(DEV), w.to(DEV), sw.to(DEV), out, exact=exact)
        torch.cuda.synchronize()
        got = _np(out)[np.ix_([0] if M == 1 else r.numpy(), c.numpy())]
        norm, err = np.linalg.norm(y), np.linalg.norm(got - y)
        bound = np.sqrt((h * norm) ** 2 / 3 + lost ** 2) + (256 + ref.kb(K) + 20) * ref.U * norm
        log(f"  {dtype}: {err / norm:.2e} of {bound / norm:.2e}")
        assert err <= 1.2 * bound


@pytest.mark.parametrize("B", [1, 8, 200])
@pytest.mark.parametrize("exact", [True, False])
def test_experts_from_end_to_end(m, B, exact):
    """Against the formula in 64 bits.  Rows are rounded to BF16 once: 2^-8 / sqrt(3).  A hidden value's FP32 form is off by 2^-15 of it
    in the mean (two sums of 276 U, or cut), which turns its rounding to BF16 in at most one of 2^6, and in one of eight of these its code:
    by 2^-3 of it at most, together 2^-3 2^-4.5; twice that for few rows, whose error scatters."""
    from moe_routed_expert_mx_amd.block import ExpertsF8, f8_weight_blocks
    log(f"experts from end to end B={B}")
    g = _gen(B + 5)
    E, topk, D, I = 12, 3, 1008, 272
    w13, s13 = f8_weight_blocks(torch.randn(E, 2 * I, D, generator=g) / D ** 0.5, halves=True)
    w2, s2 = f8_weight_blocks(torch.randn(E, D, I, generator=g) / I ** 0.5)
    x, ids = torch.randn(B, D, generator=g).to(BF), torch.rand(B, E, generator=g).argsort(1)[:, :topk].to(I32).contiguous()
    got = _np(ExpertsF8(w13, s13, w2, s2, topk=topk, B_max=B, exact=exact).forward(x.to(DEV), ids.to(DEV)))
    q, s = ref.quant(_np(x))
    want = np.empty((B * topk, D))
    for r, e in enumerate(ids.flatten().tolist()):
        t = slice(r // topk, r // topk + 1)
        h, _ = ref.linear(q[t], s[t], _np(w13[e].float()), _np(s13[e]), act="swiglu")
        hq, hs = ref.quant(torch.from_numpy(h).to(BF).double().numpy())
        want[r] = ref.linear(hq, hs, _np(w2[e].float()), _np(s2[e]))[0]
    err = np.linalg.norm(got - want) / np.linalg.norm(want)
    log(f"  {err:.2e}")
    assert err <= 2.0 ** -8 / 3 ** 0.5 + 2 * 2.0 ** -7.5

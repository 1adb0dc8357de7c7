"""The block-scaled FP8 layer's parts on the GPU, beside test_gpu_f8.py: streams, long lists, the shared expert's numbers."""
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


def _experts(g, E=12, topk=3, D=320, I=144, B_max=300):
    from moe_routed_expert_mx_amd.block import ExpertsF8, f8_weight_blocks
    w13, s13 = f8_weight_blocks(torch.randn(E, 2 * I, D, generator=g) / D ** 0.5, halves=True)
    w2, s2 = f8_weight_blocks(torch.randn(E, D, I, generator=g) / I ** 0.5)
    return ExpertsF8(w13, s13, w2, s2, topk=topk, B_max=B_max)


def _ids(B, topk, E, g):
    return torch.rand(B, E, generator=g).argsort(1)[:, :topk].to(I32).contiguous()


@pytest.mark.parametrize("raw", [False, True])
def test_combine_on_a_side_stream(m, raw):
    """On a stream that lags behind: the rows it waits for, and no buffer that the current stream allocates meanwhile."""
    log(f"combine on a side stream raw={raw}")
    g = _gen(31)
    ex = _experts(g, D=512)
    x, ids, w = torch.randn(40, 512, generator=g).to(BF).to(DEV), _ids(40, 3, 12, g).to(DEV), torch.rand(40, 3, generator=g).to(DEV)
    want = ex.combine(ex.forward(x, ids), w).clone()
    rows, big = torch.zeros(120, 512, dtype=BF, device=DEV), torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(8):
            torch.mm(big, big)
    ex.forward(x, ids, rows, stream=s)
    y = ex.combine(rows, w, stream=s.cuda_stream if raw else s)
    junk = [torch.zeros(40, 512, dtype=BF, device=DEV) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(s)
    got = y.clone()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and not any(j.any() for j in junk)


def _rows_from_end_to_end(ex, weights, x, ids, routes):
    """The formula in 64 bits for some routes (float64)."""
    w13, s13, w2, s2 = weights
    want = np.empty((len(routes), ex.D))
    for i, r in enumerate(routes):
        e = int(ids.flatten()[r])
        q, s = ref.quant(_np(x[r // ex.topk:r // ex.topk + 1]))
        h, _ = ref.linear(q, s, _np(w13[e].float()), _np(s13[e]), act="swiglu")
        hq, hs = ref.quant(torch.from_numpy(h).to(BF).double().numpy())
        want[i] = ref.linear(hq, hs, _np(w2[e].float()), _np(s2[e]))[0]
    return want


def test_more_routes_than_one_quantization_takes(m):
    """2^22 and some routes: the hidden is quantized in parts.  Bound: test_gpu_f8_sums.py, from end to end."""
    from moe_routed_expert_mx_amd.block import ExpertsF8, f8_weight_blocks
    B, D, I, E, topk = (1 << 21) + 37, 16, 32, 3, 2
    log(f"{B * topk} routes")
    g = _gen(5)
    weights = (*f8_weight_blocks(torch.randn(E, 2 * I, D, generator=g) / 4, halves=True), *f8_weight_blocks(torch.randn(E, D, I, generator=g) / 5))
    ex = ExpertsF8(*weights, topk=topk, B_max=B)
    x, ids = torch.randn(B, D, generator=g).to(BF), torch.randint(0, E, (B, topk), generator=g, dtype=I32)
    got = ex.forward(x.to(DEV), ids.to(DEV))
    torch.cuda.synchronize()
    routes = np.r_[0:20, (1 << 22) - 20:(1 << 22) + 20, B * topk - 20:B * topk, torch.randint(0, B * topk, (40,), generator=g).numpy()]
    got, want = _np(got[torch.from_numpy(routes).to(DEV)]), _rows_from_end_to_end(ex, weights, x, ids, routes)
    assert np.linalg.norm(got - want) <= (2.0 ** -8 / 3 ** 0.5 + 2 * 2.0 ** -7.5) * np.linalg.norm(want)


@pytest.mark.parametrize("B,K,E", [(200003, 16, 256), ((1 << 21) + 129, 1, 1000), (300001, 8, 1)])
@pytest.mark.parametrize("kind", ["skewed", "foreign"])
def test_lists_longer_than_a_waves_registers(m, B, K, E, kind):
    """Beyond 2^21 routes a wave's share does not stay in registers: shares of 832, 576 and 640 routes."""
    log(f"lists {B}x{K} of {E} {kind}")
    g = _gen(B)
    R = B * K
    ids = torch.randint(0, E, (B, K), generator=g, dtype=I32) if kind == "skewed" else \
        torch.randint(-E, 2 * E, (B, K), generator=g, dtype=I32)
    if kind == "skewed":
        ids = torch.where(torch.rand(B, K, generator=g) < 0.9, torch.full_like(ids, E // 2), ids)
    offsets, pairs = torch.full((E + 2,), -9, dtype=I32, device=DEV), torch.full((R + 1,), -9, dtype=I32, device=DEV)
    ws = torch.full((m.moe_lists_ws_bytes(R, E),), 0x5a, dtype=torch.uint8, device=DEV)
    m.moe_lists(ids.to(DEV), offsets[:E + 1], pairs[:R], ws=ws)
    torch.cuda.synchronize()
    flat = ids.flatten().numpy().astype(np.int64)
    flat = np.where((flat >= 0) & (flat < E), flat, E)
    order, counts = np.argsort(flat, kind="stable"), np.bincount(flat, minlength=E + 1)
    want = np.where(np.arange(R) < R - counts[E], order, -1)
    assert offsets[E + 1] == -9 and pairs[R] == -9
    assert np.array_equal(offsets[:E + 1].cpu().numpy(), np.r_[0, np.cumsum(counts[:E])])
    assert np.array_equal(pairs[:R].cpu().numpy(), want)


@pytest.mark.parametrize("B", [1, 13, 70, 520])
@pytest.mark.parametrize("how", ["rows", "codes", "add", "add in place"])
def test_shared_expert_against_the_plain_form(m, B, how):
    """SharedExpertF8 stage by stage on the values that the GPU handed on."""
    from moe_routed_expert_mx_amd.block import SharedExpertF8, f8_weight_blocks
    log(f"shared expert B={B} {how}")
    g = _gen(B)
    D, I = 400, 272
    w13, s13 = f8_weight_blocks(torch.randn(2 * I, D, generator=g) / 20, halves=True)
    w2, s2 = f8_weight_blocks(torch.randn(D, I, generator=g) / 16)
    shared = SharedExpertF8(w13, s13, w2, s2, B_max=600)
    x, add = torch.randn(B, D, generator=g).to(BF), torch.randn(B, D, generator=g).to(BF)
    q, s = ref.quant(_np(x))
    given = (torch.from_numpy(q).float().to(F8).to(DEV), torch.from_numpy(s).float().to(DEV)) if how == "codes" else x.to(DEV)
    d = add.to(DEV)
    out = shared.forward(given, add=d if "add" in how else None, out=d if how == "add in place" else None)
    torch.cuda.synchronize()
    assert how != "add in place" or out is d
    y, e = ref.linear(q, s, _np(w13.float()), _np(s13), act="swiglu", cut=False)
    hidden = _np(shared.hidden[:B])
    assert np.all(np.abs(hidden - y) <= e + 2.0 ** -8 * (np.abs(y) + e) * 1.001 + 2.0 ** -134)
    hq, hs = ref.quant(hidden)
    y, e = ref.linear(hq, hs, _np(w2.float()), _np(s2), add=_np(add) if "add" in how else None)
    assert np.all(np.abs(_np(out) - y) <= e + 2.0 ** -8 * (np.abs(y) + e) * 1.001 + 2.0 ** -134)


def test_a_ranks_part_of_the_layer(m):
    """Ids of another rank from experts to the combined output, on memory that held NaN: the parts of two ranks add up."""
    log("two ranks' parts")
    from moe_routed_expert_mx_amd.block import ExpertsF8
    g = _gen(41)
    B, E, topk, D, I = 70, 12, 3, 320, 144
    whole = _experts(g, E, topk, D, I)
    halves = [ExpertsF8(*(t[h * 6:h * 6 + 6] for t in (whole.w13, whole.s13, whole.w2, whole.s2)), topk=topk, B_max=300) for h in range(2)]
    x, ids, w = torch.randn(B, D, generator=g).to(BF).to(DEV), _ids(B, topk, E, g).to(DEV), torch.rand(B, topk, generator=g).to(DEV)
    rows = whole.forward(x, ids)
    parts, sums, left = [], 0.0, rows.clone()
    for h, ex in enumerate(halves):
        junk = torch.full((B * topk, D), float("nan"), dtype=BF, device=DEV)
        torch.cuda.synchronize()
        del junk                                        # the next buffer of its size
        part = ex.forward(x, ids - 6 * h)
        here = ((ids // 6) == h).flatten()
        assert (part[~here] == 0).all()
        left[here] -= part[here]
        parts.append(ex.combine(part, w))
        sums = sums + _np(part)
    # the same rows as the whole layer's, though by another form of the products: twice the bound of one (test_gpu_f8_sums.py)
    assert left.float().norm() <= 2 * (2.0 ** -8 / 3 ** 0.5 + 2 * 2.0 ** -7.5) * rows.float().norm()
    got, want = _np(parts[0]) + _np(parts[1]), np.einsum("bkd,bk->bd", sums.reshape(B, topk, D), _np(w))
    # each part is rounded to BF16 once; a bound by magnitudes for both
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * 1.01 * np.einsum("bkd,bk->bd", np.abs(sums).reshape(B, topk, D), _np(w)))


def test_objects_on_the_default_stream_by_its_handle(m):
    """stream=0 from another current stream: behind what the default stream, which lags, still has to do."""
    log("objects on stream 0")
    from moe_routed_expert_mx_amd.block import MoeBlock, Norm, Router, SharedExpertI8
    g = _gen(51)
    B, D, E, topk = 40, 512, 12, 3
    ex, router = _experts(g, E, topk, D), Router(torch.randn(E, D, generator=g) / 22, topk=topk, B_max=B)
    shared = SharedExpertI8.quantize(torch.randn(128, D, generator=g), torch.randn(D, 64, generator=g), B_max=B)
    block = MoeBlock(router, ex, shared, Norm(torch.ones(D)))
    x = torch.randn(B, D, generator=g).to(BF).to(DEV)
    ids, w = router.forward(x)
    rows = ex.forward(x, ids)
    calls = [lambda x, **k: router.forward(x, **k)[1], shared.forward, block.norm.forward, lambda x, **k: ex.forward(x, ids, **k), block.forward,
             lambda x, **k: ex.combine(ex.forward(x, ids, **k), w, **k)]
    want = [c(x).clone() for c in calls]
    default, side, big = torch.cuda.default_stream(), torch.cuda.Stream(), torch.randn(4096, 4096, device=DEV)
    assert default.cuda_stream == 0
    late = [torch.zeros_like(x) for _ in calls]
    torch.cuda.synchronize()
    for call, v, t in zip(calls, want, late):
        with torch.cuda.stream(default):
            for _ in range(8):
                torch.mm(big, big)
            t.copy_(x)
        with torch.cuda.stream(side):
            y = call(t, stream=0)
            side.wait_stream(default)
            got = y.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, v)
    assert rows.shape == (B * topk, D)

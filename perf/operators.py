"""The dense side of a routed-experts layer: what stands in front of and beside the experts.

Operators, each in a plain form (elementary torch operations) and as the framework's call:

  route    logits [B, E] -> the top-k expert ids and their weights (softmax or sigmoid
           scores, a balance bias, groups, renormalised weights)
  gate     x BF16 [B, D] times the router's weight [E, D] (BF16 or FP32) -> FP32 logits
  quant    x [M, K] -> int8 codes and one FP32 scale for each token
  linear   int8 product with scales for each token and channel, with SwiGLU, a channel
           bias and an added row in its epilogue (the shared expert's two products)

Definitions.
  route:  a NaN logit is read as -inf; an expert at -inf is masked and has score 0.
          softmax: m = the row's largest logit, e = exp(l - m) (1 where l = m), score = e / sum e.
          sigmoid: score = 1 / (1 + exp(-l)).
          choice = score + bias; without a bias the logit itself, since the score grows with it;
          -inf for masked experts and NaN.  Groups of E / groups consecutive experts are ranked
          by their largest choice ("max") or by the sum of their two largest choice values
          ("top2": scores where there is no bias; masked experts add nothing, a group of masked
          experts ranks last), and the first topk_groups stay.  The topk experts of the largest
          choice in them, in that order; ties go to the lowest index, of groups too.
          weight = score (renorm: / the sum of the selected scores, 0 where that is 0) * scale.
  quant:  scale = amax / 127 in FP32; code = x * 127 / amax, half to even; a row of zeros has
          scale 0 and codes 0.
  linear: y = (a . w) * a_scale * w_scale + bias, the product exact;
          swiglu: y = silu(y[:, :N/2]) * y[:, N/2:]; then + add; rounded once.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------------- cases
def _route(B, E, K, dtype, score, bias, groups=0, kept=0, group_score="max", renorm=True, scale=1.0):
    return {"op": "route", "B": B, "E": E, "K": K, "dtype": dtype, "score": score, "bias": bias, "groups": groups,
            "kept": kept, "group_score": group_score, "renorm": renorm, "scale": scale}


def _gate(B, D, E, wtype):
    return {"op": "gate", "B": B, "D": D, "E": E, "wtype": wtype}


def _quant(M, K, dtype):
    return {"op": "quant", "M": M, "K": K, "dtype": dtype}


def _linear(M, N, K, out, act="none", bias=False, add=False):
    return {"op": "linear", "M": M, "N": N, "K": K, "out": out, "act": act, "bias": bias, "add": add}


def listed():
    return [
        # one token's routing in a decode step: nothing but latency
        {"name": "route_b1", **_route(1, 160, 16, "f32", "sigmoid", True)},
        # a decode batch behind a router that keeps its logits in BF16
        {"name": "route_b256", **_route(256, 160, 16, "bf16", "softmax", False)},
        # a prompt's tokens with a balance bias and a choice of groups
        {"name": "route_prompt", **_route(16384, 160, 16, "f32", "sigmoid", True, 10, 5, "top2", True, 2.5)},
        # the router's product of a small decode batch
        {"name": "gate_b8", **_gate(8, 3584, 160, "bf16")},
        # the router's product of a prompt, its weight kept in FP32
        {"name": "gate_prompt", **_gate(8192, 3584, 160, "f32")},
        # the tokens of a decode batch before the shared expert's first product
        {"name": "quant_b8", **_quant(8, 3584, "bf16")},
        # the tokens of a prompt before it
        {"name": "quant_prompt", **_quant(8192, 3584, "bf16")},
        # the shared expert's first product for one token (gate and up rows, SwiGLU)
        {"name": "linear_b1_up", **_linear(1, 768, 3584, "bf16", "swiglu")},
        # its second product for eight tokens, added to the routed experts' rows
        {"name": "linear_b8_down", **_linear(8, 3584, 384, "bf16", add=True)},
        # a wide projection in a decode batch: the weight's bytes bound it
        {"name": "linear_b64", **_linear(64, 8192, 3584, "bf16")},
        # a piece of a prompt, ragged in its rows, with a channel bias
        {"name": "linear_chunk", **_linear(1000, 3584, 4096, "f16", bias=True)},
        # an unsharded first product over a prompt: the matrix cores bound it
        {"name": "linear_prompt_up", **_linear(8192, 7168, 3584, "bf16", "swiglu")},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "gate", "quant", "linear", "linear"])
    if op == "route":
        B = _spread(rng, 1, 16384)
        groups = rng.choice([0, 0, rng.randint(2, 12)])
        E = groups * rng.randint(4, 24) if groups else rng.randint(8, 256)
        kept = rng.randint(1, groups) if groups else 0
        K = rng.randint(1, min(16, kept * (E // groups) if groups else E))
        return _route(B, E, K, rng.choice(["f32", "bf16", "f16"]), rng.choice(["softmax", "sigmoid"]),
                      rng.random() < 0.5, groups, kept, rng.choice(["max", "top2"]) if groups else "max",
                      rng.random() < 0.7, rng.choice([1.0, 2.5]))
    if op == "gate":
        D = 512 * rng.randint(1, 10)
        E = rng.randint(8, 256)
        B = _spread(rng, 1, max(1, min(8192, 8192 * 3584 * 160 // (D * E))))
        return _gate(B, D, E, rng.choice(["bf16", "f32"]))
    if op == "quant":
        K = _spread(rng, 16, 8192)
        return _quant(_spread(rng, 1, min(8192, 8192 * 3584 // K)), K, rng.choice(["bf16", "f16", "f32"]))
    K = _spread(rng, 16, 8192)
    if rng.random() < 0.6:
        K = (K + 15) // 16 * 16
    N = 2 * _spread(rng, 8, 4096)
    M = _spread(rng, 1, max(1, min(8192, 8192 * 7168 * 3584 // (N * K))))
    return _linear(M, N, K, rng.choice(["bf16", "f16", "f32"]), rng.choice(["none", "swiglu"]), rng.random() < 0.5,
                   rng.random() < 0.5)


def work(case):
    c = case
    if c["op"] == "route":
        return {"bytes": c["B"] * (c["E"] * SIZES[c["dtype"]] + 8 * c["K"]) + (4 * c["E"] if c["bias"] else 0),
                "flops": 10 * c["B"] * c["E"]}
    if c["op"] == "gate":
        return {"bytes": 2 * c["B"] * c["D"] + c["E"] * c["D"] * SIZES[c["wtype"]] + 4 * c["B"] * c["E"],
                "flops": 2 * c["B"] * c["D"] * c["E"]}
    if c["op"] == "quant":
        return {"bytes": c["M"] * (c["K"] * (SIZES[c["dtype"]] + 1) + 4), "flops": 3 * c["M"] * c["K"]}
    M, N, K, s = c["M"], c["N"], c["K"], SIZES[c["out"]]
    No = N // 2 if c["act"] == "swiglu" else N
    return {"bytes": (M + N) * (K + 4) + M * No * s * (2 if c["add"] else 1) + (4 * N if c["bias"] else 0),
            "flops": 2 * M * N * K}


# ------------------------------------------------------------------------ inputs
def _codes(shape, g):
    """int8 codes as symmetric quantization of normal values leaves them."""
    return (torch.randn(shape, generator=g, device="cuda") * 36).round_().clamp_(-127, 127).to(torch.int8)


def prepare(case, seed):
    c = case
    g = torch.Generator("cuda").manual_seed(seed)
    s = {"case": c}

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if c["op"] == "route":
        B, E, K = c["B"], c["E"], c["K"]
        s["logits"] = (randn(B, E) * 1.5 + randn(1, E) * 0.5).to(DTYPES[c["dtype"]])
        s["bias"] = randn(E) * 0.05 if c["bias"] else None
        s["ids"] = torch.empty(B, K, dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty(B, K, device="cuda")
    elif c["op"] == "gate":
        B, D, E = c["B"], c["D"], c["E"]
        s["x"] = randn(B, D).to(torch.bfloat16)
        s["w"] = (randn(E, D) / math.sqrt(D)).to(DTYPES[c["wtype"]])
        s["logits"] = torch.empty(B, E, device="cuda")
        if own:
            import moe_routed_expert_mx_amd as moe
            s["packed"] = torch.empty(moe.moe_gate_packed_bytes(E, D, s["w"].dtype), dtype=torch.uint8, device="cuda")
            s["gate"] = moe.moe_gate_pack(s["w"], s["packed"])
    elif c["op"] == "quant":
        M, K = c["M"], c["K"]
        channel = 1 + 15 * (torch.rand(K, generator=g, device="cuda") < 0.01)     # a few channels stand out
        s["x"] = (randn(M, K) * channel).to(DTYPES[c["dtype"]])
        s["codes"] = torch.empty(M, K, dtype=torch.int8, device="cuda")
        s["scales"] = torch.empty(M, device="cuda")
    else:
        M, N, K = c["M"], c["N"], c["K"]
        No = N // 2 if c["act"] == "swiglu" else N
        s["a"], s["w"] = _codes((M, K), g), _codes((N, K), g)
        s["a_scales"] = (0.5 + torch.rand(M, generator=g, device="cuda")) * 0.03
        s["w_scales"] = (0.5 + torch.rand(N, generator=g, device="cuda")) * (0.03 / math.sqrt(K))
        s["bias"] = randn(N) * 0.1 if c["bias"] else None
        s["add"] = randn(M, No).to(DTYPES[c["out"]]) if c["add"] else None
        s["out"] = torch.empty(M, No, dtype=DTYPES[c["out"]], device="cuda")
    return s


# -------------------------------------------------------------------- plain forms
def _plain_route(s):
    c = s["case"]
    B, E, K = c["B"], c["E"], c["K"]
    logit = s["logits"].double()                  # 64 bits: a choice next to another one decides ids
    logit = torch.where(logit.isnan(), -math.inf, logit)
    masked = logit == -math.inf
    if c["score"] == "softmax":
        m = logit.amax(1, keepdim=True)
        e = torch.where(logit == m, 1.0, torch.exp(logit - m)).masked_fill(masked, 0.0)
        score = e / e.sum(1, keepdim=True).clamp_min(1.0)
    else:
        score = (1 / (1 + torch.exp(-logit))).masked_fill(masked, 0.0)
    choice = logit if s["bias"] is None else score + s["bias"].double()
    choice = torch.where(masked | choice.isnan(), -math.inf, choice)
    if c["groups"]:
        G, size = c["groups"], E // c["groups"]
        if c["group_score"] == "max":
            rank = choice.view(B, G, size).amax(2)
        else:
            v = torch.where(choice == -math.inf, -math.inf, score) if s["bias"] is None else choice
            two = v.view(B, G, size).sort(dim=2, descending=True).values[:, :, :2]
            rank = torch.where(two == -math.inf, 0.0, two).sum(2).masked_fill(two[:, :, 0] == -math.inf, -math.inf)
        kept = rank.sort(dim=1, descending=True, stable=True).indices[:, :c["kept"]].sort(dim=1).values
        ids = (kept[:, :, None] * size + torch.arange(size, device="cuda")).view(B, -1)
        order = choice.gather(1, ids).sort(dim=1, descending=True, stable=True).indices[:, :K]
        ids = ids.gather(1, order)
    else:
        ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :K]
    w = score.gather(1, ids)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return {"ids": ids.to(torch.int32), "weights": (w * c["scale"]).float()}


def _plain_gate(s):
    return s["x"].float() @ s["w"].float().T


def _plain_quant(s):
    x = s["x"].float()
    amax = x.abs().amax(1)
    # 64 bits: a code next to a half
    q = (x.double() * 127 / amax.double().clamp_min(1e-300)[:, None]).round()
    return {"codes": q.to(torch.int8), "scales": (amax.double() / 127).float()}


def _plain_linear(s):
    c = s["case"]
    acc = 0
    for k in range(0, c["K"], 1024):              # exact in 32 bits: 1024 * 128 * 128 = 2^24
        acc = acc + (s["a"][:, k:k + 1024].float() @ s["w"][:, k:k + 1024].float().T)
    y = acc * s["a_scales"][:, None] * s["w_scales"]
    if s["bias"] is not None:
        y = y + s["bias"]
    if c["act"] == "swiglu":
        gate, up = y.chunk(2, dim=1)
        y = gate / (1 + torch.exp(-gate)) * up
    if s["add"] is not None:
        y = y + s["add"].float()
    return y.to(DTYPES[c["out"]])


# --------------------------------------------------------------------- one pass
def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"route": _plain_route, "gate": _plain_gate, "quant": _plain_quant, "linear": _plain_linear}[c["op"]](s)
    import moe_routed_expert_mx_amd as moe
    if c["op"] == "route":
        moe.moe_route(s["logits"], s["ids"], s["weights"], score=c["score"], bias=s["bias"], groups=c["groups"],
                      topk_groups=c["kept"], group_score=c["group_score"], renorm=c["renorm"], scale=c["scale"])
        return {"ids": s["ids"], "weights": s["weights"]}
    if c["op"] == "gate":
        moe.moe_gate(s["gate"], s["x"], s["logits"])
        return s["logits"]
    if c["op"] == "quant":
        moe.moe_quant_i8(s["x"], s["codes"], s["scales"])
        return {"codes": s["codes"], "scales": s["scales"]}
    moe.moe_linear_i8(s["a"], s["a_scales"], s["w"], s["w_scales"], s["out"], act=c["act"], bias=s["bias"],
                      add=s["add"])
    return s["out"]


# ---------------------------------------------------- the definitions in 64 bits
def _exact_route(c, s):
    import numpy as np
    logit = s["logits"].double().cpu().numpy()
    logit[np.isnan(logit)] = -np.inf
    open_ = logit > -np.inf
    with np.errstate(all="ignore"):
        if c["score"] == "softmax":
            top = logit.max(axis=1, keepdims=True)
            score = np.where(open_, np.exp(np.where(logit == top, 0.0, logit - top)), 0.0)
            score /= np.maximum(score.sum(axis=1, keepdims=True), 1.0)
        else:
            score = np.where(open_, 1.0 / (1.0 + np.exp(-logit)), 0.0)
    choice = logit.copy()
    if s["bias"] is not None:
        choice = score + s["bias"].double().cpu().numpy()
        choice[~open_ | np.isnan(choice)] = -np.inf
    allowed = np.ones_like(open_)
    if c["groups"]:
        size = c["E"] // c["groups"]
        if c["group_score"] == "max":
            rank = choice.reshape(c["B"], c["groups"], size).max(axis=2)
        else:
            v = choice if s["bias"] is not None else np.where(open_, score, -np.inf)
            v = np.sort(v.reshape(c["B"], c["groups"], size), axis=2)[:, :, ::-1][:, :, :2]
            rank = np.where(v[:, :, 0] > -np.inf, np.where(v > -np.inf, v, 0.0).sum(axis=2), -np.inf)
        best = np.argsort(-rank, axis=1, kind="stable")[:, :c["kept"]]
        chosen = np.zeros((c["B"], c["groups"]), bool)
        np.put_along_axis(chosen, best, True, axis=1)
        allowed = np.repeat(chosen, size, axis=1)
    order = np.lexsort((np.broadcast_to(np.arange(c["E"]), choice.shape), -choice, ~allowed), axis=1)
    ids = order[:, :c["K"]]
    w = np.take_along_axis(score, ids, axis=1)
    if c["renorm"]:
        total = w.sum(axis=1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    return {"ids": torch.from_numpy(ids.astype(np.int32)), "weights": torch.from_numpy(w * c["scale"])}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "route":
        return _exact_route(c, s)
    if c["op"] == "gate":
        return torch.mm(s["w"].double(), s["x"].double().t()).t()
    if c["op"] == "quant":
        x = s["x"].double()
        amax = x.abs().max(dim=1).values
        code = torch.zeros_like(x)
        rows = amax > 0
        code[rows] = torch.round(x[rows] * 127.0 / amax[rows].unsqueeze(1))
        return {"codes": code.to(torch.int8), "scales": amax / 127.0}
    y = torch.mm(s["w"].double(), s["a"].double().t())          # [N, M], whole numbers below 2^53
    y = y * s["w_scales"].double().unsqueeze(1) * s["a_scales"].double()
    if s["bias"] is not None:
        y += s["bias"].double().unsqueeze(1)
    if c["act"] == "swiglu":
        half = c["N"] // 2
        y = y[:half] * torch.sigmoid(y[:half]) * y[half:]
    y = y.t().contiguous()
    return y if s["add"] is None else y + s["add"].double()

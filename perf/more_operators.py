"""Measured cases of the expert router and of the experts' products in 8-bit floating point.

Three operators, the ones a layer of many experts needs around its products when its weights are
held in 8 bits:

  router   softmax or sigmoid scores of the logits, a balance bias that moves the choice alone,
           groups of experts, the top k of the best groups, renormalised weights; its backward
  quant    rows, or SwiGLU of a row's halves, to E4M3 codes with a scale for each 128 of a row;
           weights with a scale for each 128 x 128 block, as stored and transposed
  product  out[r] = sum over blocks b of 128: x_scale[r, b] * w_scale[e, n / 128, b] * <x[r, b],
           w[e, n, b]> for the rows r of every expert e

``own`` False computes each operator with elementary torch operations, in fp32 (the router's scores
in fp64: close ones decide which expert is chosen), rounded once at the end; ``own`` True makes
the library's calls on the same inputs.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
BLOCK = 128


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token at the decode configuration's experts: pure latency
        dict(name="router_token", op="router", dir="fwd", T=1, E=128, k=8, score="softmax",
             bias=False, groups=1, topk_groups=1, group_top=1, renorm=True, scale=1.0, io="f32"),
        # the skewed workload's batch and experts with sigmoid scores, a balance bias and groups
        dict(name="router_groups", op="router", dir="fwd", T=8192, E=256, k=8, score="sigmoid",
             bias=True, groups=8, topk_groups=4, group_top=2, renorm=True, scale=2.5, io="f32"),
        # a training batch's backward of the full softmax's probabilities, bf16 logits
        dict(name="router_bwd", op="router", dir="bwd", T=8192, E=256, k=8, score="softmax",
             bias=False, groups=1, topk_groups=1, group_top=1, renorm=False, scale=1.0, io="bf16"),
        # a decode batch's activations
        dict(name="quant_token", op="quant", kind="rows", T=32, H=2048, io="bf16", clamp=0.0,
             interleave=0),
        # the skewed workload's activations before its first product
        dict(name="quant_rows", op="quant", kind="rows", T=8192, H=7168, io="bf16", clamp=0.0,
             interleave=0),
        # the Mixtral-shaped batch's pre-activations (top 2) before its second product
        dict(name="quant_swiglu", op="quant", kind="swiglu", T=8192, H=14336, io="bf16", clamp=0.0,
             interleave=0),
        # the second projection of the Mixtral-shaped experts, for the product and its gradient
        dict(name="quant_weights", op="quant", kind="weights", E=8, N=4096, K=14336, io="bf16",
             transposed=True),
        # one decoded token's first product at the decode configuration: eight experts' weights
        dict(name="product_token", op="product", M=8, E=128, N=1536, K=2048, out="bf16", skew=0.0,
             mix=1),
        # a decode batch's second product (T = 32): nearly every expert's weights, few rows each
        dict(name="product_batch", op="product", M=256, E=128, N=2048, K=768, out="bf16", skew=0.0,
             mix=2),
        # a ragged run: an odd width, a length of K that ends inside a block, fp32 out
        dict(name="product_odd", op="product", M=777, E=5, N=1001, K=1040, out="f32", skew=0.5,
             mix=3),
        # the skewed workload's first product: 256 experts of very different popularity
        dict(name="product_skewed", op="product", M=65536, E=256, N=4096, K=7168, out="bf16",
             skew=1.1, mix=4),
        # the Mixtral-shaped batch's first product: many rows for each of few experts
        dict(name="product_prompt", op="product", M=8192, E=8, N=28672, K=4096, out="bf16",
             skew=0.0, mix=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Multiples of 16, half of them of 128."""
    H = _log(rng, lo, hi)
    return max(lo, H // 128 * 128 if rng.random() < 0.5 else H // 16 * 16)


def draw(rng):
    op = rng.choice(["router", "router", "rows", "swiglu", "weights", "product", "product"])
    if op == "router":
        E = _log(rng, 4, 512)
        E = E // 8 * 8 if E >= 16 and rng.random() < 0.6 else E
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0 and E // g >= 2])
        topk_groups = rng.randint((groups + 1) // 2, groups)
        direction, renorm = rng.choice(["fwd", "fwd", "bwd"]), rng.random() < 0.6
        least = 2 if direction == "bwd" and renorm else 1  # one renormalised weight has no gradient
        return dict(op="router", dir=direction, T=_log(rng, 1, 16384), E=E,
                    k=rng.randint(least, min(10, topk_groups * (E // groups))),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5,
                    groups=groups, topk_groups=topk_groups, group_top=rng.choice([1, 2]),
                    renorm=renorm, scale=rng.choice([1.0, 2.5]), io=rng.choice(["bf16", "f32"]))
    if op in ("rows", "swiglu"):
        H = _width(rng, 64, 14336)
        return dict(op="quant", kind=op, T=min(_log(rng, 1, 16384), 8192 * 14336 // H), H=H,
                    io=rng.choice(["bf16", "f32"]) if op == "rows" else "bf16",
                    clamp=rng.choice([0.0, 7.0]) if op == "swiglu" else 0.0,
                    interleave=rng.choice([0, 32]) if op == "swiglu" and H % 32 == 0 else 0)
    if op == "weights":
        N, K = _width(rng, 64, 8192), _width(rng, 64, 8192)
        return dict(op="quant", kind="weights", E=min(rng.choice([1, 2, 8]), 8 * 4096 * 14336 // (N * K)),
                    N=N, K=K, io=rng.choice(["bf16", "f32"]), transposed=rng.random() < 0.5)
    N, K = _log(rng, 64, 8192), _width(rng, 128, 8192)
    E = min(_log(rng, 1, 128), (1 << 31) // (N * K))
    return dict(op="product", M=min(_log(rng, 1, 16384), 8192 * 28672 * 4096 // (N * K)), E=E, N=N, K=K,
                out=rng.choice(["bf16", "bf16", "f32"]), skew=rng.choice([0.0, 0.5, 1.1]),
                mix=rng.randint(1, 1 << 20))


# ------------------------------------------------------------------ inputs
def _counts(case):
    """Rows of every expert: popularity by rank ** -skew over shuffled experts."""
    r = random.Random(case["mix"])
    rank = list(range(1, case["E"] + 1))
    r.shuffle(rank)
    counts = [0] * case["E"]
    for e in r.choices(range(case["E"]), [i ** -case["skew"] for i in rank], k=case["M"]):
        counts[e] += 1
    return counts


def _blocks(n):
    return -(-n // BLOCK)


def _inputs(case, seed):
    """Every tensor of a case, from the seed alone (the library is not touched here)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def randn(*shape, dtype=torch.float32, std=1.0, mean=0.0):
        t = torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)
        return t.mul_(std).add_(mean).to(dtype)

    def scales(*shape, std):  # as absolute maxima of blocks of normal values spread
        return randn(*shape, std=0.2).exp_().mul_(std * 3.5 / E4M3_MAX)

    def codes(*shape):
        return randn(*shape, std=E4M3_MAX / 3.5).clamp_(-E4M3_MAX, E4M3_MAX).to(E4M3)

    s = {}
    if case["op"] == "router":
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = randn(T, E, dtype=DT[case["io"]], std=1.5)
        s["bias"] = randn(E, std=0.05) if case["bias"] else None
        if case["dir"] == "bwd":
            s["idx"] = _choose(case, s["logits"].double(), s["bias"])[1].to(torch.int32)
            s["d_w"] = randn(T, k)
    elif case["op"] == "quant" and case["kind"] == "weights":
        E, N, K = case["E"], case["N"], case["K"]
        s["src"] = torch.empty(E, N, K, dtype=DT[case["io"]], device=DEV)
        for e in range(E):
            s["src"][e] = randn(N, K, std=K ** -0.5)
    elif case["op"] == "quant":
        T, H = case["T"], case["H"] * (2 if case["kind"] == "swiglu" else 1)
        s["src"] = randn(T, H, dtype=DT[case["io"]], std=1.3)
        s["src"] *= randn(T, 1, std=0.5).exp_().to(s["src"].dtype)  # rows of different size
    else:
        M, N, K, E = (case[i] for i in "MNKE")
        s["x"], s["xs"] = codes(M, K), scales(M, _blocks(K), std=1.0)
        s["w"] = torch.empty(E, N, K, dtype=E4M3, device=DEV)
        for e in range(E):
            s["w"][e] = codes(N, K)
        s["ws"] = scales(E, _blocks(N), _blocks(K), std=K ** -0.5)
        s["counts"] = _counts(case)
        s["offsets"] = torch.tensor([0] + s["counts"]).cumsum(0).to(DEV, torch.int32)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if not own:
        return s
    import mixture_experts_ffn_permute_gb300 as moe
    if case["op"] == "router":
        T, E, k = case["T"], case["E"], case["k"]
        s["p"] = moe.RouterProblem.make(T, E, k, logits_dtype=DT[case["io"]], score=case["score"],
                                        groups=case["groups"], topk_groups=case["topk_groups"],
                                        group_top=case["group_top"], renormalize=case["renorm"],
                                        scale=case["scale"])
        if case["dir"] == "fwd":
            s["topk_idx"] = torch.empty(T, k, dtype=torch.int32, device=DEV)
            s["topk_w"] = torch.empty(T, k, device=DEV)
        else:
            s["d_logits"] = torch.empty_like(s["logits"])
    elif case["op"] == "quant" and case["kind"] == "weights":
        E, N, K = case["E"], case["N"], case["K"]
        s["codes"] = torch.empty(E, N, K, dtype=E4M3, device=DEV)
        s["scales"] = torch.empty(E, _blocks(N), _blocks(K), device=DEV)
        s["codes_t"] = torch.empty(E, K, N, dtype=E4M3, device=DEV) if case["transposed"] else None
        s["scales_t"] = (torch.empty(E, _blocks(K), _blocks(N), device=DEV) if case["transposed"]
                         else None)
        s["p"] = moe.QuantWeightsProblem.make(E, N, K, src_dtype=DT[case["io"]])
    elif case["op"] == "quant":
        T, H = case["T"], case["H"]
        s["codes"] = torch.empty(T, H, dtype=E4M3, device=DEV)
        s["scales"] = torch.empty(T, _blocks(H), device=DEV)
        s["p"] = moe.QuantProblem.make(T, H, src_dtype=DT[case["io"]], swiglu=case["kind"] == "swiglu",
                                       glu_interleave=case["interleave"], swiglu_clamp=case["clamp"])
    else:
        M, N, K, E = (case[i] for i in "MNKE")
        s["out"] = torch.empty(M, N, dtype=DT[case["out"]], device=DEV)
        s["p"] = moe.FP8Problem.make(M, N, K, E, out_dtype=DT[case["out"]])
        s["work"] = moe.alloc_fp8_matmul_workspace(s["p"])
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["op"] == "router":
        return (_router_fwd if case["dir"] == "fwd" else _router_bwd)(case, state)
    if case["op"] == "quant":
        return _quant_weights(case, state) if case["kind"] == "weights" else _quant_rows(case, state)
    return _product(case, state)


def _run_own(case, s):
    import mixture_experts_ffn_permute_gb300 as moe
    if case["op"] == "router":
        if case["dir"] == "fwd":
            moe.router_forward(s["p"], s["logits"], s["topk_idx"], s["topk_w"], bias=s["bias"])
            return {"idx": s["topk_idx"], "w": s["topk_w"]}
        moe.router_backward(s["p"], s["logits"], s["idx"], s["d_w"], s["d_logits"])
        return {"d_logits": s["d_logits"]}
    if case["op"] == "quant" and case["kind"] == "weights":
        moe.fp8_quantize_weights(s["p"], s["src"], s["codes"], s["scales"], codes_t=s["codes_t"],
                                 scales_t=s["scales_t"])
        return {n: s[n] for n in ("codes", "scales", "codes_t", "scales_t") if s[n] is not None}
    if case["op"] == "quant":
        moe.fp8_quantize_rows(s["p"], s["src"], s["codes"], s["scales"])
        return {"codes": s["codes"], "scales": s["scales"]}
    moe.fp8_matmul(s["p"], s["x"], s["xs"], s["w"], s["ws"], s["out"], s["work"],
                   expert_offsets=s["offsets"])
    return {"out": s["out"]}


def _scores(case, l):
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    ex = torch.exp(l - l.amax(1, keepdim=True))
    return ex / ex.sum(1, keepdim=True)


def _choose(case, l, bias):
    """The scores and the k experts of every row, best first, ties to the lowest id."""
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    s = _scores(case, l)
    c = s if bias is None else s + bias.double()
    if case["topk_groups"] < G:
        per = c.reshape(T, G, E // G).sort(dim=2, descending=True).values[:, :, :case["group_top"]].sum(2)
        order = per.sort(dim=1, descending=True, stable=True).indices
        out = torch.zeros(T, G, dtype=torch.bool, device=DEV)
        out.scatter_(1, order[:, case["topk_groups"]:], True)
        c = torch.where(out.repeat_interleave(E // G, 1), -math.inf, c)
    return s, c.sort(dim=1, descending=True, stable=True).indices[:, :k]


def _router_fwd(case, s):
    score, idx = _choose(case, s["logits"].double(), s["bias"])
    w = score.gather(1, idx)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"idx": idx.to(torch.int32), "w": (w * case["scale"]).to(torch.float32)}


def _router_bwd(case, s):
    l, idx, dw = s["logits"].float(), s["idx"].long(), s["d_w"] * case["scale"]
    score = _scores(case, l)
    w = score.gather(1, idx)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        dw = (dw - (dw * w).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(score).scatter_(1, idx, dw)
    if case["score"] == "sigmoid":
        dl = ds * score * (1.0 - score)
    else:
        dl = score * (ds - (ds * score).sum(1, keepdim=True))
    return {"d_logits": dl.to(s["logits"].dtype)}


def _scale_of(amax):
    scale = amax / E4M3_MAX
    return torch.where(amax > 0, scale, torch.ones_like(scale))


def _pad(t, rows, cols):
    return torch.nn.functional.pad(t, (0, -t.shape[-1] % cols, 0, -t.shape[-2] % rows))


def _codes(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(E4M3)


def _halves(case, src):
    """A row's gate and up values: its halves, or alternating blocks."""
    T, F, I = case["T"], case["H"], case["interleave"] or case["H"]
    pairs = src.reshape(T, F // I, 2, I)
    return pairs[:, :, 0].reshape(T, F), pairs[:, :, 1].reshape(T, F)


def _quant_rows(case, s):
    x = s["src"].float()
    if case["kind"] == "swiglu":
        gate, up = _halves(case, x)
        if case["clamp"] > 0:
            gate, up = gate.clamp(max=case["clamp"]), up.clamp(-case["clamp"], case["clamp"])
        x = gate / (1.0 + torch.exp(-gate)) * up
    T, H = x.shape
    b = _pad(x, 1, BLOCK).reshape(T, -1, BLOCK)
    scale = _scale_of(b.abs().amax(2))
    return {"codes": _codes(b / scale[:, :, None]).reshape(T, -1)[:, :H].contiguous(),
            "scales": scale}


def _quant_weights(case, s):
    E, N, K = case["E"], case["N"], case["K"]
    b = _pad(s["src"].float(), BLOCK, BLOCK).reshape(E, _blocks(N), BLOCK, _blocks(K), BLOCK)
    scale = _scale_of(b.abs().amax((2, 4)))
    q = _codes(b / scale[:, :, None, :, None])
    q = q.reshape(E, _blocks(N) * BLOCK, -1)[:, :N, :K].contiguous()
    res = {"codes": q, "scales": scale}
    if case["transposed"]:
        res["codes_t"] = q.transpose(1, 2).contiguous()
        res["scales_t"] = scale.transpose(1, 2).contiguous()
    return res


def _spread(scale, rows, cols):
    """Scales of blocks (rows x cols of the last two axes follow) as values of their elements."""
    if rows is not None:
        scale = scale.repeat_interleave(BLOCK, -2)[..., :rows, :]
    return scale.repeat_interleave(BLOCK, -1)[..., :cols]


def _product(case, s):
    M, N, K = case["M"], case["N"], case["K"]
    out = torch.empty(M, N, dtype=DT[case["out"]], device=DEV)
    at = 0
    for e, n in enumerate(s["counts"]):  # one product for each expert that has rows
        if n:
            x = s["x"][at:at + n].float() * _spread(s["xs"][at:at + n], None, K)
            w = s["w"][e].float() * _spread(s["ws"][e], N, K)
            out[at:at + n] = x @ w.t()
        at += n
    return {"out": out}


# ------------------------------------------------------------------ cost
def work(case):
    if case["op"] == "router":
        T, E, k, size = case["T"], case["E"], case["k"], SIZE[case["io"]]
        if case["dir"] == "fwd":  # logits, bias in; ids and weights out
            return {"bytes": T * (E * size + 8 * k) + 4 * E * case["bias"], "flops": 6 * T * E}
        return {"bytes": T * (2 * E * size + 8 * k), "flops": 8 * T * E}
    if case["op"] == "quant" and case["kind"] == "weights":
        E, N, K = case["E"], case["N"], case["K"]
        n = E * (N * K + 4 * _blocks(N) * _blocks(K)) * (2 if case["transposed"] else 1)
        return {"bytes": n + E * N * K * SIZE[case["io"]], "flops": 3 * E * N * K}
    if case["op"] == "quant":
        T, H = case["T"], case["H"]
        glu = case["kind"] == "swiglu"
        return {"bytes": T * (H * SIZE[case["io"]] * (2 if glu else 1) + H + 4 * _blocks(H)),
                "flops": T * H * (8 if glu else 3)}
    M, N, K = case["M"], case["N"], case["K"]
    live = sum(c > 0 for c in _counts(case))
    return {"bytes": M * (K + 4 * _blocks(K) + N * SIZE[case["out"]]) + 4 * (case["E"] + 1)
            + live * (N * K + 4 * _blocks(N) * _blocks(K)), "flops": 2 * M * N * K}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "router":
        return _exact_router(case, s)
    if case["op"] == "quant":
        return _exact_quant(case, s)
    M, N, K, E = (case[i] for i in "MNKE")
    out = torch.zeros(M, N, dtype=torch.float64, device=DEV)
    offsets = s["offsets"].tolist()
    for e in range(E):
        rows = slice(offsets[e], offsets[e + 1])
        if rows.start == rows.stop:
            continue
        block = torch.arange(K, device=DEV) // BLOCK
        x = s["x"][rows].double() * s["xs"][rows].double()[:, block]
        w = s["w"][e].double() * s["ws"][e].double()[torch.arange(N, device=DEV) // BLOCK][:, block]
        torch.matmul(x, w.t(), out=out[rows])
    return {"out": out}


def _exact_router(case, s):
    l = s["logits"].double()

    def weights(l, idx):
        if case["score"] == "sigmoid":
            p = torch.sigmoid(l)
        else:
            p = torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
        w = torch.take_along_dim(p, idx, 1)
        return case["scale"] * (w / w.sum(1, keepdim=True) if case["renorm"] else w)

    if case["dir"] == "bwd":
        l.requires_grad_()
        grad, = torch.autograd.grad(weights(l, s["idx"].long()), l, s["d_w"].double())
        return {"d_logits": grad}
    p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    key = p if s["bias"] is None else p + s["bias"].double()
    T, E, G = case["T"], case["E"], case["groups"]
    if case["topk_groups"] < G:
        best = key.reshape(T, G, E // G).topk(case["group_top"], 2).values.sum(2)
        keep = torch.argsort(best, dim=1, descending=True, stable=True)[:, :case["topk_groups"]]
        live = (torch.arange(G, device=DEV) == keep[:, :, None]).any(1)
        key = key.masked_fill(~live.repeat_interleave(E // G, 1), -math.inf)
    return {"idx": None, "w": weights(l, key.topk(case["k"], 1).indices)}


def _exact_quant(case, s):
    """Scales, and the codes before their rounding."""
    x = s["src"].double()
    if case["kind"] == "weights":
        E, N, K = case["E"], case["N"], case["K"]
        scale = torch.ones(E, _blocks(N), _blocks(K), dtype=torch.float64, device=DEV)
        q = torch.empty_like(x)
        for i in range(_blocks(N)):
            for j in range(_blocks(K)):
                part = x[:, i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK]
                scale[:, i, j] = part.abs().amax((1, 2)) / E4M3_MAX
                q[:, i * BLOCK:(i + 1) * BLOCK, j * BLOCK:(j + 1) * BLOCK] = part / scale[:, i, j].reshape(E, 1, 1)
        res = {"codes": q, "scales": scale}
        if case["transposed"]:
            res.update(codes_t=q.transpose(1, 2), scales_t=scale.transpose(1, 2))
        return res
    if case["kind"] == "swiglu":
        f = torch.arange(case["H"], device=DEV)
        I = case["interleave"] or case["H"]
        at = f // I * (2 * I) + f % I
        gate, up = x[:, at], x[:, at + I]
        if case["clamp"] > 0:
            gate, up = gate.minimum(torch.tensor(case["clamp"], device=DEV)), up.clamp(-case["clamp"], case["clamp"])
        x = torch.nn.functional.silu(gate) * up
    q, scale = torch.empty_like(x), []
    for j in range(0, case["H"], BLOCK):
        part = x[:, j:j + BLOCK]
        scale.append(part.abs().amax(1) / E4M3_MAX)
        q[:, j:j + BLOCK] = part / scale[-1][:, None]
    return {"codes": q, "scales": torch.stack(scale, 1)}

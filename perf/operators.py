"""Measured cases of the operators around the expert layer in a training or scoring step.

Four operators, the ones a program needs next to ``moe_forward`` / ``moe_backward``:

  norm   residual_out = residual_scale * residual + branch_scale * gate * rmsnorm(branch) * w_post
         normed       = rmsnorm(residual_out) * w_pre            (forward and backward)
  ce     loss_t = logsumexp_v(x_t . w_v) - x_t . w_label, the logits never kept whole
         (forward alone for scoring, forward and backward for training)
  clip   the L2 norm over many gradient tensors and the gradients scaled to max_norm
  embed  out_t = scale * table[id_t], and d_table summed over the tokens of each id

``own`` False computes each operator with elementary torch operations in fp32, rounded once
at the end; ``own`` True makes the library's calls on the same inputs.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token between two blocks at the decode configuration's width: pure latency
        dict(name="norm_token", op="norm", dir="fwd", T=1, H=2048, io="bf16", res="bf16", w="bf16",
             gate="none"),
        # the skewed workload's batch between two blocks in training, fp32 residual stream
        dict(name="norm_fwd", op="norm", dir="fwd", T=8192, H=7168, io="bf16", res="f32", w="f32",
             gate="channel"),
        # the Mixtral-shaped batch's backward with a learned per-channel branch gate
        dict(name="norm_bwd", op="norm", dir="bwd", T=4096, H=4096, io="bf16", res="bf16", w="f32",
             gate="channel"),
        # a small fp32 run of odd width with one gate value a token (a sigmoid gate on the block)
        dict(name="norm_bwd_odd", op="norm", dir="bwd", T=1537, H=1001, io="f32", res="f32",
             w="f32", gate="token"),
        # scoring four drafted tokens at the decode width: the vocabulary matrix streams once
        dict(name="ce_score", op="ce", dir="fwd", T=4, H=2048, V=32000, masked=0.0),
        # a ragged training batch: odd vocabulary, a width that no tile divides, masked labels
        dict(name="ce_ragged", op="ce", dir="both", T=777, H=1000, V=50021, masked=0.3),
        # the Mixtral-shaped batch's loss and gradients
        dict(name="ce_train", op="ce", dir="both", T=4096, H=4096, V=32000, masked=0.05),
        # the many small parameters of a model (norms, gates, routers) in both types, packed
        dict(name="clip_small", op="clip", n=150, lo=200, hi=70000, f32=0.3, mix=1),
        # the expert weights' gradients of the decode configuration (E=128, H=2048, F=768), both
        # projections of eight experts to a tensor
        dict(name="clip_experts", op="clip", n=16, lo=37748736, hi=37748736, f32=0.0, mix=2),
        # the embedding of one decode batch
        dict(name="embed_token", op="embed", dir="fwd", T=32, V=32000, H=2048, table="bf16",
             out="bf16", masked=0.0),
        # the embedding gradient of a training batch, natural-text token frequencies
        dict(name="embed_grad", op="embed", dir="bwd", T=16384, V=32000, H=4096, table="bf16",
             out="bf16", masked=0.02),
        # a small fp32 run: odd vocabulary and width, many padded positions
        dict(name="embed_grad_odd", op="embed", dir="bwd", T=3001, V=50021, H=1001, table="f32",
             out="f32", masked=0.4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A row width: odd ones and multiples of 64 alike."""
    H = _log(rng, lo, hi)
    H = max(64, H // 64 * 64) if rng.random() < 0.5 else H
    return H + 64 if H == 3072 else H


def draw(rng):
    kind = rng.choice(["norm_fwd", "norm_bwd", "ce_fwd", "ce_both", "clip", "embed_fwd", "embed_bwd"])
    op, _, direction = kind.partition("_")
    if op == "norm":
        H = _width(rng, 64, 8192)
        return dict(op="norm", dir=direction, T=min(_log(rng, 1, 16384), 8192 * 7168 // H), H=H,
                    io=rng.choice(["bf16", "bf16", "f32"]), res=rng.choice(["bf16", "f32"]),
                    w=rng.choice(["bf16", "f32"]),
                    gate=rng.choice(["none", "channel", "token", "element"]))
    if op == "ce":
        H = _width(rng, 128, 4096) // 8 * 8
        H = H + 8 if H == 3072 else H
        V = _log(rng, 1000, 131072)
        if direction == "fwd":
            return dict(op="ce", dir="fwd", T=_log(rng, 1, 512), H=H, V=V, masked=0.0)
        T = min(_log(rng, 16, 8192), 4096 * 4096 * 32000 // (H * V))
        return dict(op="ce", dir="both", T=max(1, T), H=H, V=V, masked=rng.choice([0.0, 0.1, 0.5]))
    if op == "clip":
        hi = _log(rng, 1000, 8000000)
        return dict(op="clip", n=rng.randint(2, 60), lo=max(1, hi // _log(rng, 1, 1000)), hi=hi,
                    f32=rng.choice([0.0, 0.3, 1.0]), mix=rng.randint(1, 1 << 20))
    H = _width(rng, 64, 4096)
    V = min(_log(rng, 1000, 131072), 32000 * 8192 // H)
    return dict(op="embed", dir=direction, T=_log(rng, 1, 16384), V=V, H=H,
                table=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]),
                masked=rng.choice([0.0, 0.1, 0.5]))


# ------------------------------------------------------------------ inputs
EPS = 1e-6
NORM_SCALES = dict(residual_scale=0.9, branch_scale=0.5)
CLIP_EPS = 1e-6
GRAD_SCALE = 1.0 / 1024.0  # loss scaling undone with the clip


def _sizes(case):
    """The elements of every gradient tensor by type: {"bf16": [...], "f32": [...]}."""
    r = random.Random(case["mix"])
    every = [(_log(r, case["lo"], case["hi"]), r.random() < case["f32"]) for _ in range(case["n"])]
    by = {"bf16": [n for n, f in every if not f], "f32": [n for n, f in every if f]}
    return {d: sizes for d, sizes in by.items() if sizes}


def _views(flat, case):
    """One parameter each: views of the packed buffers."""
    return [v for d, sizes in _sizes(case).items() for v in flat[d].split(sizes)]


def _gate_shape(case):
    return {"none": None, "channel": (case["H"],), "token": (case["T"],),
            "element": (case["T"], case["H"])}[case["gate"]]


def _zipf_ids(n, V, masked, g):
    """Token ids of natural-text frequencies (1 / rank over a shuffled vocabulary), -1 where
    masked."""
    u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
    rank = torch.exp(u * math.log(V + 1)).to(torch.int64).clamp(1, V) - 1
    ids = torch.randperm(V, generator=g, device=DEV)[rank].to(torch.int32)
    if masked:
        ids = torch.where(torch.rand(n, generator=g, device=DEV) < masked, -1, ids)
    return ids.to(torch.int32)


def _inputs(case, seed):
    """Every tensor of a case, from the seed alone (the library is not touched here)."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def randn(*shape, dtype=torch.float32, std=1.0, mean=0.0):
        t = torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)
        return t.mul_(std).add_(mean).to(dtype)

    s = {}
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        io, res, wt = DT[case["io"]], DT[case["res"]], DT[case["w"]]
        s["branch"] = randn(T, H, dtype=io, std=0.7)
        s["residual"] = randn(T, H, dtype=res, std=2.0)  # in the backward: residual_out
        s["w_post"] = randn(H, dtype=wt, std=0.1, mean=1.0)
        s["w_pre"] = randn(H, dtype=wt, std=0.1, mean=1.0)
        shape = _gate_shape(case)
        s["gate"] = None if shape is None else randn(*shape, dtype=wt, std=0.3, mean=0.6)
        if case["dir"] == "bwd":
            s["d_normed"] = randn(T, H, dtype=io)
            s["d_residual_out"] = randn(T, H, dtype=res)
    elif case["op"] == "ce":
        T, H, V = case["T"], case["H"], case["V"]
        s["x"] = randn(T, H, dtype=torch.bfloat16)
        s["w"] = randn(V, H, dtype=torch.bfloat16, std=2.0 / math.sqrt(H))
        s["labels"] = _zipf_ids(T, V, case["masked"], g)
        valid = (s["labels"] >= 0).sum().clamp(min=1).to(torch.float32)
        s["d_loss"] = (1024.0 / valid).expand(T).contiguous()  # mean over the valid, loss scale
    elif case["op"] == "clip":
        s["flat"] = {d: randn(sum(sizes), dtype=DT[d], std=30.0) for d, sizes in _sizes(case).items()}
        s["grads"] = _views(s["flat"], case)
    else:
        T, V, H = case["T"], case["V"], case["H"]
        s["ids"] = _zipf_ids(T, V, case["masked"], g)
        if case["dir"] == "fwd":
            s["table"] = randn(V, H, dtype=DT[case["table"]], std=1.0 / math.sqrt(H))
        else:
            s["d_out"] = randn(T, H, dtype=DT[case["out"]])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "clip":  # the gradients are this far above the limit
        s["max_norm"] = 1.0
    if not own:
        return s
    import mixture_experts_ffn_permute_gb300 as moe
    if case["op"] == "norm":
        p = s["p"] = moe.NormProblem.make(case["T"], case["H"], branch_dtype=DT[case["io"]],
                                          residual_dtype=DT[case["res"]],
                                          weight_dtype=DT[case["w"]], gate=case["gate"], eps=EPS,
                                          **NORM_SCALES)
        if case["dir"] == "fwd":
            s["residual_out"] = torch.empty_like(s["residual"])
            s["normed"] = torch.empty_like(s["branch"])
        else:
            s["ws"] = moe.alloc_block_norm_workspace(p)
            for k in ("branch", "w_post", "w_pre", "gate", "residual"):
                s["d_" + k] = None if s[k] is None else torch.empty_like(s[k])
    elif case["op"] == "ce":
        p = s["p"] = moe.CEProblem.make(case["T"], case["H"], case["V"])
        s["ws"] = moe.alloc_linear_ce_workspace(p, backward=case["dir"] == "both")
        s["loss"] = torch.empty(case["T"], device=DEV)
        s["lse"] = torch.empty(case["T"], device=DEV)
        if case["dir"] == "both":
            s["dx"], s["dw"] = torch.empty_like(s["x"]), torch.empty_like(s["w"])
    elif case["op"] == "clip":
        s["out"] = {d: torch.empty_like(f) for d, f in s["flat"].items()}
        s["list"] = moe.GradList(s["grads"], _views(s["out"], case))
        s["ws"] = moe.alloc_clip_workspace(s["list"])
        s["norm"] = torch.empty(2, device=DEV)
    else:
        p = s["p"] = moe.EmbedProblem.make(case["T"], case["V"], case["H"],
                                           table_dtype=DT[case["table"]],
                                           out_dtype=DT[case["out"]], scale=math.sqrt(case["H"]))
        if case["dir"] == "fwd":
            s["out"] = torch.empty(case["T"], case["H"], dtype=DT[case["out"]], device=DEV)
        else:
            s["ws"] = moe.alloc_embedding_workspace(p)
            s["d_table"] = torch.empty(case["V"], case["H"], dtype=DT[case["table"]], device=DEV)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["op"] == "norm":
        return (_norm_fwd if case["dir"] == "fwd" else _norm_bwd)(case, state)
    if case["op"] == "ce":
        return _ce(case, state)
    if case["op"] == "clip":
        return _clip(state)
    return (_embed_fwd if case["dir"] == "fwd" else _embed_bwd)(case, state)


def _run_own(case, s):
    import mixture_experts_ffn_permute_gb300 as moe
    if case["op"] == "norm":
        if case["dir"] == "fwd":
            moe.block_norm_forward(s["p"], s["residual"], branch=s["branch"], w_post=s["w_post"],
                                   gate=s["gate"], w_pre=s["w_pre"],
                                   residual_out=s["residual_out"], normed=s["normed"])
            return {"residual_out": s["residual_out"], "normed": s["normed"]}
        moe.block_norm_backward(s["p"], s["residual"], s["d_residual"], s["ws"],
                                branch=s["branch"], w_post=s["w_post"], gate=s["gate"],
                                w_pre=s["w_pre"], d_normed=s["d_normed"],
                                d_residual_out=s["d_residual_out"], d_branch=s["d_branch"],
                                d_w_post=s["d_w_post"], d_gate=s["d_gate"], d_w_pre=s["d_w_pre"])
        return {k: s["d_" + k] for k in ("residual", "branch", "w_post", "w_pre", "gate")}
    if case["op"] == "ce":
        moe.linear_ce_forward(s["p"], s["x"], s["w"], s["labels"], s["loss"], s["lse"], s["ws"])
        r = {"loss": s["loss"], "lse": s["lse"]}
        if case["dir"] == "both":
            moe.linear_ce_backward(s["p"], s["x"], s["w"], s["labels"], s["lse"], s["d_loss"],
                                   s["dx"], s["dw"], s["ws"])
            r["dx"], r["dw"] = s["dx"], s["dw"]
        return r
    if case["op"] == "clip":
        moe.clip_grad_norm(s["list"], s["max_norm"], s["norm"], s["ws"], grad_scale=GRAD_SCALE,
                           eps=CLIP_EPS)
        return {"norm": s["norm"], "out": s["out"]}
    if case["dir"] == "fwd":
        moe.embedding_forward(s["p"], s["ids"], s["table"], s["out"])
        return {"out": s["out"]}
    moe.embedding_backward(s["p"], s["ids"], s["d_out"], s["d_table"], s["ws"])
    return {"d_table": s["d_table"]}


def _gate_of(case, s):
    if s["gate"] is None:
        return 1.0
    g = s["gate"].float()
    return g[:, None] if case["gate"] == "token" else g


def _rstd(x):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _norm_fwd(case, s):
    y, r = s["branch"].float(), s["residual"].float()
    y = y * _rstd(y) * s["w_post"].float()
    r = NORM_SCALES["residual_scale"] * r + NORM_SCALES["branch_scale"] * (_gate_of(case, s) * y)
    n = r * _rstd(r) * s["w_pre"].float()
    return {"residual_out": r.to(s["residual"].dtype), "normed": n.to(s["branch"].dtype)}


def _norm_bwd(case, s):
    y, r = s["branch"].float(), s["residual"].float()  # r: the stored residual_out
    dn, dr = s["d_normed"].float(), s["d_residual_out"].float()
    w_post, w_pre, gate = s["w_post"].float(), s["w_pre"].float(), _gate_of(case, s)
    rs = _rstd(r)
    u = r * rs
    a = dn * w_pre
    g = dr + rs * (a - u * (a * u).mean(-1, keepdim=True))
    ys = _rstd(y)
    v = y * ys
    b = NORM_SCALES["branch_scale"] * g  # gradient of gate * v * w_post
    c = b * gate * w_post
    dy = ys * (c - v * (c * v).mean(-1, keepdim=True))
    res = {"residual": (NORM_SCALES["residual_scale"] * g).to(s["residual"].dtype),
           "branch": dy.to(s["branch"].dtype),
           "w_post": (b * gate * v).sum(0).to(s["w_post"].dtype),
           "w_pre": (dn * u).sum(0).to(s["w_pre"].dtype), "gate": None}
    if s["gate"] is not None:
        dg = b * v * w_post
        dg = {"channel": lambda: dg.sum(0), "token": lambda: dg.sum(1), "element": lambda: dg}[
            case["gate"]]()
        res["gate"] = dg.to(s["gate"].dtype)
    return res


def _ce(case, s):
    x, w, labels = s["x"].float(), s["w"].float(), s["labels"].long()
    valid = labels >= 0
    z = x @ w.t()
    m = z.max(1, keepdim=True).values
    lse = (z - m).exp().sum(1).log() + m[:, 0]
    at = labels.clamp(min=0)[:, None]
    loss = torch.where(valid, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    res = {"loss": loss, "lse": lse}
    if case["dir"] == "both":
        p = (z - lse[:, None]).exp()
        p.scatter_add_(1, at, torch.full_like(lse, -1.0)[:, None])
        p *= torch.where(valid, s["d_loss"], torch.zeros_like(lse))[:, None]
        res["dx"] = (p @ w).to(s["x"].dtype)
        res["dw"] = (p.t() @ x).to(s["w"].dtype)
    return res


def _clip(s):
    sq = torch.stack([(g.float() * g.float()).sum() for g in s["grads"]]).sum()
    norm = sq.sqrt() * GRAD_SCALE
    coef = (s["max_norm"] / (norm + CLIP_EPS)).clamp(max=1.0)
    outs = [(g.float() * (GRAD_SCALE * coef)).to(g.dtype) for g in s["grads"]]
    return {"norm": torch.stack([norm, coef]),
            "out": {d: torch.cat([o for o in outs if o.dtype == DT[d]]) for d in s["flat"]}}


def _embed_fwd(case, s):
    ids = s["ids"].long()
    out = s["table"][ids.clamp(min=0)].float() * math.sqrt(case["H"])
    return {"out": (out * (ids >= 0).float()[:, None]).to(DT[case["out"]])}


def _embed_bwd(case, s):
    ids = s["ids"].long()
    d = s["d_out"].float() * (ids >= 0).float()[:, None]
    table = torch.zeros(case["V"], case["H"], device=DEV)
    table.index_add_(0, ids.clamp(min=0), d)
    return {"d_table": (table * math.sqrt(case["H"])).to(DT[case["table"]])}


# ------------------------------------------------------------------ cost
def work(case):
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        io, res, wt = SIZE[case["io"]], SIZE[case["res"]], SIZE[case["w"]]
        gate = {"none": 0, "channel": H, "token": T, "element": T * H}[case["gate"]]
        if case["dir"] == "fwd":  # branch, residual in; residual_out, normed out
            return {"bytes": T * H * 2 * (io + res) + (2 * H + gate) * wt, "flops": 12 * T * H}
        # branch, residual_out, d_normed, d_residual_out in; d_branch, d_residual out
        return {"bytes": T * H * 3 * (io + res) + 2 * (2 * H + gate) * wt, "flops": 30 * T * H}
    if case["op"] == "ce":
        T, H, V = case["T"], case["H"], case["V"]
        if case["dir"] == "fwd":
            return {"bytes": 2 * (T * H + V * H) + 12 * T, "flops": 2 * T * H * V}
        # logits, d logits' two products; the logits are computed once in what cannot be spared
        return {"bytes": 4 * (T * H + V * H) + 16 * T, "flops": 6 * T * H * V}
    if case["op"] == "clip":
        n = {d: sum(sizes) for d, sizes in _sizes(case).items()}
        return {"bytes": sum(2 * n[d] * SIZE[d] for d in n), "flops": 3 * sum(n.values())}
    T, V, H = case["T"], case["V"], case["H"]
    if case["dir"] == "fwd":
        return {"bytes": T * (4 + H * (min(1.0, V / T) * SIZE[case["table"]] + SIZE[case["out"]])),
                "flops": T * H}
    return {"bytes": T * (4 + H * SIZE[case["out"]]) + V * H * SIZE[case["table"]],
            "flops": 2 * T * H}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    f = lambda t: None if t is None else t.double()  # noqa: E731
    if case["op"] == "norm":
        return _exact_norm(case, s, f)
    if case["op"] == "ce":
        return _exact_ce(case, s, f)
    if case["op"] == "clip":
        total = torch.zeros((), dtype=torch.float64, device=DEV)
        for flat in s["flat"].values():
            total += torch.linalg.vector_norm(flat.double()) ** 2
        norm = total.sqrt() * GRAD_SCALE
        coef = torch.clamp(1.0 / (norm + CLIP_EPS), max=1.0)
        return {"norm": torch.stack([norm, coef]),
                "out": {d: flat.double() * (GRAD_SCALE * coef) for d, flat in s["flat"].items()}}
    ids = s["ids"].cpu().tolist()
    if case["dir"] == "fwd":
        out = torch.zeros(case["T"], case["H"], dtype=torch.float64, device=DEV)
        keep = torch.tensor([t for t, i in enumerate(ids) if i >= 0], dtype=torch.long, device=DEV)
        src = torch.tensor([i for i in ids if i >= 0], dtype=torch.long, device=DEV)
        out[keep] = s["table"][src].double() * math.sqrt(case["H"])
        return {"out": out}
    order = sorted((i, t) for t, i in enumerate(ids) if i >= 0)
    rows = s["d_out"].double()[torch.tensor([t for _, t in order], dtype=torch.long, device=DEV)]
    # running sums at the ends of each id's run: their differences are the runs' sums
    table = torch.zeros(case["V"], case["H"], dtype=torch.float64, device=DEV)
    if order:
        ends = [k for k in range(len(order)) if k + 1 == len(order) or order[k + 1][0] != order[k][0]]
        sums = rows.cumsum(0)[torch.tensor(ends, device=DEV)]
        sums[1:] -= sums[:-1].clone()
        table[torch.tensor([order[k][0] for k in ends], device=DEV)] = sums * math.sqrt(case["H"])
    return {"d_table": table}


def _exact_norm(case, s, f):
    """The definition in 64 bits; gradients by differentiating it."""
    y, r, wo, wi, gate = (f(s[k]) for k in ("branch", "residual", "w_post", "w_pre", "gate"))
    H = case["H"]

    def norm(t, w):
        return t / torch.sqrt(t.square().sum(-1, keepdim=True) / H + EPS) * w

    def branch(y, wo, gate):
        b = norm(y, wo)
        if gate is not None:
            b = b * (gate.unsqueeze(1) if case["gate"] == "token" else gate)
        return NORM_SCALES["branch_scale"] * b

    if case["dir"] == "fwd":
        out = NORM_SCALES["residual_scale"] * r + branch(y, wo, gate)
        return {"residual_out": out, "normed": norm(out, wi)}
    leaves = [t.requires_grad_() if t is not None else None for t in (r, wi, y, wo, gate)]
    d_r, d_wi = torch.autograd.grad(norm(r, wi), leaves[:2], f(s["d_normed"]))
    g = f(s["d_residual_out"]) + d_r
    live = [t for t in leaves[2:] if t is not None]
    got = list(torch.autograd.grad(branch(y, wo, gate), live, g))
    return {"residual": NORM_SCALES["residual_scale"] * g, "branch": got[0], "w_post": got[1],
            "w_pre": d_wi, "gate": got[2] if len(got) > 2 else None}


def _exact_ce(case, s, f):
    x, w, labels = f(s["x"]), f(s["w"]), s["labels"].long()
    both = case["dir"] == "both"
    T, V = case["T"], case["V"]
    loss = torch.zeros(T, dtype=torch.float64, device=DEV)
    lse = torch.empty(T, dtype=torch.float64, device=DEV)
    dx, dw = (torch.zeros_like(x), torch.zeros_like(w)) if both else (None, None)
    step = max(1, min(T, (1 << 27) // V))
    for t0 in range(0, T, step):  # some tokens at a time: the logits in 64 bits are large
        rows = slice(t0, min(T, t0 + step))
        z = x[rows] @ w.t()
        lse[rows] = torch.logsumexp(z, 1)
        here = labels[rows]
        keep = torch.nonzero(here >= 0)[:, 0]
        loss[rows][keep] = lse[rows][keep] - z[keep, here[keep]]
        if both:
            d = torch.softmax(z, 1)
            d[keep, here[keep]] -= 1.0
            d *= (f(s["d_loss"])[rows] * (here >= 0))[:, None]
            dx[rows] = d @ w
            dw += d.t() @ x[rows]
    return {"loss": loss, "lse": lse, **({"dx": dx, "dw": dw} if both else {})}

"""GPU parity of a training step's run of the expert router and the layer of given routing:
router_forward, forward_routed, backward_routed and router_backward, against the 64-bit oracle of the
layer and the router's formulas in 64 bits.

Tolerances: the layer's own (parity.py).  A gradient of a weight is off by at most 2^-7 of its terms'
magnitude M_j; with renormalised weights d l_j = q_j f_j (g_j - sum g_i q_i), 0 < f_j <= 1, is then
off by 2^-7 scale q_j (M_j + sum M_i q_i), below 2^-6 scale q_j sum M_i, and by the router's own
rounding, some 2^-18 of the same.

The bounds of dx, dw1 and dw2 have a second part.  parity.py's magnitude of an element takes its
terms as they are; where an expert has a row or two, a term itself may be small by cancellation.
(Of the 25 million elements of dw1 in the second case four are: up value 1.99e-4 of 256 products whose
absolute values sum to 10.5, off by 1.6e-6 = 10.5 x 1.3 2^-23, eight tenths of a percent of the term,
for 2^-7.)  With u = (n + 2) 2^-23, the bound of a sum of n products in fp32 that is cut, not
rounded, A, U and G the sums of absolute values behind the gate a, the up value v and the gradient g
of h, |silu'| <= 1.1, |silu''| <= 1/2, |silu(a)| <= |a| and the exponential's part below u / 16:
  gate part  |d (g v silu'(a))| <= u (1.1 G U + 1.1 G U + G U A / 2 + G U / 16)
  up part    |d (g silu(a))|    <= u (G A + 1.1 G A + G A / 16)
  h          |d (v silu(a))|    <= u (U A + 1.1 U A + U A / 16)
summed with the absolute values of what they are multiplied with."""
import math

import pytest
import torch

import moe_inputs as mi
import oracle
import mixture_experts_ffn_permute_gb300 as moe
from mixture_experts_ffn_permute_gb300 import _build
from parity import assert_bf16_close, assert_grad_bound

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    moe.load()


def inner_bounds(shape, host, idx, w, d_out):
    """The second part of the bounds of dx, dw1 and dw2."""
    T, H, F, E, I = shape.T, shape.H, shape.F, shape.E, shape.glu_interleave or shape.F
    at = torch.arange(F) // I * (2 * I) + torch.arange(F) % I  # rows of gates; ups are I behind
    dx, dw1 = torch.zeros(T, H, dtype=torch.float64), torch.zeros(E, 2 * F, H, dtype=torch.float64)
    dw2 = torch.zeros(E, H, F, dtype=torch.float64)
    u = (max(H, F) + 2) * 2.0 ** -23
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        x, d = host["x"][t].double().abs(), d_out[t].double().abs() * w[t, j].double()[:, None]
        w1, w2 = host["w1"][e].double().abs(), host["w2"][e].double().abs()
        A, U, G = x @ w1[at].t(), x @ w1[at + I].t(), d @ w2
        gate, up, h = u * G * U * (2.3 + A / 2), 2.2 * u * G * A, 2.2 * u * U * A
        dx.index_add_(0, t, gate @ w1[at] + up @ w1[at + I])
        dw1[e, at], dw1[e, at + I] = gate.t() @ x, up.t() @ x
        dw2[e] = d.t() @ h
    return {"dx": dx.numpy(), "dw1": dw1.numpy(), "dw2": dw2.numpy()}


CASES = [(mi.MoEShape("groups", T=150, H=256, F=384, E=24, k=3, glu_interleave=32, swiglu_clamp=1.0),
          dict(score="sigmoid", groups=4, topk_groups=2, group_top=2)),
         (mi.MoEShape("odd-groups", T=90, H=256, F=256, E=192, k=6),
          dict(score="sigmoid", groups=8, topk_groups=3, group_top=2)),
         (mi.MoEShape("softmax", T=333, H=512, F=256, E=8, k=2), dict(score="softmax")),
         (mi.MoEShape("one", T=1, H=256, F=256, E=40, k=4), dict(score="softmax", groups=5, topk_groups=2))]


@pytest.mark.parametrize("shape,router", CASES, ids=[c[0].name for c in CASES])
def test_training_step_of_router_and_layer(shape, router):
    T, H, F, E, k = shape.T, shape.H, shape.F, shape.E, shape.k
    inp = {n: t.to(DEV) for n, t in mi.make_inputs(shape, seed=3).items()}
    d_out = mi.make_grad_out(shape, seed=3).to(DEV)
    bias = (0.1 * torch.randn(E, generator=torch.Generator().manual_seed(1))).to(DEV)
    logits = inp["logits"]
    pad = T - T // 8
    logits[pad:] = -math.inf  # padding: no expert
    pr = moe.RouterProblem.make(T, E, k, **router)
    p = moe.Problem.make(T, H, F, E, k, True, shape.glu_interleave, shape.swiglu_clamp)
    ws, bws = moe.alloc_workspace(p), moe.alloc_backward_workspace(p)
    moe.clear_device_status(ws)
    moe.clear_device_status(bws)
    idx = torch.empty(T, k, dtype=torch.int32, device=DEV)
    w, d_w = torch.empty(T, k, device=DEV), torch.empty(T, k, device=DEV)
    out, dx = (torch.empty(T, H, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    dw1, dw2 = torch.empty_like(inp["w1"]), torch.empty_like(inp["w2"])
    d_logits = torch.empty(T, E, device=DEV)

    def step():
        moe.router_forward(pr, logits, idx, w, bias=bias)
        moe.forward_routed(p, inp["x"], idx, w, inp["w1"], inp["w2"], out, ws)
        moe.backward_routed(p, inp["x"], idx, w, inp["w1"], inp["w2"], d_out, dx, dw1, dw2, bws, d_topk_w=d_w)
        moe.router_backward(pr, logits, idx, d_w, d_logits)

    step()
    torch.cuda.synchronize()
    assert moe.get_device_status(ws) == moe.get_device_status(bws) == moe.MOE_OK

    # the router's choice and weights by their formulas
    l = logits[:pad].double().cpu()
    s = torch.sigmoid(l) if router["score"] == "sigmoid" else torch.softmax(l, 1)
    c = s + bias.double().cpu()
    if "groups" in router:
        G = router["groups"]
        best = c.view(pad, G, E // G).topk(router.get("group_top", 1)).values.sum(2)
        kept = best.topk(router["topk_groups"]).indices
        c = c.masked_fill(~torch.zeros(pad, G, dtype=torch.bool).scatter_(1, kept, True).repeat_interleave(E // G, 1),
                          -math.inf)
    ids = c.topk(k).indices
    assert torch.equal(idx[:pad].cpu().long(), ids) and (idx[pad:] == -1).all()
    q = s.gather(1, ids)
    q = q / q.sum(1, keepdim=True)
    assert ((w[:pad].cpu().double() - q).abs() <= 2.0 ** -18 * q).all() and not w[pad:].any()

    # the layer and its gradients on that routing, by the oracle
    host = {n: t.cpu() for n, t in inp.items()}
    kw = dict(interleave=shape.glu_interleave, clamp=shape.swiglu_clamp)
    ref = oracle.moe_forward_routed(host["x"], idx.cpu(), w.cpu(), host["w1"], host["w2"], **kw)
    assert_bf16_close(out, ref["out"], "out")
    assert not out[pad:].any()
    args = (host["x"], idx.cpu(), w.cpu(), host["w1"], host["w2"], d_out.cpu())
    grad = oracle.expert_backward(*args, mask_f32=True, **kw)
    mag = oracle.expert_backward(*args, mask_f32=True, magnitude=True, **kw)
    inner = inner_bounds(shape, host, idx.cpu(), w.cpu(), d_out.cpu())
    assert_grad_bound(d_w, grad["dw_route"], mag["dw_route"], "d_topk_w")
    for name, got in (("dx", dx), ("dw1", dw1), ("dw2", dw2)):
        assert_grad_bound(got, grad[name], mag[name] + 2.0 ** 7 * inner[name], name)

    # the gradient of the logits through the weights
    lg = l.requires_grad_()
    s = torch.sigmoid(lg) if router["score"] == "sigmoid" else torch.softmax(lg, 1)
    r = s.gather(1, ids)
    want, = torch.autograd.grad(r / r.sum(1, keepdim=True), lg, torch.as_tensor(grad["dw_route"])[:pad].double())
    tol = torch.zeros(pad, E, dtype=torch.float64).scatter_(
        1, ids, (2.0 ** -6 + 2.0 ** -16) * q * torch.as_tensor(mag["dw_route"])[:pad].double().sum(1, keepdim=True))
    err = (d_logits[:pad].cpu().double() - want).abs()
    chosen = torch.zeros(pad, E, dtype=torch.bool).scatter_(1, ids, True)
    assert (err[chosen] <= tol[chosen]).all(), float((err - tol).max())
    assert not d_logits[:pad].cpu()[~chosen].any() and not d_logits[pad:].any()

    # the same step captured and replayed, bit by bit
    first = [t.clone() for t in (idx, w, out, dx, dw1, dw2, d_w, d_logits)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (w, out, dx, dw1, dw2, d_w, d_logits):
        t.fill_(7)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(first, (idx, w, out, dx, dw1, dw2, d_w, d_logits)):
        assert torch.equal(a, b)

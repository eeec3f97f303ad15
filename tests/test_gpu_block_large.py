"""The operators around the layer beyond 2^31 elements, and in a captured CUDA graph.

Large tensors are filled on the GPU with a few known rows among zeros (or with
one value), so the expected values are exact or those of a row alone; the
tolerances are the operators' own (tests of each)."""
import math

import pytest
import torch

import mixture_experts_ffn_permute_gb300 as moe
from mixture_experts_ffn_permute_gb300 import _build

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    moe.load()


@pytest.mark.parametrize("H", [8192, 8189])
def test_norm_rows_beyond_31_bits(H):
    """The last rows of a tensor of 2.3 billion elements, against the same rows alone."""
    T, n = 280_000, 5
    g = torch.Generator(device=DEV).manual_seed(H)
    small = {k: torch.randn(n, H, generator=g, device=DEV).to(BF) for k in ("y", "r", "dn", "dr")}
    w = torch.rand(H, generator=g, device=DEV) + 0.5

    def run(rows, y, r, dn, dr):
        p = moe.NormProblem.make(rows, H, weight_dtype=F32, gate="channel")
        out, nrm, d_r, d_y = (torch.empty_like(r) for _ in range(4))
        moe.block_norm_forward(p, r, branch=y, w_post=w, gate=w, w_pre=w, residual_out=out,
                               normed=nrm)
        d = [torch.empty_like(w) for _ in range(3)]
        moe.block_norm_backward(p, out, d_r, moe.alloc_block_norm_workspace(p), branch=y, w_post=w,
                                gate=w, w_pre=w, d_normed=dn, d_residual_out=dr, d_branch=d_y,
                                d_w_post=d[0], d_gate=d[1], d_w_pre=d[2])
        return out, nrm, d_r, d_y, d

    want = run(n, *small.values())
    big = []
    for t in small.values():
        b = torch.zeros(T, H, dtype=BF, device=DEV)
        b[-n:] = t
        big.append(b)
    got = run(T, *big)
    for a, b in zip(want[:4], got[:4]):
        # fewer rows take another kernel: the sums' order may differ
        assert ((a.double() - b[-n:].double()).abs() <= 2.0 ** -7 * a.double().abs() + 1e-3).all()
        assert not b[:1000].any() and not b[T // 2:T // 2 + 1000].any()
    for a, b in zip(want[4], got[4]):
        assert ((a - b).abs() <= 1e-4 * (1 + a.abs())).all()


def test_cross_entropy_weights_beyond_31_bits():
    """w and dw of 2.2 billion elements; the labels lie in the last rows."""
    T, H, V = 3, 8192, 262_400
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(T, H, generator=g, device=DEV).to(BF)
    w = torch.zeros(V, H, dtype=BF, device=DEV)
    w[-4:] = (torch.randn(4, H, generator=g, device=DEV) * 0.03).to(BF)
    labels = torch.tensor([V - 1, V - 3, 7], dtype=torch.int32, device=DEV)
    p = moe.CEProblem.make(T, H, V)
    ws = moe.alloc_linear_ce_workspace(p, backward=True)
    loss, lse = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    moe.linear_ce_forward(p, x, w, labels, loss, lse, ws)
    z = x.double() @ w[-4:].double().t()  # every other logit is 0
    want = torch.log(torch.exp(z).sum(1) + (V - 4))
    zl = torch.stack([z[0, 3], z[1, 1], torch.zeros((), dtype=torch.float64, device=DEV)])
    assert ((lse.double() - want).abs() <= 1e-4).all()
    assert ((loss.double() - (want - zl)).abs() <= 2e-4).all()
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    moe.linear_ce_backward(p, x, w, labels, lse, torch.ones(T, device=DEV), dx, dw, ws)
    prob = torch.exp(z - want[:, None])
    grad = prob.clone()
    grad[0, 3] -= 1
    grad[1, 1] -= 1
    ref = grad.t() @ x.double()
    assert float((dw[-4:].double() - ref).norm()) <= 5e-3 * float(ref.norm())
    seven = (torch.exp(-want) - torch.tensor([0., 0., 1.], device=DEV)).double() @ x.double()
    assert float((dw[7].double() - seven).norm()) <= 5e-3 * float(seven.norm())
    ref = grad @ w[-4:].double()
    assert float((dx.double() - ref).norm()) <= 5e-3 * float(ref.norm())
    assert moe.get_device_status(ws) == moe.MOE_OK


def test_clipping_a_tensor_beyond_31_bits():
    n = (1 << 31) + 12_345
    t = torch.full((n,), 2.0, dtype=BF, device=DEV)
    t[-1] = 1024.0
    lst = moe.GradList([t])
    norm = torch.empty(2, device=DEV)
    moe.clip_grad_norm(lst, 1.0, norm, moe.alloc_clip_workspace(lst), eps=0.0)
    want = math.sqrt(4.0 * (n - 1) + 2.0 ** 20)
    assert abs(float(norm[0]) - want) <= 2.0 ** -18 * want
    assert abs(float(t[-1]) * want / 1024 - 1) <= 2.0 ** -7
    for at in (0, n // 2, n - 2):
        assert abs(float(t[at]) * want / 2 - 1) <= 2.0 ** -7


def test_captured_in_a_graph():
    """All operators of a step captured once and replayed on new inputs in the same tensors."""
    T, H, V = 700, 520, 3001
    g = torch.Generator(device=DEV).manual_seed(2)

    def randn(*shape, dtype=BF):
        return torch.randn(*shape, generator=g, device=DEV).to(dtype)

    pe = moe.EmbedProblem.make(T, V, H, BF, F32)
    pn = moe.NormProblem.make(T, H, BF, F32, F32)
    pc = moe.CEProblem.make(T, H, V)
    ids = torch.randint(-1, V, (T,), generator=g, device=DEV, dtype=torch.int32)
    table, head, y, w = randn(V, H), randn(V, H), randn(T, H), randn(H, dtype=F32)
    r, out, d_r = (torch.empty(T, H, device=DEV) for _ in range(3))
    n, dn, dy = (torch.empty(T, H, dtype=BF, device=DEV) for _ in range(3))
    loss, lse, d_loss = torch.empty(T, device=DEV), torch.empty(T, device=DEV), torch.ones(T, device=DEV)
    grads = [torch.empty_like(t) for t in (table, head, w, w)]
    outs = [torch.empty_like(t) for t in grads]
    lst = moe.GradList(grads, outs)
    norm = torch.empty(2, device=DEV)
    ws = [moe.alloc_embedding_workspace(pe), moe.alloc_block_norm_workspace(pn),
          moe.alloc_linear_ce_workspace(pc, backward=True), moe.alloc_clip_workspace(lst)]

    def step():
        moe.embedding_forward(pe, ids, table, r)
        moe.block_norm_forward(pn, r, branch=y, w_post=w, w_pre=w, residual_out=out, normed=n)
        moe.linear_ce_forward(pc, n, head, ids, loss, lse, ws[2])
        moe.linear_ce_backward(pc, n, head, ids, lse, d_loss, dn, grads[1], ws[2])
        moe.block_norm_backward(pn, out, d_r, ws[1], branch=y, w_post=w, w_pre=w, d_normed=dn,
                                d_branch=dy, d_w_post=grads[2], d_w_pre=grads[3])
        moe.embedding_backward(pe, ids, d_r, grads[0], ws[0])
        moe.clip_grad_norm(lst, 1.0, norm, ws[3])
        return [loss, lse, dy, norm, *outs]

    step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for _ in range(2):
        y.copy_(randn(T, H))
        ids.copy_(torch.randint(-1, V, (T,), generator=g, device=DEV, dtype=torch.int32))
        want = [t.clone() for t in step()]
        for t in (loss, lse, dy, norm, *outs):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (loss, lse, dy, norm, *outs)):
            assert torch.equal(a, b)


def test_nothing_is_allocated():
    """The second run of every operator takes no device memory, from torch or from the driver."""
    T, H, V = 777, 1000, 5003
    x, w = (torch.randn(n, H, device=DEV).to(BF) for n in (T, V))
    ids = torch.randint(-1, V, (T,), device=DEV, dtype=torch.int32)
    pe, pc = moe.EmbedProblem.make(T, V, H), moe.CEProblem.make(T, H, V)
    pn = moe.NormProblem.make(T, H, weight_dtype=F32)
    scale = torch.ones(H, device=DEV)
    loss, lse, d_loss, norm = *(torch.ones(T, device=DEV) for _ in range(3)), torch.ones(2, device=DEV)
    a, b, c, d = (torch.empty_like(x) for _ in range(4))
    dw, g = torch.empty_like(w), [torch.empty_like(scale) for _ in range(2)]
    lst = moe.GradList([dw, *g])
    ws = [moe.alloc_embedding_workspace(pe), moe.alloc_block_norm_workspace(pn),
          moe.alloc_linear_ce_workspace(pc, backward=True), moe.alloc_clip_workspace(lst)]

    def once():
        moe.embedding_forward(pe, ids, w, a, ws=ws[0])
        moe.block_norm_forward(pn, a, branch=x, w_post=scale, w_pre=scale, residual_out=b, normed=c)
        moe.linear_ce_forward(pc, c, w, ids, loss, lse, ws[2])
        moe.linear_ce_backward(pc, c, w, ids, lse, d_loss, d, dw, ws[2])
        moe.block_norm_backward(pn, b, a, ws[1], branch=x, w_post=scale, w_pre=scale, d_normed=d,
                                d_branch=c, d_w_post=g[0], d_w_pre=g[1])
        moe.embedding_backward(pe, ids, a, dw, ws[0])
        moe.clip_grad_norm(lst, 1.0, norm, ws[3])
        torch.cuda.synchronize()
        return torch.cuda.mem_get_info()[0], torch.cuda.memory_stats()["allocation.all.allocated"]

    assert once() == once()

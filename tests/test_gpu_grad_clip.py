"""GPU parity of moe_clip_grad_norm against 64 bits on the CPU, and its edges.

Tolerances: at most 66 squares of one thread are added in fp32 (66 2^-24
relative, no cancellation) and those sums in fp64, so the norm is within
2^-18; the coefficient adds a division and the output two products and the
rounding to its type."""
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


def reference(grads, max_norm, scale, eps):
    total = math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads)) * abs(scale)
    coef = min(1.0, max_norm / (total + eps))
    return total, coef, [g.double().cpu() * (scale * coef) for g in grads]


def run(grads, outs, max_norm, scale=1.0, eps=1e-6, stream=None):
    lst = moe.GradList(grads, outs)
    norm = torch.full((2,), float("nan"), device=DEV)
    moe.clip_grad_norm(lst, max_norm, norm, moe.alloc_clip_workspace(lst), grad_scale=scale,
                       eps=eps, stream=stream)
    return norm


def check(grads, max_norm, scale=1.0, eps=1e-6, outs=None):
    total, coef, want = reference(grads, max_norm, scale, eps)
    outs = [torch.full_like(g, float("nan")) for g in grads] if outs is None else outs
    norm = run(grads, outs, max_norm, scale, eps).cpu().double()
    assert abs(float(norm[0]) - total) <= 2.0 ** -18 * total + 1e-44
    assert abs(float(norm[1]) - coef) <= 2.0 ** -17 * coef
    for o, w in zip(outs, want):
        if o is not None:
            err = (o.double().cpu() - w).abs()
            tol = (2.0 ** -8 if o.dtype is BF else 2.0 ** -16) * w.abs() + 1e-38
            assert (err <= tol).all()
    return norm


def tensors(sizes, dtypes, std=1.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * std).to(d).to(DEV) for n, d in zip(sizes, dtypes)]


# one element, round the 16-byte vector, round the 32 KB chunk, several chunks a block
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 31, 255, 2047, 2048, 8191, 8192, 8193, 16383, 16384,
                               16385, 100003, 12_345_677])
def test_one_tensor(n, dtype):
    check(tensors([n], [dtype]), 0.5)


def test_mixed_tensors_empty_ones_and_skipped_outputs():
    sizes = [0, 5, 0, 20000, 1, 16384, 0, 333333, 8, 0]
    g = tensors(sizes, [BF, F32, F32, BF, BF, F32, BF, F32, BF, F32])
    check(g, 1.0, scale=1 / 64)
    outs = [torch.full_like(t, float("nan")) if i % 2 else None for i, t in enumerate(g)]
    check(g, 1.0, outs=outs)


@pytest.mark.parametrize("n", [1, 95, 96, 97, 767, 768, 769, 1800])
def test_many_tensors(n):
    sizes = [1 + (37 * i) % 2300 for i in range(n)]
    check(tensors(sizes, [BF if i % 3 else F32 for i in range(n)]), 2.0)


@pytest.mark.parametrize("n", [63, 64, 65, 255, 256, 257, 1023, 1024, 1025, 2050])
def test_table_sizes(n):
    sizes = [1 + (41 * i) % 900 for i in range(n)]
    check(tensors(sizes, [F32 if i % 3 else BF for i in range(n)]), 2.0, scale=0.25)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_every_alignment(dtype):
    """Views at every element offset, and outputs whose 16-byte boundaries lie elsewhere."""
    g = torch.Generator().manual_seed(1)
    flat = torch.randn(400000, generator=g).to(dtype).to(DEV)
    views, outs = [], []
    out = torch.full_like(flat, float("nan"))
    for i in range(16):
        a = 20000 * i + i
        views.append(flat[a:a + 17000 + i])
        b = 20000 * i + (i if i % 2 else 3 * i + 1)
        outs.append(out[b:b + 17000 + i])
    check(views, 1.0, outs=outs)
    written = torch.zeros_like(flat, dtype=torch.bool)
    for i, o in enumerate(outs):
        b = 20000 * i + (i if i % 2 else 3 * i + 1)
        written[b:b + o.numel()] = True
    assert torch.isnan(out[~written]).all() and not torch.isnan(out[written]).any()


def test_in_place_and_no_clipping():
    g = tensors([5000, 70000], [BF, F32])
    keep = [t.clone() for t in g]
    total, coef, want = reference(keep, 1.0, 1.0, 1e-6)
    run(g, None, 1.0)
    for t, w in zip(g, want):
        assert ((t.double().cpu() - w).abs() <= 2.0 ** -8 * w.abs()).all()
    g = [t.clone() for t in keep]
    norm = run(g, None, 1e9)
    assert float(norm[1]) == 1.0 and all(torch.equal(a, b) for a, b in zip(g, keep))
    norm = run(g, None, math.inf, scale=0.5)
    assert float(norm[1]) == 1.0 and all(torch.equal(a, b * 0.5) for a, b in zip(g, keep))


def test_range():
    """Squares outside fp32: the norm itself is inside it."""
    check([torch.full((1000,), 1e25, device=DEV)], 1.0)
    check([torch.full((1000,), 1e25, device=DEV), torch.full((50000,), 3e19, device=DEV)], 1.0)
    check([torch.full((40000,), 1e-20, device=DEV)], 1e-19, eps=0.0)
    check([torch.full((40000,), 1e30, dtype=BF, device=DEV)], 1.0)
    check([torch.zeros(40000, device=DEV), torch.ones(3, dtype=BF, device=DEV)], 1.0)


def test_not_finite():
    a = torch.ones(20000, device=DEV)
    a[12345] = float("inf")
    out = torch.empty_like(a)
    norm = run([a], [out], 1.0).cpu()
    assert math.isinf(norm[0]) and norm[1] == 0.0
    out = out.cpu()
    assert math.isnan(out[12345]) and not out[:12345].any() and not out[12346:].any()
    a[12345] = float("nan")
    norm = run([a], [out.to(DEV)], 1.0).cpu()
    assert torch.isnan(norm).all()


def test_nothing_to_clip():
    norm = run([], None, 1.0).cpu()
    assert norm.tolist() == [0.0, 1.0]
    norm = run(tensors([0, 0], [BF, F32]), None, 1.0).cpu()
    assert norm.tolist() == [0.0, 1.0]


def test_reproducible_and_on_another_stream():
    g = tensors([3_000_000, 70001, 5], [BF, F32, BF])
    outs = [[torch.empty_like(t) for t in g] for _ in range(3)]
    n = [run(g, outs[0], 1.0), run(g, outs[1], 1.0)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        n.append(run(g, outs[2], 1.0))
    torch.cuda.synchronize()
    assert torch.equal(n[0], n[1]) and torch.equal(n[0], n[2])
    for a, b, c in zip(*outs):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_binding_refuses_wrong_tensors():
    a = torch.zeros(8, device=DEV)
    for grads, outs in (([a.double()], None), ([a], [a.to(BF)]), ([a], [a[:4]]),
                        ([torch.zeros(8, 8, device=DEV)[:, ::2]], None)):
        with pytest.raises(ValueError):
            moe.GradList(grads, outs)
    lst = moe.GradList([a])
    with pytest.raises(moe.MoEError):
        moe.clip_grad_norm(lst, -1.0, torch.empty(2, device=DEV), moe.alloc_clip_workspace(lst))
    with pytest.raises(ValueError):
        moe.clip_grad_norm(lst, 1.0, torch.empty(1, device=DEV), moe.alloc_clip_workspace(lst))


@pytest.mark.parametrize("value,dtype", [(1e-25, F32), (1e-30, BF), (1e-39, F32)])
def test_squares_that_vanish_in_fp32(value, dtype):
    """Every square is below fp32's smallest number, the norm is not: it is neither lost in a
    tensor of such elements nor in one that has a few of them among zeros."""
    g = torch.full((40000,), value, dtype=dtype, device=DEV)
    total, _, _ = reference([g], 1.0, 1.0, 0.0)
    check([g], total / 8, eps=0.0)
    g = torch.zeros(100003, dtype=dtype, device=DEV)
    g[[0, 77777, 100002]] = value
    check([g], value, eps=0.0)


@pytest.mark.parametrize("value", [float("inf"), float("nan"), 3e38])
def test_no_limit_and_a_norm_that_is_not_finite(value):
    """max_norm = +inf applies grad_scale and nothing else: an element that is not finite, or a
    norm beyond fp32, leaves the other gradients as they are."""
    a = torch.arange(20000, device=DEV, dtype=torch.float32)
    a[7:90] = value
    out = torch.empty_like(a)
    norm = run([a], [out], math.inf, scale=0.5).cpu()
    assert norm[1] == 1.0 and not math.isfinite(norm[0])
    assert torch.equal(out.nan_to_num(nan=-1.0), (0.5 * a).nan_to_num(nan=-1.0))
    keep = a.clone()
    norm = run([a], None, math.inf).cpu()
    assert norm[1] == 1.0 and not math.isfinite(norm[0])
    assert torch.equal(a.nan_to_num(nan=-1.0), keep.nan_to_num(nan=-1.0))

"""CPU checks of the entry points of include/moe_block.h: bad arguments are
refused on the host, before any CUDA call (no kernel is launched here)."""
import ctypes

import pytest
import torch

import mixture_experts_ffn_permute_gb300 as moe
from mixture_experts_ffn_permute_gb300 import _build

A = 1 << 20  # a 256-byte aligned address that is never dereferenced
BIG = 1 << 50


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return moe.load()


def norm(gate="none", **kw):
    fields = {k: kw.pop(k) for k in list(kw) if k in ("T", "H", "branch_dtype", "gate_kind")}
    p = moe.NormProblem.make(8, 64, gate=gate, **kw)
    for k, v in fields.items():
        setattr(p, k, v)
    return p


def norm_fwd(lib, p, **kw):
    a = dict(branch=A, w_post=A, gate=None, residual=A, w_pre=A, residual_out=A, normed=A)
    a.update(kw)
    return lib.moe_block_norm_forward(ctypes.byref(p), *a.values(), None)


def norm_bwd(lib, p, **kw):
    a = dict(branch=A, w_post=A, gate=None, residual_out=A, w_pre=A, d_residual_out=A, d_normed=A,
             d_residual=A, d_branch=A, d_w_post=A, d_gate=None, d_w_pre=A, ws=A, n=BIG)
    a.update(kw)
    return lib.moe_block_norm_backward(ctypes.byref(p), *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(H=16385), 2), (dict(branch_dtype=2), 1),
    (dict(gate_kind=4), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(ld_branch=63), 1), (dict(ld_normed=-64), 1), (dict(ld_residual=1 << 41), 1)])
def test_norm_rejects_bad_problems(lib, kw, code):
    assert norm_fwd(lib, norm(**kw)) == code
    assert norm_bwd(lib, norm(**kw)) == code
    assert lib.moe_block_norm_workspace_size(ctypes.byref(norm(**kw))) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(residual=None), 1), (dict(residual_out=None), 1), (dict(branch=None), 1),
    (dict(w_pre=None), 1), (dict(normed=None), 1), (dict(gate=A), 1),
    (dict(branch=None, residual_out=None), 1),  # a post norm without a branch
    (dict(branch=None, residual_out=None, w_post=None, w_pre=None, normed=None), 1),
    (dict(branch=A + 1), 3), (dict(w_pre=A + 1), 3), (dict(normed=A + 1), 3)])
def test_norm_forward_rejects_bad_tensors(lib, kw, code):
    assert norm_fwd(lib, norm(), **kw) == code


def test_norm_forward_rejects_missing_gate_and_in_place_strides(lib):
    assert norm_fwd(lib, norm("channel")) == 1
    assert norm_fwd(lib, norm(ld_residual=128)) == 1  # residual_out is residual, other stride
    assert lib.moe_block_norm_forward(None, *[A] * 7, None) == 1


@pytest.mark.parametrize("kw,code", [
    (dict(d_residual=None), 1), (dict(d_branch=None), 1), (dict(d_normed=None), 1),
    (dict(residual_out=None), 1), (dict(d_w_post=None), 1), (dict(d_w_pre=None), 1),
    (dict(d_gate=A), 1), (dict(ws=None), 1), (dict(ws=A + 16), 3), (dict(n=255), 4),
    (dict(d_w_post=A + 1), 3), (dict(d_residual=A + 1), 3),
    (dict(branch=None, d_branch=None), 1)])
def test_norm_backward_rejects_bad_tensors(lib, kw, code):
    assert norm_bwd(lib, norm(), **kw) == code


def test_norm_problem_rejects_unknown_options():
    with pytest.raises(ValueError):
        moe.NormProblem.make(4, 64, gate="row")
    with pytest.raises(ValueError):
        moe.NormProblem.make(4, 64, branch_dtype=torch.float16)


def test_norm_without_rows_launches_nothing(lib):
    assert norm_fwd(lib, norm(T=0), branch=None, residual=None, residual_out=None) == 0
    assert moe.last_launch_count() == 0


# ------------------------------------------------------------------ clipping
def table(*rows):
    """moe_grad_tensor rows of (grad, out, numel, dtype)."""
    t = (moe.block._GradTensor * max(1, len(rows)))()
    for e, (e.grad, e.out, e.numel, e.dtype) in zip(t, rows):
        pass
    return t


def clip(lib, rows=((A, A, 8, 0),), n=None, scale=1.0, max_norm=1.0, eps=1e-6, out=A, ws=A,
         ws_bytes=BIG):
    return lib.moe_clip_grad_norm(len(rows) if n is None else n, table(*rows), scale, max_norm,
                                  eps, out, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), 1), (dict(n=65537), 2), (dict(out=None), 1), (dict(out=A + 2), 3),
    (dict(ws=None), 1), (dict(ws=A + 128), 3), (dict(ws_bytes=256), 4), (dict(max_norm=-1.0), 1),
    (dict(max_norm=float("nan")), 1), (dict(eps=-1e-6), 1), (dict(eps=float("inf")), 1),
    (dict(scale=float("inf")), 1), (dict(rows=((A, A, 8, 2),)), 1),
    (dict(rows=((A, A, -1, 0),)), 1), (dict(rows=((None, A, 8, 0),)), 1),
    (dict(rows=((A + 1, A, 8, 0),)), 3), (dict(rows=((A, A + 2, 8, 1),)), 3),
    (dict(rows=((A, A, 1 << 43, 0),)), 2), (dict(rows=((A, A, 1 << 42, 0),) * 3), 2)])
def test_clip_rejects(lib, kw, code):
    assert clip(lib, **kw) == code


def test_clip_workspace_size(lib):
    assert lib.moe_clip_workspace_size(-1) == 0
    assert lib.moe_clip_workspace_size(65537) == 0
    assert 0 < lib.moe_clip_workspace_size(0) <= lib.moe_clip_workspace_size(65536)


def test_grad_list_refuses():
    with pytest.raises(ValueError):
        moe.GradList([torch.zeros(4)])  # not on the GPU
    with pytest.raises(ValueError):
        moe.GradList([], [None])


# ------------------------------------------------------------------ embedding
def embed(**kw):
    p = moe.EmbedProblem.make(8, 100, 64)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(V=0), 1), (dict(H=0), 1), (dict(table_dtype=5), 1),
    (dict(out_dtype=-1), 1), (dict(H=(1 << 20) + 1), 2), (dict(V=(1 << 28) + 1), 2),
    (dict(V=1 << 28, H=1 << 20), 2)])
def test_embedding_rejects_bad_problems(lib, kw, code):
    p = embed(**kw)
    assert lib.moe_embedding_forward(ctypes.byref(p), A, A, A, None, None) == code
    assert lib.moe_embedding_backward(ctypes.byref(p), A, A, A, A, BIG, None) == code
    assert lib.moe_embedding_workspace_size(ctypes.byref(p)) == 0


def test_embedding_rejects_bad_tensors(lib):
    p = ctypes.byref(embed())
    fwd, bwd = lib.moe_embedding_forward, lib.moe_embedding_backward
    for i in range(3):
        a = [A, A, A]
        a[i] = None
        assert fwd(p, *a, None, None) == 1 and bwd(p, *a, A, BIG, None) == 1
        a[i] = A + 1
        assert fwd(p, *a, None, None) == 3 and bwd(p, *a, A, BIG, None) == 3
    assert fwd(p, A, A, A, A + 4, None) == 3
    assert bwd(p, A, A, A, None, BIG, None) == 1
    assert bwd(p, A, A, A, A + 4, BIG, None) == 3
    assert bwd(p, A, A, A, A, lib.moe_embedding_workspace_size(p) - 1, None) == 4
    assert fwd(None, A, A, A, None, None) == 1


# ------------------------------------------------------------------ linear cross entropy
def ce(**kw):
    p = moe.CEProblem.make(8, 64, 100)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def ce_fwd(lib, p, **kw):
    a = dict(x=A, w=A, labels=A, loss=A, lse=A, ws=A, n=BIG)
    a.update(kw)
    return lib.moe_linear_ce_forward(ctypes.byref(p), *a.values(), None)


def ce_bwd(lib, p, **kw):
    a = dict(x=A, w=A, labels=A, lse=A, d_loss=A, d_lse=None, dx=A, dw=A, ws=A, n=BIG)
    a.update(kw)
    return lib.moe_linear_ce_backward(ctypes.byref(p), *a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(V=0), 1), (dict(logit_scale=float("nan")), 1),
    (dict(H=65), 2), (dict(H=(1 << 20) + 8), 2), (dict(V=(1 << 26) + 1), 2),
    (dict(T=1 << 26, V=1 << 26), 2)])
def test_ce_rejects_bad_problems(lib, kw, code):
    p = ce(**kw)
    assert ce_fwd(lib, p) == code and ce_bwd(lib, p) == code
    assert lib.moe_linear_ce_workspace_size(ctypes.byref(p)) == 0
    assert lib.moe_linear_ce_backward_workspace_size(ctypes.byref(p)) == 0


@pytest.mark.parametrize("name", ["x", "w", "labels", "lse"])
def test_ce_rejects_bad_tensors(lib, name):
    for f in (ce_fwd, ce_bwd):
        assert f(lib, ce(), **{name: None}) == 1
        assert f(lib, ce(), **{name: A + 2}) == 3


def test_ce_rejects_outputs_and_workspaces(lib):
    p = ce()
    assert ce_fwd(lib, p, loss=None) == 1 and ce_fwd(lib, p, loss=A + 2) == 3
    for k in ("d_loss", "dx", "dw"):
        assert ce_bwd(lib, p, **{k: None}) == 1 and ce_bwd(lib, p, **{k: A + 2}) == 3
    assert ce_bwd(lib, p, d_lse=A + 2) == 3
    for f, size in ((ce_fwd, lib.moe_linear_ce_workspace_size), (ce_bwd, None)):
        assert f(lib, p, ws=None) == 1 and f(lib, p, ws=A + 128) == 3
        assert f(lib, p, n=256) == 4
    n = lib.moe_linear_ce_workspace_size(ctypes.byref(p))
    assert ce_fwd(lib, p, n=n - 1) == 4
    # one workspace serves both directions
    assert lib.moe_linear_ce_backward_workspace_size(ctypes.byref(p)) >= n


def test_ce_workspace_does_not_hold_the_logits(lib):
    """A batch whose logits would take 17 GB in bf16."""
    p = moe.CEProblem.make(65536, 4096, 131072)
    logits = 2 * 65536 * 131072
    assert lib.moe_linear_ce_backward_workspace_size(ctypes.byref(p)) < logits / 8


def test_binding_refuses_a_gate_where_the_problem_has_none(monkeypatch):
    monkeypatch.setattr(moe.block, "_rows", lambda t, *a: None if t is None else A)
    p, r, g = norm(), torch.zeros(8, 64), torch.ones(64)
    with pytest.raises(ValueError, match="gate"):
        moe.block_norm_forward(p, r, branch=r, gate=g, residual_out=r)
    with pytest.raises(ValueError, match="gate"):
        moe.block_norm_backward(p, r, r, torch.zeros(512, dtype=torch.uint8), branch=r, d_gate=g,
                                d_branch=r)


def test_binding_refuses_workspaces_that_are_not_on_the_gpu(monkeypatch):
    """Before the library is called: the kernels would write to the host's address."""
    called = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: called.append(name) or 0

    monkeypatch.setattr(moe.block, "load", Library)
    monkeypatch.setattr(moe.block, "_raw_stream", lambda s: 0)
    for name in ("_rows", "_dense", "_gate"):
        monkeypatch.setattr(moe.block, name, lambda t, *a: None if t is None else A)
    n, e, c, t = norm(), embed(), ce(), torch.zeros(8, 64)
    grads = moe.GradList([])
    for ws in (torch.zeros(1 << 16, dtype=torch.uint8), torch.zeros(1, dtype=torch.uint8).expand(4096)):
        for f, a, kw in ((moe.block_norm_backward, (n, t, t, ws), dict(w_pre=t, d_normed=t, d_w_pre=t)),
                         (moe.clip_grad_norm, (grads, 1.0, t, ws), {}),
                         (moe.embedding_forward, (e, t, t, t, ws), {}),
                         (moe.embedding_backward, (e, t, t, t, ws), {}),
                         (moe.linear_ce_forward, (c, t, t, t, t, t, ws), {}),
                         (moe.linear_ce_backward, (c, t, t, t, t, t, t, t, ws), {})):
            with pytest.raises(ValueError, match="workspace"):
                f(*a, **kw)
    assert not called


@pytest.mark.parametrize("make", [
    lambda n: moe.NormProblem.make(n, 64), lambda n: moe.NormProblem.make(8, n),
    lambda n: moe.NormProblem.make(8, 64, ld_branch=n << 32),
    lambda n: moe.NormProblem.make(8, 64, ld_residual=n << 32),
    lambda n: moe.NormProblem.make(8, 64, ld_residual_out=n << 32),
    lambda n: moe.NormProblem.make(8, 64, ld_normed=n << 32),
    lambda n: moe.EmbedProblem.make(n, 100, 64), lambda n: moe.EmbedProblem.make(8, n, 64),
    lambda n: moe.EmbedProblem.make(8, 100, n), lambda n: moe.CEProblem.make(n, 64, 100),
    lambda n: moe.CEProblem.make(8, n, 100), lambda n: moe.CEProblem.make(8, 64, n)])
def test_problems_refuse_sizes_beyond_their_fields(make):
    """A size is not taken modulo 2^32: 2^32 + 8 rows would be 8."""
    for n in ((1 << 32) + 8, 1 << 31):
        with pytest.raises(ValueError):
            make(n)

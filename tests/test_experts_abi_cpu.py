"""CPU checks of the entry points of include/moe_experts.h: bad arguments are refused on the host,
before any CUDA call (no kernel is launched here)."""
import copy
import ctypes
import gc
import pickle
import weakref

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


def changed(p, fields):
    for k, v in fields.items():
        setattr(p, k, v)
    return ctypes.byref(p)


# ------------------------------------------------------------------ router
def router(lib, forward=True, tensors=(), **fields):
    p = changed(moe.RouterProblem.make(8, 64, 4, groups=8), fields)
    a = dict(logits=A, bias=A, idx=A, w=A) if forward else dict(logits=A, idx=A, dw=A, dl=A)
    a.update(dict(tensors))
    return (lib.moe_router_forward if forward else lib.moe_router_backward)(p, *a.values(), None)


@pytest.mark.parametrize("fields,code", [
    (dict(T=-1), 1), (dict(E=0), 1), (dict(k=0), 1), (dict(k=65), 1), (dict(logits_dtype=2), 1),
    (dict(score=2), 1), (dict(score=-1), 1), (dict(groups=0), 1), (dict(groups=7), 1),
    (dict(topk_groups=0), 1), (dict(topk_groups=9), 1), (dict(group_top=0), 1),
    (dict(group_top=3), 1), (dict(groups=64, topk_groups=64), 2), (dict(E=1032), 2),
    (dict(E=128, k=33), 2), (dict(topk_groups=1, k=9), 1), (dict(scale=float("inf")), 1),
    (dict(scale=float("nan")), 1), (dict(ld_logits=63), 1), (dict(ld_logits=-64), 1),
    (dict(ld_logits=1 << 41), 2), (dict(E=8, k=1, group_top=2), 1)])
def test_router_rejects_bad_problems(lib, fields, code):
    assert router(lib, **fields) == code
    assert router(lib, forward=False, **fields) == code


@pytest.mark.parametrize("forward", [True, False])
def test_router_rejects_bad_tensors(lib, forward):
    names = ("logits", "idx", "w") if forward else ("logits", "idx", "dw", "dl")
    for name in names:
        assert router(lib, forward, {name: None}) == 1
        assert router(lib, forward, {name: A + 2}) == 3
    assert router(lib, forward, {"logits": A + 1}, logits_dtype=0) == 3
    if forward:
        assert router(lib, forward, {"bias": A + 1}) == 3
    assert router(lib, forward, {n: None for n in names}, T=0) == 0
    assert moe.last_launch_count() == 0
    fn = lib.moe_router_forward if forward else lib.moe_router_backward
    assert fn(None, A, A, A, A, None) == 1


def test_router_problem_rejects_unknown_options():
    with pytest.raises(ValueError):
        moe.RouterProblem.make(4, 8, 2, score="tanh")
    with pytest.raises(ValueError):
        moe.RouterProblem.make(4, 8, 2, logits_dtype=torch.float16)
    with pytest.raises(ValueError):
        moe.RouterProblem.make(1 << 32, 8, 2)


# ------------------------------------------------------------------ quantisation
def rows(lib, tensors=(), **fields):
    p = changed(moe.QuantProblem.make(8, 256), fields)
    a = dict(src=A, codes=A, scales=A)
    a.update(dict(tensors))
    return lib.moe_fp8_quantize_rows(p, *a.values(), None)


@pytest.mark.parametrize("fields,code", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(H=264), 2), (dict(H=1 << 29), 2), (dict(src_dtype=2), 1),
    (dict(glu_interleave=-16), 1), (dict(swiglu=1, glu_interleave=8), 2),
    (dict(swiglu=1, glu_interleave=48), 2), (dict(ld_src=255), 1), (dict(ld_src=-256), 1),
    (dict(swiglu=1, ld_src=256), 1), (dict(ld_src=260), 2), (dict(ld_src=1 << 41), 2),
    (dict(T=(1 << 30) + 5), 2)])
def test_quantize_rows_rejects_bad_problems(lib, fields, code):
    assert rows(lib, **fields) == code


def test_quantize_rows_rejects_bad_tensors(lib):
    for name in ("src", "codes", "scales"):
        assert rows(lib, {name: None}) == 1
        assert rows(lib, {name: A + 2}) == 3
    assert rows(lib, {"src": A + 8}) == rows(lib, {"codes": A + 8}) == 3
    assert rows(lib, {n: None for n in ("src", "codes", "scales")}, T=0) == 0
    assert lib.moe_fp8_quantize_rows(None, A, A, A, None) == 1


def weights(lib, tensors=(), **fields):
    p = changed(moe.QuantWeightsProblem.make(2, 256, 384), fields)
    a = dict(src=A, codes=A, scales=A, codes_t=A, scales_t=A)
    a.update(dict(tensors))
    return lib.moe_fp8_quantize_weights(p, *a.values(), None)


@pytest.mark.parametrize("fields,code", [
    (dict(E=-1), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(src_dtype=2), 1), (dict(K=388), 2),
    (dict(N=250), 2), (dict(E=1 << 30), 2), (dict(N=1 << 30, K=1 << 30), 2)])
def test_quantize_weights_rejects_bad_problems(lib, fields, code):
    assert weights(lib, **fields) == code


def test_quantize_weights_rejects_bad_tensors(lib):
    for name in ("src", "codes", "scales", "codes_t", "scales_t"):
        assert weights(lib, {name: None}) == 1  # (one of the transposed alone as well)
        assert weights(lib, {name: A + 2}) == 3
    assert weights(lib, {n: None for n in ("src", "codes", "scales")}, E=0) == 0
    assert lib.moe_fp8_quantize_weights(None, *[A] * 5, None) == 1


# ------------------------------------------------------------------ product
def matmul(lib, tensors=(), n=BIG, **fields):
    p = changed(moe.FP8Problem.make(64, 256, 384, 4), fields)
    a = dict(x=A, xs=A, w=A, ws=A, offsets=A, out=A, work=A)
    a.update(dict(tensors))
    return lib.moe_fp8_matmul(p, *a.values(), n, None)


@pytest.mark.parametrize("fields,code", [
    (dict(M=-1), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(E=0), 1), (dict(out_dtype=2), 1),
    (dict(E=1025), 2), (dict(K=392), 2), (dict(M=(1 << 30) + 1), 2), (dict(N=(1 << 30) + 1), 2),
    (dict(K=(1 << 30) + 16), 2), (dict(M=1 << 30, N=1 << 20), 2), (dict(N=1 << 20, K=1 << 21), 2)])
def test_matmul_rejects_bad_problems(lib, fields, code):
    assert matmul(lib, **fields) == code
    p = moe.FP8Problem.make(64, 256, 384, 4)
    assert lib.moe_fp8_matmul_workspace_size(changed(p, fields)) == 0


def test_matmul_rejects_bad_tensors(lib):
    for name in ("x", "xs", "w", "ws", "out", "work"):
        assert matmul(lib, {name: None}) == 1
        assert matmul(lib, {name: A + 2}) == 3
    assert matmul(lib, {"offsets": None}) == 1  # four experts
    assert matmul(lib, {"offsets": A + 2}) == 3
    for name in ("x", "w", "out"):
        assert matmul(lib, {name: A + 8}) == 3
    assert matmul(lib, {"work": A + 128}) == 3
    assert matmul(lib, n=16) == 4
    assert matmul(lib, {n: None for n in ("x", "xs", "w", "ws", "out", "work")}, M=0) == 0
    assert lib.moe_fp8_matmul(None, *[A] * 7, BIG, None) == 1
    assert lib.moe_fp8_matmul_workspace_size(None) == 0


# ------------------------------------------------------------------ binding
def test_binding_rejects_tensors_that_are_not_the_problems():
    p = moe.RouterProblem.make(4, 8, 2)
    cpu = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        moe.router_forward(p, cpu, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    q = moe.QuantProblem.make(4, 16)
    with pytest.raises(ValueError):
        moe.fp8_quantize_rows(q, torch.zeros(4, 16), None, None)
    with pytest.raises(moe.MoEError):
        moe.alloc_fp8_matmul_workspace(moe.FP8Problem.make(4, 8, 24))
    with pytest.raises(ValueError):
        moe.FP8Experts(torch.zeros(2, 64, 256), torch.zeros(2, 256, 48), 1)


@pytest.mark.parametrize("p,field,other", [
    (moe.RouterProblem.make(8, 64, 4, scale=2.5), "E", 1032),
    (moe.QuantProblem.make(8, 256), "H", 264),
    (moe.QuantWeightsProblem.make(2, 256, 384), "K", 388),
    (moe.FP8Problem.make(64, 256, 384, 4), "K", 392)])
def test_a_copied_problem_is_the_one_that_a_call_uses(p, field, other, lib, monkeypatch):
    """A copy with a field that the library refuses: calls with it are refused, those with the
    original are not."""
    monkeypatch.setattr(moe.experts, "_dense", lambda t, *_: t)
    monkeypatch.setattr(moe.experts, "_rows", lambda t, *_: t)
    monkeypatch.setattr(moe.experts, "_codes", lambda t, *_: t)
    monkeypatch.setattr(moe.experts, "_workspace", lambda t: (t, BIG))
    monkeypatch.setattr(moe.experts, "_raw_stream", lambda s: None)
    calls = {moe.RouterProblem: [lambda q: moe.router_forward(q, None, A, A),
                                 lambda q: moe.router_backward(q, None, A, A, A)],
             moe.QuantProblem: [lambda q: moe.fp8_quantize_rows(q, A + 8, A, A)],
             moe.QuantWeightsProblem: [lambda q: moe.fp8_quantize_weights(q, A + 8, A, A)],
             moe.FP8Problem: [lambda q: moe.fp8_matmul(q, A + 8, A, A, A, A, A, expert_offsets=A)]}[type(p)]

    def status(call, q):
        with pytest.raises(moe.MoEError) as e:  # (a bad tensor: no kernel is launched)
            call(q)
        return e.value.status

    copies = [copy.copy(p), copy.deepcopy(p), pickle.loads(pickle.dumps(p))]
    for call in calls:
        want = status(call, p)
        for q in copies:
            assert bytes(q) == bytes(p) and status(call, q) == want
    for q in copies:
        setattr(q, field, other)
        for call in calls:
            assert status(call, q) == 2
            assert status(call, p) == (1 if type(p) is moe.RouterProblem else 3)


# ------------------------------------------------------------------ FP8Experts on the host
@pytest.fixture
def layer(lib, monkeypatch):
    """A layer whose kernels are records of the tensors they were given (nothing is launched)."""
    m = moe.experts
    calls = []
    for name in ("fp8_quantize_rows", "permute", "permute_rows", "fp8_matmul", "unpermute_combine"):
        monkeypatch.setattr(m, name, lambda *a, _n=name, **kw: calls.append((_n, a, kw)))
    monkeypatch.setattr(m, "_dense", lambda t, *_: t)
    monkeypatch.setattr(m, "clear_device_status", lambda ws: None)
    monkeypatch.setattr(m, "_raw_stream", lambda s=None: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    capturing = [False]
    monkeypatch.setattr(m.FP8Experts, "_quantize", staticmethod(lambda w: (w, w)))
    layer = moe.FP8Experts(torch.zeros(4, 512, 256), torch.zeros(4, 256, 256), 2)

    def call(T):
        calls.clear()
        layer(torch.zeros(T, 256), torch.zeros(T, 2, dtype=torch.int32), torch.zeros(T, 2))
        for _, args, kw in calls:  # every buffer is one of T tokens
            p = args[0]
            assert (p.T if hasattr(p, "T") else p.M) in (T, 2 * T)
            for t in (*args[1:], *kw.values()):
                if isinstance(t, torch.Tensor) and t.dim() > 1 and t.shape[0] != 4:
                    assert t.shape[0] in (T, 2 * T)
        return [t.data_ptr() for _, a, kw in calls for t in (*a[1:], *kw.values()) if isinstance(t, torch.Tensor)]

    call.layer, call.calls, call.capturing = layer, calls, capturing
    return call


@pytest.mark.parametrize("first", [False, True])
def test_a_plan_that_fails_is_not_used(layer, first, monkeypatch):
    """Memory that runs out while a plan is made: the next call makes it again, whole."""
    if not first:
        layer(8)
    real, fail_at = torch.empty, [0]

    def empty(*a, **kw):
        fail_at[0] -= 1
        if fail_at[0] == 0:
            raise torch.OutOfMemoryError("no memory left")
        return real(*a, **kw)

    monkeypatch.setattr(torch, "empty", empty)
    for n in range(1, 15):
        fail_at[0] = n
        with pytest.raises(torch.OutOfMemoryError):
            layer(32)
        fail_at[0] = 0
        layer(32)
        layer(8)



def test_rows_of_another_device_are_refused_before_a_plan(layer):
    before = layer(8)
    with pytest.raises(ValueError):
        layer.layer(torch.zeros(16, 256, device="meta"), torch.zeros(16, 2, dtype=torch.int32, device="meta"),
                    torch.zeros(16, 2, device="meta"))
    assert layer.layer._T == 8
    assert layer(8)[1:3] == before[1:3]  # (codes and scales: the plan is the same)


def test_buffers_of_a_captured_call_stay(layer):
    """Another token count frees the buffers of the one before it, but not those that a graph
    replays into."""
    def buffers():
        return [weakref.ref(t) for _, a, kw in layer.calls for t in (*a[1:], *kw.values())
                if isinstance(t, torch.Tensor) and t.dim() and any(t is b for b in vars(layer.layer).values())]

    layer(8)
    eager = buffers()
    layer.capturing[0] = True
    layer(16)
    layer.capturing[0] = False
    captured = buffers()
    layer(24)
    layer(32)
    layer.calls.clear()
    gc.collect()
    assert len(captured) > 10 and all(r() is not None for r in captured)
    weights = [layer.layer.w1, layer.layer.w2]
    assert all(r() is None or any(r() is w for w in weights) for r in eager)


def test_buffers_are_kept_for_every_stream_that_uses_them(layer, monkeypatch):
    """Calls on another stream than the one the buffers were made on say so to the allocator, which
    would else give them away, when another token count frees them, under that stream's work."""
    stream, told = [1], []
    monkeypatch.setattr(moe.experts, "_raw_stream", lambda s=None: stream[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *_: stream[0])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: told.append((t, s)))
    layer(8)
    layer(8)
    assert not told
    stream[0] = 2
    layer(8)
    used = [t for _, a, kw in layer.calls for t in (*a[1:], *kw.values()) if isinstance(t, torch.Tensor)]
    mine = [t for t in vars(layer.layer).values() if isinstance(t, torch.Tensor)]
    for t in mine:
        if any(t is u for u in used):
            assert any(t is u and s == 2 for u, s in told)
    told.clear()
    layer(8)  # (once is enough)
    assert not told
    layer(16)  # made on this stream
    assert not told
    stream[0] = 1
    layer(16)
    assert len(told) >= 14 and {s for _, s in told} == {1}


def test_the_layers_workspace_is_that_of_the_permutation(layer):
    """Of the permutation's regions alone: nothing that grows with the rows' width."""
    layer(4096)
    l = layer.layer
    routing = moe.workspace_size(moe.Problem.make(4096, 0, 0, l.E, l.k))
    assert l.ws.numel() == routing < 4096 * l.k * 100
    assert moe.workspace_size(l._p) > 4096 * l.k * (4 * l.H + 2 * l.F)


def test_buffers_made_in_a_capture_are_that_calls_alone(layer):
    """Their status words are cleared by the graph, so that no other call may read them."""
    layer.capturing[0] = True
    first = layer(8)
    second = layer(8)
    layer.capturing[0] = False
    eager = layer(8)
    again = layer(8)
    assert not set(first[1:3]) & set(second[1:3]) and not set(second[1:3]) & set(eager[1:3])
    assert eager[1:3] == again[1:3]

"""Binding of the operators around the expert layer (``include/moe_block.h``):
token embedding, the norms of a block with its gate and residual, the linear
cross entropy, and the clipping of gradients by their global norm.

As in the package's other entry points, outputs and workspaces are the
caller's tensors, work goes to the current stream (or ``stream``), and an
error status raises ``MoEError``.  Tensors that do not have the type, shape or
row stride of their problem raise ``ValueError`` before the library is called.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import MOE_OK, MoEError, load

DTYPE_BF16 = 0
DTYPE_F32 = 1
_DTYPES = {torch.bfloat16: DTYPE_BF16, torch.float32: DTYPE_F32}
GATES = {"none": 0, "channel": 1, "token": 2, "element": 3}

_vp, _sz, _ci = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int


def _dtype(d) -> int:
    if d not in _DTYPES:
        raise ValueError(f"unsupported dtype {d}: torch.bfloat16 or torch.float32")
    return _DTYPES[d]


def _sizes(*n, bits=32):
    """The sizes as integers that fit a field of so many bits (ctypes would cut them)."""
    n = tuple(int(i) for i in n)
    if any(i.bit_length() >= bits for i in n):
        raise ValueError(f"sizes {n}: beyond {bits} bits")
    return n


class NormProblem(ctypes.Structure):
    """Mirror of ``moe_norm_problem``; made with ``NormProblem.make``."""
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32),
                ("branch_dtype", ctypes.c_int32), ("residual_dtype", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("gate_kind", ctypes.c_int32),
                ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float),
                ("residual_scale", ctypes.c_float), ("branch_scale", ctypes.c_float),
                ("ld_branch", ctypes.c_int64), ("ld_residual", ctypes.c_int64),
                ("ld_residual_out", ctypes.c_int64), ("ld_normed", ctypes.c_int64)]

    @classmethod
    def make(cls, T, H, branch_dtype=torch.bfloat16, residual_dtype=torch.bfloat16,
             weight_dtype=torch.bfloat16, gate="none", eps=1e-6, weight_offset=0.0,
             residual_scale=1.0, branch_scale=1.0, ld_branch=0, ld_residual=0,
             ld_residual_out=0, ld_normed=0):
        """``gate``: "none", "channel" ([H]), "token" ([T]) or "element" ([T, H]).
        The row strides (elements) are 0 for dense rows."""
        if gate not in GATES:
            raise ValueError(f"gate must be one of {sorted(GATES)}")
        T, H = _sizes(T, H)
        lds = _sizes(ld_branch, ld_residual, ld_residual_out, ld_normed, bits=64)
        p = cls(T, H, _dtype(branch_dtype), _dtype(residual_dtype), _dtype(weight_dtype),
                GATES[gate], float(eps), float(weight_offset), float(residual_scale),
                float(branch_scale), *lds)
        p._rows, p._cols = (T, H), (H,)
        p._b, p._r, p._w = branch_dtype, residual_dtype, weight_dtype
        p._ld = tuple((ld or H, 1) for ld in lds)
        p._gate = {"none": None, "channel": (H,), "token": (T,), "element": (T, H)}[gate]
        return p


class EmbedProblem(ctypes.Structure):
    """Mirror of ``moe_embed_problem``; made with ``EmbedProblem.make``."""
    _fields_ = [("T", ctypes.c_int32), ("V", ctypes.c_int32), ("H", ctypes.c_int32),
                ("table_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("scale", ctypes.c_float)]

    @classmethod
    def make(cls, T, V, H, table_dtype=torch.bfloat16, out_dtype=torch.bfloat16, scale=1.0):
        p = cls(*_sizes(T, V, H), _dtype(table_dtype), _dtype(out_dtype), float(scale))
        p._ids, p._out, p._table = (p.T,), (p.T, p.H), (p.V, p.H)
        p._t, p._o = table_dtype, out_dtype
        return p


class CEProblem(ctypes.Structure):
    """Mirror of ``moe_ce_problem``; made with ``CEProblem.make``."""
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("V", ctypes.c_int32),
                ("logit_scale", ctypes.c_float)]

    @classmethod
    def make(cls, T, H, V, logit_scale=1.0):
        p = cls(*_sizes(T, H, V), float(logit_scale))
        p._rows, p._x, p._w = (p.T,), (p.T, p.H), (p.V, p.H)
        return p


class _GradTensor(ctypes.Structure):
    """Mirror of ``moe_grad_tensor``."""
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class GradList:
    """The gradient tensors of a model, as ``clip_grad_norm`` takes them: dense CUDA tensors of
    bf16 and fp32, and where each clipped gradient goes (``outs``; default: in place; None in the
    list: counted in the norm, not written).  It keeps the tensors alive and is made anew when
    they are replaced."""

    def __init__(self, grads, outs=None):
        self.grads = list(grads)
        self.outs = self.grads if outs is None else list(outs)
        if len(self.outs) != len(self.grads):
            raise ValueError("one output (or None) for each gradient")
        self.table = (_GradTensor * len(self.grads))()
        for e, g, o in zip(self.table, self.grads, self.outs):
            e.grad, e.numel, e.dtype = _dense(g, g.dtype, g.shape), g.numel(), _dtype(g.dtype)
            e.out = _dense(o, g.dtype, g.shape)

    def __len__(self):
        return len(self.grads)


SIGS = {
    "moe_linear_ce_workspace_size": ([_vp], _sz),
    "moe_linear_ce_backward_workspace_size": ([_vp], _sz),
    "moe_linear_ce_forward": ([_vp] * 7 + [_sz, _vp], _ci),
    "moe_linear_ce_backward": ([_vp] * 10 + [_sz, _vp], _ci),
    "moe_clip_workspace_size": ([ctypes.c_int32], _sz),
    "moe_clip_grad_norm": ([ctypes.c_int32, _vp] + [ctypes.c_float] * 3 + [_vp, _vp, _sz, _vp],
                           _ci),
    "moe_embedding_forward": ([_vp] * 6, _ci),
    "moe_embedding_workspace_size": ([_vp], _sz),
    "moe_embedding_backward": ([_vp] * 5 + [_sz, _vp], _ci),
    "moe_block_norm_forward": ([_vp] * 9, _ci),
    "moe_block_norm_workspace_size": ([_vp], _sz),
    "moe_block_norm_backward": ([_vp] * 14 + [_sz, _vp], _ci),
}


def _bad(t, what):
    raise ValueError(f"expected a CUDA tensor of {what}, got {t.dtype} {tuple(t.shape)} with "
                     f"strides {t.stride()} on {t.device}")


def _dense(t: Optional[torch.Tensor], dtype, shape):
    """The address of a dense tensor of this type and shape (None for None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda or not t.is_contiguous():
        _bad(t, f"{dtype} {tuple(shape)}, dense")
    return t.data_ptr()


def _rows(t: Optional[torch.Tensor], dtype, shape, strides):
    """The address of rows of this type, shape and stride (None for None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_cuda or t.stride() != strides:
        # the stride of a single row, or of rows of one column, says nothing
        if not (t.dtype is dtype and t.shape == shape and t.is_cuda
                and (shape[0] <= 1 or t.stride(0) == strides[0])
                and (shape[1] <= 1 or t.stride(1) == 1)):
            _bad(t, f"{dtype} {shape} with strides {strides}")
    return t.data_ptr()


def _gate(t: Optional[torch.Tensor], p):
    """The address of a gate of the problem's kind, or of its gradient (None for None)."""
    if t is not None and p._gate is None:
        raise ValueError('a gate or its gradient, for a problem of gate "none"')
    return _dense(t, p._w, p._gate)


def _workspace(ws: torch.Tensor):
    """The address and the bytes of a workspace."""
    if not (ws.is_cuda and ws.is_contiguous()):
        raise ValueError(f"expected a contiguous workspace on the GPU, got one with strides "
                         f"{ws.stride()} on {ws.device}")
    return ws.data_ptr(), ws.nbytes


# the current stream's handle without a Stream object around it (3 us of a call of 11)
_current_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw_stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _current_raw is not None:
        return _current_raw(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _ws_of(n: int, fn: str, device) -> torch.Tensor:
    """A 256-byte aligned workspace of n bytes with a cleared status word."""
    if n == 0:
        raise MoEError(fn, 1)
    ws = torch.empty(n + 256, dtype=torch.uint8, device=device)
    ws = ws[(-ws.data_ptr()) % 256:][:n]
    ws[:4].zero_()
    return ws


def block_norm_forward(p: NormProblem, residual, branch=None, w_post=None, gate=None, w_pre=None,
                       residual_out=None, normed=None, stream=None) -> None:
    """residual_out = residual_scale * residual + branch_scale * gate * rmsnorm(branch) * w_post
    and normed = rmsnorm(residual_out) * w_pre, in one pass.  Without ``w_post`` the branch is
    added unnormed; without ``branch`` only ``normed`` of the residual is computed; without
    ``w_pre`` only the residual update.  ``residual_out`` may be ``residual``."""
    b, r, ro, n = p._ld
    rc = load().moe_block_norm_forward(
        ctypes.byref(p), _rows(branch, p._b, p._rows, b), _dense(w_post, p._w, p._cols),
        _gate(gate, p), _rows(residual, p._r, p._rows, r),
        _dense(w_pre, p._w, p._cols), _rows(residual_out, p._r, p._rows, ro),
        _rows(normed, p._b, p._rows, n), _raw_stream(stream))
    if rc != MOE_OK:
        raise MoEError("moe_block_norm_forward", rc)


def alloc_block_norm_workspace(p: NormProblem, device="cuda") -> torch.Tensor:
    """The workspace of ``block_norm_backward``."""
    return _ws_of(load().moe_block_norm_workspace_size(ctypes.byref(p)),
                  "moe_block_norm_workspace_size", device)


def block_norm_backward(p: NormProblem, residual_out, d_residual, ws, branch=None, w_post=None,
                        gate=None, w_pre=None, d_normed=None, d_residual_out=None, d_branch=None,
                        d_w_post=None, d_gate=None, d_w_pre=None, stream=None) -> None:
    """Gradients of ``block_norm_forward`` from its inputs and the ``residual_out`` it stored
    (without a branch: the residual): d_residual always, d_branch, d_w_post, d_gate and d_w_pre
    for the inputs given.  ``d_residual_out`` (None: zero) is the gradient residual_out gets from
    later layers; ``d_residual`` may be the same tensor."""
    b, r, ro, n = p._ld
    rc = load().moe_block_norm_backward(
        ctypes.byref(p), _rows(branch, p._b, p._rows, b), _dense(w_post, p._w, p._cols),
        _gate(gate, p), _rows(residual_out, p._r, p._rows, ro),
        _dense(w_pre, p._w, p._cols), _rows(d_residual_out, p._r, p._rows, ro),
        _rows(d_normed, p._b, p._rows, n), _rows(d_residual, p._r, p._rows, r),
        _rows(d_branch, p._b, p._rows, b), _dense(d_w_post, p._w, p._cols),
        _gate(d_gate, p), _dense(d_w_pre, p._w, p._cols), *_workspace(ws), _raw_stream(stream))
    if rc != MOE_OK:
        raise MoEError("moe_block_norm_backward", rc)


def alloc_clip_workspace(grads: GradList, device="cuda") -> torch.Tensor:
    """The workspace of ``clip_grad_norm``."""
    return _ws_of(load().moe_clip_workspace_size(len(grads)), "moe_clip_workspace_size", device)


def clip_grad_norm(grads: GradList, max_norm: float, norm, ws, grad_scale: float = 1.0,
                   eps: float = 1e-6, stream=None) -> None:
    """Scales every gradient by ``grad_scale * min(1, max_norm / (total + eps))`` with total =
    grad_scale * their global L2 norm; ``norm`` ([2] fp32, on the GPU) gets total and the
    coefficient.  Nothing is read back to the host."""
    rc = load().moe_clip_grad_norm(len(grads.grads), ctypes.addressof(grads.table), grad_scale,
                                   max_norm, eps, _dense(norm, torch.float32, (2,)),
                                   *_workspace(ws), _raw_stream(stream))
    if rc != MOE_OK:
        raise MoEError("moe_clip_grad_norm", rc)


def embedding_forward(p: EmbedProblem, ids, table, out, ws=None, stream=None) -> None:
    """out[t] = scale * table[ids[t]] (int32 ids; a zero row where negative).  With ``ws`` (any
    workspace) an id outside the vocabulary is recorded in its status word."""
    rc = load().moe_embedding_forward(
        ctypes.byref(p), _dense(ids, torch.int32, p._ids), _dense(table, p._t, p._table),
        _dense(out, p._o, p._out), _workspace(ws)[0] if ws is not None else None,
        _raw_stream(stream))
    if rc != MOE_OK:
        raise MoEError("moe_embedding_forward", rc)


def alloc_embedding_workspace(p: EmbedProblem, device="cuda") -> torch.Tensor:
    """The workspace of ``embedding_backward``."""
    return _ws_of(load().moe_embedding_workspace_size(ctypes.byref(p)),
                  "moe_embedding_workspace_size", device)


def embedding_backward(p: EmbedProblem, ids, d_out, d_table, ws, stream=None) -> None:
    """d_table[v] = scale * sum of d_out over the tokens of id v, every row written."""
    rc = load().moe_embedding_backward(
        ctypes.byref(p), _dense(ids, torch.int32, p._ids), _dense(d_out, p._o, p._out),
        _dense(d_table, p._t, p._table), *_workspace(ws), _raw_stream(stream))
    if rc != MOE_OK:
        raise MoEError("moe_embedding_backward", rc)


def alloc_linear_ce_workspace(p: CEProblem, backward: bool = False, device="cuda") -> torch.Tensor:
    """The workspace of ``linear_ce_forward``, or of both directions."""
    fn = "moe_linear_ce_backward_workspace_size" if backward else "moe_linear_ce_workspace_size"
    return _ws_of(getattr(load(), fn)(ctypes.byref(p)), fn, device)


def linear_ce_forward(p: CEProblem, x, w, labels, loss, lse, ws, stream=None) -> None:
    """loss[t] = logsumexp_v(z) - z[labels[t]] and lse [T] fp32 of the logits z = logit_scale *
    x w^T (x [T, H], w [V, H] bf16), which are not kept.  A negative label masks its token."""
    rc = load().moe_linear_ce_forward(
        ctypes.byref(p), _dense(x, torch.bfloat16, p._x), _dense(w, torch.bfloat16, p._w),
        _dense(labels, torch.int32, p._rows), _dense(loss, torch.float32, p._rows),
        _dense(lse, torch.float32, p._rows), *_workspace(ws), _raw_stream(stream))
    if rc != MOE_OK:
        raise MoEError("moe_linear_ce_forward", rc)


def linear_ce_backward(p: CEProblem, x, w, labels, lse, d_loss, dx, dw, ws, d_lse=None,
                       stream=None) -> None:
    """dx [T, H] and dw [V, H] (bf16) from the gradients of loss and, optionally, of lse."""
    rc = load().moe_linear_ce_backward(
        ctypes.byref(p), _dense(x, torch.bfloat16, p._x), _dense(w, torch.bfloat16, p._w),
        _dense(labels, torch.int32, p._rows), _dense(lse, torch.float32, p._rows),
        _dense(d_loss, torch.float32, p._rows), _dense(d_lse, torch.float32, p._rows),
        _dense(dx, torch.bfloat16, p._x), _dense(dw, torch.bfloat16, p._w),
        *_workspace(ws), _raw_stream(stream))
    if rc != MOE_OK:
        raise MoEError("moe_linear_ce_backward", rc)


__all__ = ["NormProblem", "EmbedProblem", "CEProblem", "linear_ce_forward", "linear_ce_backward",
           "alloc_linear_ce_workspace", "GradList", "clip_grad_norm", "alloc_clip_workspace",
           "embedding_forward", "embedding_backward", "alloc_embedding_workspace", "block_norm_forward", "block_norm_backward",
           "alloc_block_norm_workspace", "DTYPE_BF16", "DTYPE_F32"]

"""Binding of the expert router and of the experts' products in 8 bits (``include/moe_experts.h``):
the router with its backward, the quantisation of rows and weights to E4M3 with a scale per block of
128, the product of the two, and ``FP8Experts``, the layer they make.

As in the package's other entry points, outputs and workspaces are the caller's tensors, work goes to
the current stream (or ``stream``), and an error status raises ``MoEError``.  Tensors that do not have
the type, shape or row stride of their problem raise ``ValueError`` before the library is called.
Codes are ``torch.float8_e4m3fn`` or ``torch.uint8`` tensors.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import (MOE_OK, MoEError, Problem, alloc_workspace, clear_device_status, load, permute,
               permute_rows, unpermute_combine)
from .block import _dense, _dtype, _raw_stream, _rows, _sizes, _workspace, _ws_of

SCORES = {"softmax": 0, "sigmoid": 1}
BLOCK = 128
_E4M3 = torch.float8_e4m3fn
_vp, _sz, _ci = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int


def _blocks(n: int) -> int:
    return -(-n // BLOCK)


class RouterProblem(ctypes.Structure):
    """Mirror of ``moe_router_problem``; made with ``RouterProblem.make``."""
    _fields_ = [("T", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("logits_dtype", ctypes.c_int32), ("score", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("topk_groups", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("scale", ctypes.c_float), ("ld_logits", ctypes.c_int64)]

    @classmethod
    def make(cls, T, E, k, logits_dtype=torch.float32, score="softmax", groups=1, topk_groups=None,
             group_top=1, renormalize=True, scale=1.0, ld_logits=0):
        """``score``: "softmax" or "sigmoid".  Of the ``groups`` the ``topk_groups`` (default: all)
        stay whose ``group_top`` (1 or 2) best experts' sum is highest.  The row stride (elements)
        is 0 for dense rows."""
        if score not in SCORES:
            raise ValueError(f"score must be one of {sorted(SCORES)}")
        T, E, k, groups, group_top = _sizes(T, E, k, groups, group_top)
        topk_groups, = _sizes(groups if topk_groups is None else topk_groups)
        ld, = _sizes(ld_logits, bits=64)
        p = cls(T, E, k, _dtype(logits_dtype), SCORES[score], groups, topk_groups, group_top,
                int(bool(renormalize)), float(scale), ld)
        p._l, p._rows, p._ld = logits_dtype, (T, E), (ld or E, 1)
        p._bias, p._topk = (E,), (T, k)
        return p


class QuantProblem(ctypes.Structure):
    """Mirror of ``moe_quant_problem``; made with ``QuantProblem.make``."""
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("src_dtype", ctypes.c_int32),
                ("swiglu", ctypes.c_int32), ("glu_interleave", ctypes.c_int32),
                ("swiglu_clamp", ctypes.c_float), ("ld_src", ctypes.c_int64)]

    @classmethod
    def make(cls, T, H, src_dtype=torch.bfloat16, swiglu=False, glu_interleave=0, swiglu_clamp=0.0,
             ld_src=0):
        """Codes [T, H] of rows [T, H], or with ``swiglu`` of rows [T, 2 H] of pre-activations."""
        T, H, glu_interleave = _sizes(T, H, glu_interleave)
        ld, = _sizes(ld_src, bits=64)
        p = cls(T, H, _dtype(src_dtype), int(bool(swiglu)), glu_interleave, float(swiglu_clamp), ld)
        width = 2 * H if swiglu else H
        p._s, p._src, p._ld = src_dtype, (T, width), (ld or width, 1)
        p._codes, p._scales = (T, H), (T, _blocks(H))
        return p


class QuantWeightsProblem(ctypes.Structure):
    """Mirror of ``moe_quant_weights_problem``; made with ``QuantWeightsProblem.make``."""
    _fields_ = [("E", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("src_dtype", ctypes.c_int32)]

    @classmethod
    def make(cls, E, N, K, src_dtype=torch.bfloat16):
        E, N, K = _sizes(E, N, K)
        p = cls(E, N, K, _dtype(src_dtype))
        p._s, p._codes, p._codes_t = src_dtype, (E, N, K), (E, K, N)
        p._scales, p._scales_t = (E, _blocks(N), _blocks(K)), (E, _blocks(K), _blocks(N))
        return p


class FP8Problem(ctypes.Structure):
    """Mirror of ``moe_fp8_problem``; made with ``FP8Problem.make``."""
    _fields_ = [("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("E", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]

    @classmethod
    def make(cls, M, N, K, E=1, out_dtype=torch.bfloat16):
        M, N, K, E = _sizes(M, N, K, E)
        p = cls(M, N, K, E, _dtype(out_dtype))
        p._o, p._out, p._x, p._xs = out_dtype, (M, N), (M, K), (M, _blocks(K))
        p._w, p._ws, p._offsets = (E, N, K), (E, _blocks(N), _blocks(K)), (E + 1,)
        return p


SIGS = {
    "moe_router_forward": ([_vp] * 6, _ci),
    "moe_router_backward": ([_vp] * 6, _ci),
    "moe_fp8_quantize_rows": ([_vp] * 5, _ci),
    "moe_fp8_quantize_weights": ([_vp] * 7, _ci),
    "moe_fp8_matmul_workspace_size": ([_vp], _sz),
    "moe_fp8_matmul": ([_vp] * 8 + [_sz, _vp], _ci),
}


def _codes(t: Optional[torch.Tensor], shape):
    """The address of a dense tensor of E4M3 codes (None for None)."""
    return _dense(t, torch.uint8 if t is not None and t.dtype is torch.uint8 else _E4M3, shape)


def router_forward(p: RouterProblem, logits, topk_idx, topk_w, bias=None, stream=None) -> None:
    """topk_idx [T, k] int32 and topk_w [T, k] fp32 of logits [T, E]: the experts of the highest
    score plus ``bias`` ([E] fp32), best first, ties to the lowest id; weights of the scores alone.
    Slots for which no expert is left (logits of -inf) get -1 and 0."""
    rc = load().moe_router_forward(
        ctypes.byref(p), _rows(logits, p._l, p._rows, p._ld),
        _dense(bias, torch.float32, p._bias), _dense(topk_idx, torch.int32, p._topk),
        _dense(topk_w, torch.float32, p._topk), _raw_stream(stream))
    if rc != MOE_OK:
        raise MoEError("moe_router_forward", rc)


def router_backward(p: RouterProblem, logits, topk_idx, d_topk_w, d_logits, stream=None) -> None:
    """d_logits [T, E] (of the logits' type and strides) from the gradients of topk_w."""
    rc = load().moe_router_backward(
        ctypes.byref(p), _rows(logits, p._l, p._rows, p._ld),
        _dense(topk_idx, torch.int32, p._topk), _dense(d_topk_w, torch.float32, p._topk),
        _rows(d_logits, p._l, p._rows, p._ld), _raw_stream(stream))
    if rc != MOE_OK:
        raise MoEError("moe_router_backward", rc)


def fp8_quantize_rows(p: QuantProblem, src, codes, scales, stream=None) -> None:
    """codes [T, H] E4M3 and scales [T, ceil(H / 128)] fp32 of the rows of src, or of the SwiGLU of
    their gate and up values: scale = max |v| / 448 of every 128 values, code = v / scale."""
    rc = load().moe_fp8_quantize_rows(
        ctypes.byref(p), _rows(src, p._s, p._src, p._ld), _codes(codes, p._codes),
        _dense(scales, torch.float32, p._scales), _raw_stream(stream))
    if rc != MOE_OK:
        raise MoEError("moe_fp8_quantize_rows", rc)


def fp8_quantize_weights(p: QuantWeightsProblem, src, codes, scales, codes_t=None, scales_t=None,
                         stream=None) -> None:
    """codes [E, N, K] E4M3 and scales [E, ceil(N / 128), ceil(K / 128)] fp32 of src [E, N, K], a
    scale for every 128 x 128; ``codes_t`` and ``scales_t`` get the same blocks transposed."""
    rc = load().moe_fp8_quantize_weights(
        ctypes.byref(p), _dense(src, p._s, p._codes), _codes(codes, p._codes),
        _dense(scales, torch.float32, p._scales), _codes(codes_t, p._codes_t),
        _dense(scales_t, torch.float32, p._scales_t), _raw_stream(stream))
    if rc != MOE_OK:
        raise MoEError("moe_fp8_quantize_weights", rc)


def alloc_fp8_matmul_workspace(p: FP8Problem, device="cuda") -> torch.Tensor:
    """The workspace of ``fp8_matmul``."""
    return _ws_of(load().moe_fp8_matmul_workspace_size(ctypes.byref(p)),
                  "moe_fp8_matmul_workspace_size", device)


def fp8_matmul(p: FP8Problem, x, x_scale, w, w_scale, out, ws, expert_offsets=None,
               stream=None) -> None:
    """out[r] = (x[r] * x_scale[r]) (w[e] * w_scale[e])^T for the rows r of every expert e, which
    are expert_offsets[e] .. expert_offsets[e + 1] (int32 [E + 1]; None: one expert has them all).
    Rows of out that are no expert's are left as they were."""
    rc = load().moe_fp8_matmul(
        ctypes.byref(p), _codes(x, p._x), _dense(x_scale, torch.float32, p._xs), _codes(w, p._w),
        _dense(w_scale, torch.float32, p._ws), _dense(expert_offsets, torch.int32, p._offsets),
        _dense(out, p._o, p._out), *_workspace(ws), _raw_stream(stream))
    if rc != MOE_OK:
        raise MoEError("moe_fp8_matmul", rc)


class FP8Experts:
    """Convenience holder: the experts' weights in 8 bits (quantised here from ``w1`` [E, 2F, H] and
    ``w2`` [E, H, F], bf16 or fp32) and the reusable workspaces of one token count.  A call runs the
    layer of given routing on bf16 rows: quantise, permute, first product, SwiGLU and quantise,
    second product, weighted sum.  H is a multiple of 256 and F one of 128, as the layer's are; the
    workspaces are its own, so one call runs at a time.  A call of another token count takes new
    ones; those of calls that a graph has captured stay as long as the layer, for its replays.  (A
    captured call that no eager one of its token count came before has buffers of its own.)
    ``get_device_status`` of ``ws`` tells of ids beyond the experts, of ``ws_matmul`` of products
    that did not finish."""

    def __init__(self, w1: torch.Tensor, w2: torch.Tensor, k: int, glu_interleave=0,
                 swiglu_clamp=0.0):
        E, twoF, H = w1.shape
        self.E, self.F, self.H, self.k = E, twoF // 2, H, k
        if w1.shape != (E, 2 * self.F, H) or w2.shape != (E, H, self.F):
            raise ValueError(f"expected w1 [E, 2F, H] and w2 [E, H, F], got {tuple(w1.shape)} and "
                             f"{tuple(w2.shape)}")
        self.glu_interleave, self.swiglu_clamp = glu_interleave, swiglu_clamp
        self.w1, self.s1 = self._quantize(w1)
        self.w2, self.s2 = self._quantize(w2)
        self._T = -1
        self._captured, self._made_captured, self._kept = False, False, []

    @staticmethod
    def _quantize(w):
        p = QuantWeightsProblem.make(*w.shape, src_dtype=w.dtype)
        codes = torch.empty(w.shape, dtype=_E4M3, device=w.device)
        scales = torch.empty(p._scales, device=w.device)
        fp8_quantize_weights(p, w, codes, scales)
        return codes, scales

    def _plan(self, T, dev):
        H, F, E, R = self.H, self.F, self.E, T * self.k

        def empty(*shape, dtype=torch.int32):
            return torch.empty(*shape, dtype=dtype, device=dev)

        self._T = -1  # no plan until all of it is there: an allocation may fail
        if self._captured:  # a graph's replays write to the buffers
            self._kept.append(self._tensors())
            self._captured = False
        self._p = Problem.make(T, H, F, E, self.k)
        self._p_in = QuantProblem.make(T, H)
        self._p_h = QuantProblem.make(R, F, swiglu=True, glu_interleave=self.glu_interleave,
                                      swiglu_clamp=self.swiglu_clamp)
        self._p1, self._p2 = FP8Problem.make(R, 2 * F, H, E), FP8Problem.make(R, H, F, E)
        self._x, self._xs = empty(T, H, dtype=_E4M3), empty(T, _blocks(H), dtype=torch.float32)
        self._xp, self._xps = empty(R, H, dtype=_E4M3), empty(R, _blocks(H), dtype=torch.float32)
        self._a, self._y = (empty(R, n, dtype=torch.bfloat16) for n in (2 * F, H))
        self._h, self._hs = empty(R, F, dtype=_E4M3), empty(R, _blocks(F), dtype=torch.float32)
        self._row_id, self._token = empty(T, self.k), empty(R)
        self.tokens_per_expert, self._offsets = empty(E), empty(E + 1)
        # of the permutation, which uses none that goes with the rows' width
        self.ws = alloc_workspace(Problem.make(T, 0, 0, E, self.k), dev)
        clear_device_status(self.ws)
        self.ws_matmul = alloc_fp8_matmul_workspace(self._p1, dev)
        self._T, self._streams = T, {_raw_stream(None)}

    def _tensors(self):
        return [t for t in vars(self).values() if isinstance(t, torch.Tensor)]

    def __call__(self, x: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
        """out [T, H] bf16 for x [T, H] bf16 and the routing that ``router_forward`` writes."""
        T = x.shape[0]
        if x.device != self.w1.device:
            raise ValueError(f"expected rows on the weights' {self.w1.device}, got {x.device}")
        if out is None:
            out = torch.empty_like(x)
        if T == 0:
            return out
        _dense(topk_idx, torch.int32, (T, self.k))
        _dense(topk_w, torch.float32, (T, self.k))
        _dense(out, torch.bfloat16, (T, self.H))
        capturing = torch.cuda.is_current_stream_capturing()
        if T != self._T or self._made_captured:
            self._plan(T, x.device)
            self._made_captured = capturing  # the graph clears the status words: no other call's
        stream = _raw_stream(None)
        if stream not in self._streams:  # (the allocator knows of the one they were made on)
            for t in self._tensors():
                t.record_stream(torch.cuda.current_stream())
            self._streams.add(stream)
        self._captured |= capturing
        fp8_quantize_rows(self._p_in, x, self._x, self._xs)
        permute(self._p, topk_idx, None, None, self._row_id, self._token, self.tokens_per_expert,
                self._offsets, self.ws)
        permute_rows(self._p, self._token, self._x, self._xp)
        permute_rows(self._p, self._token, self._xs, self._xps)
        fp8_matmul(self._p1, self._xp, self._xps, self.w1, self.s1, self._a, self.ws_matmul,
                   expert_offsets=self._offsets)
        fp8_quantize_rows(self._p_h, self._a, self._h, self._hs)
        fp8_matmul(self._p2, self._h, self._hs, self.w2, self.s2, self._y, self.ws_matmul,
                   expert_offsets=self._offsets)
        unpermute_combine(self._p, self._y, self._row_id, topk_w, out)
        return out


__all__ = ["RouterProblem", "QuantProblem", "QuantWeightsProblem", "FP8Problem", "router_forward",
           "router_backward", "fp8_quantize_rows", "fp8_quantize_weights", "fp8_matmul",
           "alloc_fp8_matmul_workspace", "FP8Experts"]

"""The operators around the expert products (second half of include/moe.h): routing rows to
experts and back with gradients, 8-bit activation checkpoints and the SwiGLU that uses them,
low-rank adapters of many requests.

As in ``api.py`` nothing here computes: tensors are checked and marshalled, in C++
(``bind/ops_bind.cpp``), because a decode step's kernels take less time than these checks do
in Python.  Matrices are cuda tensors [rows, columns] with contiguous rows (any row pitch,
offset or slice of columns); all tensors of a call live on one device, which need not be the
current one.  Outputs may be given; otherwise they are allocated on the stream of the call.
Outputs must not overlap inputs unless a call says so.  Calls run asynchronously on ``stream``
(default: the device's current stream) and can be captured into a CUDA graph.  A tensor that
does not fit raises ValueError, what the C ABI refuses MoeError.  The operators record
nothing for autograd: each gradient is a call of its own, and where autograd would record, a
tensor that takes part in a gradient raises ValueError (call under ``torch.no_grad()``, or in
a ``torch.autograd.Function`` that makes both calls).
"""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass

import torch

from . import _lib, _moe_ops
from ._lib import MoeError, check

_moe_ops.set_error(MoeError)

GROUP = 32  # columns of an 8-bit checkpoint that share a scale


# ------------------------------------------------------------------ routes
@dataclass
class Routes:
    """T*k entries sorted by group (expert or adapter), as moe_sort makes them."""
    T: int
    k: int
    E: int
    perm: torch.Tensor     # int32 [T*k]: row -> entry t*k+j; dropped entries behind the groups
    inv: torch.Tensor      # int32 [T*k]: entry -> row, -1 if dropped
    offsets: torch.Tensor  # int32 [E+1]: first row of each group; offsets[E] = rows with a group


def alloc_routes(T: int, k: int, E: int, device=None) -> Routes:
    """Memory for the routes of T tokens with k entries each in E groups."""
    p, i, o = (torch.empty(n, dtype=torch.int32, device=device or "cuda") for n in (T * k, T * k, E + 1))
    return Routes(T, k, E, p, i, o)


def sort_workspace_bytes(T: int, k: int, E: int) -> int:
    """Bytes of ws that moe_sort and moe_dispatch need (0: none)."""
    need = C.c_uint64(0)
    check("moe_sort(workspace query)", _lib.load().moe_sort(None, T, k, E, None, None, None, None, 0, C.byref(need), None))
    return need.value


def _given(routes: Routes | None, idx: torch.Tensor, E: int) -> tuple:
    if routes is None:
        return None, None, None
    T, k = idx.shape if idx.dim() == 2 else (idx.shape[0], 1)
    if routes.T != T or routes.k != k or routes.E != E:
        raise ValueError(f"routes are for {(routes.T, routes.k, routes.E)} tokens, entries and groups, need {(T, k, E)}")
    return routes.perm, routes.inv, routes.offsets


def _made(idx: torch.Tensor, E: int, made: tuple) -> Routes:
    return Routes(idx.shape[0], idx.shape[1] if idx.dim() == 2 else 1, E, *made)


def moe_sort(idx: torch.Tensor, E: int, routes: Routes | None = None, ws: torch.Tensor | None = None,
             stream: torch.cuda.Stream | None = None) -> Routes:
    """Entries of idx (cuda int32 [T, k] or [T]) sorted by group; values outside [0, E) are
    dropped.  The sort is stable."""
    made = _moe_ops.sort(idx, E, *_given(routes, idx, E), ws, stream)
    return _made(idx, E, made) if routes is None else routes


def moe_dispatch(x: torch.Tensor, idx: torch.Tensor, E: int, xs: torch.Tensor | None = None,
                 routes: Routes | None = None, ws: torch.Tensor | None = None,
                 stream: torch.cuda.Stream | None = None) -> tuple[torch.Tensor, Routes]:
    """Rows of x [T, H] sorted by expert: (xs [T*k, H], routes).  Rows of xs from
    routes.offsets[E] on are not written."""
    xs, made = _moe_ops.dispatch(x, idx, E, xs, *_given(routes, idx, E), ws, stream)
    return xs, _made(idx, E, made) if routes is None else routes


def moe_dispatch_backward(dxs: torch.Tensor, routes: Routes, dx: torch.Tensor | None = None,
                          stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """dx [T, H]: the sum of each token's rows of dxs [T*k, H]."""
    return _moe_ops.dispatch_backward(dxs, None, routes.inv, routes.T, routes.k, dx, stream)


def moe_collect(o: torch.Tensor, w: torch.Tensor, routes: Routes, y: torch.Tensor | None = None,
                stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """y [T, H]: each token's rows of o [T*k, H] summed with the weights w (float32 [T, k])."""
    return _moe_ops.collect(o, w, routes.inv, routes.T, routes.k, y, stream)


def moe_collect_backward(dy: torch.Tensor, o: torch.Tensor, w: torch.Tensor, routes: Routes,
                         do: torch.Tensor | None = None, dw: torch.Tensor | None = None,
                         stream: torch.cuda.Stream | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Gradients (do [T*k, H], dw float32 [T, k]) of moe_collect.  Rows of do from
    routes.offsets[E] on are not written; dw is 0 for dropped entries."""
    return _moe_ops.collect_backward(dy, o, w, routes.inv, routes.T, routes.k, do, dw, stream)


# ------------------------------------------------------------------ 8-bit checkpoints
class ActCkpt:
    """A matrix [R, F] of activations in 8 bits: values codes * 2**(exps - 127), one exponent
    per row and 32 columns (255: the group held an infinity or a NaN).

    codes: int8 [R, F]; exps: uint8 [R, ceil(F/32)]; dtype: type of the saved values.
    A checkpoint that an operator allocates is one piece of memory (the codes, then from the
    next multiple of 256 bytes on the exponents), of which codes and exps are views."""

    __slots__ = ("handle", "dtype")  # handle: (memory or codes, offset, None or exps, R, F)

    def __init__(self, codes: torch.Tensor, exps: torch.Tensor, dtype: torch.dtype):
        if codes.dim() != 2 or codes.dtype is not torch.int8 or not codes.is_contiguous():
            raise ValueError(f"codes must be a contiguous int8 matrix, got {codes.dtype} {list(codes.shape)}")
        R, F = codes.shape
        if tuple(exps.shape) != (R, -(-F // GROUP)) or exps.dtype is not torch.uint8 or not exps.is_contiguous() \
                or exps.device != codes.device:
            raise ValueError(f"exps must be a contiguous uint8 tensor {[R, -(-F // GROUP)]} on {codes.device}, "
                             f"got {exps.dtype} {list(exps.shape)} on {exps.device}")
        self.handle = (codes, 0, exps, R, F)
        self.dtype = dtype

    @staticmethod
    def _bytes(R: int, F: int) -> tuple[int, int]:
        """Offset of the exponents behind the codes, and the whole size."""
        e = (R * F + 255) // 256 * 256
        return e, e + (R * -(-F // GROUP) + 255) // 256 * 256

    @classmethod
    def _of(cls, handle: tuple, dtype: torch.dtype) -> "ActCkpt":
        k = cls.__new__(cls)
        k.handle = handle
        k.dtype = dtype
        return k

    @property
    def shape(self) -> tuple[int, int]:
        return self.handle[3:]

    @property
    def codes(self) -> torch.Tensor:
        mem, at, exps, R, F = self.handle
        return mem if exps is not None else mem[at:at + R * F].view(torch.int8).view(R, F)

    @property
    def exps(self) -> torch.Tensor:
        mem, at, exps, R, F = self.handle
        if exps is not None:
            return exps
        at, G = at + self._bytes(R, F)[0], -(-F // GROUP)
        return mem[at:at + R * G].view(R, G)


class SwigluCkpt:
    """What moe_swiglu_backward needs: the checkpoints of g and u."""

    __slots__ = ("handles", "dtype")

    def __init__(self, g: ActCkpt, u: ActCkpt):
        if g.dtype is not u.dtype:
            raise ValueError(f"g and u are of one type, got {g.dtype} and {u.dtype}")
        self.handles = (g.handle, u.handle)
        self.dtype = g.dtype

    @property
    def g(self) -> ActCkpt:
        return ActCkpt._of(self.handles[0], self.dtype)

    @property
    def u(self) -> ActCkpt:
        return ActCkpt._of(self.handles[1], self.dtype)


def alloc_ckpt(R: int, F: int, dtype: torch.dtype, device=None) -> ActCkpt:
    """Memory for the 8-bit checkpoint of a matrix [R, F] of dtype."""
    mem = torch.empty(ActCkpt._bytes(R, F)[1], dtype=torch.uint8, device=device or "cuda")
    return ActCkpt._of((mem, 0, None, R, F), dtype)


def _same_type(ckpt: ActCkpt | SwigluCkpt, t: torch.Tensor) -> None:
    if ckpt.dtype is not t.dtype:
        raise ValueError(f"the checkpoint is for {ckpt.dtype}, the values are {t.dtype}")


def moe_act_save(x: torch.Tensor, ckpt: ActCkpt | None = None, rows: torch.Tensor | None = None,
                 stream: torch.cuda.Stream | None = None) -> ActCkpt:
    """x [R, F] kept in 8 bits.  rows: cuda int32 [1], only rows below it are read and
    written (routes.offsets[E:] after a dispatch)."""
    if ckpt is None:
        return ActCkpt._of(_moe_ops.act_save(x, None, rows, stream), x.dtype)
    _same_type(ckpt, x)
    _moe_ops.act_save(x, ckpt.handle, rows, stream)
    return ckpt


def moe_act_load(ckpt: ActCkpt, x: torch.Tensor | None = None, rows: torch.Tensor | None = None,
                 stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The restored matrix, in the type that was saved or in that of x."""
    return _moe_ops.act_load(ckpt.handle, ckpt.dtype, x, rows, stream)


def moe_swiglu_save(g: torch.Tensor, u: torch.Tensor, h: torch.Tensor | None = None, ckpt: SwigluCkpt | None = None,
                    rows: torch.Tensor | None = None,
                    stream: torch.cuda.Stream | None = None) -> tuple[torch.Tensor, SwigluCkpt]:
    """h = silu(g) * u and the 8-bit checkpoint of g and u that moe_swiglu_backward needs."""
    if ckpt is None:
        ckpt = SwigluCkpt.__new__(SwigluCkpt)
        h, ckpt.handles = _moe_ops.swiglu_save(g, u, h, None, rows, stream)
        ckpt.dtype = g.dtype
        return h, ckpt
    _same_type(ckpt, g)
    return _moe_ops.swiglu_save(g, u, h, ckpt.handles, rows, stream)[0], ckpt


def moe_swiglu_backward(dh: torch.Tensor, ckpt: SwigluCkpt, dg: torch.Tensor | None = None,
                        du: torch.Tensor | None = None, h: torch.Tensor | None = None, rebuild_h: bool = False,
                        rows: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None
                        ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor | None]:
    """(dg, du, h) from dh and the checkpoint, all of dh's type; h, the activation again, only
    if it is given or rebuild_h is set."""
    return _moe_ops.swiglu_backward(dh, ckpt.handles, dg, du, h, rebuild_h, rows, stream)


# ------------------------------------------------------------------ adapters
def moe_adapters(x: torch.Tensor, y: torch.Tensor, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor,
                 routes: Routes, out: torch.Tensor | None = None, status: torch.Tensor | None = None,
                 stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """out = y + scale[a] * B[a] (A[a] x) for each token's adapter a (none: out = y).

    x [T, K], y and out [T, N] (out may be y), A [n, r, K] and B [n, N, r] contiguous, all
    bfloat16 or all float16; scale float32 [n]; routes = moe_sort(adapter of each token, n),
    -1 for none.  status: int32 [1], zeroed by the caller, gets MOE_ERR_TIMEOUT if a bounded
    wait of the kernel gave up (out is undefined then)."""
    return _moe_ops.adapters(x, y, A, B, scale, routes.perm, routes.inv, routes.offsets, routes.T, routes.k, routes.E,
                             out, status, stream)


__all__ = ["ActCkpt", "Routes", "SwigluCkpt", "alloc_ckpt", "alloc_routes", "moe_act_load", "moe_act_save",
           "moe_adapters", "moe_collect", "moe_collect_backward", "moe_dispatch", "moe_dispatch_backward",
           "moe_sort", "moe_swiglu_backward", "moe_swiglu_save", "sort_workspace_bytes"]

"""Python binding of the operators around the expert products (second half of
include/moe.h): routing rows to experts and back with gradients, 8-bit activation
checkpoints and the SwiGLU that uses them, low-rank adapters of many requests.

As in ``api.py`` nothing here computes: tensors are checked and marshalled.  Matrices are
cuda tensors [rows, columns] with contiguous rows (any row pitch, offset or slice of
columns); all tensors of a call live on one device, which need not be the current one.
Outputs may be given; otherwise they are allocated on the stream of the call.  Calls run
asynchronously on ``stream`` (default: the device's current stream) and can be captured
into a CUDA graph.
"""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import check

_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
GROUP = 32  # columns of an 8-bit checkpoint that share a scale


class _Call:
    """Device and stream of one call, taken from its first tensor."""

    __slots__ = ("device", "stream", "raw", "other")

    def __init__(self, t: torch.Tensor, stream: torch.cuda.Stream | None):
        if not t.is_cuda:
            raise ValueError("operands must be cuda tensors")
        self.device = t.device
        self.other = torch.cuda.current_device() != t.device.index
        self.stream = stream
        if stream is not None and stream.device != t.device:
            raise ValueError(f"the stream is on {stream.device}, the operands on {t.device}")
        self.raw = (stream or torch.cuda.current_stream(t.device)).cuda_stream

    def empty(self, shape, dtype) -> torch.Tensor:
        # on the stream of the call, so that the allocator does not hand the memory on early
        if self.stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(self.stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def run(self, fn, *args) -> None:
        if self.other:
            with torch.cuda.device(self.device):
                check(fn.__name__, fn(*args, self.raw))
        else:
            check(fn.__name__, fn(*args, self.raw))

    def workspace(self, fn, *args) -> torch.Tensor:
        need = C.c_uint64(0)
        check(f"{fn.__name__}(workspace query)", fn(*args, C.byref(need), None))
        return self.empty((need.value,), torch.uint8)

    def rows(self, t: torch.Tensor, name: str, R: int, F: int, dtype) -> tuple[int, int]:
        """Pointer and pitch of a matrix [R, F] with contiguous rows."""
        if t.dtype is not dtype or t.device != self.device or t.shape != (R, F):
            raise ValueError(f"{name} must be a {dtype} tensor {[R, F]} on {self.device}, got {t.dtype} "
                             f"{list(t.shape)} on {t.device}")
        ld, step = t.stride()
        if step != 1 and F > 1:
            raise ValueError(f"{name} must have contiguous rows, got strides {t.stride()}")
        return t.data_ptr(), (ld if R > 1 else F)

    def flat(self, t: torch.Tensor, name: str, count: int, dtype) -> int:
        if t.dtype is not dtype or t.device != self.device or t.numel() != count or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of {count} values on {self.device}, got "
                             f"{t.dtype} {list(t.shape)} on {t.device}")
        return t.data_ptr()


def _values(t: torch.Tensor, name: str) -> torch.dtype:
    if t.dtype not in _DTYPE:
        raise ValueError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, got {list(t.shape)}")
    return t.dtype


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


def _routes(c: _Call, r: Routes) -> tuple[int, int, int]:
    R = r.T * r.k
    return (c.flat(r.perm, "perm", R, torch.int32), c.flat(r.inv, "inv", R, torch.int32),
            c.flat(r.offsets, "offsets", r.E + 1, torch.int32))


def _new_routes(c: _Call, T: int, k: int, E: int, routes: Routes | None) -> Routes:
    if routes is None:
        R = T * k
        buf = c.empty((2 * R + max(E, 0) + 1,), torch.int32)
        return Routes(T, k, E, buf[:R], buf[R:2 * R], buf[2 * R:])
    if (routes.T, routes.k, routes.E) != (T, k, E):
        raise ValueError(f"routes are for {(routes.T, routes.k, routes.E)} tokens, entries and groups, need {(T, k, E)}")
    return routes


def _index(idx: torch.Tensor) -> tuple[int, int]:
    if idx.dim() not in (1, 2):
        raise ValueError(f"idx must be [T] or [T, k], got {list(idx.shape)}")
    return idx.shape[0], idx.shape[1] if idx.dim() == 2 else 1


def moe_sort(idx: torch.Tensor, E: int, routes: Routes | None = None, ws: torch.Tensor | None = None,
             stream: torch.cuda.Stream | None = None) -> Routes:
    """Entries of idx (cuda int32 [T, k] or [T]) sorted by group; values outside [0, E) are
    dropped.  The sort is stable."""
    c = _Call(idx, stream)
    T, k = _index(idx)
    ip = c.flat(idx, "idx", T * k, torch.int32)
    routes = _new_routes(c, T, k, E, routes)
    r = _routes(c, routes)
    fn = _lib.load().moe_sort
    if ws is None:
        ws = c.workspace(fn, None, T, k, E, None, None, None, None, 0)
    c.run(fn, ip, T, k, E, *r, ws.data_ptr(), ws.numel(), None)
    return routes


def moe_dispatch(x: torch.Tensor, idx: torch.Tensor, E: int, xs: torch.Tensor | None = None,
                 routes: Routes | None = None, ws: torch.Tensor | None = None,
                 stream: torch.cuda.Stream | None = None) -> tuple[torch.Tensor, Routes]:
    """Rows of x [T, H] sorted by expert: (xs [T*k, H], routes).  Rows of xs from
    routes.offsets[E] on are not written."""
    c = _Call(x, stream)
    dt = _values(x, "x")
    T, k = _index(idx)
    H = x.shape[1]
    xp, ldx = c.rows(x, "x", T, H, dt)
    ip = c.flat(idx, "idx", T * k, torch.int32)
    routes = _new_routes(c, T, k, E, routes)
    r = _routes(c, routes)
    if xs is None:
        xs = c.empty((T * k, H), dt)
    xsp, ldxs = c.rows(xs, "xs", T * k, H, dt)
    fn = _lib.load().moe_dispatch
    if ws is None:
        ws = c.workspace(fn, None, ldx, _DTYPE[dt], None, T, k, E, H, None, ldxs, None, None, None, None, 0)
    c.run(fn, xp, ldx, _DTYPE[dt], ip, T, k, E, H, xsp, ldxs, *r, ws.data_ptr(), ws.numel(), None)
    return xs, routes


def moe_dispatch_backward(dxs: torch.Tensor, routes: Routes, dx: torch.Tensor | None = None,
                          stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """dx [T, H]: the sum of each token's rows of dxs [T*k, H]."""
    c = _Call(dxs, stream)
    dt = _values(dxs, "dxs")
    T, k, H = routes.T, routes.k, dxs.shape[1]
    dp, ldd = c.rows(dxs, "dxs", T * k, H, dt)
    if dx is None:
        dx = c.empty((T, H), dt)
    xp, ldx = c.rows(dx, "dx", T, H, dt)
    c.run(_lib.load().moe_dispatch_backward, dp, ldd, _DTYPE[dt], c.flat(routes.inv, "inv", T * k, torch.int32), T, k, H,
          xp, ldx)
    return dx


def moe_collect(o: torch.Tensor, w: torch.Tensor, routes: Routes, y: torch.Tensor | None = None,
                stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """y [T, H]: each token's rows of o [T*k, H] summed with the weights w (float32 [T, k])."""
    c = _Call(o, stream)
    dt = _values(o, "o")
    T, k, H = routes.T, routes.k, o.shape[1]
    op, ldo = c.rows(o, "o", T * k, H, dt)
    if y is None:
        y = c.empty((T, H), dt)
    yp, ldy = c.rows(y, "y", T, H, dt)
    c.run(_lib.load().moe_collect, op, ldo, _DTYPE[dt], c.flat(w, "w", T * k, torch.float32),
          c.flat(routes.inv, "inv", T * k, torch.int32), T, k, H, yp, ldy)
    return y


def moe_collect_backward(dy: torch.Tensor, o: torch.Tensor, w: torch.Tensor, routes: Routes,
                         do: torch.Tensor | None = None, dw: torch.Tensor | None = None,
                         stream: torch.cuda.Stream | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Gradients (do [T*k, H], dw float32 [T, k]) of moe_collect.  Rows of do from
    routes.offsets[E] on are not written; dw is 0 for dropped entries."""
    c = _Call(o, stream)
    dt = _values(o, "o")
    T, k, H = routes.T, routes.k, o.shape[1]
    gp, ldg = c.rows(dy, "dy", T, H, dt)
    op, ldo = c.rows(o, "o", T * k, H, dt)
    if do is None:
        do = c.empty((T * k, H), dt)
    if dw is None:
        dw = c.empty((T, k), torch.float32)
    dp, ldd = c.rows(do, "do", T * k, H, dt)
    c.run(_lib.load().moe_collect_backward, gp, ldg, op, ldo, _DTYPE[dt], c.flat(w, "w", T * k, torch.float32),
          c.flat(routes.inv, "inv", T * k, torch.int32), T, k, H, dp, ldd, c.flat(dw, "dw", T * k, torch.float32))
    return do, dw


# ------------------------------------------------------------------ 8-bit checkpoints
@dataclass
class ActCkpt:
    """A matrix of activations in 8 bits: values codes * 2**(exps - 127), one exponent per
    row and 32 columns (255: the group held an infinity or a NaN)."""
    codes: torch.Tensor  # int8 [R, F]
    exps: torch.Tensor   # uint8 [R, ceil(F/32)]
    dtype: torch.dtype   # type of the saved values


@dataclass
class SwigluCkpt:
    g: ActCkpt
    u: ActCkpt


def alloc_ckpt(R: int, F: int, dtype: torch.dtype, device=None) -> ActCkpt:
    d = device or "cuda"
    return ActCkpt(torch.empty((R, F), dtype=torch.int8, device=d),
                   torch.empty((R, -(-F // GROUP)), dtype=torch.uint8, device=d), dtype)


def _ckpt(c: _Call, k: ActCkpt, R: int, F: int) -> tuple[int, int]:
    return c.flat(k.codes, "codes", R * F, torch.int8), c.flat(k.exps, "exps", R * -(-F // GROUP), torch.uint8)


def _new_ckpt(c: _Call, R: int, F: int, dt) -> ActCkpt:
    return ActCkpt(c.empty((R, F), torch.int8), c.empty((R, -(-F // GROUP)), torch.uint8), dt)


def _limit(c: _Call, rows: torch.Tensor | None) -> int | None:
    return None if rows is None else c.flat(rows, "rows", 1, torch.int32)


def moe_act_save(x: torch.Tensor, ckpt: ActCkpt | None = None, rows: torch.Tensor | None = None,
                 stream: torch.cuda.Stream | None = None) -> ActCkpt:
    """x [R, F] kept in 8 bits.  rows: cuda int32 [1], only rows below it are read and
    written (routes.offsets[E:] after a dispatch)."""
    c = _Call(x, stream)
    dt = _values(x, "x")
    R, F = x.shape
    xp, ldx = c.rows(x, "x", R, F, dt)
    if ckpt is None:
        ckpt = _new_ckpt(c, R, F, dt)
    elif ckpt.dtype is not dt:
        raise ValueError(f"the checkpoint is for {ckpt.dtype}, x is {dt}")
    c.run(_lib.load().moe_act_save, xp, ldx, _DTYPE[dt], R, F, *_ckpt(c, ckpt, R, F), _limit(c, rows))
    return ckpt


def moe_act_load(ckpt: ActCkpt, x: torch.Tensor | None = None, rows: torch.Tensor | None = None,
                 stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The restored matrix, in the type that was saved or in that of x."""
    c = _Call(ckpt.codes, stream)
    if ckpt.codes.dim() != 2:
        raise ValueError(f"codes must be a matrix, got {list(ckpt.codes.shape)}")
    R, F = ckpt.codes.shape
    if x is None:
        x = c.empty((R, F), ckpt.dtype)
    dt = _values(x, "x")
    xp, ldx = c.rows(x, "x", R, F, dt)
    c.run(_lib.load().moe_act_load, *_ckpt(c, ckpt, R, F), R, F, _DTYPE[dt], xp, ldx, _limit(c, rows))
    return x


def moe_swiglu_save(g: torch.Tensor, u: torch.Tensor, h: torch.Tensor | None = None, ckpt: SwigluCkpt | None = None,
                    rows: torch.Tensor | None = None,
                    stream: torch.cuda.Stream | None = None) -> tuple[torch.Tensor, SwigluCkpt]:
    """h = silu(g) * u and the 8-bit checkpoint of g and u that moe_swiglu_backward needs."""
    c = _Call(g, stream)
    dt = _values(g, "g")
    R, F = g.shape
    gp, ldg = c.rows(g, "g", R, F, dt)
    up, ldu = c.rows(u, "u", R, F, dt)
    if h is None:
        h = c.empty((R, F), dt)
    hp, ldh = c.rows(h, "h", R, F, dt)
    if ckpt is None:
        ckpt = SwigluCkpt(_new_ckpt(c, R, F, dt), _new_ckpt(c, R, F, dt))
    elif ckpt.g.dtype is not dt or ckpt.u.dtype is not dt:
        raise ValueError(f"the checkpoint is for {ckpt.g.dtype} and {ckpt.u.dtype}, g is {dt}")
    c.run(_lib.load().moe_swiglu_save, gp, ldg, up, ldu, _DTYPE[dt], R, F, hp, ldh, *_ckpt(c, ckpt.g, R, F),
          *_ckpt(c, ckpt.u, R, F), _limit(c, rows))
    return h, ckpt


def moe_swiglu_backward(dh: torch.Tensor, ckpt: SwigluCkpt, dg: torch.Tensor | None = None,
                        du: torch.Tensor | None = None, h: torch.Tensor | None = None, rebuild_h: bool = False,
                        rows: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None
                        ) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor | None]:
    """(dg, du, h) from dh and the checkpoint; h, the activation again, only if it is given
    or rebuild_h is set."""
    c = _Call(dh, stream)
    dt = _values(dh, "dh")
    R, F = dh.shape
    ap, lda = c.rows(dh, "dh", R, F, dt)
    if dg is None:
        dg = c.empty((R, F), dt)
    if du is None:
        du = c.empty((R, F), dt)
    if h is None and rebuild_h:
        h = c.empty((R, F), dt)
    gp, ldg = c.rows(dg, "dg", R, F, dt)
    up, ldu = c.rows(du, "du", R, F, dt)
    hp, ldh = (None, F) if h is None else c.rows(h, "h", R, F, dt)
    c.run(_lib.load().moe_swiglu_backward, ap, lda, _DTYPE[dt], *_ckpt(c, ckpt.g, R, F), *_ckpt(c, ckpt.u, R, F), R, F,
          gp, ldg, up, ldu, hp, ldh, _limit(c, rows))
    return dg, du, h


# ------------------------------------------------------------------ adapters
def moe_adapters(x: torch.Tensor, y: torch.Tensor, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor,
                 routes: Routes, out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                 stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """out = y + scale[a] * B[a] (A[a] x) for each token's adapter a (none: out = y).

    x [T, K], y and out [T, N] (out may be y), A [n, r, K] and B [n, N, r] contiguous, all
    bfloat16 or all float16; scale float32 [n]; routes = moe_sort(adapter of each token, n),
    -1 for none."""
    c = _Call(x, stream)
    dt = _values(x, "x")
    if A.dim() != 3 or B.dim() != 3:
        raise ValueError(f"A must be [n, r, K] and B [n, N, r], got {list(A.shape)} and {list(B.shape)}")
    T, K = x.shape
    n, r, N = A.shape[0], A.shape[1], B.shape[1]
    if A.shape[2] != K or B.shape[0] != n or B.shape[2] != r:
        raise ValueError(f"A must be [n, r, {K}] and B [n, N, r], got {list(A.shape)} and {list(B.shape)}")
    if (routes.T, routes.k, routes.E) != (T, 1, n):
        raise ValueError(f"routes are for {(routes.T, routes.k, routes.E)} tokens, entries and groups, need {(T, 1, n)}")
    xp, ldx = c.rows(x, "x", T, K, dt)
    yp, ldy = c.rows(y, "y", T, N, dt)
    ap, bp = c.flat(A, "A", n * r * K, dt), c.flat(B, "B", n * N * r, dt)
    sp = c.flat(scale, "scale", n, torch.float32)
    pp, _, fp = _routes(c, routes)
    if out is None:
        out = c.empty((T, N), dt)
    op, ldo = c.rows(out, "out", T, N, dt)
    fn = _lib.load().moe_adapters
    if ws is None:
        ws = c.workspace(fn, None, ldx, None, ldy, _DTYPE[dt], T, K, N, r, n, None, None, None, None, None, None, ldo,
                         None, 0)
    c.run(fn, xp, ldx, yp, ldy, _DTYPE[dt], T, K, N, r, n, ap, bp, sp, pp, fp, op, ldo, ws.data_ptr(), ws.numel(), None)
    return out


__all__ = ["ActCkpt", "Routes", "SwigluCkpt", "alloc_ckpt", "alloc_routes", "moe_act_load", "moe_act_save",
           "moe_adapters", "moe_collect", "moe_collect_backward", "moe_dispatch", "moe_dispatch_backward", "moe_sort",
           "moe_swiglu_backward", "moe_swiglu_save"]

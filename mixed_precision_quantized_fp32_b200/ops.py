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
from functools import lru_cache

import torch

from . import _lib
from ._lib import check

_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
GROUP = 32  # columns of an 8-bit checkpoint that share a scale


# The current device and stream as plain numbers: torch.cuda.current_stream() builds an
# object, 2 us of the 6 to 10 that a call takes on the host.
_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class _Call:
    """Device and stream of one call, taken from its first tensor."""

    __slots__ = ("dev", "stream")

    def __init__(self, t: torch.Tensor, stream: torch.cuda.Stream | None):
        self.dev = t.get_device()
        self.stream = stream
        if self.dev < 0:
            raise ValueError("operands must be cuda tensors")
        if stream is not None and stream.device_index != self.dev:
            raise ValueError(f"the stream is on {stream.device}, the operands on {t.device}")

    def empty(self, like: torch.Tensor, shape, dtype) -> torch.Tensor:
        # on the stream of the call, so that the allocator does not hand the memory on early
        if self.stream is None:
            return like.new_empty(shape, dtype=dtype)
        with torch.cuda.stream(self.stream):
            return like.new_empty(shape, dtype=dtype)

    def run(self, fn, *args) -> None:
        if _device() != self.dev:
            with torch.cuda.device(self.dev):
                rc = fn(*args, self.stream.cuda_stream if self.stream is not None else _raw_stream(self.dev))
        else:
            rc = fn(*args, self.stream.cuda_stream if self.stream is not None else _raw_stream(self.dev))
        if rc:
            check(fn.__name__, rc)

    def rows(self, t: torch.Tensor, name: str, R: int, F: int, dtype) -> tuple[int, int]:
        """Pointer and pitch of a matrix [R, F] with contiguous rows."""
        if t.dtype is not dtype or t.get_device() != self.dev or t.shape != (R, F):
            raise ValueError(f"{name} must be a {dtype} tensor {[R, F]} on cuda:{self.dev}, got {t.dtype} "
                             f"{list(t.shape)} on {t.device}")
        ld, step = t.stride()
        if step != 1 and F > 1:
            raise ValueError(f"{name} must have contiguous rows, got strides {t.stride()}")
        return t.data_ptr(), (ld if R > 1 else F)

    def flat(self, t: torch.Tensor, name: str, count: int, dtype) -> int:
        if t.dtype is not dtype or t.get_device() != self.dev or t.numel() != count or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of {count} values on cuda:{self.dev}, got "
                             f"{t.dtype} {list(t.shape)} on {t.device}")
        return t.data_ptr()

    def memory(self, ws: torch.Tensor | None, like: torch.Tensor, need: int) -> tuple[torch.Tensor | None, int | None, int]:
        """A workspace of at least `need` bytes: (tensor, pointer, bytes)."""
        if ws is None:
            if need == 0:
                return None, None, 0
            ws = self.empty(like, (need,), torch.uint8)
        elif ws.get_device() != self.dev or not ws.is_contiguous():
            raise ValueError(f"ws must be contiguous memory on cuda:{self.dev}")
        return ws, ws.data_ptr(), ws.numel() * ws.element_size()


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


@lru_cache(maxsize=4096)
def sort_workspace_bytes(T: int, k: int, E: int) -> int:
    """Bytes of ws that moe_sort and moe_dispatch need (0: none)."""
    need = C.c_uint64(0)
    check("moe_sort(workspace query)", _lib.load().moe_sort(None, T, k, E, None, None, None, None, 0, C.byref(need), None))
    return need.value


def _new_routes(c: _Call, idx: torch.Tensor, T: int, k: int, E: int, routes: Routes | None) -> Routes:
    if routes is None:
        R = T * k
        buf = c.empty(idx, (2 * R + max(E, 0) + 1,), torch.int32)
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
    routes = _new_routes(c, idx, T, k, E, routes)
    r = _routes(c, routes)
    ws, wp, wn = c.memory(ws, idx, sort_workspace_bytes(T, k, E))
    c.run(_lib.load().moe_sort, ip, T, k, E, *r, wp, wn, None)
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
    routes = _new_routes(c, idx, T, k, E, routes)
    r = _routes(c, routes)
    if xs is None:
        xs = c.empty(x, (T * k, H), dt)
    xsp, ldxs = c.rows(xs, "xs", T * k, H, dt)
    ws, wp, wn = c.memory(ws, idx, sort_workspace_bytes(T, k, E))
    c.run(_lib.load().moe_dispatch, xp, ldx, _DTYPE[dt], ip, T, k, E, H, xsp, ldxs, *r, wp, wn, None)
    return xs, routes


def moe_dispatch_backward(dxs: torch.Tensor, routes: Routes, dx: torch.Tensor | None = None,
                          stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """dx [T, H]: the sum of each token's rows of dxs [T*k, H]."""
    c = _Call(dxs, stream)
    dt = _values(dxs, "dxs")
    T, k, H = routes.T, routes.k, dxs.shape[1]
    dp, ldd = c.rows(dxs, "dxs", T * k, H, dt)
    if dx is None:
        dx = c.empty(dxs, (T, H), dt)
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
        y = c.empty(o, (T, H), dt)
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
        do = c.empty(o, (T * k, H), dt)
    if dw is None:
        dw = c.empty(w, (T, k), torch.float32)
    dp, ldd = c.rows(do, "do", T * k, H, dt)
    c.run(_lib.load().moe_collect_backward, gp, ldg, op, ldo, _DTYPE[dt], c.flat(w, "w", T * k, torch.float32),
          c.flat(routes.inv, "inv", T * k, torch.int32), T, k, H, dp, ldd, c.flat(dw, "dw", T * k, torch.float32))
    return do, dw


# ------------------------------------------------------------------ 8-bit checkpoints
class ActCkpt:
    """A matrix [R, F] of activations in 8 bits: values codes * 2**(exps - 127), one exponent
    per row and 32 columns (255: the group held an infinity or a NaN).

    codes: int8 [R, F]; exps: uint8 [R, ceil(F/32)]; dtype: type of the saved values.
    A checkpoint that an operator allocates is one piece of memory, of which codes and exps
    are views."""

    __slots__ = ("R", "F", "dtype", "_codes", "_exps", "_mem", "_at")

    def __init__(self, codes: torch.Tensor, exps: torch.Tensor, dtype: torch.dtype):
        if codes.dim() != 2 or codes.dtype is not torch.int8 or not codes.is_contiguous():
            raise ValueError(f"codes must be a contiguous int8 matrix, got {codes.dtype} {list(codes.shape)}")
        self.R, self.F = codes.shape
        if tuple(exps.shape) != (self.R, -(-self.F // GROUP)) or exps.dtype is not torch.uint8 \
                or not exps.is_contiguous() or exps.device != codes.device:
            raise ValueError(f"exps must be a contiguous uint8 tensor {[self.R, -(-self.F // GROUP)]} on {codes.device}, "
                             f"got {exps.dtype} {list(exps.shape)} on {exps.device}")
        self.dtype, self._codes, self._exps, self._mem, self._at = dtype, codes, exps, None, 0

    @staticmethod
    def _bytes(R: int, F: int) -> tuple[int, int]:
        """Offset of the exponents behind the codes, and the whole size (both whole 256s)."""
        e = (R * F + 255) // 256 * 256
        return e, e + (R * -(-F // GROUP) + 255) // 256 * 256

    @classmethod
    def _in(cls, mem: torch.Tensor, at: int, R: int, F: int, dtype: torch.dtype) -> "ActCkpt":
        k = cls.__new__(cls)
        k.R, k.F, k.dtype, k._codes, k._exps, k._mem, k._at = R, F, dtype, None, None, mem, at
        return k

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            self._codes = self._mem[self._at:self._at + self.R * self.F].view(torch.int8).view(self.R, self.F)
        return self._codes

    @property
    def exps(self) -> torch.Tensor:
        if self._exps is None:
            at, G = self._at + self._bytes(self.R, self.F)[0], -(-self.F // GROUP)
            self._exps = self._mem[at:at + self.R * G].view(self.R, G)
        return self._exps


@dataclass
class SwigluCkpt:
    g: ActCkpt
    u: ActCkpt


def alloc_ckpt(R: int, F: int, dtype: torch.dtype, device=None) -> ActCkpt:
    """Memory for the 8-bit checkpoint of a matrix [R, F] of dtype."""
    return ActCkpt._in(torch.empty(ActCkpt._bytes(R, F)[1], dtype=torch.uint8, device=device or "cuda"), 0, R, F, dtype)


def _ckpt(c: _Call, k: ActCkpt, R: int, F: int) -> tuple[int, int]:
    """Pointers of a checkpoint's codes and exponents."""
    mem = k._codes if k._mem is None else k._mem
    if k.R != R or k.F != F or mem.get_device() != c.dev:
        raise ValueError(f"the checkpoint must be of {[R, F]} on cuda:{c.dev}, is of {[k.R, k.F]} on {mem.device}")
    if k._mem is None:
        return k._codes.data_ptr(), k._exps.data_ptr()
    p = k._mem.data_ptr() + k._at
    return p, p + k._bytes(R, F)[0]


def _new_ckpts(c: _Call, like: torch.Tensor, R: int, F: int, dt, count: int) -> list[ActCkpt]:
    size = ActCkpt._bytes(R, F)[1]
    mem = c.empty(like, (count * size,), torch.uint8)
    return [ActCkpt._in(mem, i * size, R, F, dt) for i in range(count)]


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
        ckpt, = _new_ckpts(c, x, R, F, dt, 1)
    elif ckpt.dtype is not dt:
        raise ValueError(f"the checkpoint is for {ckpt.dtype}, x is {dt}")
    c.run(_lib.load().moe_act_save, xp, ldx, _DTYPE[dt], R, F, *_ckpt(c, ckpt, R, F), _limit(c, rows))
    return ckpt


def moe_act_load(ckpt: ActCkpt, x: torch.Tensor | None = None, rows: torch.Tensor | None = None,
                 stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The restored matrix, in the type that was saved or in that of x."""
    mem = ckpt._codes if ckpt._mem is None else ckpt._mem
    c = _Call(mem, stream)
    R, F = ckpt.R, ckpt.F
    if x is None:
        x = c.empty(mem, (R, F), ckpt.dtype)
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
        h = c.empty(g, (R, F), dt)
    hp, ldh = c.rows(h, "h", R, F, dt)
    if ckpt is None:
        ckpt = SwigluCkpt(*_new_ckpts(c, g, R, F, dt, 2))
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
        dg = c.empty(dh, (R, F), dt)
    if du is None:
        du = c.empty(dh, (R, F), dt)
    if h is None and rebuild_h:
        h = c.empty(dh, (R, F), dt)
    gp, ldg = c.rows(dg, "dg", R, F, dt)
    up, ldu = c.rows(du, "du", R, F, dt)
    hp, ldh = (None, F) if h is None else c.rows(h, "h", R, F, dt)
    c.run(_lib.load().moe_swiglu_backward, ap, lda, _DTYPE[dt], *_ckpt(c, ckpt.g, R, F), *_ckpt(c, ckpt.u, R, F), R, F,
          gp, ldg, up, ldu, hp, ldh, _limit(c, rows))
    return dg, du, h


# ------------------------------------------------------------------ adapters
def moe_adapters(x: torch.Tensor, y: torch.Tensor, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor,
                 routes: Routes, out: torch.Tensor | None = None,
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
        out = c.empty(y, (T, N), dt)
    op, ldo = c.rows(out, "out", T, N, dt)
    c.run(_lib.load().moe_adapters, xp, ldx, yp, ldy, _DTYPE[dt], T, K, N, r, n, ap, bp, sp, pp, fp, op, ldo)
    return out


__all__ = ["ActCkpt", "Routes", "SwigluCkpt", "alloc_ckpt", "alloc_routes", "moe_act_load",
           "moe_act_save", "moe_adapters", "moe_collect", "moe_collect_backward", "moe_dispatch", "moe_dispatch_backward",
           "moe_sort", "moe_swiglu_backward", "moe_swiglu_save", "sort_workspace_bytes"]

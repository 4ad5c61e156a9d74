"""The operators around the expert products on the GPU against plain 64-bit forms written
here, at the sizes and masks where they can go wrong.

Tolerances.  Every kernel works in fp32 and rounds once when it stores, so an output may
be off by half a step of its type, torch.finfo(t).eps / 2 relative to the value, plus the
fp32 error of what was summed, which each test bounds from the number of roundings
(2^-24 each) and the sum of the magnitudes.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import gen.workloads as W  # noqa: E402
import mixed_precision_quantized_fp32_b200 as moe  # noqa: E402
from tests import helpers as hp  # noqa: E402

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
F64 = torch.float64
U = 2.0 ** -24  # fp32 unit roundoff


def half_step(dt):
    return torch.finfo(dt).eps / 2


def rnd(*shape, seed=0, dtype=F32, sigma=1.0):
    g = torch.Generator().manual_seed(seed + 7919 * len(shape) + sum(shape))
    return (torch.randn(*shape, generator=g) * sigma).to(dtype).cuda()


def spaced(t, pitch, offset=0, fill=7.0):
    """t's values in a wider matrix: rows `pitch` apart, first column at `offset`; (view, memory)."""
    R, F = t.shape
    mem = torch.full((R, pitch), fill, dtype=t.dtype, device=t.device)
    mem[:, offset:offset + F] = t
    return mem[:, offset:offset + F], mem


def index(T, k, E, kind, seed=0):
    g = torch.Generator().manual_seed(seed + 31 * T + k)
    idx = torch.randint(0, E, (T, k), generator=g)
    if kind == "padded":
        idx[T - T // 3:] = -1
    elif kind == "holes":
        idx[torch.rand(T, k, generator=g) < 0.3] = -1
    elif kind == "outside":
        bad = torch.tensor([-1, E, E + 5, 2 ** 31 - 1, -2 ** 31])
        at = torch.rand(T, k, generator=g) < 0.4
        idx[at] = bad[torch.randint(0, 5, (T, k), generator=g)][at]
    elif kind == "none":
        idx[:] = -1
    elif kind == "one":
        idx[:] = E - 1
    return idx.int().cuda()


def ref_sort(idx, E):
    flat = idx.cpu().long().reshape(-1).numpy()
    key = np.where((flat >= 0) & (flat < E), flat, E)
    perm = np.argsort(key, kind="stable")
    inv = np.full(flat.size, -1, np.int64)
    total = int((key < E).sum())
    inv[perm[:total]] = np.arange(total)
    offsets = np.searchsorted(key[perm], np.arange(E + 1), side="left")
    return perm, inv, offsets


def check_routes(r, idx, E):
    perm, inv, offsets = ref_sort(idx, E)
    np.testing.assert_array_equal(r.offsets.cpu().numpy(), offsets)
    np.testing.assert_array_equal(r.perm.cpu().numpy(), perm)
    np.testing.assert_array_equal(r.inv.cpu().numpy(), inv)
    return perm, inv, int(offsets[E])


# ------------------------------------------------------------------ sort and dispatch
@pytest.mark.parametrize("T,k,E,kind", [
    (0, 2, 8, "all"), (1, 1, 1, "all"), (1, 8, 8, "all"), (16, 6, 256, "all"), (33, 3, 5, "holes"),
    (128, 8, 256, "padded"), (1024, 1, 1024, "outside"), (205, 5, 7, "holes"), (1025, 1, 1, "all"), (2048, 1, 300, "holes"),
    (2049, 1, 300, "holes"), (362, 8, 1024, "outside"), (363, 8, 256, "holes"), (1024, 2, 256, "padded"),
    (513, 2, 256, "none"), (700, 2, 64, "one"), (4097, 8, 256, "outside"), (8193, 1, 1023, "holes"),
    (3000, 3, 1024, "outside"), (16384, 1, 1024, "holes"), (16385, 1, 1024, "holes"), (16384, 3, 33, "holes"), (20000, 7, 1000, "padded"),
    (131072, 8, 128, "holes")])
def test_sort(T, k, E, kind):
    idx = index(T, k, E, kind)
    check_routes(moe.moe_sort(idx, E), idx, E)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,k,E,H,kind", [
    (0, 2, 8, 64, "all"), (1, 1, 4, 1, "all"), (16, 6, 256, 2048, "all"), (37, 3, 5, 77, "holes"),
    (200, 8, 64, 12, "outside"), (512, 8, 256, 40, "holes"), (513, 8, 256, 40, "holes"), (724, 4, 7, 24, "padded"),
    (2048, 2, 8, 16, "holes"), (2, 5, 1024, 12288, "outside"), (16385, 1, 1024, 24, "outside"), (8192, 6, 256, 64, "all"), (65536, 1, 3, 8, "padded"),
    (5471, 3, 300, 33, "holes"), (8191, 8, 256, 40, "none"), (2731, 7, 77, 520, "one"), (13108, 5, 6, 16, "holes"), (1500, 2, 8, 130, "padded"), (300, 4, 16, 1001, "holes"), (400, 3, 9, 264, "none")])
def test_dispatch(T, k, E, H, kind, dtype):
    idx, x = index(T, k, E, kind), rnd(T, H, dtype=dtype)
    xs = torch.full((T * k, H), 5.0, dtype=dtype, device="cuda")
    got, r = moe.moe_dispatch(x, idx, E, xs=xs)
    perm, _, total = check_routes(r, idx, E)
    want = torch.full((T * k, H), 5.0, dtype=dtype)
    want[:total] = x.cpu()[perm[:total] // k]
    assert got is xs and torch.equal(xs.cpu(), want)


@pytest.mark.parametrize("pitch,offset", [(300, 0), (296, 8), (264, 3), (257, 1), (512, 4)])
def test_dispatch_and_back_through_views(pitch, offset):
    # rows with any pitch and start: the bytes around them stay
    T, k, E, H = 300, 4, 16, 256
    idx, x = index(T, k, E, "holes"), rnd(T, H, dtype=BF16)
    xv, _ = spaced(x, pitch, offset)
    xs, mem = spaced(torch.zeros(T * k, H, dtype=BF16, device="cuda"), pitch, offset)
    _, r = moe.moe_dispatch(xv, idx, E, xs=xs)
    plain, _ = moe.moe_dispatch(x, idx, E, xs=torch.zeros(T * k, H, dtype=BF16, device="cuda"))
    assert torch.equal(xs, plain)
    dx, dmem = spaced(torch.zeros(T, H, dtype=BF16, device="cuda"), pitch, offset)
    moe.moe_dispatch_backward(xs, r, dx=dx)
    assert torch.equal(dx, moe.moe_dispatch_backward(plain, r))
    for m in (mem, dmem):
        m[:, offset:offset + H] = 7.0
        assert bool((m == 7.0).all())


CASES = [(1, 1, 1, 1, "all"), (1, 8, 8, 4096, "all"), (16, 6, 256, 2048, "all"), (37, 3, 5, 77, "holes"),
         (700, 2, 8, 264, "padded"), (300, 5, 16, 1001, "outside"), (64, 2, 128, 12288, "all"), (90, 7, 9, 40, "none")]


def gathered(rows, inv, T, k):
    """64-bit rows of every entry, zeros for dropped ones."""
    real = torch.from_numpy(inv >= 0).cuda().reshape(T, k)
    at = torch.from_numpy(np.maximum(inv, 0)).cuda().reshape(T, k)
    return torch.where(real[:, :, None], rows.to(F64)[at], 0.0), real


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("T,k,E,H,kind", CASES)
def test_collect_and_gradients(T, k, E, H, kind, dtype):
    idx = index(T, k, E, kind)
    r = moe.moe_sort(idx, E)
    _, inv, total = check_routes(r, idx, E)
    o, dy, w = rnd(T * k, H, dtype=dtype), rnd(T, H, dtype=dtype, seed=1), rnd(T, k, seed=2).abs()
    o[total:] = float("nan")                     # rows behind the last group's are not read
    rows, real = gathered(o, inv, T, k)
    w = torch.where(real, w, float("nan"))       # nor are the weights of dropped entries
    w64 = torch.where(real, w, 0.0).to(F64)
    # k products and sums in fp32, each off by at most U relative to the magnitudes so far
    y = (w64[:, :, None] * rows).sum(1)
    mag = (w64[:, :, None] * rows).abs().sum(1)
    got = moe.moe_collect(o, w, r).to(F64)
    assert bool(((got - y).abs() <= half_step(dtype) * y.abs() + (k + 1) * U * mag + tiny(dtype)).all())
    dx = rows.sum(1)
    got = moe.moe_dispatch_backward(o, r).to(F64)
    assert bool(((got - dx).abs() <= half_step(dtype) * dx.abs() + (k + 1) * U * rows.abs().sum(1) + tiny(dtype)).all())
    # do: one product; dw: H products, summed in any order
    do = torch.full((T * k, H), 3.0, dtype=dtype, device="cuda")
    do, dw = moe.moe_collect_backward(dy, o, w, r, do=do)
    want = torch.full((T * k, H), 3.0, dtype=F64, device="cuda")
    at = torch.from_numpy(inv).cuda().reshape(T, k)
    want[at[real]] = (w64[:, :, None] * dy.to(F64)[:, None])[real]
    assert bool(((do.to(F64) - want).abs() <= (half_step(dtype) + U) * want.abs() + tiny(dtype)).all())
    dot = (dy.to(F64)[:, None] * rows)
    assert bool(((dw.to(F64) - dot.sum(2)).abs() <= (H + 2) * U * dot.abs().sum(2)).all())
    assert bool((dw[~real] == 0).all())


# rows in accesses of 8, 4 and 2 bytes
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("k", [1, 2, 3, 8])
@pytest.mark.parametrize("H", [2, 12, 258, 1020, 1022, 1023])
def test_rows_in_fours_pairs_and_singles(H, k, dtype):
    test_collect_and_gradients(70, k, 9, H, "holes", dtype)
    test_dispatch(70, k, 9, H, "holes", dtype)


@pytest.mark.parametrize("H,pitch,offset", [(256, 260, 4), (256, 258, 2), (260, 264, 0), (258, 264, 6)])
def test_collect_through_views(H, pitch, offset):
    T, k, E = 90, 3, 7
    idx, o, dy, w = index(T, k, E, "holes"), rnd(T * k, H, dtype=F16), rnd(T, H, dtype=F16, seed=1), rnd(T, k, seed=2)
    r = moe.moe_sort(idx, E)
    total = int(r.offsets[E])
    ov, dyv = spaced(o, pitch, offset)[0], spaced(dy, pitch, offset)[0]
    y, mem = spaced(torch.zeros(T, H, dtype=F16, device="cuda"), pitch, offset)
    do, dmem = spaced(torch.zeros(T * k, H, dtype=F16, device="cuda"), pitch, offset)
    moe.moe_collect(ov, w, r, y=y)
    _, dw = moe.moe_collect_backward(dyv, ov, w, r, do=do)
    assert torch.equal(y, moe.moe_collect(o, w, r))
    do1, dw1 = moe.moe_collect_backward(dy, o, w, r)
    assert torch.equal(do[:total], do1[:total])
    # dw: H products, in another order
    dot = (dy.to(F64)[:, None] * torch.where((r.inv >= 0).reshape(T, k, 1), o.to(F64)[r.inv.clamp(min=0).long()].reshape(T, k, H), 0.0))
    assert bool(((dw - dw1).abs().to(F64) <= 2 * (H + 2) * U * dot.abs().sum(2)).all())
    for m in (mem, dmem):
        m[:, offset:offset + H] = 7.0
        assert bool((m == 7.0).all())


def tiny(dtype):
    """Half the smallest step of a type: the rounding of results below its normal range."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def test_collect_gradients_against_differences():
    # collect is linear in o and in w: <dy, y> along a direction v changes by <gradient, v>, and the
    # central difference with step 1 has no truncation error
    T, k, E, H = 50, 3, 7, 96
    idx = index(T, k, E, "holes")
    r = moe.moe_sort(idx, E)
    total = int(r.offsets[E])
    o, w, dy = rnd(T * k, H), rnd(T, k, seed=1), rnd(T, H, seed=2)
    do = torch.zeros(T * k, H, device="cuda")
    do, dw = moe.moe_collect_backward(dy, o, w, r, do=do)
    loss = lambda o, w: float((dy.to(F64) * moe.moe_collect(o, w, r).to(F64)).sum())  # noqa: E731
    v, z = rnd(T * k, H, seed=3), rnd(T, k, seed=4)
    # every loss is a sum of T*H terms, each y off by (k+1) roundings of a few units
    tol = T * H * 64 * U
    got = float((do[:total].to(F64) * v[:total].to(F64)).sum())
    assert abs((loss(o + v, w) - loss(o - v, w)) / 2 - got) <= tol
    got = float((dw.to(F64) * z.to(F64)).sum())
    assert abs((loss(o, w + z) - loss(o, w - z)) / 2 - got) <= tol


def test_inverse_outside_the_rows_counts_as_dropped():
    T, k, H = 6, 2, 64
    o, w = rnd(T * k, H), rnd(T, k, seed=1)
    inv = torch.arange(T * k, dtype=torch.int32, device="cuda")
    bad = inv.clone()
    bad[[0, 3, 7]] = torch.tensor([T * k, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    ref = inv.clone()
    ref[[0, 3, 7]] = -1
    a = moe.moe_collect(o, w, moe.Routes(T, k, 0, inv, bad, z))
    assert torch.equal(a, moe.moe_collect(o, w, moe.Routes(T, k, 0, inv, ref, z)))
    do, dw = moe.moe_collect_backward(a, o, w, moe.Routes(T, k, 0, inv, bad, z), do=torch.zeros_like(o))
    assert float(dw[0, 0]) == 0 and float(dw[1, 1]) == 0 and float(dw[3, 1]) == 0 and bool((do[3] == 0).all())


# ------------------------------------------------------------------ 8-bit checkpoints
def ref_ckpt(x):
    """Codes, exponent bytes and values of x's checkpoint, from the definition in 64 bits."""
    R, F = x.shape
    top = 9 if x.dtype == F16 else 121
    v = x.cpu().to(F64).numpy()
    G = -(-F // 32)
    codes, exps, vals = np.zeros((R, F), np.int8), np.zeros((R, G), np.uint8), np.zeros((R, F))
    for g in range(G):
        part = v[:, 32 * g:32 * g + 32]
        for i in range(R):
            big = np.abs(part[i]).max()
            if not np.isfinite(big):
                exps[i, g], vals[i, 32 * g:32 * g + 32] = 255, np.nan
                continue
            e = -126
            while e < top and 127.0 * 2.0 ** e < big:
                e += 1
            q = np.clip(np.rint(part[i] / 2.0 ** e), -127, 127)
            codes[i, 32 * g:32 * g + 32], exps[i, g], vals[i, 32 * g:32 * g + 32] = q, e + 127, q * 2.0 ** e
    return codes, exps, vals


def special(R, F, dtype, seed=0):
    """Rows of many magnitudes, with zero groups, ties, the type's extremes and groups that are not finite."""
    x = rnd(R, F, seed=seed) * torch.exp2(torch.arange(R, device="cuda")[:, None] % 37 - 18.0)
    x = x.clamp(-6e4, 6e4).to(dtype)
    fi = torch.finfo(dtype)
    x[0] = 0
    if R > 6:
        x[1] = fi.max
        x[2] = fi.tiny * fi.eps           # the smallest subnormal
        x[3] = (torch.arange(F, device="cuda") % 256 - 127.5).to(dtype)  # halves: ties
        x[4, F // 2] = float("inf")
        x[5, 0] = float("nan")
        x[6] = -fi.max
    return x


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("R,F", [(1, 1), (8, 32), (9, 40), (40, 256), (11, 77), (13, 1000), (7, 31)])
def test_checkpoint_is_exact(R, F, dtype):
    x = special(R, F, dtype)
    codes, exps, vals = ref_ckpt(x)
    c = moe.moe_act_save(x)
    np.testing.assert_array_equal(c.exps.cpu().numpy(), exps)
    np.testing.assert_array_equal(c.codes.cpu().numpy(), codes)
    back = moe.moe_act_load(c)
    assert back.dtype == dtype
    np.testing.assert_array_equal(back.cpu().to(F64).numpy(), torch.from_numpy(vals).to(dtype).to(F64).numpy())
    wide = moe.moe_act_load(c, x=torch.empty(R, F, device="cuda"))
    np.testing.assert_array_equal(wide.cpu().to(F64).numpy(), vals)
    # a finite value is off by at most half a step.  127 * 2^(e-1) < max|x| bounds the step by 2/127 of
    # the row's largest, unless e is the least there is, -126 (half a step is 2^-127 then); at the
    # type's very top the clamp may take a whole step
    fine = np.isfinite(vals)
    x64 = x.cpu().to(F64).numpy()
    amax = np.abs(np.where(fine, x64, 0)).max(axis=1, keepdims=True)
    assert np.all(np.abs(vals - np.where(fine, x64, 0))[fine] <= np.broadcast_to(amax * 2 / 127 + 2.0 ** -127, (R, F))[fine])


@pytest.mark.parametrize("F,pitch,offset", [(256, 300, 0), (256, 264, 8), (64, 67, 3), (50, 64, 8), (96, 97, 0)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_checkpoint_through_views_and_row_limits(F, pitch, offset, dtype):
    R = 37
    x = rnd(R, F, dtype=dtype)
    xv, _ = spaced(x, pitch, offset)
    codes, exps, vals = ref_ckpt(x)
    c = moe.moe_act_save(xv)
    np.testing.assert_array_equal(c.codes.cpu().numpy(), codes)
    np.testing.assert_array_equal(c.exps.cpu().numpy(), exps)
    out, mem = spaced(torch.zeros(R, F, dtype=dtype, device="cuda"), pitch, offset)
    moe.moe_act_load(c, x=out)
    np.testing.assert_array_equal(out.cpu().to(F64).numpy(), vals)
    mem[:, offset:offset + F] = 7.0
    assert bool((mem == 7.0).all())
    for n in (-3, 0, 1, 20, R, R + 9):           # rows from the limit on stay as they were
        rows = torch.tensor([n], dtype=torch.int32, device="cuda")
        m = min(max(n, 0), R)
        c = moe.alloc_ckpt(R, F, dtype)
        c.codes.fill_(3), c.exps.fill_(200)
        moe.moe_act_save(xv, ckpt=c, rows=rows)
        np.testing.assert_array_equal(c.codes[:m].cpu().numpy(), codes[:m])
        assert bool((c.codes[m:] == 3).all()) and bool((c.exps[m:] == 200).all())
        out = torch.full((R, F), 4.0, dtype=dtype, device="cuda")
        moe.moe_act_load(moe.ActCkpt(torch.from_numpy(codes).cuda(), torch.from_numpy(exps).cuda(), dtype), x=out, rows=rows)
        assert bool((out[m:] == 4.0).all())
        np.testing.assert_array_equal(out[:m].cpu().to(F64).numpy(), vals[:m])


def ref_swiglu(g, u, dh):
    s = 1 / (1 + torch.exp(-g))
    return {"h": g * s * u, "du": dh * g * s, "dg": dh * u * s * (1 + g * (1 - s))}


def swiglu_tol(g, u, dh, dtype):
    """fp32 errors of the kernels' formulas.  exp(-g) is off by at most 2 + 1.173|g| units in the
    last place, the quotient by 2, each further operation by half a one (2^-23 of the value or
    less): s is off by at most (5 + 1.2|g|) 2^-23 s.  h and du add two products.  dg has
    1 + g(1-s) with 1-s off by s's error and half a unit, so its absolute error is at most
    |dh u| s (1 + |g|)(12 + 2.4|g|) 2^-23."""
    e = 2.0 ** -23
    s = 1 / (1 + torch.exp(-g))
    rel = (7 + 1.2 * g.abs()) * e
    low = 2.0 ** -126  # s below fp32's normal range may be flushed: silu(g) is below |g| 2^-126 then
    return {"h": rel * (g * s * u).abs() + low * (1 + (g * u).abs()), "du": rel * (dh * g * s).abs() + low * (1 + (dh * g).abs()),
            "dg": (dh * u).abs() * s * (1 + g.abs()) * (12 + 2.4 * g.abs()) * e + low * (1 + (dh * u * g).abs())}


def near(got, want, extra, dtype):
    return bool(((got.to(F64) - want).abs() <= half_step(dtype) * want.abs() + extra * (1 + half_step(dtype)) + tiny(dtype)).all())


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("R,F", [(1, 1), (3, 32), (5, 8), (33, 264), (64, 768), (21, 77), (10, 1001)])
def test_swiglu_with_checkpoint(R, F, dtype):
    g, u, dh = rnd(R, F, sigma=3, dtype=dtype), rnd(R, F, seed=1, dtype=dtype), rnd(R, F, seed=2, dtype=dtype)
    g[0, 0] = -90.0
    g[0, -1] = 60.0
    h, kept = moe.moe_swiglu_save(g, u)
    g64, u64, dh64 = g.to(F64), u.to(F64), dh.to(F64)
    assert near(h, ref_swiglu(g64, u64, dh64)["h"], swiglu_tol(g64, u64, dh64, dtype)["h"], dtype)
    for t, c in ((g, kept.g), (u, kept.u)):
        codes, exps, _ = ref_ckpt(t)
        np.testing.assert_array_equal(c.codes.cpu().numpy(), codes)
        np.testing.assert_array_equal(c.exps.cpu().numpy(), exps)
    gk, uk = (moe.moe_act_load(c, x=torch.empty(R, F, device="cuda")).to(F64) for c in (kept.g, kept.u))
    want, tol = ref_swiglu(gk, uk, dh64), swiglu_tol(gk, uk, dh64, dtype)
    dg, du, again = moe.moe_swiglu_backward(dh, kept, rebuild_h=True)
    assert near(dg, want["dg"], tol["dg"], dtype) and near(du, want["du"], tol["du"], dtype)
    assert near(again, want["h"], tol["h"], dtype)
    dg2, du2, none = moe.moe_swiglu_backward(dh, kept)
    assert none is None and torch.equal(dg, dg2) and torch.equal(du, du2)


def test_swiglu_gradient_against_differences():
    # central differences of the 64-bit activation at the restored values, step 1e-5: truncation
    # 1e-10 times the third derivative (below 1), rounding 1e-16 / 1e-5 relative to values below 100
    R, F = 20, 96
    g, u, dh = rnd(R, F, sigma=2), rnd(R, F, seed=1), rnd(R, F, seed=2)
    _, kept = moe.moe_swiglu_save(g, u)
    gk, uk = (moe.moe_act_load(c).to(F64) for c in (kept.g, kept.u))
    dg, du, _ = moe.moe_swiglu_backward(dh, kept)
    f = lambda a, b: a / (1 + torch.exp(-a)) * b * dh.to(F64)  # noqa: E731
    d = 1e-5
    for got, diff in ((dg, (f(gk + d, uk) - f(gk - d, uk)) / (2 * d)), (du, (f(gk, uk + d) - f(gk, uk - d)) / (2 * d))):
        assert bool(((got.to(F64) - diff).abs() <= 2e-8 + 40 * U * (1 + diff.abs()) * (1 + uk.abs()) * (1 + gk.abs()) ** 2).all())


@pytest.mark.parametrize("F,gap", [(256, 0), (256, 8), (77, 0), (64, 3)])
def test_swiglu_on_halves_of_one_matrix_with_row_limit(F, gap):
    # gate and up as the two halves of one product, their gradients likewise; rows behind the limit stay
    R, n = 29, 17
    both, back = rnd(R, 2 * F + gap, dtype=BF16), torch.full((R, 2 * F + gap), 9.0, dtype=BF16, device="cuda")
    g, u, dh = both[:, :F], both[:, F + gap:], rnd(R, F, seed=2, dtype=BF16)
    rows = torch.tensor([n], dtype=torch.int32, device="cuda")
    kept = moe.SwigluCkpt(moe.alloc_ckpt(R, F, BF16), moe.alloc_ckpt(R, F, BF16))
    for c in (kept.g, kept.u):
        c.codes.fill_(5), c.exps.fill_(99)
    h = torch.full((R, F), 9.0, dtype=BF16, device="cuda")
    moe.moe_swiglu_save(g, u, h=h, ckpt=kept, rows=rows)
    ph, pk = moe.moe_swiglu_save(g.contiguous(), u.contiguous())
    assert torch.equal(h[:n], ph[:n]) and bool((h[n:] == 9.0).all())
    for a, b in ((kept.g, pk.g), (kept.u, pk.u)):
        assert torch.equal(a.codes[:n], b.codes[:n]) and torch.equal(a.exps[:n], b.exps[:n])
        assert bool((a.codes[n:] == 5).all()) and bool((a.exps[n:] == 99).all())
    again = torch.full((R, F), 9.0, dtype=BF16, device="cuda")
    moe.moe_swiglu_backward(dh, kept, dg=back[:, :F], du=back[:, F + gap:], h=again, rows=rows)
    dg, du, ah = moe.moe_swiglu_backward(dh, pk, rebuild_h=True)
    assert torch.equal(back[:n, :F], dg[:n]) and torch.equal(back[:n, F + gap:], du[:n]) and torch.equal(again[:n], ah[:n])
    assert bool((back[n:] == 9.0).all()) and bool((back[:, F:F + gap] == 9.0).all()) and bool((again[n:] == 9.0).all())


def test_swiglu_not_finite():
    x = rnd(4, 96, dtype=BF16)
    g, u, dh = x.clone(), rnd(4, 96, seed=1, dtype=BF16), rnd(4, 96, seed=2, dtype=BF16)
    g[0, 5], g[1, 40], u[2, 70], g[3, 64] = float("nan"), float("inf"), float("-inf"), float("-inf")
    h, kept = moe.moe_swiglu_save(g, u)
    s = g.to(F64)
    want = s / (1 + torch.exp(-s)) * u.to(F64)
    assert torch.equal(torch.isnan(h), torch.isnan(want)) and torch.equal(torch.isinf(h), torch.isinf(want))
    dg, du, _ = moe.moe_swiglu_backward(dh, kept)
    bad = torch.zeros(4, 96, dtype=torch.bool, device="cuda")
    bad[0, :32] = bad[1, 32:64] = bad[3, 64:] = True     # the group of a value that is not finite is NaN throughout
    ubad = torch.zeros_like(bad)
    ubad[2, 64:] = True
    assert torch.equal(torch.isnan(du), bad) and torch.equal(torch.isnan(dg), bad | ubad)


# widths, pitches and offsets in fours, in pairs and odd: accesses of 4, 2 and 1 values
@pytest.mark.parametrize("F,pitch,offset", [(260, 260, 0), (256, 260, 4), (28, 36, 8), (258, 258, 0), (256, 258, 2), (26, 40, 8),
                                            (260, 266, 4), (1, 2, 1), (2, 2, 0), (4, 4, 0), (33, 33, 0), (510, 513, 3)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_checkpoint_in_fours_pairs_and_singles(F, pitch, offset, dtype):
    test_checkpoint_through_views_and_row_limits(F, pitch, offset, dtype)
    test_checkpoint_is_exact(9, F, dtype)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("R,F", [(6, 2), (9, 12), (7, 30), (20, 258), (20, 260), (3, 1022), (40, 67)])
def test_swiglu_in_fours_pairs_and_singles(R, F, dtype):
    test_swiglu_with_checkpoint(R, F, dtype)


@pytest.mark.parametrize("F,gap", [(260, 0), (260, 2), (260, 1), (258, 4), (258, 1), (36, 4)])
def test_swiglu_halves_in_fours_pairs_and_singles(F, gap):
    test_swiglu_on_halves_of_one_matrix_with_row_limit(F, gap)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("F", [1921, 1922, 1924])
def test_swiglu_of_many_rows_is_that_of_few(F, dtype):
    # enough groups that a warp takes more of them; the same bits as a part of the rows alone
    R, n = 2200, 40
    g, u, dh = rnd(R, F, sigma=3, dtype=dtype), rnd(R, F, seed=1, dtype=dtype), rnd(R, F, seed=2, dtype=dtype)
    h, kept = moe.moe_swiglu_save(g, u)
    dg, du, again = moe.moe_swiglu_backward(dh, kept, rebuild_h=True)
    for at in (slice(0, n), slice(R - n, R)):
        h1, kept1 = moe.moe_swiglu_save(g[at], u[at])
        assert torch.equal(h[at], h1)
        for a, b in ((kept.g, kept1.g), (kept.u, kept1.u)):
            assert torch.equal(a.codes[at], b.codes) and torch.equal(a.exps[at], b.exps)
        for a, b in zip((dg, du, again), moe.moe_swiglu_backward(dh[at], kept1, rebuild_h=True)):
            assert torch.equal(a[at], b)


# ------------------------------------------------------------------ adapters
def ref_adapters(x, y, A, B, scale, ids):
    """64-bit result and the sum of the magnitudes behind the low-rank term."""
    out, mag = y.to(F64).clone(), torch.zeros(y.shape, dtype=F64, device="cuda")
    for a in range(A.shape[0]):
        at = torch.nonzero((ids == a).cuda()).reshape(-1)
        if at.numel():
            A64, B64, x64, s = A[a].to(F64), B[a].to(F64), x[at].to(F64), scale[a].to(F64)
            out[at] += s * ((x64 @ A64.T) @ B64.T)
            mag[at] = s.abs() * ((x64.abs() @ A64.abs().T) @ B64.abs().T)
    return out, mag


def adapters_near(got, want, mag, K, r, dtype):
    # K + r sums on the tensor cores (each off by at most a unit, 2^-23, of the magnitudes) and 64
    # more for parts, scale and y; P as hi + lo terms leaves 2^-16 (bf16: two times 8 bits) or less of |P|
    tol = half_step(dtype) * want.abs() + ((K + r + 64) * 2.0 ** -23 + 2.0 ** -16) * (mag + want.abs()) + tiny(dtype)
    return bool(((got.to(F64) - want).abs() <= tol).all())


def bank(n, r, K, N, dtype):
    return (rnd(n, r, K, dtype=dtype, sigma=K ** -0.5), rnd(n, N, r, dtype=dtype, sigma=r ** -0.5),
            torch.rand(n, generator=torch.Generator().manual_seed(n)).cuda() + 0.5)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,K,N,r,n", [
    (1, 8, 8, 8, 1), (1, 4096, 4096, 16, 32), (5, 264, 40, 8, 3), (17, 256, 1000, 24, 2), (64, 512, 256, 16, 48),
    (128, 136, 520, 64, 5), (129, 2048, 264, 32, 4), (300, 512, 512, 40, 1), (700, 320, 264, 64, 7), (400, 264, 288, 128, 3),
    (1000, 128, 128, 8, 1024), (260, 1032, 2056, 16, 6), (2100, 64, 40, 8, 2), (1500, 1000, 1048, 16, 3),
    (1030, 200, 72, 24, 5), (520, 2056, 328, 40, 2), (300, 72, 2000, 120, 6), (3000, 8, 8, 128, 9)])
def test_adapters(T, K, N, r, n, dtype):
    ids = index(T, 1, n, "holes" if T > 1 else "all")[:, 0]
    x, y = rnd(T, K, dtype=dtype), rnd(T, N, dtype=dtype, seed=1)
    A, B, scale = bank(n, r, K, N, dtype)
    x[ids < 0] = float("nan")                    # rows without an adapter are not read
    routes = moe.moe_sort(ids, n)
    want, mag = ref_adapters(x, y, A, B, scale, ids)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = moe.moe_adapters(x, y, A, B, scale, routes, status=status)
    assert adapters_near(out, want, mag, K, r, dtype) and int(status) == 0
    assert torch.equal(out[ids < 0], y[ids < 0])
    z = y.clone()
    assert moe.moe_adapters(x, z, A, B, scale, routes, out=z) is z
    assert torch.equal(z, out)                   # in place: the same bits


@pytest.mark.parametrize("T,r", [(200, 16), (700, 64)])
@pytest.mark.parametrize("kind", ["none", "one"])
def test_adapters_all_or_none(kind, T, r):
    K, N, n = 256, 264, 4
    ids = index(T, 1, n, kind)[:, 0]
    x, y = rnd(T, K, dtype=BF16), rnd(T, N, dtype=BF16, seed=1)
    A, B, scale = bank(n, r, K, N, BF16)
    out = moe.moe_adapters(x, y, A, B, scale, moe.moe_sort(ids, n))
    want, mag = ref_adapters(x, y, A, B, scale, ids)
    assert adapters_near(out, want, mag, K, r, BF16)
    if kind == "none":
        assert torch.equal(out, y)


@pytest.mark.parametrize("T,r", [(150, 32), (600, 64)])
def test_adapters_through_views(T, r):
    K, N, n = 264, 520, 5
    ids = index(T, 1, n, "holes")[:, 0]
    x, y = rnd(T, K, dtype=F16), rnd(T, N, dtype=F16, seed=1)
    A, B, scale = bank(n, r, K, N, F16)
    routes = moe.moe_sort(ids, n)
    plain = moe.moe_adapters(x, y, A, B, scale, routes)
    xv, _ = spaced(x, 400, 16)
    yv, _ = spaced(y, 600, 8)
    ov, mem = spaced(torch.zeros_like(y), 560, 24)
    moe.moe_adapters(xv, yv, A, B, scale, routes, out=ov)
    assert torch.equal(ov, plain)
    mem[:, 24:24 + N] = 7.0
    assert bool((mem == 7.0).all())


@pytest.mark.parametrize("T", [40, 600])
def test_adapters_beyond_half_range(T):
    # A x beyond 65504 in fp16 while the result is in range: it is held in 32 bits
    K, N, r, n = 512, 128, 64, 2
    ids = index(T, 1, n, "all")[:, 0]
    x = rnd(T, K, dtype=F16, sigma=300.0)
    A, B, scale = rnd(n, r, K, dtype=F16, sigma=60.0), rnd(n, N, r, dtype=F16, sigma=2e-4), torch.ones(n, device="cuda")
    y = rnd(T, N, dtype=F16, seed=1)
    assert float((x.to(F64) @ A[0].to(F64).T).abs().max()) > 65504
    want, mag = ref_adapters(x, y, A, B, scale, ids)
    assert float(want.abs().max()) < 6e4
    assert adapters_near(moe.moe_adapters(x, y, A, B, scale, moe.moe_sort(ids, n)), want, mag, K, r, F16)


@pytest.mark.parametrize("T,r", [(20, 8), (300, 128), (2100, 32)])   # tiles of 16 and of 64 tokens
def test_adapters_infinite_beside_large(T, r):
    # a low-rank term beyond 32 bits next to one of 2^79, of the other sign: infinite as the
    # formula's sum is, not the difference of two infinities
    K, N = 64, 40
    x, y = torch.zeros(T, K, dtype=F16, device="cuda"), rnd(T, N, dtype=F16)
    x[:, 0], x[:, 1] = 2.0 ** 13, 2.0 ** -24
    A, B = torch.zeros(1, r, K, dtype=F16, device="cuda"), torch.zeros(1, N, r, dtype=F16, device="cuda")
    A[0, 0, 0], A[0, 1, 1] = 1.0, 2.0 ** -24
    B[0, :, 0], B[0, :, 1] = 1.0, -1.0
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    ids[3] = -1
    out = moe.moe_adapters(x, y, A, B, torch.full((1,), 2.0 ** 127, device="cuda"), moe.moe_sort(ids, 1))
    assert bool((out[ids == 0] == float("inf")).all()) and torch.equal(out[3], y[3])


@pytest.mark.parametrize("T,r", [(33, 8), (900, 40)])
def test_adapters_keep_requests_apart(T, r):
    # one request's NaN and another's infinity stay in their rows
    K, N, n = 256, 264, 3
    ids = index(T, 1, n, "all")[:, 0]
    x, y = rnd(T, K, dtype=BF16), rnd(T, N, dtype=BF16, seed=1)
    A, B, scale = bank(n, r, K, N, BF16)
    routes = moe.moe_sort(ids, n)
    clean = moe.moe_adapters(x, y, A, B, scale, routes)
    x[7, 3], x[20, 100] = float("nan"), float("inf")
    out = moe.moe_adapters(x, y, A, B, scale, routes)
    rest = [t for t in range(T) if t not in (7, 20)]
    assert torch.equal(out[rest], clean[rest])
    assert bool(torch.isnan(out[7]).all()) and not bool(torch.isfinite(out[20]).any())


# tiles of 64 tokens: long batches, and shorter ones with more to multiply (up to eight blocks a tile)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,K,N,r,n", [
    (2049, 8, 8, 8, 1), (2100, 264, 40, 16, 3), (2060, 40, 1000, 24, 2), (2500, 320, 264, 64, 7), (2400, 264, 288, 128, 3),
    (3000, 512, 512, 40, 100), (2200, 2056, 328, 40, 2), (2300, 72, 2000, 120, 6), (1100, 2056, 1096, 64, 2), (1030, 136, 1000, 128, 4),
    (900, 2056, 3000, 72, 1), (400, 4104, 2000, 120, 1), (2048, 1552, 2000, 32, 5)])
def test_adapters_in_large_tiles(T, K, N, r, n, dtype):
    test_adapters(T, K, N, r, n, dtype)


@pytest.mark.parametrize("r", [16, 64, 128])
def test_adapters_in_large_tiles_as_programs_call_them(r):
    T = 2150
    for kind in ("none", "one"):
        test_adapters_all_or_none(kind, T, r)
    test_adapters_through_views(T, r)
    test_adapters_keep_requests_apart(T, r)
    test_adapters_beyond_half_range(T)


def test_large_tiles_on_streams_and_in_graphs():
    # two captured graphs, replayed in turn with new inputs, beside a call on another stream
    T, H, n = 2300, 264, 9
    x, y, ids = rnd(T, H, dtype=BF16), rnd(T, H, dtype=BF16, seed=1), index(T, 1, n, "holes")[:, 0]
    banks = [bank(n, r, H, H, BF16) for r in (64, 128)]

    def step(stream=None):
        routes = moe.moe_sort(ids, n, stream=stream)
        return [moe.moe_adapters(x, y, *b, routes, stream=stream) for b in banks]

    want = step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    s = torch.cuda.Stream()
    for seed in (3, 4):
        x.copy_(rnd(T, H, dtype=BF16, seed=seed))
        ids.copy_(index(T, 1, n, "holes", seed=seed)[:, 0])
        torch.cuda.synchronize()
        other = step(stream=s)
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        now = step()
        for (_, out), extra in zip(graphs, (other, now)):
            for a, b, c in zip(out, extra, now):
                assert torch.equal(a, c) and torch.equal(b, c)
        assert not torch.equal(now[0], want[0])


# ------------------------------------------------------------------ offsets beyond 32 bits
def test_rows_beyond_32_bit_offsets():
    # 2.2e9 values: the last tokens' rows lie beyond 2^31 values (and 2^32 bytes) of the matrix
    T, k, H = 33600, 8, 8192
    idx = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    idx[:, 0] = 0
    idx[T - 3:] = torch.arange(k, device="cuda").int()
    r = moe.moe_sort(idx, k)
    perm, inv, total = check_routes(r, idx, k)
    o = torch.zeros(T * k, H, dtype=F16, device="cuda")
    r.perm.copy_(torch.arange(T * k - 1, -1, -1, device="cuda"))      # rows of o from its end
    far = torch.where(r.inv >= 0, T * k - 1 - r.inv, -1).int()
    routes = moe.Routes(T, k, k, r.perm, far, r.offsets)
    v = rnd(T, H, dtype=F16)
    rows = far.reshape(T, k)[:, 0].long()
    o[rows] = v
    o[far.reshape(T, k)[T - 3:].long().reshape(-1)] = v[T - 3:].repeat_interleave(k, 0)
    w = torch.zeros(T, k, device="cuda")
    w[:, 0] = 0.5
    w[T - 3:, k - 1] = 0.25
    y = moe.moe_collect(o, w, routes)
    assert torch.equal(y[:T - 3], v[:T - 3] * 0.5) and torch.equal(y[T - 3:], v[T - 3:] * 0.75)
    do, dw = moe.moe_collect_backward(v, o, w, routes, do=o.zero_())
    assert torch.equal(do[rows], v * 0.5) and torch.equal(do[far.reshape(T, k)[T - 1, k - 1].long()], v[T - 1] * 0.25)
    xs, r2 = moe.moe_dispatch(v, idx, k, xs=do)
    assert torch.equal(xs[r2.inv.reshape(T, k)[:, 0].long()], v)


def test_checkpoints_beyond_32_bit_offsets():
    R, F = 70000, 32768                                   # 2.3e9 values
    x = torch.zeros(R, F, dtype=BF16, device="cuda")
    x[-3:] = rnd(3, F, dtype=BF16)
    c = moe.moe_act_save(x)
    codes, exps, vals = ref_ckpt(x[-3:])
    np.testing.assert_array_equal(c.codes[-3:].cpu().numpy(), codes)
    np.testing.assert_array_equal(c.exps[-3:].cpu().numpy(), exps)
    del x
    back = moe.moe_act_load(c)
    np.testing.assert_array_equal(back[-3:].cpu().to(F64).numpy(), vals)
    assert not bool(back[:4].any())
    v = moe.ActCkpt(c.codes[-3:], c.exps[-3:], BF16)      # a slice of rows is a checkpoint too
    np.testing.assert_array_equal(moe.moe_act_load(v).cpu().to(F64).numpy(), vals)


# ------------------------------------------------------------------ refusals of the binding
def test_binding_refuses_what_does_not_fit():
    T, k, E, H = 6, 2, 3, 32
    x, idx, w = rnd(T, H, dtype=BF16), index(T, k, E, "all"), rnd(T, k)
    xs, r = moe.moe_dispatch(x, idx, E)
    c, sc = moe.moe_act_save(x), moe.moe_swiglu_save(x, x)[1]
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    A, B, scale = bank(2, 8, H, H, BF16)
    ar = moe.moe_sort(ids, 2)
    bad = {
        "types": lambda: moe.moe_dispatch(x.double(), idx, E), "idx type": lambda: moe.moe_sort(idx.long(), E),
        "idx strides": lambda: moe.moe_sort(torch.stack([idx, idx], 2)[:, :, 0], E), "cpu idx": lambda: moe.moe_dispatch(x, idx.cpu(), E),
        "x rank": lambda: moe.moe_dispatch(x[0], idx, E), "tokens": lambda: moe.moe_dispatch(x[:5], idx, E),
        "xs shape": lambda: moe.moe_dispatch(x, idx, E, xs=xs[:5]), "xs type": lambda: moe.moe_dispatch(x, idx, E, xs=xs.half()),
        "routes": lambda: moe.moe_dispatch(x, idx, E + 1, routes=r), "columns": lambda: moe.moe_collect(xs.t().contiguous().t(), w, r),
        "w type": lambda: moe.moe_collect(xs, w.half(), r), "w shape": lambda: moe.moe_collect(xs, w[:, :1], r),
        "y": lambda: moe.moe_collect(xs, w, r, y=x[:, :16]), "dy": lambda: moe.moe_collect_backward(xs, xs, w, r),
        "not a tensor": lambda: moe.moe_collect(xs, 1.0, r), "E": lambda: moe.moe_sort(idx, 2 ** 40),
        "ckpt type": lambda: moe.moe_act_save(x.half(), ckpt=c), "ckpt shape": lambda: moe.moe_act_save(x[:3], ckpt=c),
        "load shape": lambda: moe.moe_act_load(c, x=x[:3]), "swiglu": lambda: moe.moe_swiglu_save(x, x[:3]),
        "swiglu ckpt": lambda: moe.moe_swiglu_backward(x[:3], sc), "swiglu type": lambda: moe.moe_swiglu_save(x.float(), x.float(), ckpt=sc),
        "rows": lambda: moe.moe_act_save(x, rows=ids), "A": lambda: moe.moe_adapters(x, x, A[:, :, :16], B, scale, ar),
        "B": lambda: moe.moe_adapters(x, x, A, B[:1], scale, ar), "scale": lambda: moe.moe_adapters(x, x, A, B, scale[:1], ar),
        "adapter routes": lambda: moe.moe_adapters(x, x, A, B, scale, r), "adapters' ws": lambda: moe.moe_sort(idx, E, ws=ids.cpu()),
    }
    for name, call in bad.items():
        with pytest.raises(ValueError):
            call()
            pytest.fail(name)
    refused = {
        "E": (lambda: moe.moe_sort(idx, 1025), "MOE_ERR_SHAPE"), "k": (lambda: moe.moe_sort(torch.zeros(2, 9, dtype=torch.int32, device="cuda"), 3), "MOE_ERR_SHAPE"),
        "pitch 0": (lambda: moe.moe_act_save(x[:1].expand(4, H)), "MOE_ERR_SHAPE"),
        "fp32 adapters": (lambda: moe.moe_adapters(x.float(), x.float(), A.float(), B.float(), scale, ar), "MOE_ERR_FORMAT"),
        "rank": (lambda: moe.moe_adapters(x, x, A[:, :4].contiguous(), B[:, :, :4].contiguous(), scale, ar), "MOE_ERR_SHAPE"),
        "alignment": (lambda: moe.moe_adapters(spaced(x, 64, 4)[0], x, A, B, scale, ar), "MOE_ERR_ALIGN"),
        "pitch": (lambda: moe.moe_adapters(spaced(x, 36)[0], x, A, B, scale, ar), "MOE_ERR_ALIGN"),
    }
    for name, (call, status) in refused.items():
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.name == status, name
    torch.cuda.synchronize()


def test_two_calls_at_once():
    # two streams, two host threads: calls share nothing
    import threading
    T, k, E, H = 3000, 8, 64, 512                          # 24000 entries: the sort that needs a workspace
    A, B, scale = bank(4, 64, H, H, BF16)
    jobs = [(rnd(T, H, dtype=BF16, seed=i), index(T, k, E, "holes", seed=i), index(T, 1, 4, "holes", seed=i)[:, 0]) for i in (1, 2)]

    def work(x, idx, ids, stream=None):
        xs, r = moe.moe_dispatch(x, idx, E, xs=None, stream=stream)
        return r.perm, moe.moe_dispatch_backward(xs, r, stream=stream), moe.moe_adapters(x, x, A, B, scale, moe.moe_sort(ids, 4, stream=stream), stream=stream)

    want = [work(*j) for j in jobs]
    torch.cuda.synchronize()
    got, streams = [None, None], [torch.cuda.Stream() for _ in jobs]

    def run(i):
        for _ in range(20):
            got[i] = work(*jobs[i], stream=streams[i])
        streams[i].synchronize()

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    for g, w in zip(got, want):
        for a, b in zip(g, w):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ calls as programs make them
def test_two_runs_give_the_same_bits():
    T, k, E, H = 2500, 4, 64, 512
    idx = index(T, k, E, "holes")
    o, w, dy = rnd(T * k, H, dtype=BF16), rnd(T, k), rnd(T, H, dtype=BF16, seed=1)
    ids = index(T, 1, 30, "holes")[:, 0]
    A, B, scale = bank(30, 16, H, H, BF16)
    wide = bank(3, 64, H, H, BF16)
    wids = index(T, 1, 3, "holes")[:, 0]

    def go():
        r = moe.moe_sort(idx, E)
        do = torch.zeros(T * k, H, dtype=BF16, device="cuda")
        return [r.perm, r.inv, r.offsets, moe.moe_collect(o, w, r), *moe.moe_collect_backward(dy, o, w, r, do=do),
                moe.moe_adapters(dy, o[:T], A, B, scale, moe.moe_sort(ids, 30)),
                moe.moe_adapters(dy, o[:T], *wide, moe.moe_sort(wids, 3))]

    first = go()
    for _ in range(3):
        for a, b in zip(first, go()):
            assert torch.equal(a, b)


def test_side_stream_and_graph_replay():
    # on a stream of its own, then captured with the workspaces of the capture; replays see new inputs
    T, k, E, H = 900, 3, 40, 264
    x, idx, w = rnd(T, H, dtype=BF16), index(T, k, E, "holes"), rnd(T, k)
    ids = index(T, 1, 9, "holes")[:, 0]
    A, B, scale = bank(9, 16, H, H, BF16)
    wide = bank(9, 64, H, H, BF16)

    def step(stream=None):
        xs, r = moe.moe_dispatch(x, idx, E, xs=torch.zeros(T * k, H, dtype=BF16, device="cuda"), stream=stream)
        y = moe.moe_collect(xs, w, r, stream=stream)
        h, kept = moe.moe_swiglu_save(xs, xs, rows=r.offsets[E:], stream=stream)
        y2 = moe.moe_adapters(x, y, A, B, scale, moe.moe_sort(ids, 9, stream=stream), stream=stream)
        y3 = moe.moe_adapters(x, y, *wide, moe.moe_sort(ids, 9, stream=stream), stream=stream)
        return y, y2, y3, xs, r.perm

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(stream=s)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for seed in (5, 6):
        x.copy_(rnd(T, H, dtype=BF16, seed=seed))
        idx.copy_(index(T, k, E, "outside", seed=seed))
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = step()
        for _, out in graphs:
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_training_step_of_routed_experts():
    # dispatch -> expert products -> SwiGLU kept in 8 bits -> products -> collect, and back: against the
    # chain's formulas in 64 bits with the activations that the checkpoint restores
    T, k, E, H, F = 96, 2, 5, 64, 80
    x, dy, w = rnd(T, H), rnd(T, H, seed=1), rnd(T, k, seed=2).abs()
    idx = index(T, k, E, "padded")
    Wg, Wu, Wd = rnd(E, F, H, sigma=H ** -0.5), rnd(E, F, H, seed=3, sigma=H ** -0.5), rnd(E, H, F, seed=4, sigma=F ** -0.5)
    xs, r = moe.moe_dispatch(x, idx, E, xs=torch.zeros(T * k, H, device="cuda"))
    off = r.offsets.tolist()
    total, rows = off[E], r.offsets[E:]

    def products(a, Ws):
        out = torch.zeros(T * k, Ws.shape[1], dtype=a.dtype, device="cuda")
        for e in range(E):
            out[off[e]:off[e + 1]] = a[off[e]:off[e + 1]] @ Ws[e].to(a.dtype).T
        return out

    g, u = products(xs, Wg), products(xs, Wu)
    h, kept = moe.moe_swiglu_save(g, u, rows=rows)
    o = products(h, Wd)
    y = moe.moe_collect(o, w, r)
    do, dw = moe.moe_collect_backward(dy, o, w, r, do=torch.zeros(T * k, H, device="cuda"))
    dh = products(do, Wd.transpose(1, 2))
    dg, du, again = moe.moe_swiglu_backward(dh, kept, rebuild_h=True, rows=rows)
    dxs = products(dg, Wg.transpose(1, 2)) + products(du, Wu.transpose(1, 2))
    dx = moe.moe_dispatch_backward(dxs, r)

    # 64 bits
    tok = (r.perm[:total].long() // k)
    ent = r.perm[:total].long()
    gi, ui = (moe.moe_act_load(c).to(F64)[:total] for c in (kept.g, kept.u))
    X, DY, w64 = x.to(F64), dy.to(F64), w.to(F64).reshape(-1)
    of = torch.repeat_interleave(torch.arange(E), torch.tensor([off[e + 1] - off[e] for e in range(E)])).cuda()
    mul = lambda a, Ws: torch.einsum("rh,rfh->rf", a, Ws.to(F64)[of])  # noqa: E731
    G, Uu = mul(X[tok], Wg), mul(X[tok], Wu)
    O = mul(G / (1 + torch.exp(-G)) * Uu, Wd)
    Y = torch.zeros(T, H, dtype=F64, device="cuda").index_add_(0, tok, w64[ent][:, None] * O)
    DO = w64[ent][:, None] * DY[tok]
    DW = torch.zeros(T * k, dtype=F64, device="cuda")
    DW[ent] = (DY[tok] * O).sum(1)
    DH = mul(DO, Wd.transpose(1, 2))
    S = 1 / (1 + torch.exp(-gi))
    DG, DU = DH * ui * S * (1 + gi * (1 - S)), DH * gi * S
    DX = torch.zeros(T, H, dtype=F64, device="cuda").index_add_(0, tok, mul(DG, Wg.transpose(1, 2)) + mul(DU, Wu.transpose(1, 2)))
    # about 2(H + F) + 20 fp32 roundings along the longest path; the values are of order 1 to 10, so
    # 400 roundings of a magnitude of 32 bound every one of them
    for got, want in ((y, Y), (dw.reshape(-1), DW), (do[:total], DO), (dg[:total], DG), (du[:total], DU),
                      (again[:total], gi * S * ui), (dx, DX)):
        assert float(want.abs().max()) < 32
        assert float((got.to(F64) - want).abs().max()) <= 400 * U * 32


def test_adapters_beside_the_packed_layer():
    # many requests served at once: the packed layer's output plus each request's adapter, against the oracle
    L = W.layer("tiny")
    layer = hp.gpu_pack(L)
    Wr, b = W.device_router(L)
    T, n, r = 16, 4, 8
    x = W.device_x(T, L.H)
    ids = torch.tensor([-1, 0, 1, 2, 3, 3, 2, 0] * 2, dtype=torch.int32, device="cuda")
    A, B, scale = bank(n, r, L.H, L.H, BF16)
    y = moe.moe_layer_forward(x, Wr, b, layer, L.k)
    out = moe.moe_adapters(x, y, A, B, scale, moe.moe_sort(ids, n))
    base = hp.orc.moe_forward(hp.oracle_pack(L, range(L.E)), W.x_bf16_bits(T, L.H), W.router_w(L.E, L.H), None, L.k)
    base = torch.from_numpy((base.astype(np.uint32) << 16).view(np.float32).astype(np.float64)).cuda()
    want, mag = ref_adapters(x, base, A, B, scale, ids)
    # the layer's own tolerance, and what the adapters add
    tol = hp.TOL * float(base.abs().max()) + half_step(BF16) * want.abs() + 2.0 ** -12 * mag
    assert bool(((out.to(F64) - want).abs() <= tol).all())


def test_layer_routing_matches_sort():
    # the layer's own permutation and moe_sort of its choice agree
    L = W.layer("tiny")
    layer = hp.gpu_pack(L)
    Wr, b = W.device_router(L)
    T = 300
    dbg = {f: torch.empty(T * L.k, dtype=torch.int32, device="cuda") for f in ("topk_idx", "perm", "inv")}
    dbg["counts"] = torch.empty(L.E, dtype=torch.int32, device="cuda")
    moe.moe_layer_forward(W.device_x(T, L.H), Wr, b, layer, L.k, debug=dbg)
    r = moe.moe_sort(dbg["topk_idx"].reshape(T, L.k), L.E)
    assert torch.equal(r.perm, dbg["perm"]) and torch.equal(r.inv, dbg["inv"])
    assert torch.equal(r.offsets[1:] - r.offsets[:-1], dbg["counts"])

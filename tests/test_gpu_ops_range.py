"""The operators around the expert products at the ends of their types' ranges and of their waits.  Tolerances count
roundings: 2^-24 of the value for one in fp32, half a step of the type for the stored value.
"""
import ctypes as C

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import mixed_precision_quantized_fp32_b200 as moe  # noqa: E402
from mixed_precision_quantized_fp32_b200 import _lib  # noqa: E402
from tests.test_gpu_ops import BF16, F16, F32, F64, U, adapters_near, bank, half_step, index, ref_adapters, rnd  # noqa: E402


# ------------------------------------------------------------------ adapters: small low-rank terms
@pytest.mark.parametrize("small", [0, 14, 20, 24, 100])
@pytest.mark.parametrize("T,r", [(40, 16), (40, 128), (300, 32), (2100, 16), (2100, 64), (2100, 128)])  # tiles of 16 and of 64 tokens
def test_adapters_of_small_terms_in_fp16(T, r, small):
    # scale * A x near 2^-small, far below fp16's normal range, and B large enough that their product
    # is an ordinary number of the type: it has the bits that a product in 32 bits gives
    K, N, n = 64, 72, 2
    ids = index(T, 1, n, "all")[:, 0]
    x, y = rnd(T, K, dtype=F16), torch.zeros(T, N, dtype=F16, device="cuda")
    A, B, _ = bank(n, r, K, N, F16)
    up = min(small - 10, 13)
    B = (B.float() * (r ** 0.5 * 2.0 ** up)).clamp(-6e4, 6e4).half()
    x[3], x[5, 1:] = 0, 0                        # a row without a term, one with a single product
    scale = torch.full((n,), 2.0 ** -small, device="cuda")
    out = moe.moe_adapters(x, y, A, B, scale, moe.moe_sort(ids, n)).to(F64)
    want, mag = ref_adapters(x, y, A, B, scale, ids)
    # the magnitudes of P and of B, for what its two terms leave
    P, b = torch.empty(T, r, dtype=F64, device="cuda"), torch.empty(T, N, dtype=F64, device="cuda")
    for a in range(n):
        at = torch.nonzero(ids == a).reshape(-1)
        P[at] = (x[at].to(F64) @ A[a].to(F64).T).abs() * 2.0 ** -small
        b[at] = B[a].to(F64).abs().sum(1)
    # K products summed on the tensor cores (each sum off by at most 2^-23 of the magnitudes), 2r terms
    # summed again, scale and y; two fp16 terms of P: 2^-22 of a value, 2^-38 of its row's largest
    tol = half_step(F16) * want.abs() + 2.0 ** -25 + (K + 2 * r + 8) * 2.0 ** -23 * mag + 2.0 ** -22 * mag \
        + 2.0 ** -38 * P.max(1, keepdim=True).values * b
    assert bool(((out - want).abs() <= tol).all())
    assert not bool(out[3].any())
    if small < 100:                              # ordinary numbers, so that half a step is what counts
        assert float(want.abs().median()) > 2.0 ** -12


# ------------------------------------------------------------------ SwiGLU: far gates, large factors
def swiglu_errors(g, u, dh, dtype):
    """Bounds on the fp32 errors of h, du and dg, in 64 bits.  The kernels take v = 2^-32 exp(-g), 2^32 s = 1/(2^-32 + v)
    and 1 - s = v * 2^32 s.  v is off by
      fp32: twice 2 units in the last place of exp(-g/2), 8 U, and U for the square: 9 U;
      16-bit: the exponent 32 + 1.443 |g| is rounded once and its factor once before, (32 + 1.8 |g|) U ln 2, and
        the power is off by 2^-22: (27 + 1.3 |g|) U.
    The sum adds U and the reciprocal, one unit in the last place, 2 U to s; its product another U to 1 - s.  s
    is held in steps of 2^-149 where it is subnormal.  Products and sums behind it add U each."""
    v = 9.0 if dtype is F32 else 27 + 1.3 * g.abs()
    s, o = torch.sigmoid(g), torch.sigmoid(-g)
    low = 2.0 ** -148
    h = (v + 5) * U * (g * s * u).abs() + low * (1 + g.abs()) * u.abs()
    du = (v + 5) * U * (g * s * dh).abs() + low * (1 + g.abs()) * dh.abs()
    # d = s (1 + g (1 - s)): s's error, that of 1 - s times g, one rounding of the sum and one of the product; then two products
    inner = 1 + (g * o).abs()
    dg = ((v + 3) + (v + 4) + 4) * U * (dh * u).abs() * s * inner + low * inner * (dh * u).abs() \
        + low * torch.minimum(dh.abs(), u.abs())
    return h, du, dg


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("F", [256, 264, 260, 258, 257])     # 8 values a lane without and with gaps, fours, pairs, single
def test_swiglu_of_far_gates_and_large_factors(F, dtype):
    # the sigmoid at -104 to 90 beside factors up to 1e30: a finite result stays finite and keeps its bits,
    # also where exp(-g) or dh * u pass fp32's range
    R = 48
    lo, hi = torch.linspace(-104, 80, R, device="cuda")[:, None], torch.linspace(0, 10, F, device="cuda")
    g = (lo + hi).to(dtype)
    top = 4.0 if dtype is F16 else 30.0
    ten = torch.full((), 10.0, dtype=F64, device="cuda")
    far = torch.pow(ten, torch.linspace(-4, top, R, device="cuda", dtype=F64))[:, None]
    u = (rnd(R, F, seed=1).to(F64) * far).to(dtype)
    dh = (rnd(R, F, seed=2).to(F64) * far.flip(0)[torch.randperm(R, generator=torch.Generator().manual_seed(3))]).to(dtype)
    u[:8], dh[:8] = (v[:8].to(F64).sign().to(dtype) * float(10 ** top) for v in (u, dh))     # both large where s is least
    h, kept = moe.moe_swiglu_save(g, u)
    wide = torch.empty(R, F, device="cuda")
    gk, uk = (moe.moe_act_load(c, x=wide.clone()).to(F64) for c in (kept.g, kept.u))
    dg, du, again = moe.moe_swiglu_backward(dh, kept, rebuild_h=True)

    def close(got, want, err):
        top = torch.finfo(dtype)
        fits = want.abs() < top.max * (1 - top.eps)
        assert bool(fits.any())
        tol = half_step(dtype) * want.abs() + (1 + half_step(dtype)) * err + top.tiny * top.eps / 2
        return bool((~fits | ((got.to(F64) - want).abs() <= tol)).all())

    def formulas(g, u, dh):
        s = torch.sigmoid(g)
        return g * s * u, dh * g * s, dh * u * s * (1 + g * torch.sigmoid(-g))

    d64 = dh.to(F64)
    want, err = formulas(g.to(F64), u.to(F64), d64), swiglu_errors(g.to(F64), u.to(F64), d64, dtype)
    assert close(h, want[0], err[0])
    want, err = formulas(gk, uk, d64), swiglu_errors(gk, uk, d64, dtype)
    assert close(again, want[0], err[0]) and close(du, want[1], err[1]) and close(dg, want[2], err[2])


# ------------------------------------------------------------------ adapters: waits that run out
@pytest.mark.parametrize("K,r", [(40, 16), (264, 64), (2056, 64), (1096, 128)])   # one stage a block to more than the ring holds
def test_adapters_wait_that_runs_out_is_reported_and_leaves_the_context_usable(K, r):
    # the kernel of long batches keeps the completion of its first products back and its waits get 200k cycles
    # (0.1 ms): every block ends by itself, the status says so, and a call after it is right.  A status that
    # nothing timed out for stays as it was.
    T, N, n = 2100, 520, 3
    ids = index(T, 1, n, "holes")[:, 0]
    x, y = rnd(T, K, dtype=BF16), rnd(T, N, dtype=BF16, seed=1)
    A, B, scale = bank(n, r, K, N, BF16)
    routes = moe.moe_sort(ids, n)
    want, mag = ref_adapters(x, y, A, B, scale, ids)
    status, out = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty_like(y)

    def call(**hooks):
        d = _lib.MoeDebug(status=status.data_ptr(), **hooks)
        _lib.check("moe_adapters_debug", _lib.load().moe_adapters_debug(
            x.data_ptr(), K, y.data_ptr(), N, 0, T, K, N, r, n, A.data_ptr(), B.data_ptr(), scale.data_ptr(),
            routes.perm.data_ptr(), routes.offsets.data_ptr(), out.data_ptr(), N, C.byref(d),
            torch.cuda.current_stream().cuda_stream))
        torch.cuda.synchronize()
        return _lib.STATUS[int(status)]

    assert call() == "MOE_OK" and adapters_near(out, want, mag, K, r, BF16)
    assert call(test_withhold=1, wait_cycles=200_000) == "MOE_ERR_TIMEOUT"
    status.zero_()
    for _ in range(3):
        out.zero_()
        assert call() == "MOE_OK" and adapters_near(out, want, mag, K, r, BF16)
    again = moe.moe_adapters(x, y, A, B, scale, routes, status=status)
    assert torch.equal(again, out) and int(status) == 0


# ------------------------------------------------------------------ adapters: every bit
SHAPES = [(1, 4096, 4096, 16, 3), (40, 1032, 264, 8, 3), (130, 4096, 520, 32, 4), (64, 4104, 2000, 120, 2), (300, 2056, 1096, 64, 2),
          (128, 136, 520, 56, 5), (260, 1000, 40, 24, 40),                                            # tiles of 16 tokens
          (2100, 1096, 520, 32, 5), (2100, 8, 72, 8, 3), (2060, 2056, 328, 40, 2), (2049, 4104, 2000, 120, 1), (2500, 1000, 72, 128, 9),
          (1100, 2056, 1096, 64, 2)]                                                                   # and of 64


def whole(shape, top, seed):
    return torch.randint(-top, top + 1, shape, generator=torch.Generator().manual_seed(seed + sum(shape)))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,K,N,r,n", SHAPES)
def test_adapters_are_exact_where_every_sum_is(T, K, N, r, n, dtype):
    # whole numbers: A x needs up to 16 bits, more than the type has, and the outputs are differences of two of
    # its elements, which are small.  Rows 2i and 2i+1 of A differ by one at the places k = i mod r/2, so
    # a bit of A x that is lost, or a k, an element of the rank or a block's share left out, shows in the outputs.
    ids = index(T, 1, n, "holes" if T > 1 else "all")[:, 0]
    x = whole((T, K), 1, 1).to(dtype)
    A = whole((n, r // 2, 1, K), 126, 2).expand(n, r // 2, 2, K).clone()
    pair = torch.arange(K) % (r // 2)
    A[:, pair, 1, torch.arange(K)] += 2 * whole((n, K), 1, 3).ne(0) - 1
    A = A.reshape(n, r, K).to(dtype)
    take = torch.zeros(n, N, r // 2)
    for seed in (4, 5):                          # each output takes two pairs, with either sign
        at = torch.randint(0, r // 2, (n, N, 1), generator=torch.Generator().manual_seed(seed + N))
        take.scatter_(2, at, (2 * (whole((n, N, 1), 1, seed) > 0) - 1).float())
    B = torch.stack([take, -take], 3).reshape(n, N, r).to(dtype)
    y, scale = whole((T, N), 8, 6).to(dtype), torch.tensor([1.0, 0.5, -1.0, 2.0])[torch.arange(n) % 4]
    x, A, B, y, scale = (t.cuda() for t in (x, A, B, y, scale))
    routes = moe.moe_sort(ids, n)
    want, _ = ref_adapters(x, y, A, B, scale, ids)
    P = torch.stack([x.to(F64) @ a.to(F64).T for a in A])
    # P in 16 bits, so that its two terms hold all of it (and more than the type's bits); results in the type's
    assert float(P.abs().max()) < 2 ** 15 and (K < 100 or float(P.abs().max()) > 2 ** 11)
    assert torch.equal(want.to(dtype).to(F64), want) and float((want - y.to(F64)).abs().max()) >= 1
    assert torch.equal(moe.moe_adapters(x, y, A, B, scale, routes).to(F64), want)
    z = y.clone()
    assert torch.equal(moe.moe_adapters(x, z, A, B, scale, routes, out=z).to(F64), want)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,K,N,r,n", SHAPES)
def test_adapters_as_a_whole(T, K, N, r, n, dtype):
    # the term alone (y = 0), over all outputs: each is off by at most half a step of itself, by P's two terms
    # (2^-17 of each product) and by fp32 sums, whose errors, about 2^-24 times a few, are far below 2^-14 of their root mean square
    ids = index(T, 1, n, "all")[:, 0]
    x, y = rnd(T, K, dtype=dtype), torch.zeros(T, N, dtype=dtype, device="cuda")
    A, B, scale = bank(n, r, K, N, dtype)
    want, _ = ref_adapters(x, y, A, B, scale, ids)
    err = moe.moe_adapters(x, y, A, B, scale, moe.moe_sort(ids, n)).to(F64) - want
    rms = lambda t: float(t.square().mean().sqrt())  # noqa: E731
    assert rms(err) <= (half_step(dtype) + 2.0 ** -14) * rms(want)


# ------------------------------------------------------------------ adapters: the largest low-rank terms
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,r", [(40, 16), (300, 128), (2100, 32), (2100, 128)])      # tiles of 16 and of 64 tokens
def test_adapters_of_the_largest_terms(T, r, dtype):
    # scale * A x at fp32's largest numbers, which the value type rounds to an infinity, beside a B that brings
    # them back: the outputs are finite.  An infinity and a NaN stay what they are.
    K, N = 64, 40
    x, y = torch.zeros(T, K, dtype=dtype, device="cuda"), torch.zeros(T, N, dtype=dtype, device="cuda")
    x[:, 0], x[1::2, 0] = 1.0, -1.0
    A, B = torch.zeros(1, r, K, dtype=dtype, device="cuda"), torch.zeros(1, N, r, dtype=dtype, device="cuda")
    A[0, 0, 0], A[0, 1, 1] = 1.0, 2.0
    low = 2.0 ** (-100 if dtype is BF16 else -24)
    B[0, :, 0] = low
    B[0, :, 1] = torch.tensor([low, -low], device="cuda").repeat(N // 2)
    x[5, 1], x[6, 1], x[7, 1] = 1.0, float("nan"), -1.0       # 2 * scale: beyond fp32
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    out = moe.moe_adapters(x, y, A, B, torch.full((1,), torch.finfo(F32).max, device="cuda"), moe.moe_sort(ids, 1)).to(F64)
    inf = float("inf")
    want = x[:, :1].to(F64) * torch.finfo(F32).max * low + torch.zeros(N, dtype=F64, device="cuda")
    want[5, ::2], want[5, 1::2], want[7, ::2], want[7, 1::2] = inf, -inf, -inf, inf
    if dtype is F16:
        want[want.abs() > 65504] *= inf          # 2^104: beyond the type, with its sign
    rest = torch.arange(T, device="cuda") != 6
    assert bool(torch.isnan(out[6]).all())
    # P's terms leave 2^-17 of it, and the product with a power of two is exact
    near = (out - want).abs() <= (half_step(dtype) + 2.0 ** -16) * want.abs()
    assert bool(((out == want) | (torch.isfinite(want) & near))[rest].all())

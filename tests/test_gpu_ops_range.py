"""The operators around the expert products at the ends of their types' ranges.  Tolerances count
roundings: 2^-24 of the value for one in fp32, half a step of the type for the stored value.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

import mixed_precision_quantized_fp32_b200 as moe  # noqa: E402
from tests.test_gpu_ops import F16, F64, bank, half_step, index, ref_adapters, rnd  # noqa: E402


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

// Activations kept in 8 bits for a backward pass, and the SwiGLU that keeps its inputs
// that way (the layer's integer formats applied to activations: symmetric codes, one
// scale per row and group of 32).
//
//   save   e = smallest whole number with max|x| <= 127 * 2^e over the group, at least
//          -126 and at most 121 (fp16: 9); q = rint(x * 2^-e), clamped to [-127, 127]
//   load   x^ = q * 2^e
//   SwiGLU forward   h = silu(g) * u, codes of g and u
//   backward         s = 1/(1+exp(-g^));  du = dh * g^ s;  dg = dh * u^ * s (1 + g^ (1-s));
//                    h^ = g^ s u^ (for the down projection's weight gradient)
//
// The scale is a power of two, so that x * 2^-e and q * 2^e are exact: a code is the
// correctly rounded one whatever computes it, no value needs a division, and q * 2^e is
// exact in bf16.  The price is a step of up to 2/127 of the group's maximum, where a
// free scale has 1/127.  A group that holds an infinity or a NaN keeps that as exponent
// byte 255 with zero codes: it is restored as NaN (0 * inf), never as finite values.
//
// Memory bounds all of these.  A quad of lanes takes one group, eight values a lane, so
// bf16 loads are 16 bytes and code stores 8 bytes a lane, consecutive over the warp, and
// the group's maximum takes two shuffles.  Rows whose pitch or start does not allow that
// run with fewer values a lane.  Of the measured copy rate:
//   save and load, 8192 x 4096 bf16 (203 MB)               31.2 us, 101%
//   SwiGLU forward and backward, 4096 x 14336 bf16 (1.06 GB)  162 us, 102%
//   widths in fours, in pairs and odd: save and load of 8192 x 4092, 4094, 4095 47, 49, 68 us
//   (67, 64, 46%), SwiGLU of 4096 x 5004, 5002, 5001 71, 82, 113 us (81, 70, 51%)
#include <initializer_list>
#include <type_traits>

#include "ops_common.cuh"

namespace moe {

constexpr int kGroup = 32;
constexpr int kEmin = -126;

template <typename T> __device__ __forceinline__ constexpr int emax() { return 121; }  // 127 * 2^121 < 2^128
template <> __device__ __forceinline__ constexpr int emax<__half>() { return 9; }       // 127 * 2^9 < 65504

// Exponent byte (e + 127; 255: not finite) of a group whose largest |x| has these fp32 bits.
template <typename T>
__device__ __forceinline__ uint32_t group_exp(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return 255u;
  // exponent of amax - 6, one more if its significand is above 127/64
  const int e = (int)((amax_bits + 0x1FFFFu) >> 23) - 127 - 6;
  return (uint32_t)(min(max(e, kEmin), emax<T>()) + 127);
}

// 2^-e of an exponent byte; 0 for the byte of a group that is not finite.
__device__ __forceinline__ float inv_step(uint32_t eb) { return eb == 255u ? 0.0f : __uint_as_float((254u - eb) << 23); }
// 2^e; infinity for byte 255, which makes 0 * step a NaN.
__device__ __forceinline__ float step_of(uint32_t eb) { return __uint_as_float(eb << 23); }

// The code sits in the low byte of x * 2^-e + 1.5 * 2^23: that sum is rounded to a whole
// number, to nearest even, by the addition itself.
__device__ __forceinline__ uint32_t code_bits(float x, float inv) {
  return __float_as_uint(fmaf(x, inv, 12582912.0f));
}
__device__ __forceinline__ float clamp127(float x) { return fminf(fmaxf(x, -127.0f), 127.0f); }

// Codes of N values, up to four in a word.  Only the highest exponent can leave values beyond 127
// steps, and only 255 stands for values without codes: both take the branch.
template <typename T, int N>
__device__ __forceinline__ void encode(const float (&v)[N], uint32_t eb, uint32_t (&q)[(N + 3) / 4]) {
  uint32_t c[N];
  if (eb < (uint32_t)(emax<T>() + 127)) {
    const float inv = inv_step(eb);
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = code_bits(v[i], inv);
  } else {
    const float inv = inv_step(eb);
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = eb == 255u ? 0u : code_bits(clamp127(v[i] * inv), 1.0f);
  }
  if constexpr (N < 4) {
    q[0] = N == 1 ? c[0] & 0xFFu : __byte_perm(c[0], c[N - 1], 0x4440) & 0xFFFFu;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      q[i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040), __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040), 0x5410);
  }
}
template <typename T>
__device__ __forceinline__ uint2 encode8(const float (&v)[8], uint32_t eb) {
  uint32_t q[2];
  encode<T, 8>(v, eb, q);
  return make_uint2(q[0], q[1]);
}

// Eight values as they lie in memory.
template <typename T> struct Eight { uint4 a[sizeof(T) / 2]; };
template <typename T>
__device__ __forceinline__ Eight<T> load8(const T* p) {
  Eight<T> e;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) e.a[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  return e;
}
template <typename T>
__device__ __forceinline__ void values8(const Eight<T>& e, float (&v)[8]) {
  constexpr int N = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
    float f[N];
    decode_raw<T, N>(e.a[i], f);
#pragma unroll
    for (int j = 0; j < N; ++j) v[N * i + j] = f[j];
  }
}

// Largest |x| over the quad's 32 values as fp32 bits.  Magnitudes order as their bits do,
// infinities and NaN on top, so the maximum is an integer one: of 16-bit halves two at once.
template <typename T>
__device__ __forceinline__ uint32_t quad_amax(const Eight<T>& e) {
  if constexpr (sizeof(T) == 4) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      m = max(m, max(max(e.a[i].x & 0x7FFFFFFFu, e.a[i].y & 0x7FFFFFFFu), max(e.a[i].z & 0x7FFFFFFFu, e.a[i].w & 0x7FFFFFFFu)));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  } else {
    constexpr uint32_t A = 0x7FFF7FFFu;
    uint32_t m = __vmaxu2(__vmaxu2(e.a[0].x & A, e.a[0].y & A), __vmaxu2(e.a[0].z & A, e.a[0].w & A));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    m = max(m & 0xFFFFu, m >> 16);
    return __float_as_uint(unpack2<T>(m).x);
  }
}

// q * 2^e of N codes.  One byte permute makes 2^23 + 128 + q as a float, one fused
// multiply-add takes the offset off and scales; both are exact.  Steps of 2^103 and more,
// where the offset times the step would overflow, and NaN groups multiply afterwards.
template <int N>
__device__ __forceinline__ void decode(const uint32_t (&q)[(N + 3) / 4], uint32_t eb, float (&v)[N]) {
  const float step = step_of(eb);
  uint32_t w[(N + 3) / 4];
#pragma unroll
  for (int i = 0; i < (N + 3) / 4; ++i) w[i] = q[i] ^ 0x80808080u;
  if (eb < 230u) {
    const float off = -8388736.0f * step;
#pragma unroll
    for (int i = 0; i < N; ++i)
      v[i] = fmaf(__uint_as_float(__byte_perm(w[i / 4], 0x4B000000u, 0x7440 + i % 4)), step, off);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      v[i] = (__uint_as_float(__byte_perm(w[i / 4], 0x4B000000u, 0x7440 + i % 4)) - 8388736.0f) * step;
  }
}
__device__ __forceinline__ void decode8(uint2 c, uint32_t eb, float (&v)[8]) {
  const uint32_t q[2] = {c.x, c.y};
  decode<8>(q, eb, v);
}

// Arithmetic on one value or on two, which share an instruction (f32x2).  What there is to compute for a
// value takes as long as its bytes, so pairs are taken (backward of 4096 x 14336 bf16 92 us, with single
// values 96; forward of 4096 x 5001 bf16 54, 56), but for the backward pass with fewer than eight values
// a lane, which they do not help (4096 x 5002 bf16: 52 us for 47).
__device__ __forceinline__ uint64_t join(float2 v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
  return r;
}
__device__ __forceinline__ float2 split(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float mul_add(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float2 add(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(join(a)), "l"(join(b)));
  return split(r);
}
__device__ __forceinline__ float2 mul(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(join(a)), "l"(join(b)));
  return split(r);
}
__device__ __forceinline__ float2 mul_add(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(join(a)), "l"(join(b)), "l"(join(c)));
  return split(r);
}
template <typename F> __device__ __forceinline__ F all(float v);
template <> __device__ __forceinline__ float all<float>(float v) { return v; }
template <> __device__ __forceinline__ float2 all<float2>(float v) { return make_float2(v, v); }
template <float (*Op)(float)> __device__ __forceinline__ float each(float a) { return Op(a); }
template <float (*Op)(float)> __device__ __forceinline__ float2 each(float2 a) { return make_float2(Op(a.x), Op(a.y)); }
template <float (*Op)(float, float)> __device__ __forceinline__ float each(float a, float b) { return Op(a, b); }
template <float (*Op)(float, float)> __device__ __forceinline__ float2 each(float2 a, float2 b) {
  return make_float2(Op(a.x, b.x), Op(a.y, b.y));
}

__device__ __forceinline__ float exp2_fast(float x) {  // to 2^-22 of the value
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float reciprocal(float x) {  // to a unit of the last place
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ float not_below_110(float x) { return fmaxf(x, -110.0f); }
// The larger magnitude with the sign of a * b (NaN if either is one), and the smaller.
__device__ __forceinline__ float larger(float a, float b) {
  float r;
  asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float smaller(float a, float b) { return fminf(fabsf(a), fabsf(b)); }

// s = 1/(1+exp(-g)) and 1 - s.  With v = 2^-32 exp(-g), which stays below 2^127 (from -110 on s is zero),
//   2^32 s = 1/(2^-32 + v)   and   1 - s = v * 2^32 s:
// nothing overflows, s keeps its bits down to fp32's least numbers (1/(1+exp(-g)) would be zero from
// -88 on), and 1 - s loses none to a subtraction.  fp32 values: s to 12 * 2^-24 of it, by the library's
// exponential (its square, since of -g it would overflow).  16-bit values: to (31 + 1.3 |g|) 2^-24, as v is a
// power of two of one rounded product; 2^-16.5 at -104, far below their own steps.
template <typename F> struct Sigmoid {
  F s, rest;
};
template <typename T, typename F>
__device__ __forceinline__ Sigmoid<F> sigmoid(F g) {
  const F b = each<not_below_110>(g);
  F v;
  if constexpr (sizeof(T) == 4) {
    const F root = mul(each<exp_of>(mul(b, all<F>(-0.5f))), all<F>(0x1p-16f));
    v = mul(root, root);
  } else {
    v = each<exp2_fast>(mul_add(b, all<F>(-1.44269504f), all<F>(-32.0f)));  // 1/ln 2
  }
  const F s32 = each<reciprocal>(add(v, all<F>(0x1p-32f)));
  return {mul(s32, all<F>(0x1p-32f)), mul(v, s32)};
}

// silu(g) * u.  At g = -inf this is -inf * 0: NaN, as the formula says.
template <typename T, typename F>
__device__ __forceinline__ F swiglu(F g, F u) {
  return mul(mul(g, sigmoid<T>(g).s), u);
}

// From g, u and dh: du in g, h in u and dg in dh.  dg = d * dh * u with d = s (1 + g (1 - s)), at most 1.1: dh * u
// may pass fp32's range where the whole does not, and d times the smaller of the two may fall below it, so
// d takes the larger one first.  (In fp16 neither can happen.)
template <typename T, typename F>
__device__ __forceinline__ void swiglu_grad(F& g, F& u, F& dh) {
  const Sigmoid<F> y = sigmoid<T>(g);
  const F a = mul(g, y.s), d = mul(y.s, mul_add(g, y.rest, all<F>(1.0f)));
  F dg;
  if constexpr (std::is_same<T, __half>::value) dg = mul(mul(d, dh), u);
  else dg = mul(mul(d, each<larger>(dh, u)), each<smaller>(dh, u));
  g = mul(dh, a), u = mul(a, u), dh = dg;
}

// Eight values, in pairs.
template <typename T>
__device__ __forceinline__ void swiglu8(float (&g)[8], const float (&u)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 h = swiglu<T>(make_float2(g[i], g[i + 1]), make_float2(u[i], u[i + 1]));
    g[i] = h.x, g[i + 1] = h.y;
  }
}
template <typename T>
__device__ __forceinline__ void swiglu_grad8(float (&g)[8], float (&u)[8], float (&dh)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    float2 a = make_float2(g[i], g[i + 1]), b = make_float2(u[i], u[i + 1]), d = make_float2(dh[i], dh[i + 1]);
    swiglu_grad<T>(a, b, d);
    g[i] = a.x, g[i + 1] = a.y, u[i] = b.x, u[i + 1] = b.y, dh[i] = d.x, dh[i + 1] = d.y;
  }
}

// Where a lane works: group `at` of the rows in order, value `col` of row `row`.
struct Place {
  int64_t row, col;
  int grp;
  bool in;  // the lane has values there
};

// ---------------------------------------------------------------- eight values a lane
// FLAT: F is a multiple of 32 and every matrix is without gaps, so the groups of all rows
// follow one another and a lane's place needs no division by the groups a row.
// A thread takes two places, 64 groups apart, with both places' loads in flight at once.
constexpr int kPlaces = 2;
constexpr int kGroupsPerBlock = 64 * kPlaces;

__device__ __forceinline__ int row_count(int R, const int32_t* n_rows) {
  return n_rows ? min(R, max(0, __ldg(n_rows))) : R;
}

template <bool FLAT>
__device__ __forceinline__ Place place8(int i, int G, int rows, int F) {
  Place p;
  const uint32_t at = blockIdx.x * (uint32_t)kGroupsPerBlock + i * 64u + (threadIdx.x >> 2);
  if (FLAT) {
    p.row = 0;
    p.grp = (int)at;
    p.col = (int64_t)at * kGroup + (threadIdx.x & 3) * 8;
    p.in = at < (uint32_t)rows * (uint32_t)G;
  } else {
    const uint32_t row = at / (uint32_t)G;
    p.row = row;
    p.grp = (int)(at - row * (uint32_t)G);
    p.col = p.grp * kGroup + (threadIdx.x & 3) * 8;
    p.in = row < (uint32_t)rows && p.col < F;
  }
  return p;
}

template <typename T, bool FLAT>
__global__ void __launch_bounds__(256) act_save_kernel(const T* __restrict__ x, int64_t ldx, int R, int F,
                                                       int8_t* __restrict__ q, uint8_t* __restrict__ ex,
                                                       const int32_t* __restrict__ n_rows) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  const int G = (F + kGroup - 1) / kGroup, rows = row_count(R, n_rows);
  Place p[kPlaces];
  Eight<T> e[kPlaces];
#pragma unroll
  for (int i = 0; i < kPlaces; ++i) {
    p[i] = place8<FLAT>(i, G, rows, F);
    e[i] = Eight<T>{};
    if (p[i].in) e[i] = load8(x + p[i].row * ldx + p[i].col);
  }
#pragma unroll
  for (int i = 0; i < kPlaces; ++i) {
    const uint32_t eb = group_exp<T>(quad_amax(e[i]));
    if (!p[i].in) continue;
    float v[8];
    values8(e[i], v);
    *reinterpret_cast<uint2*>(q + p[i].row * F + p[i].col) = encode8<T>(v, eb);
    if ((threadIdx.x & 3) == 0) ex[p[i].row * G + p[i].grp] = (uint8_t)eb;
  }
}

template <typename T, bool FLAT>
__global__ void __launch_bounds__(256) act_load_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ ex,
                                                       int R, int F, T* __restrict__ x, int64_t ldx,
                                                       const int32_t* __restrict__ n_rows) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  const int G = (F + kGroup - 1) / kGroup, rows = row_count(R, n_rows);
  Place p[kPlaces];
  uint2 c[kPlaces];
  uint32_t eb[kPlaces];
#pragma unroll
  for (int i = 0; i < kPlaces; ++i) {
    p[i] = place8<FLAT>(i, G, rows, F);
    if (p[i].in) {
      c[i] = __ldg(reinterpret_cast<const uint2*>(q + p[i].row * F + p[i].col));
      eb[i] = __ldg(ex + p[i].row * G + p[i].grp);
    }
  }
#pragma unroll
  for (int i = 0; i < kPlaces; ++i) {
    if (!p[i].in) continue;
    float v[8];
    decode8(c[i], eb[i], v);
    store_vec<T, 8>(x + p[i].row * ldx + p[i].col, v);
  }
}

template <typename T, bool FLAT>
__global__ void __launch_bounds__(256) swiglu_save_kernel(const T* __restrict__ g, int64_t ldg, const T* __restrict__ u,
                                                          int64_t ldu, int R, int F, T* __restrict__ h, int64_t ldh,
                                                          int8_t* __restrict__ gq, uint8_t* __restrict__ ge,
                                                          int8_t* __restrict__ uq, uint8_t* __restrict__ ue,
                                                          const int32_t* __restrict__ n_rows) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  const int G = (F + kGroup - 1) / kGroup, rows = row_count(R, n_rows);
  Place p[kPlaces];
  Eight<T> e[kPlaces], f[kPlaces];
#pragma unroll
  for (int i = 0; i < kPlaces; ++i) {
    p[i] = place8<FLAT>(i, G, rows, F);
    e[i] = f[i] = Eight<T>{};
    if (p[i].in) {
      e[i] = load8(g + p[i].row * ldg + p[i].col);
      f[i] = load8(u + p[i].row * ldu + p[i].col);
    }
  }
#pragma unroll
  for (int i = 0; i < kPlaces; ++i) {
    const uint32_t ea = group_exp<T>(quad_amax(e[i])), eb = group_exp<T>(quad_amax(f[i]));
    if (!p[i].in) continue;
    const int64_t at = p[i].row * F + p[i].col, ge_at = p[i].row * G + p[i].grp;
    float a[8], b[8];
    values8(e[i], a);
    values8(f[i], b);
    *reinterpret_cast<uint2*>(gq + at) = encode8<T>(a, ea);
    *reinterpret_cast<uint2*>(uq + at) = encode8<T>(b, eb);
    if ((threadIdx.x & 3) == 0) {
      ge[ge_at] = (uint8_t)ea;
      ue[ge_at] = (uint8_t)eb;
    }
    swiglu8<T>(a, b);
    store_vec<T, 8>(h + p[i].row * ldh + p[i].col, a);
  }
}

// Five blocks an SM for 16-bit values (48 registers; without the bound 58, and 101 us for 92).
template <typename T, bool FLAT>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 5 : 4) swiglu_backward_kernel(
    const T* __restrict__ dh, int64_t lddh, const int8_t* __restrict__ gq, const uint8_t* __restrict__ ge,
    const int8_t* __restrict__ uq, const uint8_t* __restrict__ ue, int R, int F, T* __restrict__ dg, int64_t lddg,
    T* __restrict__ du, int64_t lddu, T* __restrict__ h, int64_t ldh, const int32_t* __restrict__ n_rows) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  const int G = (F + kGroup - 1) / kGroup, rows = row_count(R, n_rows);
  Place p[kPlaces];
  Eight<T> e[kPlaces];
  uint2 cg[kPlaces], cu[kPlaces];
  uint32_t eg[kPlaces], eu[kPlaces];
#pragma unroll
  for (int i = 0; i < kPlaces; ++i) {
    p[i] = place8<FLAT>(i, G, rows, F);
    if (!p[i].in) continue;
    const int64_t at = p[i].row * F + p[i].col, ge_at = p[i].row * G + p[i].grp;
    e[i] = load8(dh + p[i].row * lddh + p[i].col);
    cg[i] = __ldg(reinterpret_cast<const uint2*>(gq + at));
    cu[i] = __ldg(reinterpret_cast<const uint2*>(uq + at));
    eg[i] = __ldg(ge + ge_at);
    eu[i] = __ldg(ue + ge_at);
  }
#pragma unroll
  for (int i = 0; i < kPlaces; ++i) {
    if (!p[i].in) continue;
    float d[8], a[8], b[8];
    values8(e[i], d);
    decode8(cg[i], eg[i], a);
    decode8(cu[i], eu[i], b);
    swiglu_grad8<T>(a, b, d);
    store_vec<T, 8>(dg + p[i].row * lddg + p[i].col, d);
    store_vec<T, 8>(du + p[i].row * lddu + p[i].col, a);
    if (h) store_vec<T, 8>(h + p[i].row * ldh + p[i].col, b);
  }
}

// ---------------------------------------------------------------- fewer values a lane
// Any width, pitch and alignment: a lane has N consecutive values in accesses of V (4, 2 or 1,
// what widths, rows and codes are aligned to; N >= V).  A warp takes N groups of a row at once,
// S times, with all loads in flight, and finds the row once.  The number of instructions bounds
// these kernels, and few lanes a group save what each of them computes for it; but a larger N
// spreads an access over more lines.  Single values: save and load of 8192 x 4095 bf16 take 68 us
// with N = 2 (1: 76, 4: 71); the SwiGLU kernels, with more to do for a value, 113 for 4096 x 5001
// with N = 1 (4: 135).  Pairs take N = 4: save and load of 8192 x 4094 49 us, with N = 2 58.
template <int V> constexpr int kMany = V == 1 ? 2 : 4;  // N of save and load
template <int V> constexpr int kSpan = 8 / kMany<V>;    // their S
template <int V> constexpr int kFew = V == 1 ? 1 : 4;   // N of the SwiGLU kernels

// The lane's first group and column and what is left of the row from there; its next group
// lies N groups further.
struct Span {
  int64_t row;
  int grp, col, left;
  bool in;  // the warp has a row
};
template <int N, int S>
__device__ __forceinline__ Span span_of(int G, int rows, int F) {
  const uint32_t spans = (uint32_t)(G + N * S - 1) / (N * S), at = blockIdx.x * 8u + (threadIdx.x >> 5);
  const uint32_t row = at / spans, lane = threadIdx.x & 31;
  Span s;
  s.row = row;
  s.grp = (int)(at - row * spans) * N * S;
  s.col = s.grp * kGroup + lane * N;
  s.grp += lane * N / kGroup;
  s.left = F - s.col;
  s.in = row < (uint32_t)rows;
  return s;
}

// V values at p, zeros where there are none.
template <typename T, int V>
__device__ __forceinline__ void load_v(const T* p, bool in, float* v) {
  if constexpr (V == 1) {
    v[0] = in ? to_f32<T>(__ldg(p)) : 0.0f;
  } else if constexpr (sizeof(T) * V == 16) {
    const float4 f = in ? __ldg(reinterpret_cast<const float4*>(p)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    v[0] = f.x, v[1] = f.y, v[V - 2] = f.z, v[V - 1] = f.w;
  } else if constexpr (sizeof(T) == 4) {
    const float2 f = in ? __ldg(reinterpret_cast<const float2*>(p)) : make_float2(0.0f, 0.0f);
    v[0] = f.x, v[1] = f.y;
  } else if constexpr (V == 2) {
    const float2 f = unpack2<T>(in ? __ldg(reinterpret_cast<const uint32_t*>(p)) : 0u);
    v[0] = f.x, v[1] = f.y;
  } else {
    const uint2 q = in ? __ldg(reinterpret_cast<const uint2*>(p)) : make_uint2(0u, 0u);
    const float2 f = unpack2<T>(q.x), g = unpack2<T>(q.y);
    v[0] = f.x, v[1] = f.y, v[V - 2] = g.x, v[V - 1] = g.y;
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float* v) {
  if constexpr (V == 1) *p = from_f32<T>(v[0]);
  else if constexpr (sizeof(T) * V == 16) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[V - 2], v[V - 1]);
  else if constexpr (sizeof(T) == 4) *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
  else if constexpr (V == 2) *reinterpret_cast<uint32_t*>(p) = pack2<T>(v[0], v[1]);
  else *reinterpret_cast<uint2*>(p) = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[V - 2], v[V - 1]));
}
template <int V> struct CodesOf;
template <> struct CodesOf<1> { using type = uint8_t; };
template <> struct CodesOf<2> { using type = uint16_t; };
template <> struct CodesOf<4> { using type = uint32_t; };

// A span's values from p on, zeros behind the row's end, and back.
template <int V, typename T, int N, int S>
__device__ __forceinline__ void load_span(const T* p, int left, float (&v)[S][N]) {
#pragma unroll
  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int j = 0; j < N; j += V) load_v<T, V>(p + i * N * kGroup + j, i * N * kGroup + j < left, v[i] + j);
}
template <int V, typename T, int N, int S>
__device__ __forceinline__ void store_span(T* p, int left, const float (&v)[S][N]) {
#pragma unroll
  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int j = 0; j < N; j += V)
      if (i * N * kGroup + j < left) store_v<T, V>(p + i * N * kGroup + j, v[i] + j);
}

// A span's codes and exponents; a group's largest value is found by its 32 / N lanes.
template <typename T, int V, int N, int S>
__device__ __forceinline__ void encode_span(const float (&v)[S][N], int left, int8_t* q, uint8_t* ex) {
  using C = typename CodesOf<V>::type;
  const int lane = threadIdx.x & 31;
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < S; ++i) {
    uint32_t m = 0, c[1];
#pragma unroll
    for (int j = 0; j < N; ++j) m = max(m, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
    if constexpr (N == 1) {
      m = __reduce_max_sync(0xffffffffu, m);
    } else {
#pragma unroll
      for (int o = 1; o < 32 / N; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    const uint32_t eb = group_exp<T>(m);
    encode<T, N>(v[i], eb, c);
#pragma unroll
    for (int j = 0; j < N; j += V)
      if (i * N * kGroup + j < left) *reinterpret_cast<C*>(q + i * N * kGroup + j) = (C)(c[0] >> (8 * j));
    if (N > 1 && lane % (32 / N) == 0 && i * N * kGroup < left) ex[N * i] = (uint8_t)eb;
    if (N == 1 && lane == i) mine = eb;
  }
  // single values: the first S lanes store one each (left counts from column `lane` on)
  if (N == 1 && lane < S && lane * kGroup < left + lane) ex[lane] = (uint8_t)mine;
}
template <int V, int N, int S>
__device__ __forceinline__ void load_codes(const int8_t* __restrict__ q, const uint8_t* __restrict__ ex, int left,
                                           uint32_t (&c)[S][1], uint32_t (&eb)[S]) {
  using C = typename CodesOf<V>::type;
#pragma unroll
  for (int i = 0; i < S; ++i) {
    c[i][0] = 0;
#pragma unroll
    for (int j = 0; j < N; j += V)
      if (i * N * kGroup + j < left)
        c[i][0] |= (uint32_t)__ldg(reinterpret_cast<const C*>(q + i * N * kGroup + j)) << (8 * j);
    eb[i] = i * N * kGroup < left ? __ldg(ex + N * i) : 0u;
  }
}

template <typename T, int V>
__global__ void __launch_bounds__(256) act_save_v_kernel(const T* __restrict__ x, int64_t ldx, int R, int F,
                                                         int8_t* __restrict__ q, uint8_t* __restrict__ ex,
                                                         const int32_t* __restrict__ n_rows) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  constexpr int N = kMany<V>, S = kSpan<V>;
  const int G = (F + kGroup - 1) / kGroup;
  const Span s = span_of<N, S>(G, row_count(R, n_rows), F);
  if (!s.in) return;
  float v[S][N];
  load_span<V>(x + s.row * ldx + s.col, s.left, v);
  encode_span<T, V>(v, s.left, q + s.row * F + s.col, ex + s.row * G + s.grp);
}

template <typename T, int V>
__global__ void __launch_bounds__(256) act_load_v_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ ex,
                                                         int R, int F, T* __restrict__ x, int64_t ldx,
                                                         const int32_t* __restrict__ n_rows) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  constexpr int N = kMany<V>, S = kSpan<V>;
  const int G = (F + kGroup - 1) / kGroup;
  const Span s = span_of<N, S>(G, row_count(R, n_rows), F);
  if (!s.in) return;
  uint32_t c[S][1], eb[S];
  load_codes<V, N>(q + s.row * F + s.col, ex + s.row * G + s.grp, s.left, c, eb);
#pragma unroll
  for (int i = 0; i < S; ++i) {
    float v[1][N];
    decode<N>(c[i], eb[i], v[0]);
    store_span<V>(x + s.row * ldx + s.col + i * N * kGroup, s.left - i * N * kGroup, v);
  }
}

template <typename T, int V, int S>
__global__ void __launch_bounds__(256) swiglu_save_v_kernel(const T* __restrict__ g, int64_t ldg,
                                                            const T* __restrict__ u, int64_t ldu, int R, int F,
                                                            T* __restrict__ h, int64_t ldh, int8_t* __restrict__ gq,
                                                            uint8_t* __restrict__ ge, int8_t* __restrict__ uq,
                                                            uint8_t* __restrict__ ue,
                                                            const int32_t* __restrict__ n_rows) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  constexpr int N = kFew<V>;
  const int G = (F + kGroup - 1) / kGroup;
  const Span s = span_of<N, S>(G, row_count(R, n_rows), F);
  if (!s.in) return;
  float a[S][N], b[S][N];
  load_span<V>(g + s.row * ldg + s.col, s.left, a);
  load_span<V>(u + s.row * ldu + s.col, s.left, b);
  const int64_t at = s.row * F + s.col, e_at = s.row * G + s.grp;
  encode_span<T, V>(a, s.left, gq + at, ge + e_at);
  encode_span<T, V>(b, s.left, uq + at, ue + e_at);
#pragma unroll
  for (int i = 0; i < S * N; i += 2) {
    float &p = a[i / N][i % N], &q = a[(i + 1) / N][(i + 1) % N];
    const float2 y = swiglu<T>(make_float2(p, q), make_float2(b[i / N][i % N], b[(i + 1) / N][(i + 1) % N]));
    p = y.x, q = y.y;
  }
  store_span<V>(h + s.row * ldh + s.col, s.left, a);
}

template <typename T, int V, int S>
__global__ void __launch_bounds__(256) swiglu_backward_v_kernel(
    const T* __restrict__ dh, int64_t lddh, const int8_t* __restrict__ gq, const uint8_t* __restrict__ ge,
    const int8_t* __restrict__ uq, const uint8_t* __restrict__ ue, int R, int F, T* __restrict__ dg, int64_t lddg,
    T* __restrict__ du, int64_t lddu, T* __restrict__ h, int64_t ldh, const int32_t* __restrict__ n_rows) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  constexpr int N = kFew<V>;
  const int G = (F + kGroup - 1) / kGroup;
  const Span s = span_of<N, S>(G, row_count(R, n_rows), F);
  if (!s.in) return;
  const int64_t at = s.row * F + s.col, e_at = s.row * G + s.grp;
  float d[S][N], a[S][N], b[S][N];
  uint32_t cg[S][1], cu[S][1], eg[S], eu[S];
  load_span<V>(dh + s.row * lddh + s.col, s.left, d);
  load_codes<V, N>(gq + at, ge + e_at, s.left, cg, eg);
  load_codes<V, N>(uq + at, ue + e_at, s.left, cu, eu);
#pragma unroll
  for (int i = 0; i < S; ++i) {
    decode<N>(cg[i], eg[i], a[i]);
    decode<N>(cu[i], eu[i], b[i]);
#pragma unroll
    for (int j = 0; j < N; ++j) swiglu_grad<T>(a[i][j], b[i][j], d[i][j]);
  }
  store_span<V>(dg + s.row * lddg + s.col, s.left, d);
  store_span<V>(du + s.row * lddu + s.col, s.left, a);
  if (h) store_span<V>(h + s.row * ldh + s.col, s.left, b);
}

// ---------------------------------------------------------------- host
namespace {

// How a call runs: one, two, four or eight values a lane, or eight with all rows in one.
enum class Way { kOne, kTwo, kFour, kEight, kFlat };

struct Matrix {
  const void* p;
  int64_t ld;
};
// The widest that widths, rows (in values of es bytes) and codes allow.  Eight values want
// rows on 16 bytes and codes on 8.
Way way_of(int es, int F, std::initializer_list<Matrix> rows, std::initializer_list<const void*> codes) {
  uint64_t bytes = 0, values = (uint64_t)F;
  bool flat = F % kGroup == 0;
  for (const Matrix& m : rows) {
    if (!m.p) continue;
    bytes |= (uint64_t)(uintptr_t)m.p | (uint64_t)(m.ld * es);
    flat = flat && m.ld == F;
  }
  for (const void* c : codes) values |= (uint64_t)(uintptr_t)c;
  auto allow = [&](int v) { return values % v == 0 && bytes % (v * es < 16 ? v * es : 16) == 0; };
  if (allow(8)) return flat ? Way::kFlat : Way::kEight;
  return allow(4) ? Way::kFour : allow(2) ? Way::kTwo : Way::kOne;
}

// span: groups a warp takes where it has fewer than eight values a lane.
dim3 grid_of(Way w, int R, int F, int span) {
  const uint64_t G = (F + kGroup - 1) / kGroup;
  if (w < Way::kEight) return dim3((unsigned)((R * ((G + span - 1) / span) + 7) / 8));
  return dim3((unsigned)((R * G + kGroupsPerBlock - 1) / kGroupsPerBlock));
}

// SwiGLU of pairs and fours: S = 2 where there are groups enough for all warps the machine holds
// (4096 x 5002 bf16 82 us, S = 1 92), else 1 (1000 x 1022 7.3 us, S = 2 8.4; 333 x 778 fp32 4.3 / 5.0).
bool long_spans(int R, int F) { return (int64_t)R * ((F + kGroup - 1) / kGroup) >= 1 << 17; }
int swiglu_span(Way w, int R, int F) { return w == Way::kOne || !long_spans(R, F) ? 4 : 8; }

#define MOE_PICK(w, name, T)                          \
  ((w) == Way::kOne     ? name##_v_kernel<T, 1>        \
   : (w) == Way::kTwo   ? name##_v_kernel<T, 2>        \
   : (w) == Way::kFour  ? name##_v_kernel<T, 4>        \
   : (w) == Way::kEight ? name##_kernel<T, false>     \
                        : name##_kernel<T, true>)
#define MOE_PICK_SWIGLU(w, many, name, T)                                             \
  ((w) == Way::kOne     ? name##_v_kernel<T, 1, 4>                                     \
   : (w) == Way::kTwo   ? ((many) ? name##_v_kernel<T, 2, 2> : name##_v_kernel<T, 2, 1>) \
   : (w) == Way::kFour  ? ((many) ? name##_v_kernel<T, 4, 2> : name##_v_kernel<T, 4, 1>) \
   : (w) == Way::kEight ? name##_kernel<T, false>                                     \
                        : name##_kernel<T, true>)

template <typename T>
cudaError_t save_as(ConstRows x, int R, int F, Ckpt c, const int32_t* n_rows, cudaStream_t s) {
  const Way w = way_of(sizeof(T), F, {{x.p, x.ld}}, {c.q});
  return launch_chained(MOE_PICK(w, act_save, T), grid_of(w, R, F, 8), dim3(256), 0, s, (const T*)x.p, x.ld, R, F, c.q, c.e,
                        n_rows);
}
template <typename T>
cudaError_t load_as(Ckpt c, int R, int F, Rows x, const int32_t* n_rows, cudaStream_t s) {
  const Way w = way_of(sizeof(T), F, {{x.p, x.ld}}, {c.q});
  return launch_chained(MOE_PICK(w, act_load, T), grid_of(w, R, F, 8), dim3(256), 0, s, (const int8_t*)c.q,
                        (const uint8_t*)c.e, R, F, (T*)x.p, x.ld, n_rows);
}
template <typename T>
cudaError_t swiglu_save_as(ConstRows g, ConstRows u, int R, int F, Rows h, Ckpt cg, Ckpt cu, const int32_t* n_rows,
                           cudaStream_t s) {
  const Way w = way_of(sizeof(T), F, {{g.p, g.ld}, {u.p, u.ld}, {h.p, h.ld}}, {cg.q, cu.q});
  return launch_chained(MOE_PICK_SWIGLU(w, long_spans(R, F), swiglu_save, T), grid_of(w, R, F, swiglu_span(w, R, F)), dim3(256), 0, s, (const T*)g.p, g.ld,
                        (const T*)u.p, u.ld, R, F, (T*)h.p, h.ld, cg.q, cg.e, cu.q, cu.e, n_rows);
}
template <typename T>
cudaError_t swiglu_backward_as(ConstRows dh, Ckpt cg, Ckpt cu, int R, int F, Rows dg, Rows du, Rows h,
                               const int32_t* n_rows, cudaStream_t s) {
  const Way w = way_of(sizeof(T), F, {{dh.p, dh.ld}, {dg.p, dg.ld}, {du.p, du.ld}, {h.p, h.ld}}, {cg.q, cu.q});
  return launch_chained(MOE_PICK_SWIGLU(w, long_spans(R, F), swiglu_backward, T), grid_of(w, R, F, swiglu_span(w, R, F)), dim3(256), 0, s, (const T*)dh.p, dh.ld,
                        (const int8_t*)cg.q, (const uint8_t*)cg.e, (const int8_t*)cu.q, (const uint8_t*)cu.e, R, F,
                        (T*)dg.p, dg.ld, (T*)du.p, du.ld, (T*)h.p, h.ld, n_rows);
}
#undef MOE_PICK
#undef MOE_PICK_SWIGLU

}  // namespace

cudaError_t launch_act_save(ConstRows x, int dtype, int R, int F, Ckpt c, const int32_t* n_rows, cudaStream_t s) {
  if (dtype == MOE_F32) return save_as<float>(x, R, F, c, n_rows, s);
  return dtype == MOE_F16 ? save_as<__half>(x, R, F, c, n_rows, s) : save_as<__nv_bfloat16>(x, R, F, c, n_rows, s);
}
cudaError_t launch_act_load(Ckpt c, int R, int F, int dtype, Rows x, const int32_t* n_rows, cudaStream_t s) {
  if (dtype == MOE_F32) return load_as<float>(c, R, F, x, n_rows, s);
  return dtype == MOE_F16 ? load_as<__half>(c, R, F, x, n_rows, s) : load_as<__nv_bfloat16>(c, R, F, x, n_rows, s);
}
cudaError_t launch_swiglu_save(ConstRows g, ConstRows u, int dtype, int R, int F, Rows h, Ckpt cg, Ckpt cu,
                               const int32_t* n_rows, cudaStream_t s) {
  if (dtype == MOE_F32) return swiglu_save_as<float>(g, u, R, F, h, cg, cu, n_rows, s);
  return dtype == MOE_F16 ? swiglu_save_as<__half>(g, u, R, F, h, cg, cu, n_rows, s)
                          : swiglu_save_as<__nv_bfloat16>(g, u, R, F, h, cg, cu, n_rows, s);
}
cudaError_t launch_swiglu_backward(ConstRows dh, int dtype, Ckpt cg, Ckpt cu, int R, int F, Rows dg, Rows du, Rows h,
                                   const int32_t* n_rows, cudaStream_t s) {
  if (dtype == MOE_F32) return swiglu_backward_as<float>(dh, cg, cu, R, F, dg, du, h, n_rows, s);
  return dtype == MOE_F16 ? swiglu_backward_as<__half>(dh, cg, cu, R, F, dg, du, h, n_rows, s)
                          : swiglu_backward_as<__nv_bfloat16>(dh, cg, cu, R, F, dg, du, h, n_rows, s);
}

}  // namespace moe

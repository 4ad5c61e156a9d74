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
// run one lane per value.
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
template <typename T>
__device__ __forceinline__ uint32_t code_bits(float x, float inv, bool top) {
  if (top) x = fminf(fmaxf(x * inv, -127.0f), 127.0f), inv = 1.0f;
  return __float_as_uint(fmaf(x, inv, 12582912.0f));
}

template <typename T>
__device__ __forceinline__ uint2 encode8(const float (&v)[8], uint32_t eb) {
  const float inv = inv_step(eb);
  if (eb == 255u) return make_uint2(0u, 0u);
  const bool top = eb == (uint32_t)(emax<T>() + 127);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = code_bits<T>(v[i], inv, top);
  uint2 q;
  q.x = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
  q.y = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
  return q;
}

__device__ __forceinline__ uint32_t abs_bits8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return max(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// q * 2^e of four codes: byte + 2^23 as a float by one byte permute, then the offset off.
__device__ __forceinline__ void decode4(uint32_t q, float step, float* v) {
  q ^= 0x80808080u;  // q + 128
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = (__uint_as_float(__byte_perm(q, 0x4B000000u, 0x7440 + i)) - 8388736.0f) * step;
}
__device__ __forceinline__ void decode8(uint2 q, float step, float (&v)[8]) {
  decode4(q.x, step, v);
  decode4(q.y, step, v + 4);
}

__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

// silu(g) * u.  At g = -inf this is -inf * 0: NaN, as the formula says.
__device__ __forceinline__ float swiglu(float g, float u) { return g * sigmoid(g) * u; }

struct Grads {
  float dg, du, h;
};
__device__ __forceinline__ Grads swiglu_grad(float g, float u, float dh) {
  const float s = sigmoid(g), a = g * s;
  return {dh * u * (s * fmaf(g, 1.0f - s, 1.0f)), dh * a, a * u};
}

// Where a lane works: group `at` of the rows in order, value `col` of row `row`.
struct Place {
  int64_t row;
  int grp, col;
  bool in;  // the lane has values there
};

// ---------------------------------------------------------------- eight values a lane
__device__ __forceinline__ Place place8(uint32_t at, int G, int rows, int F) {
  Place p;
  p.row = at / (uint32_t)G;
  p.grp = (int)(at - (uint32_t)p.row * (uint32_t)G);
  p.col = p.grp * kGroup + (threadIdx.x & 3) * 8;
  p.in = p.row < rows && p.col < F;
  return p;
}

__device__ __forceinline__ int row_count(int R, const int32_t* n_rows) {
  return n_rows ? min(R, max(0, __ldg(n_rows))) : R;
}

template <typename T>
__global__ void __launch_bounds__(256) act_save_kernel(const T* __restrict__ x, int64_t ldx, int R, int F,
                                                       int8_t* __restrict__ q, uint8_t* __restrict__ ex,
                                                       const int32_t* __restrict__ n_rows) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  const int G = (F + kGroup - 1) / kGroup, rows = row_count(R, n_rows);
  const Place p = place8(blockIdx.x * 64u + (threadIdx.x >> 2), G, rows, F);
  float v[8] = {};
  if (p.in) load_vec<T, 8>(x + p.row * ldx + p.col, v);
  const uint32_t eb = group_exp<T>(quad_max(abs_bits8(v)));
  if (!p.in) return;
  *reinterpret_cast<uint2*>(q + p.row * F + p.col) = encode8<T>(v, eb);
  if ((threadIdx.x & 3) == 0) ex[p.row * G + p.grp] = (uint8_t)eb;
}

template <typename T>
__global__ void __launch_bounds__(256) act_load_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ ex,
                                                       int R, int F, T* __restrict__ x, int64_t ldx,
                                                       const int32_t* __restrict__ n_rows) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  const int G = (F + kGroup - 1) / kGroup, rows = row_count(R, n_rows);
  const Place p = place8(blockIdx.x * 64u + (threadIdx.x >> 2), G, rows, F);
  if (!p.in) return;
  float v[8];
  decode8(__ldg(reinterpret_cast<const uint2*>(q + p.row * F + p.col)), step_of(__ldg(ex + p.row * G + p.grp)), v);
  store_vec<T, 8>(x + p.row * ldx + p.col, v);
}

template <typename T>
__global__ void __launch_bounds__(256) swiglu_save_kernel(const T* __restrict__ g, int64_t ldg, const T* __restrict__ u,
                                                          int64_t ldu, int R, int F, T* __restrict__ h, int64_t ldh,
                                                          int8_t* __restrict__ gq, uint8_t* __restrict__ ge,
                                                          int8_t* __restrict__ uq, uint8_t* __restrict__ ue,
                                                          const int32_t* __restrict__ n_rows) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  const int G = (F + kGroup - 1) / kGroup, rows = row_count(R, n_rows);
  const Place p = place8(blockIdx.x * 64u + (threadIdx.x >> 2), G, rows, F);
  float a[8] = {}, b[8] = {};
  if (p.in) {
    load_vec<T, 8>(g + p.row * ldg + p.col, a);
    load_vec<T, 8>(u + p.row * ldu + p.col, b);
  }
  const uint32_t ea = group_exp<T>(quad_max(abs_bits8(a))), eb = group_exp<T>(quad_max(abs_bits8(b)));
  if (!p.in) return;
  const int64_t at = p.row * F + p.col;
  *reinterpret_cast<uint2*>(gq + at) = encode8<T>(a, ea);
  *reinterpret_cast<uint2*>(uq + at) = encode8<T>(b, eb);
  if ((threadIdx.x & 3) == 0) {
    ge[p.row * G + p.grp] = (uint8_t)ea;
    ue[p.row * G + p.grp] = (uint8_t)eb;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = swiglu(a[i], b[i]);
  store_vec<T, 8>(h + p.row * ldh + p.col, a);
}

template <typename T>
__global__ void __launch_bounds__(256) swiglu_backward_kernel(
    const T* __restrict__ dh, int64_t lddh, const int8_t* __restrict__ gq, const uint8_t* __restrict__ ge,
    const int8_t* __restrict__ uq, const uint8_t* __restrict__ ue, int R, int F, T* __restrict__ dg, int64_t lddg,
    T* __restrict__ du, int64_t lddu, T* __restrict__ h, int64_t ldh, const int32_t* __restrict__ n_rows) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  const int G = (F + kGroup - 1) / kGroup, rows = row_count(R, n_rows);
  const Place p = place8(blockIdx.x * 64u + (threadIdx.x >> 2), G, rows, F);
  if (!p.in) return;
  float d[8], a[8], b[8];
  const int64_t at = p.row * F + p.col;
  load_vec<T, 8>(dh + p.row * lddh + p.col, d);
  decode8(__ldg(reinterpret_cast<const uint2*>(gq + at)), step_of(__ldg(ge + p.row * G + p.grp)), a);
  decode8(__ldg(reinterpret_cast<const uint2*>(uq + at)), step_of(__ldg(ue + p.row * G + p.grp)), b);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const Grads r = swiglu_grad(a[i], b[i], d[i]);
    d[i] = r.dg, a[i] = r.du, b[i] = r.h;
  }
  store_vec<T, 8>(dg + p.row * lddg + p.col, d);
  store_vec<T, 8>(du + p.row * lddu + p.col, a);
  if (h) store_vec<T, 8>(h + p.row * ldh + p.col, b);
}

// ---------------------------------------------------------------- one value a lane
__device__ __forceinline__ Place place1(uint32_t at, int G, int rows, int F) {
  Place p;
  p.row = at / (uint32_t)G;
  p.grp = (int)(at - (uint32_t)p.row * (uint32_t)G);
  p.col = p.grp * kGroup + (threadIdx.x & 31);
  p.in = p.row < rows && p.col < F;
  return p;
}

template <typename T>
__device__ __forceinline__ uint32_t warp_exp(float v) {
  return group_exp<T>(__reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7FFFFFFFu));
}
template <typename T>
__device__ __forceinline__ int8_t encode1(float v, uint32_t eb) {
  if (eb == 255u) return 0;
  return (int8_t)(code_bits<T>(v, inv_step(eb), eb == (uint32_t)(emax<T>() + 127)) & 0xFFu);
}

template <typename T>
__global__ void __launch_bounds__(256) act_save1_kernel(const T* __restrict__ x, int64_t ldx, int R, int F,
                                                        int8_t* __restrict__ q, uint8_t* __restrict__ ex,
                                                        const int32_t* __restrict__ n_rows) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  const int G = (F + kGroup - 1) / kGroup, rows = row_count(R, n_rows);
  const Place p = place1(blockIdx.x * 8u + (threadIdx.x >> 5), G, rows, F);
  const float v = p.in ? to_f32<T>(__ldg(x + p.row * ldx + p.col)) : 0.0f;
  const uint32_t eb = warp_exp<T>(v);
  if (!p.in) return;
  q[p.row * F + p.col] = encode1<T>(v, eb);
  if ((threadIdx.x & 31) == 0) ex[p.row * G + p.grp] = (uint8_t)eb;
}

template <typename T>
__global__ void __launch_bounds__(256) act_load1_kernel(const int8_t* __restrict__ q, const uint8_t* __restrict__ ex,
                                                        int R, int F, T* __restrict__ x, int64_t ldx,
                                                        const int32_t* __restrict__ n_rows) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  const int G = (F + kGroup - 1) / kGroup, rows = row_count(R, n_rows);
  const Place p = place1(blockIdx.x * 8u + (threadIdx.x >> 5), G, rows, F);
  if (!p.in) return;
  x[p.row * ldx + p.col] = from_f32<T>((float)q[p.row * F + p.col] * step_of(__ldg(ex + p.row * G + p.grp)));
}

template <typename T>
__global__ void __launch_bounds__(256) swiglu_save1_kernel(const T* __restrict__ g, int64_t ldg,
                                                           const T* __restrict__ u, int64_t ldu, int R, int F,
                                                           T* __restrict__ h, int64_t ldh, int8_t* __restrict__ gq,
                                                           uint8_t* __restrict__ ge, int8_t* __restrict__ uq,
                                                           uint8_t* __restrict__ ue,
                                                           const int32_t* __restrict__ n_rows) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  const int G = (F + kGroup - 1) / kGroup, rows = row_count(R, n_rows);
  const Place p = place1(blockIdx.x * 8u + (threadIdx.x >> 5), G, rows, F);
  const float a = p.in ? to_f32<T>(__ldg(g + p.row * ldg + p.col)) : 0.0f;
  const float b = p.in ? to_f32<T>(__ldg(u + p.row * ldu + p.col)) : 0.0f;
  const uint32_t ea = warp_exp<T>(a), eb = warp_exp<T>(b);
  if (!p.in) return;
  gq[p.row * F + p.col] = encode1<T>(a, ea);
  uq[p.row * F + p.col] = encode1<T>(b, eb);
  if ((threadIdx.x & 31) == 0) {
    ge[p.row * G + p.grp] = (uint8_t)ea;
    ue[p.row * G + p.grp] = (uint8_t)eb;
  }
  h[p.row * ldh + p.col] = from_f32<T>(swiglu(a, b));
}

template <typename T>
__global__ void __launch_bounds__(256) swiglu_backward1_kernel(
    const T* __restrict__ dh, int64_t lddh, const int8_t* __restrict__ gq, const uint8_t* __restrict__ ge,
    const int8_t* __restrict__ uq, const uint8_t* __restrict__ ue, int R, int F, T* __restrict__ dg, int64_t lddg,
    T* __restrict__ du, int64_t lddu, T* __restrict__ h, int64_t ldh, const int32_t* __restrict__ n_rows) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  const int G = (F + kGroup - 1) / kGroup, rows = row_count(R, n_rows);
  const Place p = place1(blockIdx.x * 8u + (threadIdx.x >> 5), G, rows, F);
  if (!p.in) return;
  const int64_t at = p.row * F + p.col, ge_at = p.row * G + p.grp;
  const Grads r = swiglu_grad((float)gq[at] * step_of(__ldg(ge + ge_at)), (float)uq[at] * step_of(__ldg(ue + ge_at)),
                              to_f32<T>(__ldg(dh + p.row * lddh + p.col)));
  dg[p.row * lddg + p.col] = from_f32<T>(r.dg);
  du[p.row * lddu + p.col] = from_f32<T>(r.du);
  if (h) h[p.row * ldh + p.col] = from_f32<T>(r.h);
}

// ---------------------------------------------------------------- host
namespace {

// Eight values a lane need 16-byte rows and codes on 8-byte boundaries.
bool vec_rows(const void* p, int64_t ld, int es) { return on16(p) && (ld * es) % 16 == 0; }
bool vec_ckpt(const Ckpt& c, int F) { return F % 8 == 0 && ((uintptr_t)c.q & 7) == 0; }

unsigned blocks(int R, int F, int per) {
  return (unsigned)(((uint64_t)R * ((F + kGroup - 1) / kGroup) + per - 1) / per);
}

template <typename T>
cudaError_t save_as(ConstRows x, int R, int F, Ckpt c, const int32_t* n_rows, cudaStream_t s) {
  const bool v = vec_rows(x.p, x.ld, sizeof(T)) && vec_ckpt(c, F);
  return launch_chained(v ? act_save_kernel<T> : act_save1_kernel<T>, dim3(blocks(R, F, v ? 64 : 8)), dim3(256), 0, s,
                        (const T*)x.p, x.ld, R, F, c.q, c.e, n_rows);
}
template <typename T>
cudaError_t load_as(Ckpt c, int R, int F, Rows x, const int32_t* n_rows, cudaStream_t s) {
  const bool v = vec_rows(x.p, x.ld, sizeof(T)) && vec_ckpt(c, F);
  return launch_chained(v ? act_load_kernel<T> : act_load1_kernel<T>, dim3(blocks(R, F, v ? 64 : 8)), dim3(256), 0, s,
                        (const int8_t*)c.q, (const uint8_t*)c.e, R, F, (T*)x.p, x.ld, n_rows);
}
template <typename T>
cudaError_t swiglu_save_as(ConstRows g, ConstRows u, int R, int F, Rows h, Ckpt cg, Ckpt cu, const int32_t* n_rows,
                           cudaStream_t s) {
  const bool v = vec_rows(g.p, g.ld, sizeof(T)) && vec_rows(u.p, u.ld, sizeof(T)) && vec_rows(h.p, h.ld, sizeof(T)) &&
                 vec_ckpt(cg, F) && vec_ckpt(cu, F);
  return launch_chained(v ? swiglu_save_kernel<T> : swiglu_save1_kernel<T>, dim3(blocks(R, F, v ? 64 : 8)), dim3(256),
                        0, s, (const T*)g.p, g.ld, (const T*)u.p, u.ld, R, F, (T*)h.p, h.ld, cg.q, cg.e, cu.q, cu.e,
                        n_rows);
}
template <typename T>
cudaError_t swiglu_backward_as(ConstRows dh, Ckpt cg, Ckpt cu, int R, int F, Rows dg, Rows du, Rows h,
                               const int32_t* n_rows, cudaStream_t s) {
  const bool v = vec_rows(dh.p, dh.ld, sizeof(T)) && vec_rows(dg.p, dg.ld, sizeof(T)) &&
                 vec_rows(du.p, du.ld, sizeof(T)) && (!h.p || vec_rows(h.p, h.ld, sizeof(T))) && vec_ckpt(cg, F) &&
                 vec_ckpt(cu, F);
  return launch_chained(v ? swiglu_backward_kernel<T> : swiglu_backward1_kernel<T>, dim3(blocks(R, F, v ? 64 : 8)),
                        dim3(256), 0, s, (const T*)dh.p, dh.ld, (const int8_t*)cg.q, (const uint8_t*)cg.e,
                        (const int8_t*)cu.q, (const uint8_t*)cu.e, R, F, (T*)dg.p, dg.ld, (T*)du.p, du.ld, (T*)h.p,
                        h.ld, n_rows);
}

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

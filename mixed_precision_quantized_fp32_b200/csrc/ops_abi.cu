// Host side of the operators around the expert products (declared in include/moe.h):
// arguments are checked before anything is launched.
#include "kernels.cuh"
#include "ops_common.cuh"

namespace moe {
namespace {

bool known_type(int dtype) { return dtype == MOE_BF16 || dtype == MOE_F16 || dtype == MOE_F32; }
bool on(const void* p, int es) { return ((uintptr_t)p & (uintptr_t)(es - 1)) == 0; }

bool entries_ok(int T, int k) { return T >= 0 && k >= 1 && k <= kMaxK && (long long)T * k <= (1LL << 20); }
bool width_ok(int H) { return H >= 1 && H <= (1 << 20); }
bool ckpt_ok(int R, int F) {
  return R >= 0 && width_ok(F) && (long long)R * ((F + 31) / 32) < (1LL << 31) - 64;
}

moe_status launched(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

moe_status sort_rows(const void* x, int64_t ldx, int32_t dtype, const int32_t* idx, int T, int k, int E, int H, void* xs,
                     int64_t ldxs, int32_t* perm, int32_t* inv, int32_t* offsets, void* ws, uint64_t ws_bytes,
                     uint64_t* ws_bytes_out, cudaStream_t stream) {
  const uint64_t need = sort_ws_bytes(T * k, E);
  if (ws_bytes_out) *ws_bytes_out = need;
  if (!ws && (ws_bytes_out || need > 0)) return ws_bytes_out ? MOE_OK : MOE_ERR_ARG;
  if (!offsets || (T > 0 && (!idx || !perm || !inv))) return MOE_ERR_ARG;
  if (!on(idx, 4) || !on(perm, 4) || !on(inv, 4) || !on(offsets, 4) || !on(ws, 256)) return MOE_ERR_ALIGN;
  if (ws_bytes < need) return MOE_ERR_WORKSPACE;
  const moe_status ds = check_device();
  if (ds != MOE_OK) return ds;
  return launched(launch_dispatch(idx, T, k, E, perm, inv, offsets, {x, ldx}, {xs, ldxs}, H, dtype, ws, stream));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_sort(const int32_t* idx, int32_t T, int32_t k, int32_t E, int32_t* perm, int32_t* inv,
                               int32_t* offsets, void* ws, uint64_t ws_bytes, uint64_t* ws_bytes_out,
                               cudaStream_t stream) {
  if (!entries_ok(T, k) || E < 1 || E > kMaxGroups) return MOE_ERR_SHAPE;
  return sort_rows(nullptr, 0, MOE_F32, idx, T, k, E, 0, nullptr, 0, perm, inv, offsets, ws, ws_bytes, ws_bytes_out,
                   stream);
}

extern "C" moe_status moe_dispatch(const void* x, int64_t ldx, int32_t dtype, const int32_t* idx, int32_t T, int32_t k,
                                   int32_t E, int32_t H, void* xs, int64_t ldxs, int32_t* perm, int32_t* inv,
                                   int32_t* offsets, void* ws, uint64_t ws_bytes, uint64_t* ws_bytes_out,
                                   cudaStream_t stream) {
  if (!entries_ok(T, k) || E < 1 || E > kMaxGroups || !width_ok(H)) return MOE_ERR_SHAPE;
  if (!known_type(dtype)) return MOE_ERR_FORMAT;
  if (ws || !ws_bytes_out) {  // not a size query
    const int es = dtype_size(dtype);
    if (T > 0 && (!x || !xs)) return MOE_ERR_ARG;
    if (ldx < H || ldxs < H) return MOE_ERR_SHAPE;
    if (!on(x, es) || !on(xs, es)) return MOE_ERR_ALIGN;
  }
  return sort_rows(x, ldx, dtype, idx, T, k, E, H, xs, ldxs, perm, inv, offsets, ws, ws_bytes, ws_bytes_out, stream);
}

static moe_status collect(const void* o, int64_t ldo, int32_t dtype, const float* w, const int32_t* inv, int32_t T,
                          int32_t k, int32_t H, void* y, int64_t ldy, cudaStream_t stream) {
  if (!entries_ok(T, k) || !width_ok(H) || ldo < H || ldy < H) return MOE_ERR_SHAPE;
  if (!known_type(dtype)) return MOE_ERR_FORMAT;
  if (T == 0) return MOE_OK;
  const int es = dtype_size(dtype);
  if (!o || !inv || !y) return MOE_ERR_ARG;
  if (!on(o, es) || !on(y, es) || !on(w, 4) || !on(inv, 4)) return MOE_ERR_ALIGN;
  const moe_status ds = check_device();
  if (ds != MOE_OK) return ds;
  return launched(launch_collect({o, ldo}, w, inv, T, k, H, dtype, {y, ldy}, stream));
}

extern "C" moe_status moe_dispatch_backward(const void* dxs, int64_t lddxs, int32_t dtype, const int32_t* inv,
                                            int32_t T, int32_t k, int32_t H, void* dx, int64_t lddx,
                                            cudaStream_t stream) {
  return collect(dxs, lddxs, dtype, nullptr, inv, T, k, H, dx, lddx, stream);
}

extern "C" moe_status moe_collect(const void* o, int64_t ldo, int32_t dtype, const float* w, const int32_t* inv,
                                  int32_t T, int32_t k, int32_t H, void* y, int64_t ldy, cudaStream_t stream) {
  if (!w && T > 0) return MOE_ERR_ARG;
  return collect(o, ldo, dtype, w, inv, T, k, H, y, ldy, stream);
}

extern "C" moe_status moe_collect_backward(const void* dy, int64_t lddy, const void* o, int64_t ldo, int32_t dtype,
                                           const float* w, const int32_t* inv, int32_t T, int32_t k, int32_t H,
                                           void* d_o, int64_t lddo, float* dw, cudaStream_t stream) {
  if (!entries_ok(T, k) || !width_ok(H) || lddy < H || ldo < H || lddo < H) return MOE_ERR_SHAPE;
  if (!known_type(dtype)) return MOE_ERR_FORMAT;
  if (T == 0) return MOE_OK;
  const int es = dtype_size(dtype);
  if (!dy || !o || !w || !inv || !d_o || !dw) return MOE_ERR_ARG;
  if (!on(dy, es) || !on(o, es) || !on(d_o, es) || !on(w, 4) || !on(inv, 4) || !on(dw, 4)) return MOE_ERR_ALIGN;
  const moe_status ds = check_device();
  if (ds != MOE_OK) return ds;
  return launched(launch_collect_backward({dy, lddy}, {o, ldo}, w, inv, T, k, H, dtype, {d_o, lddo}, dw, stream));
}

extern "C" moe_status moe_act_save(const void* x, int64_t ldx, int32_t dtype, int32_t R, int32_t F, int8_t* codes,
                                   uint8_t* exps, const int32_t* n_rows, cudaStream_t stream) {
  if (!ckpt_ok(R, F) || ldx < F) return MOE_ERR_SHAPE;
  if (!known_type(dtype)) return MOE_ERR_FORMAT;
  if (R == 0) return MOE_OK;
  if (!x || !codes || !exps) return MOE_ERR_ARG;
  if (!on(x, dtype_size(dtype)) || !on(n_rows, 4)) return MOE_ERR_ALIGN;
  const moe_status ds = check_device();
  if (ds != MOE_OK) return ds;
  return launched(launch_act_save({x, ldx}, dtype, R, F, {codes, exps}, n_rows, stream));
}

extern "C" moe_status moe_act_load(const int8_t* codes, const uint8_t* exps, int32_t R, int32_t F, int32_t dtype,
                                   void* x, int64_t ldx, const int32_t* n_rows, cudaStream_t stream) {
  if (!ckpt_ok(R, F) || ldx < F) return MOE_ERR_SHAPE;
  if (!known_type(dtype)) return MOE_ERR_FORMAT;
  if (R == 0) return MOE_OK;
  if (!x || !codes || !exps) return MOE_ERR_ARG;
  if (!on(x, dtype_size(dtype)) || !on(n_rows, 4)) return MOE_ERR_ALIGN;
  const moe_status ds = check_device();
  if (ds != MOE_OK) return ds;
  return launched(launch_act_load({(int8_t*)codes, (uint8_t*)exps}, R, F, dtype, {x, ldx}, n_rows, stream));
}

extern "C" moe_status moe_swiglu_save(const void* g, int64_t ldg, const void* u, int64_t ldu, int32_t dtype, int32_t R,
                                      int32_t F, void* h, int64_t ldh, int8_t* g_codes, uint8_t* g_exps,
                                      int8_t* u_codes, uint8_t* u_exps, const int32_t* n_rows, cudaStream_t stream) {
  if (!ckpt_ok(R, F) || ldg < F || ldu < F || ldh < F) return MOE_ERR_SHAPE;
  if (!known_type(dtype)) return MOE_ERR_FORMAT;
  if (R == 0) return MOE_OK;
  const int es = dtype_size(dtype);
  if (!g || !u || !h || !g_codes || !g_exps || !u_codes || !u_exps) return MOE_ERR_ARG;
  if (!on(g, es) || !on(u, es) || !on(h, es) || !on(n_rows, 4)) return MOE_ERR_ALIGN;
  const moe_status ds = check_device();
  if (ds != MOE_OK) return ds;
  return launched(launch_swiglu_save({g, ldg}, {u, ldu}, dtype, R, F, {h, ldh}, {g_codes, g_exps}, {u_codes, u_exps},
                                     n_rows, stream));
}

extern "C" moe_status moe_swiglu_backward(const void* dh, int64_t lddh, int32_t dtype, const int8_t* g_codes,
                                          const uint8_t* g_exps, const int8_t* u_codes, const uint8_t* u_exps,
                                          int32_t R, int32_t F, void* dg, int64_t lddg, void* du, int64_t lddu, void* h,
                                          int64_t ldh, const int32_t* n_rows, cudaStream_t stream) {
  if (!ckpt_ok(R, F) || lddh < F || lddg < F || lddu < F || (h && ldh < F)) return MOE_ERR_SHAPE;
  if (!known_type(dtype)) return MOE_ERR_FORMAT;
  if (R == 0) return MOE_OK;
  const int es = dtype_size(dtype);
  if (!dh || !dg || !du || !g_codes || !g_exps || !u_codes || !u_exps) return MOE_ERR_ARG;
  if (!on(dh, es) || !on(dg, es) || !on(du, es) || !on(h, es) || !on(n_rows, 4)) return MOE_ERR_ALIGN;
  const moe_status ds = check_device();
  if (ds != MOE_OK) return ds;
  return launched(launch_swiglu_backward({dh, lddh}, dtype, {(int8_t*)g_codes, (uint8_t*)g_exps},
                                         {(int8_t*)u_codes, (uint8_t*)u_exps}, R, F, {dg, lddg}, {du, lddu}, {h, ldh},
                                         n_rows, stream));
}

static moe_status adapters(const void* x, int64_t ldx, const void* y, int64_t ldy, int32_t dtype, int32_t T, int32_t K,
                           int32_t N, int32_t r, int32_t n, const void* A, const void* B, const float* scale,
                           const int32_t* perm, const int32_t* offsets, void* out, int64_t ldo, int32_t* status,
                           uint32_t withhold, uint32_t wait_cycles, cudaStream_t stream) {
  if (!entries_ok(T, 1) || n < 1 || n > kMaxGroups || r < 8 || r > 128 || r % 8 != 0) return MOE_ERR_SHAPE;
  if (!width_ok(K) || !width_ok(N) || K % 8 != 0 || N % 8 != 0) return MOE_ERR_SHAPE;
  if (dtype != MOE_BF16 && dtype != MOE_F16) return MOE_ERR_FORMAT;
  if (ldx < K || ldy < N || ldo < N) return MOE_ERR_SHAPE;
  if (T == 0) return MOE_OK;
  if (!x || !y || !A || !B || !scale || !perm || !offsets || !out) return MOE_ERR_ARG;
  if (out == y && ldo != ldy) return MOE_ERR_ARG;
  if (!on(x, 16) || !on(y, 16) || !on(A, 16) || !on(B, 16) || !on(out, 16) || ldx % 8 != 0 || ldy % 8 != 0 ||
      ldo % 8 != 0 || !on(scale, 4) || !on(perm, 4) || !on(offsets, 4) || !on(status, 4))
    return MOE_ERR_ALIGN;
  const moe_status ds = check_device();
  if (ds != MOE_OK) return ds;
  AdapterArgs a{};
  a.x = {x, ldx};
  a.y = {y, ldy};
  a.out = {out, ldo};
  a.T = T, a.K = K, a.N = N, a.r = r, a.n = n;
  a.A = A, a.B = B, a.scale = scale, a.perm = perm, a.offsets = offsets;
  a.status = status, a.withhold = withhold, a.wait_cycles = wait_cycles;
  return launched(launch_adapters(a, dtype, stream));
}

extern "C" moe_status moe_adapters(const void* x, int64_t ldx, const void* y, int64_t ldy, int32_t dtype, int32_t T,
                                   int32_t K, int32_t N, int32_t r, int32_t n, const void* A, const void* B,
                                   const float* scale, const int32_t* perm, const int32_t* offsets, void* out,
                                   int64_t ldo, int32_t* status, cudaStream_t stream) {
  return adapters(x, ldx, y, ldy, dtype, T, K, N, r, n, A, B, scale, perm, offsets, out, ldo, status, 0, 0, stream);
}

extern "C" moe_status moe_adapters_debug(const void* x, int64_t ldx, const void* y, int64_t ldy, int32_t dtype,
                                         int32_t T, int32_t K, int32_t N, int32_t r, int32_t n, const void* A,
                                         const void* B, const float* scale, const int32_t* perm,
                                         const int32_t* offsets, void* out, int64_t ldo, const moe_debug* dbg,
                                         cudaStream_t stream) {
  const moe_debug d = dbg ? *dbg : moe_debug{};
  return adapters(x, ldx, y, ldy, dtype, T, K, N, r, n, A, B, scale, perm, offsets, out, ldo, d.status, d.test_withhold,
                  d.wait_cycles, stream);
}

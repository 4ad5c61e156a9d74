// Shared by the operators around the expert products (routes.cu, ckpt8.cu,
// adapters.cu): value types, vector loads and stores, and the launchers that the
// host ABI (ops_abi.cu) calls.  All arithmetic is in fp32; a value is rounded once
// (to nearest even) when it is stored in a 16-bit type.
#pragma once
#include "moe_common.cuh"

namespace moe {

// ---------------------------------------------------------------- value types
template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32(float v) { return v; }
template <> __device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }

template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t v);
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<__half2*>(&v));
}
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

// N consecutive values as they lie in memory, in one access of 2 to 16 bytes (N = 8 only of a
// 16-bit type), so that many loads are on their way before the first is used.
template <int B> struct Access;
template <> struct Access<4> { using type = uint32_t; };
template <> struct Access<8> { using type = uint2; };
template <> struct Access<16> { using type = uint4; };
template <typename T, int N> struct Raw { using type = typename Access<N * (int)sizeof(T)>::type; };
template <typename T> struct Raw<T, 1> { using type = T; };

template <typename T, int N>
__device__ __forceinline__ void decode_raw(const typename Raw<T, N>::type& q, float (&v)[N]) {
  if constexpr (N == 1) {
    v[0] = to_f32<T>(q);
  } else {
    constexpr int W = N * sizeof(T) / 4;
    uint32_t w[4] = {};
    if constexpr (W == 1) w[0] = q;
    else w[0] = q.x, w[1] = q.y;
    if constexpr (W == 4) w[2] = q.z, w[3] = q.w;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      if constexpr (sizeof(T) == 4) {
        v[j] = __uint_as_float(w[j]);
      } else {
        const float2 f = unpack2<T>(w[j]);
        v[2 * j] = f.x, v[2 * j + 1] = f.y;
      }
    }
  }
}
template <typename R> __device__ __forceinline__ R zero_raw() {
  if constexpr (sizeof(R) == 16) return make_uint4(0, 0, 0, 0);
  else if constexpr (sizeof(R) == 8) return make_uint2(0, 0);
  else return R(0.0f);
}

// N values rounded and stored, in accesses of up to 16 bytes.
template <typename T, int N>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[N]) {
  if constexpr (N == 1) {
    *p = from_f32<T>(v[0]);
  } else {
    constexpr int W = N * sizeof(T) / 4;
    uint32_t w[W];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(v[j]);
      else w[j] = pack2<T>(v[2 * j], v[2 * j + 1]);
    }
    if constexpr (W == 1) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else if constexpr (W == 2) {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < W / 4; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
  }
}

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
// A word of block `rank`'s shared memory at the place that p has in this block's.
__device__ __forceinline__ uint32_t load_remote(const void* p, uint32_t rank) {
  uint32_t at, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

__device__ __forceinline__ float4 load_remote4(const float* p, uint32_t rank) {
  uint32_t at;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

// launch_chained with clusters of `cluster` blocks.
template <typename... Exp, typename... Act>
inline cudaError_t launch_cluster(void (*kern)(Exp...), dim3 grid, dim3 block, int cluster, size_t smem,
                                  cudaStream_t stream, Act&&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Act>(args)...);
}

inline int dtype_size(int dtype) { return dtype == MOE_F32 ? 4 : 2; }

// A row-major matrix as the operators take it: `ld` values from one row to the next.
struct ConstRows {
  const void* p;
  int64_t ld;
};
struct Rows {
  void* p;
  int64_t ld;
};

constexpr int kMaxGroups = 1024;  // groups of a sort: experts, or the adapters of a bank

// ---------------------------------------------------------------- launchers
// Entries (t, j) sorted by group: workspace bytes and the launch; with x the rows follow.
uint64_t sort_ws_bytes(int R, int E);
cudaError_t launch_dispatch(const int32_t* idx, int T, int k, int E, int32_t* perm, int32_t* inv, int32_t* offsets,
                            ConstRows x, Rows xs, int H, int dtype, void* ws, cudaStream_t stream);
// y[t] = sum_j w[t,j] * o[inv[t,j]] (w null: 1)
cudaError_t launch_collect(ConstRows o, const float* w, const int32_t* inv, int T, int k, int H, int dtype, Rows y,
                           cudaStream_t stream);
cudaError_t launch_collect_backward(ConstRows dy, ConstRows o, const float* w, const int32_t* inv, int T, int k, int H,
                                    int dtype, Rows d_o, float* dw, cudaStream_t stream);


// 8-bit checkpoints (codes [R][F], exps [R][ceil(F/32)]); n_rows null: all R rows.
struct Ckpt {
  int8_t* q;
  uint8_t* e;
};
cudaError_t launch_act_save(ConstRows x, int dtype, int R, int F, Ckpt c, const int32_t* n_rows, cudaStream_t stream);
cudaError_t launch_act_load(Ckpt c, int R, int F, int dtype, Rows x, const int32_t* n_rows, cudaStream_t stream);
cudaError_t launch_swiglu_save(ConstRows g, ConstRows u, int dtype, int R, int F, Rows h, Ckpt cg, Ckpt cu,
                               const int32_t* n_rows, cudaStream_t stream);
cudaError_t launch_swiglu_backward(ConstRows dh, int dtype, Ckpt cg, Ckpt cu, int R, int F, Rows dg, Rows du, Rows h,
                                   const int32_t* n_rows, cudaStream_t stream);

// out = y + scale * B (A x) per token's adapter; out.p == y.p: in place.
struct AdapterArgs {
  ConstRows x, y;
  Rows out;
  int T, K, N, r, n;
  const void *A, *B;
  const float* scale;
  const int32_t *perm, *offsets;
  int32_t* status;  // null, or where MOE_ERR_TIMEOUT goes
  uint32_t withhold, wait_cycles;  // test hooks (moe_debug.test_withhold / wait_cycles)
};
cudaError_t launch_adapters(const AdapterArgs& a, int dtype, cudaStream_t stream);

}  // namespace moe

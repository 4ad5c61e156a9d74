// Rows sorted by expert and brought back: the permutation, gather and combine of the
// layer forward as operators of their own, with their gradients (expert-routing section
// of the quantized MoE inference page: tokens go to their chosen experts and the output
// is the weighted sum of what the experts return).
//
//   sort             key(i) = idx[i] if 0 <= idx[i] < E, else E (dropped); a stable order
//                    of the entries i = t*k + j by key
//   dispatch         xs[row] = x[perm[row] / k]                  row < offsets[E]
//   its gradient     dx[t]   = sum_j dxs[inv[t,j]]               (collect with weights 1)
//   collect          y[t]    = sum_j w[t,j] * o[inv[t,j]]        ascending j, fp32
//   its gradient     do[inv[t,j]] = w[t,j] * dy[t],  dw[t,j] = <dy[t], o[inv[t,j]]>
//
// Every kernel moves rows and computes next to nothing on them, so memory bounds it, and
// latency where there are few.  Rows are walked token by token: a token's row is read (or
// written) once, its k expert rows once each, and nothing is accumulated in memory, so
// results do not depend on the order in which blocks run.  Of the measured copy rate:
//   dispatch, 8192 tokens x 6, 2048 bf16 (235 MB)         47.2 us, 77% (rows alone 38 us, 94%)
//   its gradient, 4096 x 8, 2048 bf16 (141 MB)            24.2 us, 90%
//   collect, 8192 x 2, 4096 bf16 (201 MB)                 31.3 us, 99%
//   its gradient, 2048 x 2, 4096 bf16 (81 MB)             16.0 us, 78%
//   dispatch of 16 x 6 entries 2.8 us, collect of 64 x 2 rows of 12288 fp32 2.9 us
// Rows whose width, pitch or start is no multiple of 16 bytes go in accesses of 8, 4 or 2 (collect
// of 8192 x 2 rows of 4092, 4094 and 4095 bf16: 34, 36 and 59 us).
#include "ops_common.cuh"

namespace moe {

constexpr int kSortBlock = 1024;
constexpr int kSortMaxBlocks = 128;
constexpr int kSortCluster = 8;    // blocks of the cluster that sorts more
constexpr int kSortRounds = 2;     // keys a lane of it holds
constexpr int kSortMedium = kSortCluster * kSortBlock * kSortRounds;
static_assert(kMaxGroups <= kSortBlock, "the cluster's scan takes the keys in at most two steps");

__device__ __forceinline__ int sort_key(int32_t e, int E) { return (unsigned)e < (unsigned)E ? e : E; }

// Few entries in one launch: the row of an entry is the number of entries with a smaller
// key, or an equal key and a smaller index, so each block counts its own token's rows (every
// thread looks at its share of all keys) and copies the token's row there.  Key and index
// are compared as one number.  Block 0 makes the offsets; blockIdx.y shares a long row.
// At these sizes latency is all there is: 256 tokens x 8, rows of 4 KB, take 4.4 us, a sort and
// the rows behind it 8.4 and a second launch on the host.  K: entries a token has at most.
template <typename U, int K>
__global__ void __launch_bounds__(256) dispatch_small_kernel(const int32_t* __restrict__ idx, int R, int k, int E,
                                                             int32_t* __restrict__ perm, int32_t* __restrict__ inv,
                                                             int32_t* __restrict__ offsets, const U* __restrict__ x,
                                                             int64_t ldx, U* __restrict__ xs, int64_t ldxs, int n) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (blockIdx.x == 0) {
    if (blockIdx.y != 0) return;
    __shared__ int32_t hist[kMaxGroups + 1];
    __shared__ int32_t wsum[8];
    for (int e = tid; e <= E; e += 256) hist[e] = 0;
    __syncthreads();
    for (int i = tid; i < R; i += 256) atomicAdd(&hist[sort_key(__ldg(idx + i), E)], 1);  // integer counts: any order
    __syncthreads();
    int run = 0;
    for (int e0 = 0; e0 <= E; e0 += 256) {  // exclusive scan, 256 groups at a time
      const int e = e0 + tid;
      const int v = e <= E ? hist[e] : 0;
      int s = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
      }
      if (lane == 31) wsum[warp] = s;
      __syncthreads();
      int before = run;
      for (int w = 0; w < warp; ++w) before += wsum[w];
      if (e <= E) offsets[e] = before + s - v;
      for (int w = 0; w < 8; ++w) run += wsum[w];
      __syncthreads();
    }
    return;
  }
  __shared__ int32_t part[8][K];
  const int t = blockIdx.x - 1, c0 = blockIdx.y * 256 + tid, cstep = gridDim.y * 256;
  const U* src = x + (int64_t)t * ldx;
  U piece{};
  if (x && c0 < n) piece = __ldg(src + c0);  // on its way while the rows are counted
  uint32_t own[K];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const int i = t * k + j;
    own[j] = j < k ? (uint32_t)sort_key(__ldg(idx + i), E) << 20 | (uint32_t)i : 0u;
  }
  int count[K] = {};
#pragma unroll 4
  for (int i = tid; i < R; i += 256) {
    const uint32_t that = (uint32_t)sort_key(__ldg(idx + i), E) << 20 | (uint32_t)i;
#pragma unroll
    for (int j = 0; j < K; ++j) count[j] += that < own[j];
  }
#pragma unroll
  for (int j = 0; j < K; ++j) {
    count[j] = __reduce_add_sync(0xffffffffu, count[j]);
    if (lane == 0) part[warp][j] = count[j];
  }
  __syncthreads();
  U* dst[K];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    int row = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) row += part[w][j];
    const bool kept = j < k && (own[j] >> 20) < (uint32_t)E;
    dst[j] = kept && x ? xs + (int64_t)row * ldxs : nullptr;
    if (tid == j && j < k && blockIdx.y == 0) {
      perm[row] = t * k + j;
      inv[t * k + j] = kept ? row : -1;
    }
  }
  if (!x) return;
  for (int c = c0; c < n; c += cstep) {
    const U v = c == c0 ? piece : __ldg(src + c);
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (dst[j]) dst[j][c] = v;
  }
}

// Inclusive scan over a block of 1024 threads.  wsum: 32 words of shared memory.
__device__ __forceinline__ int block_scan(int v, int32_t* wsum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto warp_scan = [&](int s) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    return s;
  };
  const int s = warp_scan(v);
  if (lane == 31) wsum[warp] = s;
  __syncthreads();
  if (warp == 0) {  // the warps' sums become what lies before each warp
    const int w = wsum[lane];
    wsum[lane] = warp_scan(w) - w;
  }
  __syncthreads();
  return wsum[warp] + s;
}

// Up to 16384 entries in one launch of one cluster, without a workspace.  Each of its 256
// warps owns consecutive entries and keeps its lanes' keys (at most two) in registers:
//   - a warp ranks its entries among its own, 32 at a time, with a count per key;
//   - per key, the warps' counts become offsets within the block, the blocks' totals are
//     read over distributed shared memory, and the totals are scanned over the keys;
//   - row = start of the key + earlier blocks + earlier warps + rank.
// The scattered stores of perm bound it to what 8 SMs can do: at 16384 entries of 256 groups
// it takes as long as the two launches below, at 49152 4 us more.
__global__ void __launch_bounds__(kSortBlock) sort_cluster_kernel(const int32_t* __restrict__ idx, int R, int per,
                                                                  int E, int32_t* __restrict__ perm,
                                                                  int32_t* __restrict__ inv,
                                                                  int32_t* __restrict__ offsets) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  extern __shared__ uint16_t wcount[];  // [32][E+1]: entries of each key in each warp, then the earlier warps'
  __shared__ int32_t total[kMaxGroups + 1], base[kMaxGroups + 1];
  __shared__ int32_t wsum[kSortBlock / 32], carry;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int lo = (int)(rank * (kSortBlock / 32) + warp) * per, hi = min(R, lo + per);
  int key[kSortRounds], below[kSortRounds];
#pragma unroll
  for (int i = 0; i < kSortRounds; ++i) {
    const int at = lo + 32 * i + lane;
    key[i] = 32 * i < per && at < hi ? sort_key(__ldg(idx + at), E) : -1;
  }
  for (int c = tid; c < 16 * (E + 1); c += kSortBlock) reinterpret_cast<uint32_t*>(wcount)[c] = 0;
  __syncthreads();
  uint16_t* mine = wcount + warp * (E + 1);
#pragma unroll
  for (int i = 0; i < kSortRounds; ++i) {
    if (32 * i >= per) break;
    const unsigned same = __match_any_sync(0xffffffffu, key[i]);
    const int lower = __popc(same & ((1u << lane) - 1u));
    const int before = key[i] >= 0 ? mine[key[i]] : 0;
    below[i] = before + lower;
    __syncwarp();
    if (key[i] >= 0 && lower == 0) mine[key[i]] = (uint16_t)(before + __popc(same));
    __syncwarp();
  }
  __syncthreads();
  for (int e = tid; e <= E; e += kSortBlock) {
    int run = 0;
#pragma unroll 8
    for (int w = 0; w < kSortBlock / 32; ++w) {
      const int c = wcount[w * (E + 1) + e];
      wcount[w * (E + 1) + e] = (uint16_t)run;
      run += c;
    }
    total[e] = run;
  }
  cluster_arrive();
  cluster_wait();
  int run = 0;
  for (int e0 = 0; e0 <= E; e0 += kSortBlock) {
    const int e = e0 + tid;
    int all = 0, earlier = 0;
    if (e <= E) {
#pragma unroll
      for (int b = 0; b < kSortCluster; ++b) {
        const int v = (int)load_remote(&total[e], b);
        all += v;
        earlier += b < (int)rank ? v : 0;
      }
    }
    const int off = run + block_scan(all, wsum) - all;
    if (e <= E) {
      base[e] = off + earlier;
      if (rank == 0) offsets[e] = off;
    }
    if (tid == kSortBlock - 1) carry = off + all;  // read again only where E = 1024: one more key follows
    __syncthreads();
    run = carry;
  }
  cluster_arrive();  // totals have been read; a block may not leave before the others have
#pragma unroll
  for (int i = 0; i < kSortRounds; ++i) {
    if (key[i] < 0) continue;
    const int at = lo + 32 * i + lane;
    const int row = base[key[i]] + mine[key[i]] + below[i];
    perm[row] = at;
    inv[at] = key[i] < E ? row : -1;
  }
  cluster_wait();
}

// More entries: pass 1 over `per` entries a block, histogram of the keys.
__global__ void __launch_bounds__(kSortBlock) sort_hist_kernel(const int32_t* __restrict__ idx, int R, int per, int E,
                                                               int32_t* __restrict__ blk_hist) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  __shared__ int32_t hist[kMaxGroups + 1];
  for (int e = threadIdx.x; e <= E; e += kSortBlock) hist[e] = 0;
  __syncthreads();
  const int lo = blockIdx.x * per, hi = min(R, lo + per);
  for (int i = lo + threadIdx.x; i < hi; i += kSortBlock) atomicAdd(&hist[sort_key(idx[i], E)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += kSortBlock) blk_hist[(size_t)blockIdx.x * (E + 1) + e] = hist[e];
}

// Pass 2: every block sums the histograms of all blocks, and of those before its own, with
// its threads in groups of blocks; then it ranks its entries 1024 at a time as the cluster does.
__global__ void __launch_bounds__(kSortBlock) sort_rank_kernel(const int32_t* __restrict__ idx, int R, int per, int E,
                                                               const int32_t* __restrict__ blk_hist,
                                                               int32_t* __restrict__ perm, int32_t* __restrict__ inv,
                                                               int32_t* __restrict__ offsets) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  extern __shared__ uint8_t wcnt[];  // [32][E+1]: entries of each key in each warp
  __shared__ int32_t total[kMaxGroups + 1], base[kMaxGroups + 1];
  __shared__ int32_t wsum[kSortBlock / 32], carry;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int lo = blockIdx.x * per, hi = min(R, lo + per);
  int next = lo + tid < hi ? __ldg(idx + lo + tid) : 0;  // the first entries, on their way meanwhile
  for (int e = tid; e <= E; e += kSortBlock) total[e] = base[e] = 0;
  __syncthreads();
  // warps w, w + 32/groups, ... of one part of the keys each sum a share of the blocks
  const int parts = (E + 32) / 32;                   // 32 keys a warp at once
  const int shares = max(1, (kSortBlock / 32) / parts);
  for (int job = warp; job < parts * shares; job += kSortBlock / 32) {
    const int e = (job % parts) * 32 + lane, share = job / parts;
    int all = 0, before = 0;
    if (e <= E) {
#pragma unroll 8
      for (int b = share; b < (int)gridDim.x; b += shares) {
        const int v = __ldg(blk_hist + (size_t)b * (E + 1) + e);
        all += v;
        before += b < (int)blockIdx.x ? v : 0;
      }
      atomicAdd(&total[e], all);  // integer sums: any order
      atomicAdd(&base[e], before);
    }
  }
  __syncthreads();
  int run = 0;
  for (int e0 = 0; e0 <= E; e0 += kSortBlock) {
    const int e = e0 + tid;
    const int all = e <= E ? total[e] : 0;
    const int off = run + block_scan(all, wsum) - all;
    if (e <= E) {
      base[e] += off;
      if (blockIdx.x == 0) offsets[e] = off;
    }
    if (tid == kSortBlock - 1) carry = off + all;  // read again only where E = 1024: one more key follows
    __syncthreads();
    run = carry;
  }
  for (int i0 = lo; i0 < hi; i0 += kSortBlock) {
    for (int c = tid; c < 8 * (E + 1); c += kSortBlock) reinterpret_cast<uint32_t*>(wcnt)[c] = 0;  // 32 * (E+1) bytes
    const int i = i0 + tid;
    const int key = i < hi ? sort_key(next, E) : -1;
    next = i + kSortBlock < hi ? __ldg(idx + i + kSortBlock) : 0;
    __syncthreads();
    const unsigned same = __match_any_sync(0xffffffffu, key);
    const int below = __popc(same & ((1u << lane) - 1u));
    if (key >= 0 && below == 0) wcnt[warp * (E + 1) + key] = (uint8_t)__popc(same);
    __syncthreads();
    if (key >= 0) {
      int row = base[key] + below;
#pragma unroll 4
      for (int w = 0; w < warp; ++w) row += wcnt[w * (E + 1) + key];
      perm[row] = i;
      inv[i] = key < E ? row : -1;
    }
    if (i0 + kSortBlock >= hi) break;
    __syncthreads();
    for (int e = tid; e <= E; e += kSortBlock) {
      int s = 0;
#pragma unroll 8
      for (int w = 0; w < kSortBlock / 32; ++w) s += wcnt[w * (E + 1) + e];
      base[e] += s;
    }
    __syncthreads();
  }
}

// Where a thread of the row kernels works.  A token's row is walked by P consecutive
// threads (a power of two up to the block), so short rows share a block.
struct Walk {
  int64_t t;
  int lane, P;
};
__device__ __forceinline__ Walk walk(int shift) {
  return {(int64_t)blockIdx.x * (blockDim.x >> shift) + (threadIdx.x >> shift), (int)(threadIdx.x & ((1u << shift) - 1)),
          1 << shift};
}

// A token's row goes to each of its experts' rows.  K: entries a token has at most, so
// that the rows stay in registers.  Small accesses want more of them in flight: rows of 2047
// bf16, 8192 x 1 and 8192 x 6, take 30.3 and 74 us with 2, 25.2 and 69.7 with 8; of 302, 8192 x 2,
// 11.9 with 2 and 10.3 with 4 accesses of 4 bytes.
constexpr int row_pieces(int bytes) { return bytes >= 8 ? 2 : bytes == 4 ? 4 : 8; }
template <typename U, int K>
__global__ void __launch_bounds__(256) dispatch_rows_kernel(const U* __restrict__ x, int64_t ldx,
                                                            const int32_t* __restrict__ inv, int T, int k,
                                                            U* __restrict__ xs, int64_t ldxs, int n, int shift) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  const Walk w = walk(shift);
  if (w.t >= T) return;
  const U* src = x + w.t * ldx;
  U* dst[K];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const int row = j < k ? __ldg(inv + w.t * k + j) : -1;
    dst[j] = row >= 0 ? xs + (int64_t)row * ldxs : nullptr;
  }
  constexpr int V = row_pieces(sizeof(U));
  for (int c = w.lane; c < n; c += V * w.P) {
    U v[V];
#pragma unroll
    for (int u = 0; u < V; ++u)
      if (c + u * w.P < n) v[u] = __ldg(src + c + u * w.P);
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (dst[j]) {
#pragma unroll
        for (int u = 0; u < V; ++u)
          if (c + u * w.P < n) dst[j][c + u * w.P] = v[u];
      }
  }
}

// Rows and weights of a token's entries; an entry without a row gets weight 0 and is not read.
template <int K>
__device__ __forceinline__ void entries_of(int64_t t, const int32_t* inv, const float* w, int R, int k, int (&rows)[K],
                                           float (&wt)[K]) {
#pragma unroll
  for (int j = 0; j < K; ++j) {
    rows[j] = j < k ? __ldg(inv + t * k + j) : -1;
    if ((unsigned)rows[j] >= (unsigned)R) rows[j] = -1;
    wt[j] = rows[j] < 0 ? 0.0f : w ? __ldg(w + t * k + j) : 1.0f;
  }
}

// Sum of a token's expert rows, weighted or not.  U pieces of J rows are on their way
// before the first sum.  Blocks an SM by measurement, each the best of three or four budgets:
// with 16-byte accesses K = 2 wants many light threads (8: 31.3 us, 6: 33.8, 5: 36.2 for 8192 x 2
// rows of 4096 bf16), K = 8 few with all their loads in flight (1: 24.2 us, the compiler's own
// choice 32.5, for 4096 x 8 rows of 2048 bf16); smaller accesses want more threads (rows of 2046
// and 2047: 30.9 and 47.6 us with 6, 40.1 and 67.5 with 8).
constexpr int collect_blocks(int bytes, int K) {  // bytes: of an access
  if (bytes == 16) return K <= 2 ? 8 : K <= 4 ? 4 : 1;
  return bytes == 8 ? (K <= 4 ? 6 : 3) : bytes == 4 && K <= 4 ? 8 : 6;
}
template <typename T, int N, int K, int U>
__global__ void __launch_bounds__(256, collect_blocks(N * sizeof(T), K))
    collect_rows_kernel(const T* __restrict__ o, int64_t ldo, const float* __restrict__ w,
                        const int32_t* __restrict__ inv, int T_, int k, int cols, T* __restrict__ y, int64_t ldy,
                        int shift) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  using R = typename Raw<T, N>::type;
  constexpr int J = K < 4 ? K : 4;
  const Walk at = walk(shift);
  if (at.t >= T_) return;
  int rows[K];
  float wt[K];
  entries_of<K>(at.t, inv, w, T_ * k, k, rows, wt);
  bool any = false;
#pragma unroll
  for (int j = 0; j < K; ++j) any |= rows[j] >= 0;
  if (!any) {  // a token behind the batch's end
    const float zero[N] = {};
    for (int c = blockIdx.y * at.P + at.lane; c < cols; c += gridDim.y * at.P)
      store_vec<T, N>(y + at.t * ldy + (int64_t)c * N, zero);
    return;
  }
  for (int c = blockIdx.y * U * at.P + at.lane; c < cols; c += gridDim.y * U * at.P) {
    float acc[U][N] = {};
#pragma unroll
    for (int j0 = 0; j0 < K; j0 += J) {
      R v[U][J];
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < J; ++j)
          v[u][j] = rows[j0 + j] >= 0 && c + u * at.P < cols
                        ? __ldg(reinterpret_cast<const R*>(o + (int64_t)rows[j0 + j] * ldo) + c + u * at.P)
                        : zero_raw<R>();
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < J; ++j) {
          float f[N];
          decode_raw<T, N>(v[u][j], f);
#pragma unroll
          for (int i = 0; i < N; ++i) acc[u][i] = fmaf(wt[j0 + j], f[i], acc[u][i]);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (c + u * at.P < cols) store_vec<T, N>(y + at.t * ldy + (int64_t)(c + u * at.P) * N, acc[u]);
  }
}

// Gradient of collect: dy's row is read once, scaled into each expert row, and its dot
// product with each expert's output summed over the token's threads in a fixed order.
// 2048 x 2 rows of 4096 bf16: 16.0 us; 18.5 with one piece in flight, 18 to 19 with fewer
// or more registers a thread.  Blocks an SM by measurement, as above (4096 x 8 rows of 2046
// fp16: 77.8 us with 3, 84.2 with 4, 124 with 5; 4096 x 2 of 2047 bf16: 28.7 with 8, 32.0 with 6).
constexpr int gradient_blocks(int bytes, int K) {
  if (bytes == 16) return K <= 2 ? 5 : K <= 4 ? 4 : 3;
  return K <= 4 ? (bytes == 8 ? 6 : 8) : bytes == 2 ? 4 : 3;
}
template <typename T, int N, int K, int U>
__global__ void __launch_bounds__(256, gradient_blocks(N * sizeof(T), K))
    collect_backward_kernel(const T* __restrict__ dy, int64_t lddy, const T* __restrict__ o, int64_t ldo,
                            const float* __restrict__ w, const int32_t* __restrict__ inv, int T_, int k, int cols,
                            T* __restrict__ d_o, int64_t lddo, float* __restrict__ dw, int shift) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  using R = typename Raw<T, N>::type;
  constexpr int J = K < 8 ? 2 : 4;
  __shared__ float part[8][K];
  const Walk at = walk(shift);
  const bool real = at.t < T_;
  int rows[K];
  float wt[K], dot[K] = {};
  if (real) {
    entries_of<K>(at.t, inv, w, T_ * k, k, rows, wt);
    bool any = false;
#pragma unroll
    for (int j = 0; j < K; ++j) any |= rows[j] >= 0;
    for (int c = any ? at.lane : cols; c < cols; c += U * at.P) {
      R g[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        g[u] = c + u * at.P < cols ? __ldg(reinterpret_cast<const R*>(dy + at.t * lddy) + c + u * at.P) : zero_raw<R>();
#pragma unroll
      for (int j0 = 0; j0 < K; j0 += J) {
        R v[U][J];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int j = 0; j < J; ++j)
            v[u][j] = rows[j0 + j] >= 0 && c + u * at.P < cols
                          ? __ldg(reinterpret_cast<const R*>(o + (int64_t)rows[j0 + j] * ldo) + c + u * at.P)
                          : zero_raw<R>();
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (c + u * at.P >= cols) break;
          float a[N];
          decode_raw<T, N>(g[u], a);
#pragma unroll
          for (int j = 0; j < J; ++j) {
            if (rows[j0 + j] < 0) continue;
            float f[N], d[N];
            decode_raw<T, N>(v[u][j], f);
#pragma unroll
            for (int i = 0; i < N; ++i) {
              dot[j0 + j] = fmaf(a[i], f[i], dot[j0 + j]);
              d[i] = wt[j0 + j] * a[i];
            }
            store_vec<T, N>(d_o + (int64_t)rows[j0 + j] * lddo + (int64_t)(c + u * at.P) * N, d);
          }
        }
      }
    }
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int within = at.P < 32 ? at.P : 32;  // threads of the token in this warp
#pragma unroll
  for (int j = 0; j < K; ++j)
    for (int s = within / 2; s > 0; s >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], s);
  if (at.P > 32) {  // the token's warps: their sums in order
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (lane == 0) part[warp][j] = dot[j];
    __syncthreads();
    if (at.lane == 0)
#pragma unroll
      for (int j = 0; j < K; ++j) {
        dot[j] = 0.0f;
        for (int q = 0; q < at.P / 32; ++q) dot[j] += part[warp + q][j];
      }
  }
  if (real && at.lane == 0)
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (j < k) dw[at.t * k + j] = dot[j];
}

// ---------------------------------------------------------------- host
namespace {

int sort_per_block(int R) {  // entries per block: a multiple of 1024, at most 128 blocks
  const int per = (R + kSortMaxBlocks - 1) / kSortMaxBlocks;
  return (per + kSortBlock - 1) / kSortBlock * kSortBlock;
}

cudaError_t sort_medium(const int32_t* idx, int R, int E, int32_t* perm, int32_t* inv, int32_t* offsets,
                        cudaStream_t stream) {
  const int warps = kSortCluster * kSortBlock / 32, per = ((R + warps - 1) / warps + 31) / 32 * 32;
  const size_t smem = (size_t)64 * (E + 1);
  const cudaError_t e = cudaFuncSetAttribute(sort_cluster_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             64 * (kMaxGroups + 1));
  if (e != cudaSuccess) return e;
  return launch_cluster(sort_cluster_kernel, dim3(kSortCluster), dim3(kSortBlock), kSortCluster, smem, stream, idx, R,
                        per, E, perm, inv, offsets);
}

cudaError_t sort_large(const int32_t* idx, int R, int E, int32_t* perm, int32_t* inv, int32_t* offsets, int32_t* hist,
                       cudaStream_t stream) {
  const int per = sort_per_block(R), nblk = (R + per - 1) / per;
  const cudaError_t e = launch_chained(sort_hist_kernel, dim3(nblk), dim3(kSortBlock), 0, stream, idx, R, per, E, hist);
  if (e != cudaSuccess) return e;
  return launch_chained(sort_rank_kernel, dim3(nblk), dim3(kSortBlock), (size_t)32 * (E + 1), stream, idx, R, per, E,
                        (const int32_t*)hist, perm, inv, offsets);
}

// Whether the blocks count their rows themselves: up to 2^24 comparisons over all of them (512
// tokens x 8: 8.5 us with rows of 4 KB where sort and rows take 9.6, 1024 x 8: 15.8 / 12.8),
// without rows 2^23 (2048 entries 4.8 / 4.8 us, 4096 11.3 / 4.9).
bool counts_rows(int T, int k, bool rows) {
  return (int64_t)T * k * T * (k <= 2 ? 2 : k <= 4 ? 4 : 8) <= (rows ? 1 << 24 : 1 << 23);
}

// Threads that walk a row of n pieces, U at a time: a power of two from 8 to `most`, as its shift.
int walk_shift(int n, int U, int most) {
  int s = 3;
  while ((1 << s) < most && (int64_t)(1 << s) * U < n) ++s;
  return s;
}
unsigned walk_blocks(int T, int threads, int shift) { return (unsigned)((T + (threads >> shift) - 1) / (threads >> shift)); }

template <typename U>
cudaError_t dispatch_as(const int32_t* idx, int T, int k, int E, int32_t* perm, int32_t* inv, int32_t* offsets,
                        ConstRows x, Rows xs, int es, int H, void* ws, cudaStream_t stream) {
  const int R = T * k;
  const int unit = sizeof(U);
  const int64_t ldx = x.ld * es / unit, ldxs = xs.ld * es / unit;
  const int n = (int)((int64_t)H * es / unit);
  const U* xp = (const U*)x.p;
  U* xsp = (U*)xs.p;
  if (counts_rows(T, k, xp != nullptr)) {
    unsigned ny = 1;  // column blocks: more parallelism for few tokens
    while (T * ny < 148 && (int64_t)ny * 256 < n) ny *= 2;
    auto kern = k <= 2   ? dispatch_small_kernel<U, 2>
                : k <= 4 ? dispatch_small_kernel<U, 4>
                         : dispatch_small_kernel<U, 8>;
    return launch_chained(kern, dim3(T + 1, ny), dim3(256), 0, stream, idx, R, k, E, perm, inv, offsets, xp, ldx, xsp,
                          ldxs, n);
  }
  cudaError_t e = R <= kSortMedium ? sort_medium(idx, R, E, perm, inv, offsets, stream)
                                   : sort_large(idx, R, E, perm, inv, offsets, (int32_t*)ws, stream);
  if (e != cudaSuccess || !xp) return e;
  const int shift = walk_shift(n, row_pieces(sizeof(U)), 256);
  auto kern = k <= 2 ? dispatch_rows_kernel<U, 2> : k <= 4 ? dispatch_rows_kernel<U, 4> : dispatch_rows_kernel<U, 8>;
  return launch_chained(kern, dim3(walk_blocks(T, 256, shift)), dim3(256), 0, stream, xp, ldx, (const int32_t*)inv, T,
                        k, xsp, ldxs, n, shift);
}

// U: pieces of each row in flight.
template <typename T, int N, int K>
cudaError_t collect_as(ConstRows o, const float* w, const int32_t* inv, int T_, int k, int H, Rows y,
                       cudaStream_t stream) {
  constexpr int U = N * sizeof(T) < 16 && K <= 2 ? 4 : 2;
  const int cols = H / N, shift = walk_shift(cols, U, 256);
  const unsigned blocks = walk_blocks(T_, 256, shift);
  unsigned ny = 1;  // column blocks: more parallelism for few tokens
  while (blocks * ny < 2 * 148 && (int64_t)ny * U * 256 < cols) ny *= 2;
  return launch_chained(collect_rows_kernel<T, N, K, U>, dim3(blocks, ny), dim3(256), 0, stream, (const T*)o.p, o.ld, w,
                        inv, T_, k, cols, (T*)y.p, y.ld, shift);
}

template <typename T, int N, int K>
cudaError_t collect_backward_as(ConstRows dy, ConstRows o, const float* w, const int32_t* inv, int T_, int k, int H,
                                Rows d_o, float* dw, cudaStream_t stream) {
  constexpr int U = N * sizeof(T) < 16 && K > 4 ? 4 : 2;
  const int cols = H / N;
  const int shift = walk_shift(cols, U, 256);
  return launch_chained(collect_backward_kernel<T, N, K, U>, dim3(walk_blocks(T_, 256, shift)), dim3(256), 0, stream,
                        (const T*)dy.p, dy.ld, (const T*)o.p, o.ld, w, inv, T_, k, cols, (T*)d_o.p, d_o.ld, dw,
                        shift);
}

template <typename T, int N>
cudaError_t collect_k(ConstRows o, const float* w, const int32_t* inv, int T_, int k, int H, Rows y, cudaStream_t s) {
  return k <= 2   ? collect_as<T, N, 2>(o, w, inv, T_, k, H, y, s)
         : k <= 4 ? collect_as<T, N, 4>(o, w, inv, T_, k, H, y, s)
                  : collect_as<T, N, 8>(o, w, inv, T_, k, H, y, s);
}
template <typename T, int N>
cudaError_t collect_backward_k(ConstRows dy, ConstRows o, const float* w, const int32_t* inv, int T_, int k, int H,
                               Rows d_o, float* dw, cudaStream_t s) {
  return k <= 2   ? collect_backward_as<T, N, 2>(dy, o, w, inv, T_, k, H, d_o, dw, s)
         : k <= 4 ? collect_backward_as<T, N, 4>(dy, o, w, inv, T_, k, H, d_o, dw, s)
                  : collect_backward_as<T, N, 8>(dy, o, w, inv, T_, k, H, d_o, dw, s);
}

// The most values, a power of two up to 16 bytes, that all these bits (addresses, pitches and
// widths in bytes) are multiples of.
int values_at_once(uint64_t bits, int es) {
  int n = 16 / es;
  while (bits % (uint64_t)(n * es) != 0) n /= 2;
  return n;
}

template <typename T>
cudaError_t collect_n(int n, ConstRows o, const float* w, const int32_t* inv, int T_, int k, int H, Rows y, cudaStream_t s) {
  if constexpr (sizeof(T) == 2)
    if (n == 8) return collect_k<T, 8>(o, w, inv, T_, k, H, y, s);
  return n == 4   ? collect_k<T, 4>(o, w, inv, T_, k, H, y, s)
         : n == 2 ? collect_k<T, 2>(o, w, inv, T_, k, H, y, s)
                  : collect_k<T, 1>(o, w, inv, T_, k, H, y, s);
}
template <typename T>
cudaError_t collect_backward_n(int n, ConstRows dy, ConstRows o, const float* w, const int32_t* inv, int T_, int k, int H,
                               Rows d_o, float* dw, cudaStream_t s) {
  if constexpr (sizeof(T) == 2)
    if (n == 8) return collect_backward_k<T, 8>(dy, o, w, inv, T_, k, H, d_o, dw, s);
  return n == 4   ? collect_backward_k<T, 4>(dy, o, w, inv, T_, k, H, d_o, dw, s)
         : n == 2 ? collect_backward_k<T, 2>(dy, o, w, inv, T_, k, H, d_o, dw, s)
                  : collect_backward_k<T, 1>(dy, o, w, inv, T_, k, H, d_o, dw, s);
}

}  // namespace

uint64_t sort_ws_bytes(int R, int E) {
  if (R <= kSortMedium) return 0;
  const int per = sort_per_block(R);
  return up256((uint64_t)((R + per - 1) / per) * (E + 1) * 4);
}

cudaError_t launch_dispatch(const int32_t* idx, int T, int k, int E, int32_t* perm, int32_t* inv, int32_t* offsets,
                            ConstRows x, Rows xs, int H, int dtype, void* ws, cudaStream_t stream) {
  const int es = dtype_size(dtype);
  const uint64_t all = (uintptr_t)x.p | (uintptr_t)xs.p | (uint64_t)(x.ld * es) | (uint64_t)(xs.ld * es) |
                       (uint64_t)((int64_t)H * es);
  if ((all & 15) == 0) return dispatch_as<uint4>(idx, T, k, E, perm, inv, offsets, x, xs, es, H, ws, stream);
  if ((all & 7) == 0) return dispatch_as<uint2>(idx, T, k, E, perm, inv, offsets, x, xs, es, H, ws, stream);
  if ((all & 3) == 0) return dispatch_as<uint32_t>(idx, T, k, E, perm, inv, offsets, x, xs, es, H, ws, stream);
  return dispatch_as<uint16_t>(idx, T, k, E, perm, inv, offsets, x, xs, es, H, ws, stream);
}

cudaError_t launch_collect(ConstRows o, const float* w, const int32_t* inv, int T, int k, int H, int dtype, Rows y,
                           cudaStream_t stream) {
  const int es = dtype_size(dtype);
  const int n = values_at_once((uintptr_t)o.p | (uintptr_t)y.p | (uint64_t)(o.ld * es) | (uint64_t)(y.ld * es) |
                                   (uint64_t)((int64_t)H * es), es);
  if (dtype == MOE_F32) return collect_n<float>(n, o, w, inv, T, k, H, y, stream);
  return dtype == MOE_F16 ? collect_n<__half>(n, o, w, inv, T, k, H, y, stream)
                          : collect_n<__nv_bfloat16>(n, o, w, inv, T, k, H, y, stream);
}

cudaError_t launch_collect_backward(ConstRows dy, ConstRows o, const float* w, const int32_t* inv, int T, int k, int H,
                                    int dtype, Rows d_o, float* dw, cudaStream_t stream) {
  const int es = dtype_size(dtype);
  const int n = values_at_once((uintptr_t)dy.p | (uintptr_t)o.p | (uintptr_t)d_o.p | (uint64_t)(dy.ld * es) |
                                   (uint64_t)(o.ld * es) | (uint64_t)(d_o.ld * es) | (uint64_t)((int64_t)H * es), es);
  if (dtype == MOE_F32) return collect_backward_n<float>(n, dy, o, w, inv, T, k, H, d_o, dw, stream);
  return dtype == MOE_F16 ? collect_backward_n<__half>(n, dy, o, w, inv, T, k, H, d_o, dw, stream)
                          : collect_backward_n<__nv_bfloat16>(n, dy, o, w, inv, T, k, H, d_o, dw, stream);
}

}  // namespace moe

// Low-rank adapters of many requests at once beside a shared projection or the whole
// layer: out[t] = y[t] + scale[a] * B_a (A_a x[t]) for the adapter a of token t, and
// out[t] = y[t] for a token without one.
//
// Tokens come sorted by adapter (routes.cu), so a tile of rows shares its adapter and
// both products are matrix products of a tile of tokens with A_a and B_a.  A cluster of
// 1 to 8 blocks takes one tile: each block has a share of the k values for
//   P[row][r] = sum_k x[k] A_a[r][k]
// in fp32, the blocks read one another's shares from distributed shared memory and add
// them in order, and each block then has a share of the outputs for scale * P B_a^T + y.
// One launch, no workspace, nothing added in global memory.  (Down and up product as two
// launches with partial sums in a workspace took 9.6 us for 64 requests where this takes
// 6.6, and 104 us for the long batch below.)
//
// The up product's fp32 operand P goes in as two terms of the value type, P = hi + lo: to within
// 2^-17 of a value in bf16 and 2^-23 in fp16, so its rounding stays far below that of the stored
// result.  In fp16 a row's largest magnitude is first brought to 2^13 .. 2^14 by a power of two,
// since P may pass fp16's range at either end: unscaled, lo would be subnormal for values below
// 2^-3, and terms near 2^-20 keep 5 bits.  Values far below their row's largest are off by at
// most 2^-38 of that.
//
// Two kernels.  Decode batches: tiles of 16 tokens on mma.sync, operands from memory straight
// to fragments (the contraction index may be permuted if both operands are permuted alike,
// so a lane takes eight consecutive values, 16 bytes, of its row).  What bounds it is the
// chain of latencies: finding the tile 0.8 us, loads and product 0.9, the cluster's meeting
// 1.3, the second product 0.9.  K = N = 4096, r 16: 1 token 4.9 us, 64 requests of 48 adapters
// 6.6 us; 64 requests of r 64 (69 MB of adapters) 12.0 us, 89% of the copy rate.
// Long batches: tiles of 64 tokens on tcgen05 (adapter_wide_kernel).  8192 tokens, K = N =
// 2048, r 64 (113 MB): 31 us, 56% of the copy rate; r 128 43 us.  Each block goes through
// finding its tile, the down product, the cluster's meeting and the up product once, all blocks
// at the same time, so memory idles in the meetings; mma.sync in its place took 38 and 76 us.
#include <algorithm>

#include "ops_common.cuh"
#include "tc_ptx.cuh"

namespace moe {

constexpr int kAdWarps = 8;
constexpr int kAdThreads = 32 * kAdWarps;
constexpr int kAdMaxCluster = 8;
constexpr long long kWideWait = 2000000000ll;  // cycles a wait on the tensor cores may take, about a second

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T> constexpr bool is_f16 = false;
template <> constexpr bool is_f16<__half> = true;

struct Tile {
  int adapter, row0, rows;  // rows 0: none
};

// Tile `want` of the sorted rows: each adapter's rows in tiles of TM, adapters in order.
// Every thread takes a run of adapters and the block scans their tile counts.  first: shared
// memory for the first kAdThreads entries of perm, which short batches take from there, so
// that they are loaded together with the offsets and not after them.
__device__ Tile find_tile(int want, int TM, const int32_t* __restrict__ offsets, int n, int T,
                          const int32_t* __restrict__ perm, int32_t* first) {
  __shared__ int wsum[kAdWarps];
  __shared__ Tile found;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (n + kAdThreads - 1) / kAdThreads;
  if (tid == 0) found = {0, 0, 0};
  const int mine_of_perm = first && tid < T ? __ldg(perm + tid) : -1;
  auto lo_of = [&](int a) { return min(max(__ldg(offsets + a), 0), T); };
  auto hi_of = [&](int a, int lo) { return min(max(__ldg(offsets + a + 1), lo), T); };
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int a = tid * per + i;
    if (a >= n) break;
    const int lo = lo_of(a);
    mine += (hi_of(a, lo) - lo + TM - 1) / TM;
  }
  int s = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  if (lane == 31 && warp < kAdWarps) wsum[warp] = s;
  if (first) first[tid] = mine_of_perm;
  __syncthreads();
  int before = s - mine;
  for (int w = 0; w < min(warp, kAdWarps); ++w) before += wsum[w];
  if (want >= before && want < before + mine) {
    for (int i = 0; i < per; ++i) {
      const int a = tid * per + i;
      if (a >= n) break;
      const int lo = lo_of(a), hi = hi_of(a, lo), tiles = (hi - lo + TM - 1) / TM;
      if (want < before + tiles) {
        const int r0 = lo + (want - before) * TM;
        found = {a, r0, min(TM, hi - r0)};
        break;
      }
      before += tiles;
    }
  }
  __syncthreads();
  return found;
}

// 16 bytes of y, which may be the output itself: not through the read-only path.
__device__ __forceinline__ uint4 load_y16(const void* p) {
  uint4 v;
  asm("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// out = y for the rows without an adapter, those from `first` on: a share of them for every
// warp, whether its block has a tile or not.  The shares, 128 pieces of 16 bytes, start at the
// last blocks, which have no tile if any has none.
template <typename T>
__device__ void copy_rest(const T* y, int64_t ldy, T* out, int64_t ldo, int N, int first, int T_,
                          const int32_t* __restrict__ perm) {
  const int lane = threadIdx.x & 31, pieces = N / 8, shares = (pieces + 127) / 128;
  const int64_t all = (int64_t)(T_ - first) * shares;
  for (int64_t i = (int64_t)(gridDim.x - 1 - blockIdx.x) * kAdWarps + (threadIdx.x >> 5); i < all;
       i += (int64_t)gridDim.x * kAdWarps) {
    const int row = (int)(i / shares), t = __ldg(perm + first + row);
    if ((unsigned)t >= (unsigned)T_) continue;
    const int c0 = (int)(i - (int64_t)row * shares) * 128 + lane;
    const uint4* from = reinterpret_cast<const uint4*>(y + (int64_t)t * ldy) + c0;
    uint4* to = reinterpret_cast<uint4*>(out + (int64_t)t * ldo) + c0;
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c0 + 32 * k < pieces) v[k] = __ldg(from + 32 * k);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c0 + 32 * k < pieces) to[32 * k] = v[k];
  }
}

// Two values as hi and lo terms of T.  hi stays finite: a finite value next to T's largest would round to an
// infinity, and an infinity goes to lo alone (inf - inf would be NaN), where a NaN goes too.
template <typename T>
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  constexpr float top = is_f16<T> ? 65504.0f : 0x1.FEp127f;
  hi = pack2<T>(fminf(fmaxf(a, -top), top), fminf(fmaxf(b, -top), top));
  const float2 f = unpack2<T>(hi);
  lo = pack2<T>(a - f.x, b - f.y);
}

// The power of two 2^-e that brings a row of P, whose largest magnitude has these bits, into
// [2^13, 2^14), and 2^e, which takes it back.  An infinity is taken for the largest finite value: it
// stays infinite, and the finite terms beside it stay finite.  Rows below 2^-87 go up by 2^100 only,
// so that both powers are ordinary numbers: no B makes such a row more than 2^-63.
struct RowScale {
  float down, back;
};
__device__ __forceinline__ RowScale row_scale(uint32_t big) {
  const int e = max((int)(min(big, 0x7F7FFFFFu) >> 23) - 127 - 13, -100);
  return {__uint_as_float((uint32_t)(127 - e) << 23), __uint_as_float((uint32_t)(127 + e) << 23)};
}

// Eight values of a lane, its share of 32 of the rank, as the MMA's first operand (h: row g or
// g + 8): pairs 0, 1 to the first MMA, 2, 3 to the second, as B's.
template <typename T>
__device__ __forceinline__ void split8(const float (&p)[8], int h, uint32_t (&hi)[2][4], uint32_t (&lo)[2][4]) {
  split2<T>(p[0], p[1], hi[0][h], lo[0][h]);
  split2<T>(p[2], p[3], hi[0][2 + h], lo[0][2 + h]);
  split2<T>(p[4], p[5], hi[1][h], lo[1][h]);
  split2<T>(p[6], p[7], hi[1][2 + h], lo[1][2 + h]);
}

// Adds the blocks' shares of P in order: every thread takes 16-byte pieces, whose remote
// loads are consecutive over the warp.  mine: [TM][RP] in every block; P: [TM][KB*32 + 4],
// zeros beyond the rank and behind the tile's rows.
template <int TM, int KB, int RP>
__device__ __forceinline__ void gather_p(const float* mine, int cluster, float scale, int r, int rows, float* P) {
  constexpr int LD = KB * 32 + 4, PIECES = KB * 8;
#pragma unroll
  for (int c0 = 0; c0 < TM * PIECES; c0 += kAdThreads) {
    const int c = c0 + threadIdx.x, row = c / PIECES, i = (c % PIECES) * 4;
    if (TM * PIECES % kAdThreads != 0 && c >= TM * PIECES) break;
    float4 s = make_float4(0, 0, 0, 0);
    if (i < r && row < rows) {  // the rank is a multiple of 8
      float4 v[kAdMaxCluster];
#pragma unroll
      for (int k = 0; k < kAdMaxCluster; ++k)
        if (k < cluster) v[k] = load_remote4(mine + row * RP + i, k);
#pragma unroll
      for (int k = 0; k < kAdMaxCluster; ++k)
        if (k < cluster) s.x += v[k].x, s.y += v[k].y, s.z += v[k].z, s.w += v[k].w;
      s.x *= scale, s.y *= scale, s.z *= scale, s.w *= scale;
    }
    *reinterpret_cast<float4*>(P + row * LD + i) = s;
  }
}

// A lane's share of P as the up product's operand: rows g and g + 8 of the token tile at P.
// back: what takes a row's power of two back (fp16; else 1).
template <typename T, int KB>
__device__ __forceinline__ void operand_p(const float* P, uint32_t (&hi)[KB][2][4], uint32_t (&lo)[KB][2][4],
                                          float (&back)[2]) {
  constexpr int LD = KB * 32 + 4;
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float p[KB][8];
    uint32_t big = 0;
#pragma unroll
    for (int b = 0; b < KB; ++b)
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(P + (8 * h + g) * LD + 32 * b + 8 * q + i);
        p[b][i] = v.x, p[b][i + 1] = v.y, p[b][i + 2] = v.z, p[b][i + 3] = v.w;
      }
    back[h] = 1.0f;
    if constexpr (is_f16<T>) {  // the row's four lanes agree on its power of two
#pragma unroll
      for (int b = 0; b < KB; ++b)
#pragma unroll
        for (int i = 0; i < 8; ++i) big = max(big, __float_as_uint(p[b][i]) & 0x7FFFFFFFu);
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
      const RowScale by = row_scale(big);
      back[h] = by.back;
#pragma unroll
      for (int b = 0; b < KB; ++b)
#pragma unroll
        for (int i = 0; i < 8; ++i) p[b][i] *= by.down;
    }
#pragma unroll
    for (int b = 0; b < KB; ++b) split8<T>(p[b], h, hi[b], lo[b]);
  }
}

// 32 of the rank times 32 outputs, small terms first; the four sums are independent.
template <typename T>
__device__ __forceinline__ void mma_hi_lo(float (&acc)[4][4], const uint32_t (&hi)[2][4], const uint32_t (&lo)[2][4],
                                          const uint4 (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) mma16816<T>(acc[i], lo[0], w[i].x, w[i].y);
#pragma unroll
  for (int i = 0; i < 4; ++i) mma16816<T>(acc[i], lo[1], w[i].z, w[i].w);
#pragma unroll
  for (int i = 0; i < 4; ++i) mma16816<T>(acc[i], hi[0], w[i].x, w[i].y);
#pragma unroll
  for (int i = 0; i < 4; ++i) mma16816<T>(acc[i], hi[1], w[i].z, w[i].w);
}

// y + back * acc for a lane's eight outputs of row g (h = 0) or g + 8 (h = 1).
template <typename T>
__device__ __forceinline__ void store_sum(T* out, const uint4& y, const float (&acc)[4][4], int h, float back) {
  const uint32_t w[4] = {y.x, y.y, y.z, y.w};
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<T>(w[i]);
    v[i] = pack2<T>(fmaf(back, acc[i][2 * h], f.x), fmaf(back, acc[i][2 * h + 1], f.y));
  }
  *reinterpret_cast<uint4*>(out) = make_uint4(v[0], v[1], v[2], v[3]);
}

// ---------------------------------------------------------------- decode batches
// Tiles of 16 tokens; NR: n8 tiles of the rank (r <= 8*NR).  The 8 warps share the block's k
// values, 32 at a time, then its outputs.
template <typename T, int NR>
__global__ void __launch_bounds__(kAdThreads, NR <= 8 ? 2 : 1)
    adapter_kernel(const T* __restrict__ x, int64_t ldx, const T* y, int64_t ldy, int T_, int K, int N, int r, int n,
                   const T* __restrict__ A, const T* __restrict__ B, const float* __restrict__ scale,
                   const int32_t* __restrict__ perm, const int32_t* __restrict__ offsets, bool rest, int cluster,
                   int kslice, int nslice, T* out, int64_t ldo) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  constexpr int TM = 16, KG = kAdWarps, KB = (NR + 3) / 4, RP = NR * 8;
  extern __shared__ __align__(16) float sm[];
  float* red = sm;                  // [KG][TM][RP] shares of the warps
  float* mine = red + KG * TM * RP;  // [TM][RP] this block's share of P
  float* P = mine + TM * RP;         // [TM][KB*32 + 4]
  __shared__ int32_t first[kAdThreads];
  const uint32_t rank = cluster_rank();
  const int rest0 = rest ? min(max(__ldg(offsets + n), 0), T_) : T_;
  const bool few = T_ <= kAdThreads;
  const Tile tile = find_tile(blockIdx.x / cluster, TM, offsets, n, T_, perm, few ? first : nullptr);
  if (tile.rows == 0) {  // all blocks of the cluster alike
    if (rest) copy_rest(y, ldy, out, ldo, N, rest0, T_, perm);
    return;
  }
  const float sc = __ldg(scale + tile.adapter);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const int n0 = rank * nslice, n1 = min(N, n0 + nslice);
  int tok[2];  // tokens of the lane's rows, -1: none
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = tile.row0 + 8 * h + g;
    const int t = 8 * h + g >= tile.rows ? -1 : few ? first[row] : __ldg(perm + row);
    tok[h] = (unsigned)t < (unsigned)T_ ? t : -1;
  }
  const T* Ba = B + (int64_t)tile.adapter * N * r;
  {  // B's slice is on its way to L2 while A's is multiplied
    const int64_t bytes = (int64_t)(n1 - n0) * r * sizeof(T);
    const char* p = reinterpret_cast<const char*>(Ba + (int64_t)n0 * r);
    for (int64_t c = threadIdx.x * 128; c < bytes; c += kAdThreads * 128)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p + c));
  }
  uint32_t hi[KB][2][4], lo[KB][2][4];
  {
    float acc[NR][4];
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[i][c] = 0.0f;
    const T* x0 = x + (int64_t)tok[0] * ldx;
    const T* x1 = x + (int64_t)tok[1] * ldx;
    const T* Ar = A + ((int64_t)tile.adapter * r + g) * K;
    const int k0 = rank * kslice, k1 = min(K, k0 + kslice);
#pragma unroll 2
    for (int kk = k0 + warp * 32 + q * 8; kk - q * 8 < k1; kk += KG * 32) {
      const bool in = kk < k1;  // k1 and kk are multiples of 8
      const uint4 zero = make_uint4(0, 0, 0, 0);
      const uint4 a = in && tok[0] >= 0 ? __ldg(reinterpret_cast<const uint4*>(x0 + kk)) : zero;
      const uint4 b = in && tok[1] >= 0 ? __ldg(reinterpret_cast<const uint4*>(x1 + kk)) : zero;
      uint4 w[NR];
#pragma unroll
      for (int i = 0; i < NR; ++i)
        w[i] = in && 8 * i < r ? __ldg(reinterpret_cast<const uint4*>(Ar + (int64_t)8 * i * K + kk)) : zero;
      const uint32_t a0[4] = {a.x, b.x, a.y, b.y}, a1[4] = {a.z, b.z, a.w, b.w};
#pragma unroll
      for (int i = 0; i < NR; ++i) mma16816<T>(acc[i], a0, w[i].x, w[i].y);
#pragma unroll
      for (int i = 0; i < NR; ++i) mma16816<T>(acc[i], a1, w[i].z, w[i].w);
    }
    // the warps' shares added in order, then (gather_p) the blocks'
    float* mr = red + warp * TM * RP;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < NR; ++i)
        *reinterpret_cast<float2*>(mr + (8 * h + g) * RP + 8 * i + 2 * q) = make_float2(acc[i][2 * h], acc[i][2 * h + 1]);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < TM * RP; c += kAdThreads) {
    float s = red[c];
#pragma unroll
    for (int p = 1; p < KG; ++p) s += red[p * TM * RP + c];
    mine[c] = s;
  }
  cluster_arrive();
  // column c of MMA tile i is output nn + 8*(c/2) + 2*i + c%2, so that a lane ends up with
  // outputs nn + 8q .. nn + 8q + 7 of its rows
  auto load_y = [&](int nn, uint4 (&v)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      v[h] = tok[h] >= 0 && nn + 8 * q < n1
                 ? load_y16(y + (int64_t)tok[h] * ldy + nn + 8 * q)
                 : make_uint4(0, 0, 0, 0);
  };
  auto load_b = [&](int nn, int b, uint4 (&v)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int o = nn + 8 * (g >> 1) + 2 * i + (g & 1), kk = 32 * b + 8 * q;
      v[i] = o < n1 && kk < r ? __ldg(reinterpret_cast<const uint4*>(Ba + (int64_t)o * r + kk)) : make_uint4(0, 0, 0, 0);
    }
  };
  // the first step's operands are on their way while the cluster meets (of B the first 32 or 64 of the rank)
  constexpr int AHEAD = KB < 2 ? KB : 2;
  int nn = n0 + warp * 32;
  uint4 yv[2], bv[AHEAD][4];
  load_y(nn, yv);
#pragma unroll
  for (int b = 0; b < AHEAD; ++b) load_b(nn, b, bv[b]);
  cluster_wait();
  float back[2];
  gather_p<TM, KB, RP>(mine, cluster, sc, r, tile.rows, P);
  cluster_arrive();  // this warp has read; no block may leave before all have
  __syncthreads();
  operand_p<T, KB>(P, hi, lo, back);
  while (nn < n1) {
    float acc[4][4] = {};
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      if (b >= AHEAD) load_b(nn, b, bv[b % AHEAD]);
      mma_hi_lo<T>(acc, hi[b], lo[b], bv[b % AHEAD]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (tok[h] >= 0 && nn + 8 * q < n1)
        store_sum<T>(out + (int64_t)tok[h] * ldo + nn + 8 * q, yv[h], acc, h, back[h]);
    nn += KG * 32;
    if (nn >= n1) break;
    load_y(nn, yv);
#pragma unroll
    for (int b = 0; b < AHEAD; ++b) load_b(nn, b, bv[b]);
  }
  if (rest) copy_rest(y, ldy, out, ldo, N, rest0, T_, perm);
  cluster_wait();
}

// ---------------------------------------------------------------- long batches
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {  // zeros where `in` is false
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// 16 tensor-memory lanes x 8*X 32-bit columns: lane (g, q) of the warp gets, for every 8
// columns, columns 2q and 2q + 1 of row g, then of row g + 8 (an m16n8 accumulator).
template <int X>
__device__ __forceinline__ void tmem_rows16(uint32_t taddr, float (&r)[X][4]) {
  static_assert(X == 2 || X == 4 || X == 8, "");
  float* f = &r[0][0];
  if constexpr (X == 2)
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
                 : "r"(taddr));
  else if constexpr (X == 4)
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7]), "=f"(f[8]),
          "=f"(f[9]), "=f"(f[10]), "=f"(f[11]), "=f"(f[12]), "=f"(f[13]), "=f"(f[14]), "=f"(f[15])
        : "r"(taddr));
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7]), "=f"(f[8]),
          "=f"(f[9]), "=f"(f[10]), "=f"(f[11]), "=f"(f[12]), "=f"(f[13]), "=f"(f[14]), "=f"(f[15]), "=f"(f[16]),
          "=f"(f[17]), "=f"(f[18]), "=f"(f[19]), "=f"(f[20]), "=f"(f[21]), "=f"(f[22]), "=f"(f[23]), "=f"(f[24]),
          "=f"(f[25]), "=f"(f[26]), "=f"(f[27]), "=f"(f[28]), "=f"(f[29]), "=f"(f[30]), "=f"(f[31])
        : "r"(taddr));
}

// Tiles of 64 tokens of one adapter.  The same two products and the same split over a
// cluster, on tcgen05 with accumulators in tensor memory: at ranks of 64 the mma.sync form
// spent half its time feeding and running the tensor cores beside the loads.  Operands come
// through one ring of 64-wide stages in shared memory over both products: x and A, then y and
// B.  Eight warps copy (cp.async: tokens are gathered, so there is no box for a TMA load) and
// drain; a ninth issues the MMAs.  One block barrier a stage says that the stage has landed
// and that the stage two before it has been drained, which is the one copied into next but two.
//   D1[64][RP]  = sum over k of x A^T        tensor memory columns 0 .. 127
//   D2[64][64]  = P_lo B^T + P_hi B^T        two buffers, columns 128 .. 255; one is drained
//                                            and added to y while the next is computed
// x, A, B and P lie in 128-byte swizzled rows (16-byte chunk c of row j at c ^ (j % 8)), as the
// matrix descriptors say.  Row j of a B stage is output 8*(c/2) + 2*i + c%2 of its half of the
// 64, with i = j/8 % 4 and c = j % 8, so that a lane of the epilogue has eight outputs in a row.
// Two blocks share an SM; each asks for 256 of its 512 tensor-memory columns and for more than
// a third of its shared memory, so that a third block never waits for columns.  Every wait is bounded;
// where one gives up, all later ones of the block do, and it ends when its MMAs have.  withhold (a test
// hook): the first stage's completion is not reported.
constexpr int kWideStages = 5;
constexpr int kWideAhead = 3;  // stages copied ahead
constexpr int kWideThreads = kAdThreads + 32;
constexpr int kWideTokens = 64;
constexpr uint32_t kWideTmem = 256;
constexpr int kWideTile = 64 * 128;  // 64 rows of 128 bytes

template <int NR> constexpr int wide_stage_bytes() { return kWideTile + (NR <= 8 ? kWideTile : 2 * kWideTile); }
template <int NR> constexpr int wide_smem_bytes() {
  return 1024 + kWideStages * wide_stage_bytes<NR>() + 2 * (NR <= 8 ? 1 : 2) * kWideTile + kWideTokens * 4 +
         (NR <= 8 ? 0 : kWideTokens * NR * 8 * 4);
}

static_assert(wide_smem_bytes<4>() > 76 * 1024, "two blocks an SM, not three");

template <typename T> __host__ __device__ constexpr uint32_t wide_idesc(int N) {
  const uint32_t type = is_f16<T> ? 0u : 1u;  // of A and of B
  return (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kWideTokens >> 4) << 24);
}

template <typename T, int NR>
__global__ void __launch_bounds__(kWideThreads, NR <= 8 ? 2 : 1)
    adapter_wide_kernel(const T* __restrict__ x, int64_t ldx, const T* y, int64_t ldy, int T_, int K, int N, int r,
                        int n, const T* __restrict__ A, const T* __restrict__ B, const float* __restrict__ scale,
                        const int32_t* __restrict__ perm, const int32_t* __restrict__ offsets, bool rest, int cluster,
                        int kslice, int nslice, T* out, int64_t ldo, int32_t* status, long long wait, bool withhold) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  constexpr int TM = kWideTokens, RP = NR * 8, KBLK = NR <= 8 ? 1 : 2, HALF = RP / 16;  // HALF: n8 tiles of half of P
  constexpr int STAGE = wide_stage_bytes<NR>();
  extern __shared__ uint8_t wide_sm[];
  __shared__ uint64_t done[kWideStages];  // the MMAs that read a stage have completed
  __shared__ uint64_t all_done;           // after a wait that gave up: all MMAs have
  __shared__ uint64_t spare;              // takes the report that withhold keeps from `done`
  __shared__ uint32_t tmem_at;
  __shared__ int given_up;
  const uint32_t ring = (ptx::smem_u32(wide_sm) + 1023u) & ~1023u;  // swizzled tiles start at multiples of 1024
  const uint32_t p_hi = ring + kWideStages * STAGE, p_lo = p_hi + KBLK * kWideTile;
  auto at_smem = [&](uint32_t a) { return reinterpret_cast<float*>(wide_sm + (a - ptx::smem_u32(wide_sm))); };
  float* undo = at_smem(p_lo + KBLK * kWideTile);  // [TM] fp16: what takes a row's power of two back
  const uint32_t rank = cluster_rank();
  const int rest0 = rest ? min(max(__ldg(offsets + n), 0), T_) : T_;
  const Tile tile = find_tile(blockIdx.x / cluster, TM, offsets, n, T_, perm, nullptr);
  if (tile.rows == 0) {  // all blocks of the cluster alike
    if (rest && threadIdx.x < kAdThreads) copy_rest(y, ldy, out, ldo, N, rest0, T_, perm);
    return;
  }
  const float sc = __ldg(scale + tile.adapter);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const bool drains = warp < kAdWarps;
  const int m = warp & 3, half = (warp >> 2) & 1;  // a warp reads 16 tokens' lanes of tensor memory, half of the columns
  const int k0 = rank * kslice, k1 = min(K, k0 + kslice), n0 = rank * nslice, n1 = min(N, n0 + nslice);
  auto token = [&](int row) {
    const int t = row < tile.rows ? __ldg(perm + tile.row0 + row) : -1;
    return (unsigned)t < (unsigned)T_ ? t : -1;
  };
  const int chunk = tid & 7, row8 = (tid >> 3) & 31;  // what the thread copies: 16-byte chunk of rows row8, row8 + 32
  const int src[2] = {token(row8), token(row8 + 32)};
  const int tok[2] = {token(16 * m + g), token(16 * m + 8 + g)};
  // the same number of k stages in every block (zeros behind K), so that their shares of P lie alike
  const int down = (kslice + 63) / 64, up = n1 > n0 ? (n1 - n0 + 63) / 64 : 0;
  auto swizzled = [](int row, int c) { return (uint32_t)(row * 128 + ((c ^ (row & 7)) << 4)); };
  auto stage_at = [&](int st) { return ring + (uint32_t)(st % kWideStages) * STAGE; };
  // Stages are issued in order: what a thread copies next is kept in pointers that advance.
  // Of x, A and y it copies one chunk of rows row8 + 32 i, 32 rows being 4096 bytes of a tile.
  const uint32_t at_row = swizzled(row8, chunk);
  int k_next = k0 + chunk * 8, n_next = n0 + chunk * 8;
  const T* x_next[2] = {x + (int64_t)max(src[0], 0) * ldx + k_next, x + (int64_t)max(src[1], 0) * ldx + k_next};
  const T* y_next[2] = {y + (int64_t)max(src[0], 0) * ldy + n_next, y + (int64_t)max(src[1], 0) * ldy + n_next};
  const T* a_next = A + ((int64_t)tile.adapter * r + row8) * K + k_next;
  const int64_t a_rows = (int64_t)32 * K;
  // of B chunk b_chunk of outputs b_out + b_step i, which lie in permuted rows
  constexpr int b_step = kAdThreads / NR;
  const int b_chunk = tid % NR, b_out = (tid % kAdThreads) / NR;
  int b_left = n1 - n0 - b_out;
  const T* b_next = B + ((int64_t)tile.adapter * N + n0 + b_out) * r + b_chunk * 8;
  uint32_t at_b[NR / 4];
#pragma unroll
  for (int j = 0; j < NR / 4; ++j) {
    const int o = b_out + b_step * j;
    at_b[j] = kWideTile + (b_chunk >> 3) * kWideTile +
              swizzled((o & 32) + ((o >> 1) & 3) * 8 + ((o >> 3) & 3) * 2 + (o & 1), b_chunk & 7);
  }
  auto issue = [&](int st) {
    const uint32_t base = stage_at(st);
    if (st < down) {
      const bool in = k_next < k1;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        copy16(base + at_row + 4096 * h, x_next[h], in && src[h] >= 0);
        x_next[h] += 64;
      }
#pragma unroll
      for (int j = 0; j < NR / 4; ++j)
        copy16(base + kWideTile + at_row + 4096 * j, a_next + a_rows * j, in && row8 + 32 * j < r);
      a_next += 64;
      k_next += 64;
    } else if (st < down + up) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        copy16(base + at_row + 4096 * h, y_next[h], n_next < n1 && src[h] >= 0);
        y_next[h] += 64;
      }
#pragma unroll
      for (int j = 0; j < NR / 4; ++j)
        copy16(base + at_b[j], b_next + (int64_t)b_step * j * r, b_step * j < b_left && b_chunk * 8 < r);
      b_next += (int64_t)64 * r;
      b_left -= 64;
      n_next += 64;
    }
    copy_commit();
  };
  auto wait_done = [&](int st) {  // of the stage's MMAs; bounded
    if (!ptx::mbar_wait(&done[st % kWideStages], (st / kWideStages) & 1, &given_up, wait)) given_up = 1;
  };
  if (drains) {
#pragma unroll
    for (int st = 0; st < kWideAhead; ++st) issue(st);
  } else {
    ptx::tmem_alloc(&tmem_at, kWideTmem);
    ptx::tmem_relinquish();  // at once: the SM's other block waits for the permit
    if (lane == 0) {
      for (int i = 0; i < kWideStages; ++i) ptx::mbar_init(&done[i], 1);
      ptx::mbar_init(&all_done, 1);
      ptx::mbar_init(&spare, 1);
      ptx::fence_mbar_init();
      given_up = 0;
    }
  }
  if (rest && drains) copy_rest(y, ldy, out, ldo, N, rest0, T_, perm);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_at, my_lanes = (uint32_t)(m * 32) << 16;
  for (int st = 0; st < down; ++st) {
    copy_wait<kWideAhead - 1>();
    ptx::fence_proxy_async_smem();
    __syncthreads();
    if (drains) {
      if (st > 1) wait_done(st - 2);
      issue(st + kWideAhead);
    } else {
      const uint64_t xd = ptx::sw128_desc(stage_at(st)), ad = ptx::sw128_desc(stage_at(st) + kWideTile);
#pragma unroll
      for (int k = 0; k < 4; ++k)  // 16 values, 32 bytes, at a time
        ptx::mma_f16_ss_warp(tmem, xd + 2 * k, ad + 2 * k, wide_idesc<T>(RP), st || k ? 1u : 0u);
      ptx::mma_commit_warp(withhold && st == 0 ? &spare : &done[st % kWideStages]);
    }
  }
  // This block's share of P lies behind the ring's last filled stage: there, unless it is too
  // small for it, nothing is copied before the cluster has met again.
  float* mine = at_smem(NR <= 8 ? stage_at(down + kWideStages - 1) : p_lo + KBLK * kWideTile + TM * 4);  // [TM][RP]
  wait_done(down - 1);
  if (drains) {
    float acc[HALF][4];
    ptx::tc_fence_after();
    tmem_rows16<HALF>(tmem + my_lanes + half * (RP / 2), acc);
    ptx::tmem_ld_wait();
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < HALF; ++i)
        *reinterpret_cast<float2*>(mine + (16 * m + 8 * h + g) * RP + half * (RP / 2) + 8 * i + 2 * q) =
            make_float2(acc[i][2 * h], acc[i][2 * h + 1]);
  }
  cluster_arrive();
  cluster_wait();
  // P: the blocks' shares added in order, in 16-byte pieces, and split into hi and lo terms
  constexpr int PIECES = RP / 4;  // lanes of a row, a power of two up to 32
  if (drains)
#pragma unroll 2
    for (int c = tid; c < TM * PIECES; c += kAdThreads) {
      const int row = c / PIECES, piece = c % PIECES;
      float4 s = make_float4(0, 0, 0, 0);
      if (piece * 4 < r && row < tile.rows) {  // the rank is a multiple of 8
        float4 v[kAdMaxCluster];
#pragma unroll
        for (int k = 0; k < kAdMaxCluster; ++k)
          if (k < cluster) v[k] = load_remote4(mine + c * 4, k);
#pragma unroll
        for (int k = 0; k < kAdMaxCluster; ++k)
          if (k < cluster) s.x += v[k].x, s.y += v[k].y, s.z += v[k].z, s.w += v[k].w;
        s.x *= sc, s.y *= sc, s.z *= sc, s.w *= sc;
      }
      if constexpr (is_f16<T>) {  // the row's lanes agree on its power of two
        uint32_t big = max(max(__float_as_uint(s.x) & 0x7FFFFFFFu, __float_as_uint(s.y) & 0x7FFFFFFFu),
                           max(__float_as_uint(s.z) & 0x7FFFFFFFu, __float_as_uint(s.w) & 0x7FFFFFFFu));
#pragma unroll
        for (int o = PIECES / 2; o > 0; o >>= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
        const RowScale by = row_scale(big);
        s.x *= by.down, s.y *= by.down, s.z *= by.down, s.w *= by.down;
        if (piece == 0) undo[row] = by.back;
      }
      uint32_t hi[2], lo[2];
      split2<T>(s.x, s.y, hi[0], lo[0]);
      split2<T>(s.z, s.w, hi[1], lo[1]);
      const uint32_t at = (piece >> 4) * kWideTile + swizzled(row, (piece & 15) >> 1) + (piece & 1) * 8;
      asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(p_hi + at), "r"(hi[0]), "r"(hi[1]) : "memory");
      asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(p_lo + at), "r"(lo[0]), "r"(lo[1]) : "memory");
    }
  cluster_arrive();  // this warp has read; no block may overwrite its share or leave before all have
  // the lane's outputs of a stage: eight in a row of two tokens
  const uint32_t at_y = swizzled(16 * m + g, 4 * half + q);  // eight rows further: 1024 bytes
  int col = n0 + 32 * half + 8 * q;
  T* o_next[2] = {out + (int64_t)max(tok[0], 0) * ldo + col, out + (int64_t)max(tok[1], 0) * ldo + col};
  float back[2] = {1.0f, 1.0f};
  for (int st = down; st < down + up + 1; ++st) {
    if (st == down + 1) cluster_wait();
    if (st < down + up) {
      copy_wait<kWideAhead - 1>();
      ptx::fence_proxy_async_smem();  // the first time of P's terms too
      ptx::tc_fence_before();
      __syncthreads();
      if (drains) {
        issue(st + kWideAhead);
      } else {
        ptx::tc_fence_after();
        const uint32_t d2 = tmem + 128 + (st & 1) * 64;
        const uint64_t bd = ptx::sw128_desc(stage_at(st) + kWideTile);
#pragma unroll
        for (int term = 0; term < 2; ++term) {  // small terms first
          const uint64_t pd = ptx::sw128_desc(term == 0 ? p_lo : p_hi);
#pragma unroll
          for (int k = 0; k < RP / 16; ++k) {
            const uint64_t at = (uint64_t)((k >> 2) * (kWideTile >> 4) + (k & 3) * 2);
            ptx::mma_f16_ss_warp(d2, pd + at, bd + at, wide_idesc<T>(64), term || k ? 1u : 0u);
          }
        }
        ptx::mma_commit_warp(&done[st % kWideStages]);
      }
    }
    if (st > down && drains) {  // y + what the stage before came to
      const int was = st - 1;
      wait_done(was);
      ptx::tc_fence_after();
      float acc[4][4];
      tmem_rows16<4>(tmem + my_lanes + 128 + (was & 1) * 64 + 32 * half, acc);
      const uint32_t ys = stage_at(was) + at_y;
      const uint4 yv[2] = {ptx::lds_v4(ys), ptx::lds_v4(ys + 1024)};
      if (is_f16<T> && was == down) back[0] = undo[16 * m + g], back[1] = undo[16 * m + 8 + g];
      ptx::tmem_ld_wait();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (tok[h] >= 0 && col < n1) store_sum<T>(o_next[h], yv[h], acc, h, back[h]);
        o_next[h] += 64;
      }
      col += 64;
    }
  }
  if (up == 0) cluster_wait();
  copy_wait<0>();
  ptx::tc_fence_before();
  __syncthreads();  // all waits are over: given_up stands
  if (given_up && tid == 0 && status) *status = MOE_ERR_TIMEOUT;
  if (!drains) {
    ptx::tc_fence_after();
    if (given_up) {  // MMAs may be in flight still, whatever the stages' barriers say: they must not outlive their memory
      ptx::mma_commit_warp(&all_done);
      ptx::mbar_drain(&all_done, 0, kWideWait);
    }
    ptx::tmem_dealloc(tmem, kWideTmem);
  }
}

// ---------------------------------------------------------------- host
namespace {

struct Shares {
  int tiles, cluster, kslice, nslice;
};
// tiles: an upper bound on the tiles of TM rows; half of the last tiles of the adapters are
// expected.  A tile gets blocks, each with at least a step of k or of outputs, while the
// kernel's rule has room for all of them.
template <typename Fits>
Shares shares_of(const AdapterArgs& a, int TM, int kstep, Fits fits) {
  const int most = a.T < a.n ? a.T : a.n, full = a.T / TM, likely = full + (most + 1) / 2;
  Shares s{most + full, 1, 0, 0};
  while (s.cluster < kAdMaxCluster && std::max(a.K, a.N) > s.cluster * kstep && fits(2 * likely * s.cluster, s.cluster))
    s.cluster *= 2;
  s.kslice = ((a.K + s.cluster - 1) / s.cluster + 31) / 32 * 32;
  s.nslice = ((a.N + s.cluster - 1) / s.cluster + 31) / 32 * 32;
  return s;
}

template <typename Kern>
cudaError_t allow_smem(Kern kern, int smem) {
  return smem > 48 * 1024 ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) : cudaSuccess;
}

// 16-token tiles: a block an SM, since two share the path from L2 that the adapters take (300
// tokens of 2 adapters, K = N = 2048, r 128, 4 blocks a tile 11.7 us, 8 14.2; 600 of 8, 4096 ->
// 1000, r 64, 2 blocks 11.3, 8 15.9; 100 of 60, 2048, r 32, 4 blocks 7.2, 8 8.4).  Two an SM, and a
// tenth more since some tokens have no adapter, at ranks up to 16, where latency counts for more
// (K = N = 4096, r 16: 1024 tokens of 32 adapters 17.8 us with 2 blocks a tile, 12.0 with 4; 64 of 48
// 7.8 with 4, 6.3 with 8), and where each tile brings much of an adapter of its own from memory
// (64 of 48, r 64: 14.9 with 4, 10.9 with 8).
template <typename T, int NR>
cudaError_t adapters_short(const AdapterArgs& a, cudaStream_t s) {
  constexpr int KB = (NR + 3) / 4, smem = ((kAdWarps + 1) * 16 * NR * 8 + 16 * (KB * 32 + 4)) * (int)sizeof(float);
  const bool own = a.T <= 16 * a.n;
  const Shares p = shares_of(a, 16, kAdWarps * 32, [&](int blocks, int cluster) {
    if (blocks <= 148) return true;
    const bool much = own && (int64_t)a.r * (a.K + a.N) * 2 / cluster > 96 * 1024;
    return NR <= 8 && (NR <= 2 || much) && blocks <= 2 * 148 * 11 / 10;
  });
  const cudaError_t e = allow_smem(adapter_kernel<T, NR>, smem);
  if (e != cudaSuccess) return e;
  return launch_cluster(adapter_kernel<T, NR>, dim3((unsigned)p.tiles * p.cluster), dim3(kAdThreads), p.cluster, smem, s,
                        (const T*)a.x.p, a.x.ld, (const T*)a.y.p, a.y.ld, a.T, a.K, a.N, a.r, a.n, (const T*)a.A,
                        (const T*)a.B, a.scale, a.perm, a.offsets, a.out.p != a.y.p, p.cluster, p.kslice, p.nslice,
                        (T*)a.out.p, a.out.ld);
}
// 64-token tiles: as many as an SM holds.  8192 tokens of 24 adapters, r 64, take 31.2 us with 2
// blocks a tile and 37.6 with 1; of 32 adapters, r 128, one block an SM, 42.8 with 1 and 49.7 with 2;
// 2048 tokens of 16, K = N = 4096, r 64, each token with one of them, 29.3 with 4 and 33.6 with 8, more
// than fit.
template <typename T, int NR>
cudaError_t adapters_wide(const AdapterArgs& a, cudaStream_t s) {
  const Shares p = shares_of(a, kWideTokens, 64, [](int blocks, int) { return blocks <= 148 * (NR <= 8 ? 2 : 1); });
  const cudaError_t e = allow_smem(adapter_wide_kernel<T, NR>, wide_smem_bytes<NR>());
  if (e != cudaSuccess) return e;
  return launch_cluster(adapter_wide_kernel<T, NR>, dim3((unsigned)p.tiles * p.cluster), dim3(kWideThreads), p.cluster,
                        (size_t)wide_smem_bytes<NR>(), s, (const T*)a.x.p, a.x.ld, (const T*)a.y.p, a.y.ld, a.T, a.K, a.N,
                        a.r, a.n, (const T*)a.A, (const T*)a.B, a.scale, a.perm, a.offsets, a.out.p != a.y.p, p.cluster,
                        p.kslice, p.nslice, (T*)a.out.p, a.out.ld, a.status,
                        a.wait_cycles ? (long long)a.wait_cycles : kWideWait, a.withhold != 0);
}

// Tiles of 16 tokens where every row may be a request of its own (decode batches, banks of
// many adapters) and where there is little to multiply; tiles of 64 where adapters have rows
// enough to fill them.  16- against 64-token tiles (T, K, N, r, adapters; a few requests more than
// adapters, of which an eighth has none):
//   350, 2896, 2896, 96, 1    13.8 / 16.9 us       2048, 1024, 1024, 64, 16   11.8 / 10.8
//   512, 2048, 2048, 128, 4   11.8 / 16.4          2048, 2048, 2048, 32, 16   17.3 / 13.3
//   1024, 2048, 2048, 64, 8   11.8 / 14.5          1000, 4096, 4096, 32, 8    16.7 / 15.6 (*)
//   1024, 4096, 4096, 16, 32  12.0 / 16.3          8192, 256, 256, 64, 24     15.7 / 10.7
//   2048, 1024, 1024, 32, 16   8.6 /  9.5          2048, 4096, 4096, 64, 16   42.9 / 24.3
//   512, 4096, 4096, 16, 64   10.4 / 22.2          8192, 128, 128, 8, 24       9.8 / 8.2
// The rule is two cuts through these points, and time moves in waves of blocks.  It takes the slower side at
// (*), and where every token has an adapter at 512, 2048, 2048, 128, 4 (20.8 / 17.3, the 16-token tiles
// just beyond one wave) and 640 or 800, 4096, 4096, 32, 4 to 8 (18.2 / 15): up to a fifth more.
template <typename T>
cudaError_t adapters_of(const AdapterArgs& a, cudaStream_t s) {
  const int64_t products = (int64_t)a.T * a.r * (a.K + a.N);
  if (a.T <= 128 || a.T < 16 * a.n || (a.T <= 1024 && products <= 275000000) ||
      (a.T <= 2048 && products <= 150000000)) {
    if (a.r <= 16) return adapters_short<T, 2>(a, s);
    if (a.r <= 32) return adapters_short<T, 4>(a, s);
    return a.r <= 64 ? adapters_short<T, 8>(a, s) : adapters_short<T, 16>(a, s);
  }
  if (a.r <= 32) return adapters_wide<T, 4>(a, s);
  return a.r <= 64 ? adapters_wide<T, 8>(a, s) : adapters_wide<T, 16>(a, s);
}

}  // namespace

cudaError_t launch_adapters(const AdapterArgs& a, int dtype, cudaStream_t stream) {
  return dtype == MOE_F16 ? adapters_of<__half>(a, stream) : adapters_of<__nv_bfloat16>(a, stream);
}

}  // namespace moe

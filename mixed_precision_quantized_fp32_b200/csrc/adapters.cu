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
// One launch, no workspace, nothing added in global memory.
//
// Arithmetic per byte is about the rank, far below what the tensor cores need to be the
// bound, so operands go from memory straight to mma.sync fragments: the contraction
// index may be permuted if both operands are permuted alike, and with a lane taking
// eight consecutive values (16 bytes) of its row as its share of 32, every load is a
// full 16 bytes and nothing is staged in shared memory.  The up product's fp32 operand P
// goes in as two terms of the value type (P = hi + lo, 16 or more bits), so its rounding
// stays far below that of the stored result; in fp16 a row is first brought to at most
// 2^14 by a power of two, since P may pass fp16's range.
#include "ops_common.cuh"

namespace moe {

constexpr int kAdWarps = 8;
constexpr int kAdThreads = 32 * kAdWarps;
constexpr int kAdMaxCluster = 8;
#ifndef XSHORT
#define XSHORT 128
#define XPER 16
#endif

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
  if (lane == 31) wsum[warp] = s;
  if (first) first[tid] = mine_of_perm;
  __syncthreads();
  int before = s - mine;
  for (int w = 0; w < warp; ++w) before += wsum[w];
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

// Two values as hi and lo terms of T; an infinity stays one (inf - inf would be NaN).
template <typename T>
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack2<T>(a, b);
  const float2 f = unpack2<T>(hi);
  lo = pack2<T>(isinf(f.x) ? 0.0f : a - f.x, isinf(f.y) ? 0.0f : b - f.y);
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
      const int e = (int)(big >> 23) - 127 - 13;  // 2^e: the row's largest is in [2^13, 2^14) after
      if (big < 0x7F800000u && e > 0) {
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        back[h] = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
          for (int i = 0; i < 8; ++i) p[b][i] *= down;
      }
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
                 ? __ldg(reinterpret_cast<const uint4*>(y + (int64_t)tok[h] * ldy + nn + 8 * q))
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
__device__ __forceinline__ void copy16(void* dst, const void* src, bool in) {  // zeros where `in` is false
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
               "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Tiles of 64 tokens of one adapter.  The same two products and the same split over a
// cluster, but operands come through a ring of 64-wide stages in shared memory (x and A,
// then y and B, one ring over both products), since a tile's loads no longer fit in
// registers ahead of their use.  Warps: 4 token tiles times 2 halves of a stage.
// Rows of a stage are 128 bytes (B's: the rank); a lane reads the 16 bytes at chunk q of
// its half in row g, and odd rows have their halves swapped, so the eight lanes of a
// phase hit eight different 16-byte columns.
constexpr int kWideStages = 4;
constexpr int kWideTokens = 64;

template <int NR> constexpr int wide_stage_bytes() { return kWideTokens * 128 + NR * 8 * 128; }
template <int NR> constexpr int wide_smem_bytes() {
  return kWideStages * wide_stage_bytes<NR>() + kWideTokens * (2 * NR * 8 + 4) * 4;
}

template <typename T, int NR>
__global__ void __launch_bounds__(kAdThreads, NR <= 8 ? 2 : 1)
    adapter_wide_kernel(const T* __restrict__ x, int64_t ldx, const T* y, int64_t ldy, int T_, int K, int N, int r,
                        int n, const T* __restrict__ A, const T* __restrict__ B, const float* __restrict__ scale,
                        const int32_t* __restrict__ perm, const int32_t* __restrict__ offsets, bool rest, int cluster,
                        int kslice, int nslice, T* out, int64_t ldo) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  constexpr int TM = kWideTokens, KB = NR / 4, RP = NR * 8, BROW = RP * 2;  // B's row in bytes
  constexpr int STAGE = wide_stage_bytes<NR>();
  extern __shared__ __align__(128) uint8_t wide_sm[];
  uint8_t* ring = wide_sm;
  float* mine = reinterpret_cast<float*>(ring + kWideStages * STAGE);  // [TM][RP] this block's share of P
  float* P = mine + TM * RP;                                          // [TM][KB*32 + 4]
  const uint32_t rank = cluster_rank();
  const int rest0 = rest ? min(max(__ldg(offsets + n), 0), T_) : T_;
  const Tile tile = find_tile(blockIdx.x / cluster, TM, offsets, n, T_, perm, nullptr);
  if (tile.rows == 0) {  // all blocks of the cluster alike
    if (rest) copy_rest(y, ldy, out, ldo, N, rest0, T_, perm);
    return;
  }
  const float sc = __ldg(scale + tile.adapter);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const int m = warp & 3, half = warp >> 2;
  const int k0 = rank * kslice, k1 = min(K, k0 + kslice), n0 = rank * nslice, n1 = min(N, n0 + nslice);
  auto token = [&](int row) {
    const int t = row < tile.rows ? __ldg(perm + tile.row0 + row) : -1;
    return (unsigned)t < (unsigned)T_ ? t : -1;
  };
  const int chunk = tid & 7, row8 = tid >> 3;  // what the thread copies: 16-byte chunk of rows row8, row8 + 32
  const int src[2] = {token(row8), token(row8 + 32)};
  const int tok[2] = {token(16 * m + g), token(16 * m + 8 + g)};
  const T* Aa = A + (int64_t)tile.adapter * r * K;
  const T* Ba = B + (int64_t)tile.adapter * N * r;
  const int down = k1 > k0 ? (k1 - k0 + 63) / 64 : 0, up = n1 > n0 ? (n1 - n0 + 63) / 64 : 0;
  auto issue = [&](int st) {
    uint8_t* base = ring + (st & (kWideStages - 1)) * STAGE;
    if (st < down) {
      const int k = k0 + st * 64 + chunk * 8;
      const bool in = k < k1;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = row8 + 32 * h;
        copy16(base + row * 128 + ((chunk ^ ((row & 1) * 4)) * 16), src[h] >= 0 ? x + (int64_t)src[h] * ldx + (in ? k : 0) : x,
               in && src[h] >= 0);
      }
#pragma unroll
      for (int j = 0; j < NR / 4; ++j) {
        const int row = row8 + 32 * j;
        const bool real = in && row < r;
        copy16(base + TM * 128 + row * 128 + ((chunk ^ ((row & 1) * 4)) * 16), real ? Aa + (int64_t)row * K + k : Aa, real);
      }
    } else if (st < down + up) {
      const int c0 = n0 + (st - down) * 64, c = c0 + chunk * 8;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = row8 + 32 * h;
        const bool in = c < n1 && src[h] >= 0;
        copy16(base + row * 128 + ((chunk ^ ((row & 1) * 4)) * 16), in ? y + (int64_t)src[h] * ldy + c : y, in);
      }
      // NR chunks a row: NR/4 a thread
#pragma unroll
      for (int j = 0; j < NR / 4; ++j) {
        const int i = tid + kAdThreads * j, row = i / NR, b = i % NR;
        const bool in = c0 + row < n1 && b * 8 < r;
        copy16(base + TM * 128 + row * BROW + ((NR >= 8 ? b ^ ((row & 1) * 4) : b) * 16),
               in ? Ba + (int64_t)(c0 + row) * r + b * 8 : Ba, in);
      }
    }
    copy_commit();
  };
  // 16 bytes at chunk c of row `row` of a tile with `pitch` bytes a row
  auto piece = [](const uint8_t* base, int row, int c, int pitch) {
    return *reinterpret_cast<const uint4*>(base + row * pitch + ((pitch >= 128 ? c ^ ((row & 1) * 4) : c) * 16));
  };
#pragma unroll
  for (int st = 0; st < kWideStages - 1; ++st) issue(st);
  if (rest) copy_rest(y, ldy, out, ldo, N, rest0, T_, perm);
  uint32_t hi[KB][2][4], lo[KB][2][4];
  {
    float acc[NR][4];
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[i][c] = 0.0f;
    for (int st = 0; st < down; ++st) {
      copy_wait<kWideStages - 2>();
      __syncthreads();
      issue(st + kWideStages - 1);
      const uint8_t* xs = ring + (st & (kWideStages - 1)) * STAGE;
      const uint8_t* as = xs + TM * 128;
      const uint4 a = piece(xs, 16 * m + g, 4 * half + q, 128), b = piece(xs, 16 * m + 8 + g, 4 * half + q, 128);
      const uint32_t a0[4] = {a.x, b.x, a.y, b.y}, a1[4] = {a.z, b.z, a.w, b.w};
      constexpr int PART = NR < 8 ? NR : 8;  // independent sums between two that depend on one another
#pragma unroll
      for (int i0 = 0; i0 < NR; i0 += PART) {
        uint4 w[PART];
#pragma unroll
        for (int i = 0; i < PART; ++i) w[i] = piece(as, 8 * (i0 + i) + g, 4 * half + q, 128);
#pragma unroll
        for (int i = 0; i < PART; ++i) mma16816<T>(acc[i0 + i], a0, w[i].x, w[i].y);
#pragma unroll
        for (int i = 0; i < PART; ++i) mma16816<T>(acc[i0 + i], a1, w[i].z, w[i].w);
      }
    }
    // the two halves, then the blocks, each added in order
    auto share = [&](int h, int i) {
      return reinterpret_cast<float2*>(mine + (16 * m + 8 * h + g) * RP + 8 * i + 2 * q);
    };
    if (half == 1)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < NR; ++i) *share(h, i) = make_float2(acc[i][2 * h], acc[i][2 * h + 1]);
    __syncthreads();
    if (half == 0)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const float2 o = *share(h, i);
          *share(h, i) = make_float2(acc[i][2 * h] + o.x, acc[i][2 * h + 1] + o.y);
        }
  }
  cluster_arrive();
  cluster_wait();
  float back[2];
  gather_p<TM, KB, RP>(mine, cluster, sc, r, tile.rows, P);
  cluster_arrive();  // this warp has read; no block may leave before all have
  __syncthreads();
  operand_p<T, KB>(P + 16 * m * (KB * 32 + 4), hi, lo, back);
  for (int st = down; st < down + up; ++st) {
    copy_wait<kWideStages - 2>();
    __syncthreads();
    issue(st + kWideStages - 1);
    const uint8_t* ys = ring + (st & (kWideStages - 1)) * STAGE;
    const uint8_t* bs = ys + TM * 128;
    float acc[4][4] = {};
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      uint4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = piece(bs, 32 * half + 8 * (g >> 1) + 2 * i + (g & 1), 4 * b + q, BROW);
      mma_hi_lo<T>(acc, hi[b], lo[b], w);
    }
    const int col = n0 + (st - down) * 64 + 32 * half + 8 * q;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (tok[h] < 0 || col >= n1) continue;
      store_sum<T>(out + (int64_t)tok[h] * ldo + col, piece(ys, 16 * m + 8 * h + g, 4 * half + q, 128), acc, h, back[h]);
    }
  }
  copy_wait<0>();
  cluster_wait();
}

// ---------------------------------------------------------------- host
namespace {

template <typename T, typename Kern>
cudaError_t adapters_with(Kern kern, int TM, int kstep, int smem, const AdapterArgs& a, cudaStream_t stream) {
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  const bool rest = a.out.p != a.y.p;  // rows without an adapter still have to be copied
  const int tiles = (a.T < a.n ? a.T : a.n) + a.T / TM;  // at most this many
  // as many blocks a tile as the machine holds at once and still have a step of k each
  int cluster = 1;
  while (cluster < kAdMaxCluster && 2 * tiles * cluster <= 3 * 148 && a.K > cluster * kstep) cluster *= 2;
  const int kslice = ((a.K + cluster - 1) / cluster + 31) / 32 * 32;
  const int nslice = ((a.N + cluster - 1) / cluster + 31) / 32 * 32;
  return launch_cluster(kern, dim3((unsigned)tiles * cluster), dim3(kAdThreads), cluster, smem, stream,
                        (const T*)a.x.p, a.x.ld, (const T*)a.y.p, a.y.ld, a.T, a.K, a.N, a.r, a.n, (const T*)a.A,
                        (const T*)a.B, a.scale, a.perm, a.offsets, rest, cluster, kslice, nslice, (T*)a.out.p,
                        a.out.ld);
}

template <typename T, int NR>
cudaError_t adapters_short(const AdapterArgs& a, cudaStream_t s) {
  constexpr int KB = (NR + 3) / 4, smem = ((kAdWarps + 1) * 16 * NR * 8 + 16 * (KB * 32 + 4)) * (int)sizeof(float);
  return adapters_with<T>(adapter_kernel<T, NR>, 16, kAdWarps * 32, smem, a, s);
}
template <typename T, int NR>
cudaError_t adapters_wide(const AdapterArgs& a, cudaStream_t s) {
  return adapters_with<T>(adapter_wide_kernel<T, NR>, kWideTokens, 64, wide_smem_bytes<NR>(), a, s);
}

// Tiles of 16 tokens where every row may be a request of its own (decode batches, banks of
// many adapters); tiles of 64 where adapters have rows enough to fill them.
template <typename T>
cudaError_t adapters_of(const AdapterArgs& a, cudaStream_t s) {
  if (a.T <= XSHORT || a.T < XPER * a.n) {
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

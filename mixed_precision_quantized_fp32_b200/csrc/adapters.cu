// Low-rank adapters of many requests at once beside a shared projection or the whole
// layer: out[t] = y[t] + scale[a] * B_a (A_a x[t]) for the adapter a of token t, and
// out[t] = y[t] for a token without one.
//
// Tokens come sorted by adapter (routes.cu), so a tile of rows shares its adapter and
// both products are matrix products of a tile of tokens with A_a and B_a:
//   adapter_down_kernel   P[row][r] = sum_k x[k] A_a[r][k], split over k where there are
//                         few tiles; each part is written in fp32 and nothing is added
//                         in memory
//   adapter_up_kernel     sums the parts in order, scales, multiplies by B_a and adds y
// Arithmetic per byte is about the rank, far below what the tensor cores need to be the
// bound, so the operands go from memory straight to mma.sync fragments: the contraction
// index may be permuted if both operands are permuted alike, and with a lane taking
// eight consecutive values (16 bytes) of its row as its share of 32, every load is a
// full 16 bytes and no shared memory is staged.  The up product's fp32 operand P goes
// in as two terms of the value type (P = hi + lo, 16 or more bits), so its rounding
// stays far below that of the stored result; in fp16 a row is first brought to at most
// 2^14 by a power of two, since P may pass fp16's range.
#include "ops_common.cuh"

namespace moe {

constexpr int kAdWarps = 8;
constexpr int kAdThreads = 32 * kAdWarps;
constexpr int kAdStep = 32 * kAdWarps;  // k values a block takes at once

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <typename T> constexpr bool is_f16 = false;
template <> constexpr bool is_f16<__half> = true;

struct Tile {
  int adapter, row0, rows;  // rows 0: none
};

// Tile `want` of the sorted rows: each adapter's rows in tiles of TM, adapters in order;
// with `rest`, the rows behind the last adapter's follow as adapter n.  Every thread
// takes a run of adapters and the block scans their tile counts.
__device__ Tile find_tile(int want, int TM, const int32_t* __restrict__ offsets, int n, int T, bool rest) {
  __shared__ int wsum[kAdWarps];
  __shared__ Tile found;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int segs = n + (rest ? 1 : 0), per = (segs + kAdThreads - 1) / kAdThreads;
  if (tid == 0) found = {0, 0, 0};
  auto lo_of = [&](int a) { return min(max(__ldg(offsets + a), 0), T); };
  auto hi_of = [&](int a, int lo) { return a < n ? min(max(__ldg(offsets + a + 1), lo), T) : T; };
  int mine = 0;
  for (int i = 0; i < per; ++i) {
    const int a = tid * per + i;
    if (a >= segs) break;
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
  __syncthreads();
  int before = s - mine;
  for (int w = 0; w < warp; ++w) before += wsum[w];
  if (want >= before && want < before + mine) {
    for (int i = 0; i < per; ++i) {
      const int a = tid * per + i;
      if (a >= segs) break;
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

// NR: n8 tiles of the rank (r <= 8*NR), MT: m16 tiles of tokens.
template <typename T, int NR, int MT>
__global__ void __launch_bounds__(kAdThreads) adapter_down_kernel(const T* __restrict__ x, int64_t ldx, int T_, int K,
                                                                  int r, int n, const T* __restrict__ A,
                                                                  const int32_t* __restrict__ perm,
                                                                  const int32_t* __restrict__ offsets, int kslice,
                                                                  float* __restrict__ part) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  constexpr int TM = 16 * MT;
  __shared__ float red[kAdWarps / 2][TM * NR * 8];
  const Tile tile = find_tile(blockIdx.x, TM, offsets, n, T_, false);
  if (tile.rows == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const T* xr[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = 16 * m + 8 * h + g;
      const int t = i < tile.rows ? perm[tile.row0 + i] : -1;
      xr[m][h] = (unsigned)t < (unsigned)T_ ? x + (int64_t)t * ldx : nullptr;
    }
  const T* Ar = A + ((int64_t)tile.adapter * r + g) * K;
  float acc[MT][NR][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[m][i][c] = 0.0f;
  const int k0 = blockIdx.y * kslice, k1 = min(K, k0 + kslice);
#pragma unroll 2
  for (int kk = k0 + warp * 32 + q * 8; kk - q * 8 < k1; kk += kAdStep) {
    const bool in = kk < k1;  // K is a multiple of 8
    uint4 av[MT][2], bv[NR];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        av[m][h] = in && xr[m][h] ? __ldg(reinterpret_cast<const uint4*>(xr[m][h] + kk)) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < NR; ++i)
      bv[i] = in && 8 * i < r ? __ldg(reinterpret_cast<const uint4*>(Ar + (int64_t)8 * i * K + kk))
                              : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const uint32_t a0[4] = {av[m][0].x, av[m][1].x, av[m][0].y, av[m][1].y};
      const uint32_t a1[4] = {av[m][0].z, av[m][1].z, av[m][0].w, av[m][1].w};
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        mma16816<T>(acc[m][i], a0, bv[i].x, bv[i].y);
        mma16816<T>(acc[m][i], a1, bv[i].z, bv[i].w);
      }
    }
  }
  // sum over the warps: upper half to shared memory, lower half adds, three times
#pragma unroll
  for (int half = kAdWarps / 2; half > 0; half >>= 1) {
    if (warp >= half && warp < 2 * half) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) red[warp - half][((m * NR + i) * 4 + c) * 32 + lane] = acc[m][i][c];
    }
    __syncthreads();
    if (warp < half) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) acc[m][i][c] += red[warp][((m * NR + i) * 4 + c) * 32 + lane];
    }
    __syncthreads();
  }
  if (warp == 0) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 16 * m + 8 * h + g;
        if (row >= tile.rows) continue;
        float* out = part + ((int64_t)blockIdx.y * T_ + tile.row0 + row) * r + 2 * q;
#pragma unroll
        for (int i = 0; i < NR; ++i)
          if (8 * i < r) *reinterpret_cast<float2*>(out + 8 * i) = make_float2(acc[m][i][2 * h], acc[m][i][2 * h + 1]);
      }
  }
}

// Two values as hi and lo terms of T; an infinity stays one (inf - inf would be NaN).
template <typename T>
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack2<T>(a, b);
  const float2 f = unpack2<T>(hi);
  lo = pack2<T>(isinf(f.x) ? 0.0f : a - f.x, isinf(f.y) ? 0.0f : b - f.y);
}

template <typename T, int NR, int MT>
__global__ void __launch_bounds__(kAdThreads) adapter_up_kernel(const T* y, int64_t ldy, int T_, int N,
                                                                int r, int n, const T* __restrict__ B,
                                                                const float* __restrict__ scale,
                                                                const int32_t* __restrict__ perm,
                                                                const int32_t* __restrict__ offsets, bool rest,
                                                                int parts, const float* __restrict__ part,
                                                                int nslice, T* out, int64_t ldo) {
  pdl_enter();  // before any global memory access (see moe_common.cuh)
  constexpr int TM = 16 * MT, KB = (NR + 3) / 4, LD = KB * 32 + 4;
  __shared__ float P[TM][LD];
  __shared__ float undo[TM];
  const Tile tile = find_tile(blockIdx.x, TM, offsets, n, T_, rest);
  if (tile.rows == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const bool has = tile.adapter < n;
  const T* yr[MT][2];
  T* orow[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = 16 * m + 8 * h + g;
      const int t = i < tile.rows ? perm[tile.row0 + i] : -1;
      const bool ok = (unsigned)t < (unsigned)T_;
      yr[m][h] = ok ? y + (int64_t)t * ldy : nullptr;
      orow[m][h] = ok ? out + (int64_t)t * ldo : nullptr;
    }
  uint32_t hi[MT][KB][2][4], lo[MT][KB][2][4];
  if (has) {
    const float sc = __ldg(scale + tile.adapter);
    for (int c = threadIdx.x; c < TM * KB * 32; c += kAdThreads) {
      const int row = c / (KB * 32), i = c % (KB * 32);
      float s = 0.0f;
      if (row < tile.rows && i < r)
        for (int p = 0; p < parts; ++p) s += part[((int64_t)p * T_ + tile.row0 + row) * r + i];
      P[row][i] = row < tile.rows && i < r ? s * sc : 0.0f;
    }
    __syncthreads();
    if (is_f16<T>) {  // fp16: bring each row to at most 2^14
      for (int row = warp; row < TM; row += kAdWarps) {
        uint32_t m = 0;
        for (int i = lane; i < KB * 32; i += 32) m = max(m, __float_as_uint(P[row][i]) & 0x7FFFFFFFu);
        m = __reduce_max_sync(0xffffffffu, m);
        const int e = (int)(m >> 23) - 127 - 13;  // 2^e: the row's largest is in [2^13, 2^14) after
        const bool scaled = m > 0 && m < 0x7F800000u && e > 0;
        if (scaled)
          for (int i = lane; i < KB * 32; i += 32) P[row][i] *= __uint_as_float((uint32_t)(127 - e) << 23);
        if (lane == 0) undo[row] = scaled ? __uint_as_float((uint32_t)(127 + e) << 23) : 1.0f;
      }
      __syncthreads();
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int b = 0; b < KB; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float* p = &P[16 * m + 8 * h + g][32 * b + 8 * q];
          // lane's eight values: pairs 0, 1 to the first MMA, 2, 3 to the second (as B's)
          split2<T>(p[0], p[1], hi[m][b][0][h], lo[m][b][0][h]);
          split2<T>(p[2], p[3], hi[m][b][0][2 + h], lo[m][b][0][2 + h]);
          split2<T>(p[4], p[5], hi[m][b][1][h], lo[m][b][1][h]);
          split2<T>(p[6], p[7], hi[m][b][1][2 + h], lo[m][b][1][2 + h]);
        }
  }
  const T* Ba = B + (int64_t)(has ? tile.adapter : 0) * N * r;
  const int n0 = blockIdx.y * nslice, n1 = min(N, n0 + nslice);
  for (int nn = n0 + warp * 32; nn < n1; nn += kAdStep) {
    // column c of MMA tile i is output nn + 8*(c/2) + 2*i + c%2, so that a lane ends up
    // with outputs nn + 8q .. nn + 8q + 7 of its rows
    float acc[MT][4][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[m][i][c] = 0.0f;
    const int col = nn + 8 * q;
    uint4 yv[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        yv[m][h] = yr[m][h] && col < n1 ? __ldg(reinterpret_cast<const uint4*>(yr[m][h] + col)) : make_uint4(0, 0, 0, 0);
    if (has) {
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        uint4 bv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int o = nn + 8 * (g >> 1) + 2 * i + (g & 1), kk = 32 * b + 8 * q;
          bv[i] = o < n1 && kk < r ? __ldg(reinterpret_cast<const uint4*>(Ba + (int64_t)o * r + kk)) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mma16816<T>(acc[m][i], lo[m][b][0], bv[i].x, bv[i].y);
            mma16816<T>(acc[m][i], lo[m][b][1], bv[i].z, bv[i].w);
            mma16816<T>(acc[m][i], hi[m][b][0], bv[i].x, bv[i].y);
            mma16816<T>(acc[m][i], hi[m][b][1], bv[i].z, bv[i].w);
          }
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!orow[m][h] || col >= n1) continue;
        const float s = is_f16<T> && has ? undo[16 * m + 8 * h + g] : 1.0f;
        const uint32_t w[4] = {yv[m][h].x, yv[m][h].y, yv[m][h].z, yv[m][h].w};
        uint32_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = unpack2<T>(w[i]);
          v[i] = has ? pack2<T>(fmaf(s, acc[m][i][2 * h], f.x), fmaf(s, acc[m][i][2 * h + 1], f.y)) : w[i];
        }
        *reinterpret_cast<uint4*>(orow[m][h] + col) = make_uint4(v[0], v[1], v[2], v[3]);
      }
  }
}

// ---------------------------------------------------------------- host
namespace {

struct AdapterPlan {
  int nr, mt;      // kernel variant
  int tiles;       // upper bound on the tiles of adapters
  int parts, kslice;
};

// Tiles of 16 tokens for decode batches; for longer ones as many rows as 64 accumulators
// a lane allow, so that an adapter's matrices are read less often.  Parts of k fill the
// machine when there are few tiles.
AdapterPlan adapter_plan(int T, int K, int r, int n) {
  AdapterPlan p;
  p.nr = r <= 16 ? 2 : r <= 32 ? 4 : r <= 64 ? 8 : 16;
  p.mt = T <= 128 ? 1 : p.nr <= 4 ? 4 : 16 / p.nr;
  const int tm = 16 * p.mt;
  p.tiles = (T < n ? T : n) + T / tm;
  if (p.tiles < 1) p.tiles = 1;  // T = 0: sizes only
  const int steps = (K + kAdStep - 1) / kAdStep;
  int parts = (4 * 148 + p.tiles - 1) / p.tiles;
  if (parts > steps) parts = steps;
  p.kslice = (steps + parts - 1) / parts * kAdStep;
  p.parts = (K + p.kslice - 1) / p.kslice;
  return p;
}

template <typename T, int NR, int MT>
cudaError_t adapters_as(const AdapterPlan& p, const AdapterArgs& a, cudaStream_t stream) {
  cudaError_t e = launch_chained(adapter_down_kernel<T, NR, MT>, dim3(p.tiles, p.parts), dim3(kAdThreads), 0, stream,
                                 (const T*)a.x.p, a.x.ld, a.T, a.K, a.r, a.n, (const T*)a.A, a.perm, a.offsets,
                                 p.kslice, a.part);
  if (e != cudaSuccess) return e;
  const bool rest = a.out.p != a.y.p;  // rows without an adapter still have to be copied
  const int tiles = p.tiles + (rest ? 1 : 0);  // one more segment of the same T rows
  const int steps = (a.N + kAdStep - 1) / kAdStep;
  int slices = (4 * 148 + p.tiles - 1) / p.tiles;
  if (slices > steps) slices = steps;
  const int nslice = (steps + slices - 1) / slices * kAdStep;
  return launch_chained(adapter_up_kernel<T, NR, MT>, dim3(tiles, (a.N + nslice - 1) / nslice), dim3(kAdThreads), 0,
                        stream, (const T*)a.y.p, a.y.ld, a.T, a.N, a.r, a.n, (const T*)a.B, a.scale, a.perm, a.offsets,
                        rest, p.parts, (const float*)a.part, nslice, (T*)a.out.p, a.out.ld);
}

template <typename T>
cudaError_t adapters_of(const AdapterPlan& p, const AdapterArgs& a, cudaStream_t s) {
  switch (p.nr) {
    case 2: return p.mt == 1 ? adapters_as<T, 2, 1>(p, a, s) : adapters_as<T, 2, 4>(p, a, s);
    case 4: return p.mt == 1 ? adapters_as<T, 4, 1>(p, a, s) : adapters_as<T, 4, 4>(p, a, s);
    case 8: return p.mt == 1 ? adapters_as<T, 8, 1>(p, a, s) : adapters_as<T, 8, 2>(p, a, s);
    default: return adapters_as<T, 16, 1>(p, a, s);
  }
}

}  // namespace

uint64_t adapters_ws_bytes(int T, int K, int r, int n) {
  const AdapterPlan p = adapter_plan(T, K, r, n);
  return up256((uint64_t)p.parts * T * r * 4 + 4);
}

cudaError_t launch_adapters(const AdapterArgs& a, int dtype, cudaStream_t stream) {
  const AdapterPlan p = adapter_plan(a.T, a.K, a.r, a.n);
  return dtype == MOE_F16 ? adapters_of<__half>(p, a, stream) : adapters_of<__nv_bfloat16>(p, a, stream);
}

}  // namespace moe

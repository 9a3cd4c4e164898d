// Low-rank adapters of many requests beside a shared projection:
//   Y[m] = base[m] + s[a] (X[m] A[a]^T) B[a]^T,   a = adapter[m];  a = -1: Y[m] = base[m].
//
// Two kernels: the shrink V = s X A^T [M, r], and the expand Y = base + V B^T.  Both are bound by
// bytes (a decode batch by the adapters' A and B, a prefill batch by X, base and Y), so the
// contractions run on mma.sync m16n8k16 straight from global memory into registers: no operand is
// staged, every load is 16 bytes a lane.
//   Both operands are contiguous along the contracted index.  A lane holds 8 neighbouring values of
//   it (one load) and gives four to each of two products; which k a fragment slot stands for is
//   free as long as both operands agree.
//   Rows of different adapters share a 16-row block: for each adapter that occurs in it (the lowest
//   of its rows leads), the products run with the rows of all others set to zero, into the same
//   accumulators.
// The sum over K is split over warps and over the CTAs of a cluster; partial sums meet in shared
// memory and are added in a fixed order.  V is kept in the element type (rounded once, after the
// scale): it is an operand of the second product, which takes 16 bits.
#include <algorithm>

#include "elem16.cuh"
#include "internal.h"

namespace wq {

__device__ uint32_t g_lora_err;

uint32_t lora_read_and_clear_error() {
  uint32_t v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_lora_err, sizeof(v));
  cudaMemcpyToSymbol(g_lora_err, &z, sizeof(z));
  return v;
}

namespace {

template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 32 values of the contracted index: lane 4g + q holds values 8q .. 8q + 7 of rows g and g + 8 (x)
// and of column g (w).
template <bool F16>
__device__ __forceinline__ void mma_k32(float (&c)[4], const uint4& lo, const uint4& hi, const uint4& w) {
  mma16816<F16>(c, lo.x, hi.x, lo.y, hi.y, w.x, w.y);
  mma16816<F16>(c, lo.z, hi.z, lo.w, hi.w, w.z, w.w);
}

__device__ __forceinline__ uint4 ld_stream(const uint16_t* p) {     // read once: leave L1 to the shared operand
  uint4 v;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ld_shared_operand(const uint16_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }

// Adapter of row m: -1 for none (and for rows past M); out of range: reported, none.
__device__ __forceinline__ int row_adapter(const LoraArgs& p, int m) {
  if (m >= p.M) return -1;
  const int a = __ldg(p.adapter + m);
  if (a < -1 || a >= p.L) {
    atomicOr(&g_lora_err, kErrIndex);
    return -1;
  }
  return a;
}
// Its rank rounded up to 8.
__device__ __forceinline__ int adapter_rank(const LoraArgs& p, int a) {
  int rank = p.ranks ? __ldg(p.ranks + a) : p.r;
  if (rank < 0 || rank > p.r) {
    atomicOr(&g_lora_err, kErrIndex);
    rank = min(max(rank, 0), p.r);
  }
  return (rank + 7) & ~7;
}
// Lanes whose adapter occurs in the warp's rows for the first time (lanes with -1 never lead).
__device__ __forceinline__ uint32_t leaders(int a) {
  const uint32_t same = __match_any_sync(0xffffffffu, a);
  return __ballot_sync(0xffffffffu, a >= 0 && (same & ((1u << (threadIdx.x & 31)) - 1)) == 0);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// The float at shared address `addr` of CTA `rank` of the cluster.
__device__ __forceinline__ float ld_cluster(const float* p, uint32_t rank) {
  uint32_t a;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

// Steps of 32 of the contracted index that slice i of n takes.
__device__ __forceinline__ void slice(int steps, int i, int n, int& lo, int& hi) {
  lo = static_cast<int>(static_cast<int64_t>(steps) * i / n);
  hi = static_cast<int>(static_cast<int64_t>(steps) * (i + 1) / n);
}

// acc[b][t] += X rows (16 b + g, + 8) . A row (8 t + g) over steps [lo, hi) of 32, for the rows that
// `on` marks (bits 2b: row 16 b + g, 2b + 1: row 16 b + g + 8); NT tiles of 8 ranks, `tiles` live.
template <bool F16, int RB, int NT, int U>
__device__ __forceinline__ void shrink_loop(float (&acc)[RB][NT][4], const LoraArgs& p, const uint16_t* x, const uint16_t* a,
                                            uint32_t on, int tiles, int lo, int hi) {
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  for (int s = lo; s < hi; s += U) {
    uint4 xv[U][RB][2], av[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (s + u) * 32 + 8 * q;
      const bool in = s + u < hi && k < p.K;
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          xv[u][b][h] = make_uint4(0, 0, 0, 0);
          if (in && ((on >> (2 * b + h)) & 1u)) xv[u][b][h] = ld_stream(x + static_cast<int64_t>(16 * b + 8 * h + g) * p.K + k);
        }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        av[u][t] = make_uint4(0, 0, 0, 0);
        if (in && t < tiles) av[u][t] = ld_shared_operand(a + static_cast<int64_t>(8 * t + g) * p.K + k);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (t < tiles)
#pragma unroll
          for (int b = 0; b < RB; ++b) mma_k32<F16>(acc[b][t], xv[u][b][0], xv[u][b][1], av[u][t]);
  }
}

// Few rows: one cluster for each row that leads its adapter in its 16-row block; 8 warps a CTA, each
// a slice of K.
constexpr int kRowWarps = 8;
template <bool F16, int NT>
__global__ void __launch_bounds__(32 * kRowWarps) k_lora_shrink_rows(const LoraArgs p, uint16_t* V) {
  extern __shared__ float red[];              // [warp][16][8 NT], then the CTA's sum over [0]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
  pdl_wait();
  pdl_launch_dependents();                    // the expand may read all but V from here on
  const int m = blockIdx.y, m0 = m & ~15;
  const int mine = lane < 16 ? row_adapter(p, m0 + lane) : -1;
  const uint32_t lead = leaders(mine);
  if (!((lead >> (m & 15)) & 1u)) return;     // the same for all CTAs of the cluster
  const int a = __shfl_sync(0xffffffffu, mine, m & 15);
  const int rank = adapter_rank(p, a), tiles = rank / 8;
  const uint32_t rows = __ballot_sync(0xffffffffu, mine == a);
  float acc[1][NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[0][t][e] = 0.f;
  int lo, hi;
  slice((p.K + 31) / 32, blockIdx.x * kRowWarps + warp, gridDim.x * kRowWarps, lo, hi);
  const uint32_t on = ((rows >> g) & 1u) | (((rows >> (g + 8)) & 1u) << 1);
  shrink_loop<F16, 1, NT, NT <= 4 ? 4 : 2>(acc, p, p.X + static_cast<int64_t>(m0) * p.K,
                                            p.A + static_cast<int64_t>(a) * p.r * p.K, on, tiles, lo, hi);
  constexpr int W = 8 * NT;
  float* part = red + warp * 16 * W;
  const int q = lane & 3;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    *reinterpret_cast<float2*>(part + g * W + 8 * t + 2 * q) = make_float2(acc[0][t][0], acc[0][t][1]);
    *reinterpret_cast<float2*>(part + (g + 8) * W + 8 * t + 2 * q) = make_float2(acc[0][t][2], acc[0][t][3]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * W; i += blockDim.x) {
    float v = red[i];
#pragma unroll
    for (int w = 1; w < kRowWarps; ++w) v += red[w * 16 * W + i];
    red[i] = v;
  }
  const uint32_t n = gridDim.x;
  if (n > 1) cluster_sync();
  else __syncthreads();
  const float s = __ldg(p.scales + a);
  for (int i = threadIdx.x * n + cluster_rank(); i < 16 * W; i += blockDim.x * n) {
    const int row = i / W, j = i % W;
    if (!((rows >> row) & 1u) || j >= rank) continue;
    float v = 0.f;
    for (uint32_t c = 0; c < n; ++c) v += n > 1 ? ld_cluster(red + i, c) : red[i];
    V[static_cast<int64_t>(m0 + row) * p.r + j] = round1<F16>(v * s);
  }
  if (n > 1) cluster_sync();                  // the others have read this CTA's sums
}

// Many rows: a cluster for each 128 rows (and each 64 ranks); a warp has 32 rows and half of the
// CTA's slice of K, and runs through the adapters of its rows.  Four warps read the same A, from L1.
constexpr int kTileRows = 128;
template <bool F16>
__global__ void __launch_bounds__(256) k_lora_shrink_tile(const LoraArgs p, uint16_t* V) {
  constexpr int W = 64, RB = 2, NT = 8, LD = W + 4;
  __shared__ float red[kTileRows * LD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int part = warp >> 2, r0 = (warp & 3) * 32;            // K half, first row in the tile
  pdl_wait();
  pdl_launch_dependents();
  const int m0 = blockIdx.y * kTileRows + r0, j0 = blockIdx.z * W;
  const int mine = row_adapter(p, m0 + lane);
  float acc[RB][NT][4];
#pragma unroll
  for (int b = 0; b < RB; ++b)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[b][t][e] = 0.f;
  int lo, hi;
  slice((p.K + 31) / 32, blockIdx.x * 2 + part, gridDim.x * 2, lo, hi);
  for (uint32_t todo = leaders(mine); todo; todo &= todo - 1) {
    const int a = __shfl_sync(0xffffffffu, mine, __ffs(todo) - 1);
    const uint32_t rows = __ballot_sync(0xffffffffu, mine == a) >> g;
    const uint32_t on = (rows & 1u) | ((rows >> 7) & 2u) | ((rows >> 14) & 4u) | ((rows >> 21) & 8u);
    const int tiles = min(NT, (adapter_rank(p, a) - j0) / 8);
    if (tiles > 0)
      shrink_loop<F16, RB, NT, 1>(acc, p, p.X + static_cast<int64_t>(m0) * p.K,
                                  p.A + (static_cast<int64_t>(a) * p.r + j0) * p.K, on, tiles, lo, hi);
  }
#pragma unroll
  for (int h = 1; h >= 0; --h) {               // half 1 writes, half 0 adds its own
    if (part == h) {
#pragma unroll
      for (int b = 0; b < RB; ++b)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            float2* d = reinterpret_cast<float2*>(red + (r0 + 16 * b + 4 * e + g) * LD + 8 * t + 2 * q);
            const float2 o = h ? make_float2(0.f, 0.f) : *d;
            *d = make_float2(acc[b][t][e] + o.x, acc[b][t][e + 1] + o.y);
          }
    }
    __syncthreads();
  }
  const uint32_t n = gridDim.x;
  if (n > 1) cluster_sync();
  // each CTA of the cluster finishes its share of the rows, a warp a row at a time
  for (int row = cluster_rank() * 8 + warp; row < kTileRows; row += 8 * n) {
    const int m = blockIdx.y * kTileRows + row;
    const int a = row_adapter(p, m);
    if (a < 0) continue;
    const float s = __ldg(p.scales + a);
    const int rank = adapter_rank(p, a) - j0;
    float2 v = make_float2(0.f, 0.f);
    for (uint32_t c = 0; c < n; ++c) {
      const float* src = red + row * LD + 2 * lane;
      v.x += n > 1 ? ld_cluster(src, c) : src[0];
      v.y += n > 1 ? ld_cluster(src + 1, c) : src[1];
    }
    if (2 * lane < rank)
      *reinterpret_cast<uint32_t*>(V + static_cast<int64_t>(m) * p.r + j0 + 2 * lane) = pack2<F16>(v.x * s, v.y * s);
  }
  if (n > 1) cluster_sync();
}

// The expand: a warp has 16 rows and 64 output columns.  Output tile t of 8 columns stands for the
// columns 32 (t / 4) + 8 (c / 2) + 2 (t % 4) + c % 2, c = 0 .. 7, so that a lane's results of four
// tiles are 8 neighbouring columns: base and Y move 16 bytes a lane.
constexpr int kCols = 64;
template <bool F16, int CH>     // CH: chunks of 32 ranks
__global__ void __launch_bounds__(256) k_lora_expand(const LoraArgs p, const uint16_t* V, int row_warps) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int col_warps = (blockDim.x >> 5) / row_warps;
  const int m0 = (blockIdx.y * row_warps + warp % row_warps) * 16;
  const int n0 = (blockIdx.x * col_warps + warp / row_warps) * kCols;
  pdl_launch_dependents();
  if (m0 >= p.M || n0 >= p.N) return;          // whole warps
  const int mine = lane < 16 ? row_adapter(p, m0 + lane) : -1;
  uint32_t todo = leaders(mine);
  // B of one adapter and chunk of ranks: column of tile t, 8 ranks a lane
  const auto load_b = [&](uint4 (&b)[8], int a, int rank, int ch) {
    const int k = 32 * ch + 8 * q;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int n = n0 + 32 * (t >> 2) + 8 * (g >> 1) + 2 * (t & 3) + (g & 1);
      b[t] = make_uint4(0, 0, 0, 0);
      if (k < rank && n < p.N) b[t] = ld_shared_operand(p.B + (static_cast<int64_t>(a) * p.N + n) * p.r + k);
    }
  };
  int a = 0, rank = 0;
  uint4 b[8];
  if (todo) {
    a = __shfl_sync(0xffffffffu, mine, __ffs(todo) - 1);
    rank = adapter_rank(p, a);
    load_b(b, a, rank, 0);                     // on its way while the shrink finishes
  }
  pdl_wait();
  const int id[2] = {__shfl_sync(0xffffffffu, mine, g), __shfl_sync(0xffffffffu, mine, g + 8)};
  uint4 v[CH][2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int own = id[h] >= 0 ? adapter_rank(p, id[h]) : 0;
#pragma unroll
    for (int ch = 0; ch < CH; ++ch) {
      v[ch][h] = make_uint4(0, 0, 0, 0);
      if (32 * ch + 8 * q < own)
        v[ch][h] = __ldcg(reinterpret_cast<const uint4*>(V + static_cast<int64_t>(m0 + 8 * h + g) * p.r + 32 * ch + 8 * q));
    }
  }
  const bool vec = p.N % 8 == 0;
  uint4 base[2][2];                            // [row half][32 columns]
  if (vec) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int m = m0 + 8 * h + g, n = n0 + 32 * c + 8 * q;
        if (m < p.M && n < p.N) base[h][c] = *reinterpret_cast<const uint4*>(p.base + static_cast<int64_t>(m) * p.N + n);
      }
  }
  float acc[8][4];
#pragma unroll
  for (int t = 0; t < 8; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
  while (todo) {
    todo &= todo - 1;
    const int next = todo ? __shfl_sync(0xffffffffu, mine, __ffs(todo) - 1) : a;
    const int next_rank = todo ? adapter_rank(p, next) : 0;
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int ch = 0; ch < CH; ++ch) {
      uint4 nb[8];
      if (ch + 1 < CH) load_b(nb, a, rank, ch + 1);
      else load_b(nb, next, next_rank, 0);
      const uint4 lo = id[0] == a ? v[ch][0] : zero, hi = id[1] == a ? v[ch][1] : zero;
#pragma unroll
      for (int t = 0; t < 8; ++t) mma_k32<F16>(acc[t], lo, hi, b[t]);
#pragma unroll
      for (int t = 0; t < 8; ++t) b[t] = nb[t];
    }
    a = next, rank = next_rank;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int m = m0 + 8 * h + g;
    if (m >= p.M) continue;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int n = n0 + 32 * c + 8 * q;
      const int64_t at = static_cast<int64_t>(m) * p.N + n;
      if (vec) {
        if (n >= p.N) continue;
        uint32_t w[4] = {base[h][c].x, base[h][c].y, base[h][c].z, base[h][c].w};
        if (id[h] >= 0) {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const float2 f = unpack2<F16>(w[t]);
            w[t] = pack2<F16>(f.x + acc[4 * c + t][2 * h], f.y + acc[4 * c + t][2 * h + 1]);
          }
        }
        *reinterpret_cast<uint4*>(p.Y + at) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int64_t i = at + 2 * t + e;
            if (n + 2 * t + e >= p.N) continue;
            p.Y[i] = id[h] >= 0 ? round1<F16>(load1<F16>(p.base + i) + acc[4 * c + t][2 * h + e]) : p.base[i];
          }
      }
    }
  }
}

// Launch with programmatic serialization, and clusters of `cluster` CTAs along x.
template <typename... P, typename... A>
cudaError_t launch_cluster(void (*kern)(P...), dim3 grid, unsigned threads, size_t smem, unsigned cluster, cudaStream_t stream,
                           A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Up to this many rows a cluster for each leading row; above, for each 128 rows.
constexpr int kRowsMax = 1024;

template <bool F16, int NT>
cudaError_t launch_rows(const LoraArgs& a, uint16_t* V, cudaStream_t stream) {
  // at least four steps of 32 a warp, up to 8 CTAs
  const int steps = (a.K + 31) / 32;
  unsigned c = 1;
  while (c < 8 && steps >= static_cast<int>(2 * c) * kRowWarps * 4) c *= 2;
  const size_t smem = static_cast<size_t>(kRowWarps) * 16 * 8 * NT * sizeof(float);
  if (smem > 48 * 1024) {
    const cudaError_t e = set_smem_attr_once(reinterpret_cast<const void*>(k_lora_shrink_rows<F16, NT>), smem);
    if (e != cudaSuccess) return e;
  }
  return launch_cluster(k_lora_shrink_rows<F16, NT>, dim3(c, a.M), 32 * kRowWarps, smem, c, stream, a, V);
}

template <bool F16>
cudaError_t shrink_t(const LoraArgs& a, uint16_t* V, cudaStream_t stream) {
  if (a.M <= kRowsMax) {
    if (a.r <= 32) return launch_rows<F16, 4>(a, V, stream);
    if (a.r <= 64) return launch_rows<F16, 8>(a, V, stream);
    return launch_rows<F16, 16>(a, V, stream);
  }
  const int tiles = (a.M + kTileRows - 1) / kTileRows, steps = (a.K + 31) / 32;
  unsigned c = 1;
  while (c < 8 && tiles * c < 2u * device_sm_count() && steps >= static_cast<int>(2 * c) * 8) c *= 2;
  return launch_cluster(k_lora_shrink_tile<F16>, dim3(c, tiles, (a.r + 63) / 64), 256, 0, c, stream, a, V);
}

template <bool F16>
cudaError_t expand_t(const LoraArgs& a, const uint16_t* V, cudaStream_t stream) {
  const int blocks = (a.M + 15) / 16, cols = (a.N + kCols - 1) / kCols;
  // 8 warps a CTA: as many row blocks as there are (they share B through L1), then columns
  int rw = 1;
  while (rw < 8 && rw < blocks) rw *= 2;
  const int cw = 8 / rw;
  const dim3 grid((cols + cw - 1) / cw, (blocks + rw - 1) / rw);
  if (a.r <= 32) return launch_pdl(k_lora_expand<F16, 1>, grid, 256, 0, stream, a, V, rw);
  if (a.r <= 64) return launch_pdl(k_lora_expand<F16, 2>, grid, 256, 0, stream, a, V, rw);
  return launch_pdl(k_lora_expand<F16, 4>, grid, 256, 0, stream, a, V, rw);
}

}  // namespace

size_t lora_scratch_bytes(int64_t M, int64_t K, int64_t N, int64_t r) {
  (void)K;
  (void)N;
  return (static_cast<size_t>(M) * r * sizeof(uint16_t) + 255) / 256 * 256;
}

cudaError_t launch_lora_shrink(int dtype, const LoraArgs& a, void* scratch, cudaStream_t stream) {
  uint16_t* V = static_cast<uint16_t*>(scratch);
  return dtype == kF16 ? shrink_t<true>(a, V, stream) : shrink_t<false>(a, V, stream);
}

cudaError_t launch_lora_expand(int dtype, const LoraArgs& a, void* scratch, cudaStream_t stream) {
  const uint16_t* V = static_cast<const uint16_t*>(scratch);
  return dtype == kF16 ? expand_t<true>(a, V, stream) : expand_t<false>(a, V, stream);
}

}  // namespace wq

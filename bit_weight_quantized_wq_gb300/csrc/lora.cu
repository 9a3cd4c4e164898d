// Low-rank adapters of many requests beside a shared projection:
//   Y[m] = base[m] + s[a] (X[m] A[a]^T) B[a]^T,   a = adapter[m];  a = -1: Y[m] = base[m].
//
// Two kernels, the shrink V = s X A^T [M, r] and the expand Y = base + V B^T, each in a form for few rows and
// one for many (lora_many_rows, below).  All are bound by bytes: a decode batch by the adapters' A and B, a prefill
// batch by X, base and Y.
//
// Few rows: mma.sync m16n8k16 with the operands straight from global memory (A, B of the shrink; the
// expand's B through per-thread queues); every load is 16 bytes a lane.
//   Both operands are contiguous along the contracted index.  A lane holds 8 neighbouring values of
//   it (one load) and gives four to each of two products; which k a fragment slot stands for is
//   free as long as both operands agree.
//   Rows of different adapters share a 16-row block: for each adapter that occurs in it (the lowest
//   of its rows leads) the products run for all 16 rows, and its own rows take them.
// Many rows: tcgen05 with TMA on tiles of 128 rows, an accumulator for each adapter that occurs in them; each
// row takes its own.
// The sum over K is split over warps and over the CTAs of a cluster; partial sums meet in shared
// memory and are added in a fixed order.  V is kept in the element type (rounded once, after the
// scale): it is an operand of the second product, which takes 16 bits.  For few rows, and where base itself
// comes rounded from the quantized layer of the same call, V is kept in two such parts, itself and what
// its rounding left (`lo`): base's rounding and the result's are then the only ones that count.
// fp16 has no room for inner products from 65520 on, where Y may well be ordinary: each row of V, by halves of
// 64 ranks, is kept divided by a power of two that brings its largest value below 2^15 (1 where it is already),
// and the expand multiplies its sums by it in float32.
// For many rows V is rounded once: in two parts there the expand has room for one CTA an SM only and takes twice
// the products (4001 rows of rank 64, 8192 x 8192: 60.1 us instead of 47.6; 1024 rows, K 4096, N 4096, rank 16:
// 19.6 instead of 18.3).  Y's error is then some 1.2 times that of its own rounding alone.
//
// Measured, whole calls in a graph, cold adapters (as all figures below): 3 rows 4096 x 4096 5.9 us (launches and
// dependent loads); 64 rows of 48 adapters of rank 32 on 4096 x 28672 22.5 us, 3.9 TB/s; 4001 rows of 11
// requests, rank 64, 8192 x 8192 47.3 us, 4.5 TB/s.
#include <algorithm>
#include <type_traits>

#include "elem16.cuh"
#include "internal.h"
#include "tcgen05.cuh"

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
// Its rank, forced into range.
__device__ __forceinline__ int checked_rank(const LoraArgs& p, int rank) {
  if (rank < 0 || rank > p.r) {
    atomicOr(&g_lora_err, kErrIndex);
    rank = min(max(rank, 0), p.r);
  }
  return rank;
}
__device__ __forceinline__ int adapter_rank(const LoraArgs& p, int a) { return checked_rank(p, p.ranks ? __ldg(p.ranks + a) : p.r); }
__device__ __forceinline__ int up8(int rank) { return (rank + 7) & ~7; }
// What v's rounding to `hi` left: nothing where that is infinite (inf - inf would make the sum of the parts NaN).
__device__ __forceinline__ float rest(float v, float hi) { return fabsf(hi) == INFINITY ? 0.f : v - hi; }
// fp16: the power of two by which a row of V is divided, from the largest finite size in each lane.  All lanes.
__device__ __forceinline__ float row_power(float most) {
  if (!__any_sync(0xffffffffu, most >= 32768.f)) return 1.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  return __uint_as_float(((__float_as_uint(most) >> 23) - 14) << 23);      // most is in 2^14 .. 2^15 of it
}
__device__ __forceinline__ float inverse_power(float p) { return __uint_as_float((254u << 23) - __float_as_uint(p)); }
__device__ __forceinline__ float finite_size(float v) { return fabsf(v) < INFINITY ? fabsf(v) : 0.f; }
// The rows' powers follow V in the scratch: [2][M], by halves of 64 ranks.
__host__ __device__ inline int64_t v_elements(const LoraArgs& p) { return (static_cast<int64_t>(p.M) * (p.r + p.lo) + 7) / 8 * 8; }
__device__ __forceinline__ float* powers(const LoraArgs& p, uint16_t* V) { return reinterpret_cast<float*>(V + v_elements(p)); }
__device__ __forceinline__ const float* powers(const LoraArgs& p, const uint16_t* V) { return reinterpret_cast<const float*>(V + v_elements(p)); }
// 8 fp16 values times a power of two of at most 1.
__device__ __forceinline__ void scale_f16(uint4& x, float by) {
  const auto each = [&](uint32_t& w) {
    const float2 f = unpack2<true>(w);
    w = pack2<true>(f.x * by, f.y * by);
  };
  each(x.x), each(x.y), each(x.z), each(x.w);
}
// Row m's, of all its ranks.
__device__ __forceinline__ float row_power(const LoraArgs& p, const uint16_t* V, int m) {
  const float* at = powers(p, V) + m;
  const float a = __ldcg(at);
  return p.r > 64 ? fmaxf(a, __ldcg(at + p.M)) : a;
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

// The sum, in the CTAs' order, of the floats at p in the n (2, 4 or 8) CTAs of the cluster; all
// loads under way at once (one after the other they took some 300 cycles each).
__device__ __forceinline__ float sum_cluster(const float* p, uint32_t n) {
  const auto sum = [&](auto count) {
    float part[decltype(count)::value];
#pragma unroll
    for (uint32_t c = 0; c < decltype(count)::value; ++c) part[c] = ld_cluster(p, c);
    float v = part[0];
#pragma unroll
    for (uint32_t c = 1; c < decltype(count)::value; ++c) v += part[c];
    return v;
  };
  if (n == 8) return sum(std::integral_constant<uint32_t, 8>{});
  if (n == 4) return sum(std::integral_constant<uint32_t, 4>{});
  return sum(std::integral_constant<uint32_t, 2>{});
}

// Steps of 32 of the contracted index that slice i of n takes.
__device__ __forceinline__ void slice(int steps, int i, int n, int& lo, int& hi) {
  lo = static_cast<int>(static_cast<int64_t>(steps) * i / n);
  hi = static_cast<int>(static_cast<int64_t>(steps) * (i + 1) / n);
}

// acc[t] += X rows (g, g + 8) . A row (8 t + g) over steps [lo, hi) of 32, for the rows that `on` marks (bit 0:
// row g, bit 1: row g + 8); NT tiles of 8 ranks, `tiles` live; U steps' loads under way at a time.
template <bool F16, int NT, int U>
__device__ __forceinline__ void shrink_loop(float (&acc)[NT][4], const LoraArgs& p, const uint16_t* x, const uint16_t* a,
                                            uint32_t on, int tiles, int lo, int hi) {
  const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  for (int s = lo; s < hi; s += U) {
    uint4 xv[U][2], av[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (s + u) * 32 + 8 * q;
      const bool in = s + u < hi && k < p.K;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        xv[u][h] = make_uint4(0, 0, 0, 0);
        if (in && ((on >> h) & 1u)) xv[u][h] = ld_stream(x + static_cast<int64_t>(8 * h + g) * p.K + k);
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
        if (t < tiles) mma_k32<F16>(acc[t], xv[u][0], xv[u][1], av[u][t]);
  }
}

// Few rows: one cluster for each row that leads its adapter in its 16-row block; 8 warps a CTA, each
// a slice of K.  9 us by itself for 48 adapters of rank 32, K 4096 (10 MB of A): adapter, rank and A are
// loads that wait for one another, and the cluster meets twice.
// Two CTAs an SM are asked for so that the compiler keeps a step's loads in registers, all under way; left to
// itself it took 86 to 114 registers, by what else stood in the kernel, and loaded in turns (13 rows of rank 48,
// K 4992: 13.9 us instead of 9.6; 64 rows of rank 32: 23.1 instead of 22.5).
constexpr int kRowWarps = 8;
template <bool F16, int NT>
__global__ void __launch_bounds__(32 * kRowWarps, NT <= 8 ? 2 : 1) k_lora_shrink_rows(const LoraArgs p, uint16_t* V) {
  extern __shared__ float red[];              // [warp][16][8 NT], then the CTA's sum over [0]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
  pdl_wait();
  pdl_launch_dependents();                    // the expand may read all but V from here on
  const int m = blockIdx.y, m0 = m & ~15;
  // Up to 128 adapters: their ranks come beside the rows' adapters, not after them (after / beside, in us: 16
  // rows 7.6 / 7.3, 64 rows of 48 adapters 22.7 / 22.4, 200 rows 40.6 / 39.9).
  const bool ahead = p.ranks && p.L <= 128;
  int all_ranks[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) all_ranks[i] = ahead && lane + 32 * i < p.L ? __ldg(p.ranks + lane + 32 * i) : 0;
  const int mine = lane < 16 ? row_adapter(p, m0 + lane) : -1;
  const uint32_t lead = leaders(mine);
  if (!((lead >> (m & 15)) & 1u)) return;     // the same for all CTAs of the cluster
  const int a = __shfl_sync(0xffffffffu, mine, m & 15);
  int rank;
  if (ahead) {
    const int i = a >> 5;                     // the same in all lanes
    rank = checked_rank(p, __shfl_sync(0xffffffffu, i == 0 ? all_ranks[0] : i == 1 ? all_ranks[1] : i == 2 ? all_ranks[2] : all_ranks[3], a & 31));
  } else {
    rank = adapter_rank(p, a);
  }
  const int tiles = up8(rank) / 8;
  const uint32_t rows = __ballot_sync(0xffffffffu, mine == a);
  float acc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
  int lo, hi;
  slice((p.K + 31) / 32, blockIdx.x * kRowWarps + warp, gridDim.x * kRowWarps, lo, hi);
  const uint32_t on = ((rows >> g) & 1u) | (((rows >> (g + 8)) & 1u) << 1);
  shrink_loop<F16, NT, NT <= 4 ? 4 : 2>(acc, p, p.X + static_cast<int64_t>(m0) * p.K,
                                            p.A + static_cast<int64_t>(a) * p.r * p.K, on, tiles, lo, hi);
  constexpr int W = 8 * NT;
  float* part = red + warp * 16 * W;
  const int q = lane & 3;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    *reinterpret_cast<float2*>(part + g * W + 8 * t + 2 * q) = make_float2(acc[t][0], acc[t][1]);
    *reinterpret_cast<float2*>(part + (g + 8) * W + 8 * t + 2 * q) = make_float2(acc[t][2], acc[t][3]);
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
  for (int row = cluster_rank() + n * warp; row < 16; row += n * kRowWarps) {     // a warp a row
    if (!((rows >> row) & 1u)) continue;
    float v[W / 32], most = 0.f;
#pragma unroll
    for (int c = 0; c < W / 32; ++c) {
      const int j = 32 * c + lane;
      v[c] = 0.f;                             // past the rank: the expand of many rows takes all r
      if (j < rank) v[c] = (n > 1 ? sum_cluster(red + row * W + j, n) : red[row * W + j]) * s;
      if constexpr (F16) most = fmaxf(most, finite_size(v[c]));
    }
    if constexpr (F16) {
      const float up = row_power(most);
#pragma unroll
      for (int c = 0; c < W / 32; ++c) v[c] *= inverse_power(up);
      if (lane < 2) powers(p, V)[static_cast<int64_t>(lane) * p.M + m0 + row] = up;
    }
    uint16_t* to = V + static_cast<int64_t>(m0 + row) * (p.r + p.lo) + lane;
#pragma unroll
    for (int c = 0; c < W / 32; ++c) {
      if (32 * c + lane >= p.r) continue;
      const uint32_t hi = pack2<F16>(v[c], 0.f);
      to[32 * c] = static_cast<uint16_t>(hi);
      if (p.lo) to[32 * c + p.lo] = round1<F16>(rest(v[c], unpack2<F16>(hi).x));
    }
  }
  if (n > 1) cluster_sync();                  // the others have read this CTA's sums
}

// Many rows: a cluster for each 128 rows (and each 64 ranks), its CTAs a slice of K each, on the
// tensor cores: tcgen05.mma with X [128 rows, 64 k] and A [ranks, 64 k] by TMA (128-byte swizzle), one
// accumulator in tensor memory for each adapter that occurs in the rows, two adapters a pass over
// the slice.  Three stages of 32 KB and two CTAs an SM keep some 150 KB of loads under way; the
// same contraction on mma.sync, with A prefetched one step ahead, waited for L2 at every step.  24 us by
// itself at 4001 rows, K 8192, rank 64: 72 MB, 3.0 TB/s; a CTA has only 16 steps of 64 between its start
// and the cluster's sum.
constexpr int kTileRows = 128, kTileStages = 3, kTilePass = 2;
constexpr int kTileLd = 64 + 4;
// The different adapters of 128 rows, in order of their first row.
struct Found {
  int lead[4][32], place[4][32], n_lead[4];    // a warp's leading rows: adapter, place in `id`
  int id[kTileRows];
  int n[4];
  __device__ __forceinline__ int count() const { return n[0] + n[1] + n[2] + n[3]; }
};
// Fills `f`, and gives each row's place in it (-1: none).  All threads of the CTA; rw: 0 .. 3 for the
// four warps that have a row a thread, else -1.  Within a warp by a match; then the leaders of warp rw
// look for themselves among those of the warps before it.
__device__ __forceinline__ int find_adapters(Found& f, int rw, int mine) {
  const int lane = threadIdx.x & 31;
  const uint32_t lead = leaders(mine), same = __match_any_sync(0xffffffffu, mine);
  const bool leads = rw >= 0 && ((lead >> lane) & 1u);
  const int nth = __popc(lead & ((1u << lane) - 1));
  if (leads) f.lead[rw][nth] = mine;
  if (rw >= 0 && lane == 0) f.n_lead[rw] = __popc(lead);
  __syncthreads();
  int before = -1, place = -1;                 // 32 w + i: warp w's i-th leader has it already
  if (leads)
    for (int w = 0; w < rw && before < 0; ++w)
      for (int i = 0; i < f.n_lead[w] && before < 0; ++i)
        if (f.lead[w][i] == mine) before = 32 * w + i;
  const uint32_t fresh = __ballot_sync(0xffffffffu, leads && before < 0);
  if (rw >= 0 && lane == 0) f.n[rw] = __popc(fresh);
  __syncthreads();
  if ((fresh >> lane) & 1u) {
    place = __popc(fresh & ((1u << lane) - 1));
    for (int w = 0; w < rw; ++w) place += f.n[w];
    f.id[place] = mine;
  }
  if (leads) f.place[rw][nth] = place;
  __syncthreads();
  if (before >= 0) place = f.place[before >> 5][before & 31];
  place = __shfl_sync(0xffffffffu, place, __ffs(same) - 1);
  return mine < 0 ? -1 : place;
}

struct TileSmem {
  union {
    struct {
      uint8_t x[kTileStages][kTileRows * 128];
      uint8_t a[kTileStages][kTilePass][64 * 128];
    } ring;
    float red[kTileRows * kTileLd];            // after the last product
  };
  uint64_t full[kTileStages], empty[kTileStages], acc_full[2], acc_empty[2], drain;
  Found who;
  float scale[kTileRows];                      // of each row's adapter
  int rank[kTileRows];                         // -1: no adapter
  uint32_t tmem_base;
};

template <bool F16>
__global__ void __launch_bounds__(192) k_lora_shrink_tile(const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap ta,
                                                          const LoraArgs p, uint16_t* V, int box_ranks) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  TileSmem& sm = *reinterpret_cast<TileSmem*>(smem_raw + smem_align_pad(smem_raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kTileStages; ++s) mbar_init(&sm.full[s], 1), mbar_init(&sm.empty[s], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&sm.acc_full[i], 1), mbar_init(&sm.acc_empty[i], 4);
    mbar_init(&sm.drain, 1);
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem_base, 256);            // two sets of two accumulators of 64 columns
    tmem_relinquish();
  }
  pdl_wait();
  pdl_launch_dependents();
  const int m0 = blockIdx.y * kTileRows, j0 = blockIdx.z * 64;
  const int row = (warp & 3) * 32 + lane;      // warps 2 .. 5: a row a thread, its tensor-memory lane
  const int mine = warp >= 2 ? row_adapter(p, m0 + row) : -1;
  if (warp >= 2) {                             // for the end, when a row is any warp's
    sm.scale[row] = mine >= 0 ? __ldg(p.scales + mine) : 0.f;
    sm.rank[row] = mine >= 0 ? adapter_rank(p, mine) : -1;
  }
  tc_fence_before();
  const int place = find_adapters(sm.who, warp >= 2 ? warp & 3 : -1, mine);
  tc_fence_after();
  const int found = sm.who.count();
  const int passes = (found + kTilePass - 1) / kTilePass;
  int lo, hi;
  slice((p.K + 63) / 64, blockIdx.x, gridDim.x, lo, hi);
  const uint32_t tmem = sm.tmem_base;
  float res[64];
#pragma unroll
  for (int e = 0; e < 64; ++e) res[e] = 0.f;

  if (warp == 0) {
    uint32_t ord = 0;
    bool ok = true;
    const uint64_t once = l2_policy_evict_first(), keep = l2_policy_evict_last();
    for (int ps = 0; ps < passes && ok; ++ps) {
      const int n = min(kTilePass, found - ps * kTilePass);
      for (int s = lo; s < hi; ++s, ++ord) {
        const int st = ord % kTileStages;
        ok = __all_sync(0xffffffffu, mbar_wait_short(&sm.empty[st], ((ord / kTileStages) & 1) ^ 1, &g_lora_err, kErrWaitEmpty));
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&sm.full[st], kTileRows * 128 + n * box_ranks * 128);
          tma_load_2d(sm.ring.x[st], &tx, s * 64, m0, &sm.full[st], passes > 1 ? keep : once);
          for (int d = 0; d < n; ++d)
            tma_load_2d(sm.ring.a[st][d], &ta, s * 64, sm.who.id[ps * kTilePass + d] * p.r + j0, &sm.full[st], keep);
        }
        __syncwarp();
      }
    }
    for (uint32_t i = ord > kTileStages ? ord - kTileStages : 0; i < ord; ++i)
      mbar_wait_short(&sm.full[i % kTileStages], (i / kTileStages) & 1, &g_lora_err, kErrDrain);
  } else if (warp == 1) {
    constexpr uint32_t fmt = F16 ? 0u : 1u;
    const uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | (static_cast<uint32_t>(box_ranks >> 3) << 17) | ((kTileRows >> 4) << 24);
    uint32_t ord = 0;
    bool ok = true;
    for (int ps = 0; ps < passes && ok; ++ps) {
      const int n = min(kTilePass, found - ps * kTilePass), set = ps & 1;
      ok = __all_sync(0xffffffffu, mbar_wait_short(&sm.acc_empty[set], ((ps >> 1) & 1) ^ 1, &g_lora_err, kErrWaitAccum));
      for (int s = lo; s < hi && ok; ++s, ++ord) {
        const int st = ord % kTileStages;
        ok = __all_sync(0xffffffffu, mbar_wait_short(&sm.full[st], (ord / kTileStages) & 1, &g_lora_err, kErrWaitFull));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t xd = smem_desc_sw128(smem_u32(sm.ring.x[st]));
          for (int d = 0; d < n; ++d) {
            const uint64_t ad = smem_desc_sw128(smem_u32(sm.ring.a[st][d]));
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc_mma_ss_f16(tmem + 128 * set + 64 * d, xd + 2 * k, ad + 2 * k, idesc, (s > lo || k) ? 1u : 0u);
          }
          tc_commit(&sm.empty[st]);
        }
        __syncwarp();
      }
      if (ok && elect_one()) tc_commit(&sm.acc_full[set]);
      __syncwarp();
    }
    if (elect_one()) tc_commit(&sm.drain);     // nothing under way any more, whatever happened
    mbar_wait_short(&sm.drain, 0, &g_lora_err, kErrDrain);
  } else {
    for (int ps = 0; ps < passes; ++ps) {
      const int n = min(kTilePass, found - ps * kTilePass), set = ps & 1;
      if (!__all_sync(0xffffffffu, mbar_wait_short(&sm.acc_full[set], (ps >> 1) & 1, &g_lora_err, kErrWaitAccum))) break;
      tc_fence_after();
      for (int d = 0; d < n && lo < hi; ++d) {
        const bool own = place == ps * kTilePass + d;
        if (!__any_sync(0xffffffffu, own)) continue;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t v[32];
          tmem_ld32(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 128 * set + 64 * d + 32 * h, v);
          tc_wait_ld();
          if (own)
#pragma unroll
            for (int e = 0; e < 32; ++e) res[32 * h + e] = __uint_as_float(v[e]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.acc_empty[set]);
    }
  }
  __syncwarp();
  __syncthreads();                             // the ring is idle: its memory holds the sums now
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
  if (warp >= 2) {
    float4* d = reinterpret_cast<float4*>(sm.red + row * kTileLd);
#pragma unroll
    for (int e = 0; e < 16; ++e) d[e] = make_float4(res[4 * e], res[4 * e + 1], res[4 * e + 2], res[4 * e + 3]);
  }
  const uint32_t n = gridDim.x;
  if (n > 1) cluster_sync();
  else __syncthreads();
  // each CTA of the cluster finishes its share of the rows, a warp a row at a time
  for (int r = cluster_rank() * 6 + warp; r < kTileRows; r += 6 * n) {
    const int m = m0 + r;
    if (sm.rank[r] < 0) continue;
    const float s = sm.scale[r];
    const int rank = sm.rank[r] - j0;
    const float* src = sm.red + r * kTileLd + 2 * lane;
    float2 v = n > 1 ? make_float2(sum_cluster(src, n), sum_cluster(src + 1, n)) : make_float2(src[0], src[1]);
    v = make_float2(2 * lane < rank ? v.x * s : 0.f, 2 * lane + 1 < rank ? v.y * s : 0.f);
    if constexpr (F16) {
      const float up = row_power(fmaxf(finite_size(v.x), finite_size(v.y))), down = inverse_power(up);
      v.x *= down, v.y *= down;
      if (lane == 0) powers(p, V)[static_cast<int64_t>(blockIdx.z) * p.M + m] = up;
    }
    if (2 * lane < p.r - j0) {
      uint16_t* to = V + static_cast<int64_t>(m) * (p.r + p.lo) + j0 + 2 * lane;
      const uint32_t hi = pack2<F16>(v.x, v.y);
      const float2 f = unpack2<F16>(hi);
      *reinterpret_cast<uint32_t*>(to) = hi;
      if (p.lo) *reinterpret_cast<uint32_t*>(to + p.lo) = pack2<F16>(rest(v.x, f.x), rest(v.y, f.y));
    }
  }
  if (n > 1) cluster_sync();                   // the others have read this CTA's sums
}

// The expand: a warp has 16 rows, 32 output columns at a time, and every `subsets`-th adapter of
// those rows (their rows are its own to write; rows without an adapter are the first warp's).
// Output tile t of 8 columns stands for the columns 8 (c / 2) + 2 t + c % 2, c = 0 .. 7, so that a
// lane's results of four tiles are 8 neighbouring columns: base and Y move 16 bytes a lane.  21 us by itself
// for 64 rows of 48 adapters of rank 32, N 28672: 84 MB, 4.1 TB/s.
//   B (32 columns and 32 ranks a step) and base come through queues in shared memory, each thread
//   its own place, so that steps ahead are under way without registers: with B one step ahead in
//   registers a decode batch of 48 adapters ran at 2.5 TB/s.
//   `span` column tiles a warp: 1 for few rows; many rows keep their set-up over several.
constexpr int kCols = 32;
constexpr int kBQueue = 4, kBaseQueue = 4;   // see the waits below
constexpr int kStageLd = 33;
static_assert(8 * 16 * kStageLd * 4 <= kBaseQueue * 2 * 256 * 16, "the staged rows take the base queue's place");
template <bool F16, int CH, bool LO>     // CH: chunks of 32 ranks; LO: V in two parts
__global__ void __launch_bounds__(256, CH * (LO ? 2 : 1) <= 2 ? 2 : 1) k_lora_expand(const LoraArgs p, const uint16_t* V, int log_rows, int log_subsets, int span) {
  extern __shared__ __align__(16) uint8_t expand_smem[];
  uint4* bq = reinterpret_cast<uint4*>(expand_smem) + threadIdx.x;              // [step][4][256]
  uint4* baseq = bq + kBQueue * 4 * 256;                                        // [tile][2][256]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  // warps of a CTA: row blocks first (they share B through L1), then subsets, then columns
  const int subset = (warp >> log_rows) & ((1 << log_subsets) - 1);
  const int m0 = ((blockIdx.y << log_rows) + (warp & ((1 << log_rows) - 1))) * 16;
  const int col_warps = 8 >> (log_rows + log_subsets);
  const int ct0 = (blockIdx.x * col_warps + (warp >> (log_rows + log_subsets))) * span;
  const int ct1 = min(ct0 + span, (p.N + kCols - 1) / kCols);
  pdl_launch_dependents();
  if (m0 >= p.M || ct0 >= ct1) return;         // whole warps
  const int mine = lane < 16 ? row_adapter(p, m0 + lane) : -1;
  const int my_rank = mine >= 0 ? up8(adapter_rank(p, mine)) : 0;
  uint32_t list = 0;                           // this subset's leading rows
  {
    uint32_t lead = leaders(mine);
    for (int i = 0; lead; ++i, lead &= lead - 1)
      if ((i & ((1 << log_subsets) - 1)) == subset) list |= lead & (0u - lead);
  }
  const int first = __ffs(__match_any_sync(0xffffffffu, mine)) - 1;
  const bool own_row = lane < 16 && (mine >= 0 ? ((list >> first) & 1u) != 0 : subset == 0);
  const uint32_t own_rows = __ballot_sync(0xffffffffu, own_row);
  if (!own_rows) return;

  // The steps: column tile, leading row, chunk of ranks -- walked twice, by the copies and, kBQueue
  // steps behind, by the products.
  struct Step {
    int ct, ch;
    uint32_t todo;                             // leading rows from this step's on
  };
  const auto next_step = [&](Step& s) {
    if (++s.ch < CH) return;
    s.ch = 0;
    s.todo &= s.todo - 1;
    if (!s.todo) s.todo = list, ++s.ct;
  };
  // The walk of the copies costs as much as the products: a row's lane keeps where its adapter's B
  // begins, a lane where its four columns are in the tile.
  Step fs{ct0, 0, list};
  int f_at = 0;
  const int64_t b_of = mine >= 0 ? static_cast<int64_t>(mine) * p.N * p.r : 0;
  const int c_lane = 8 * (g >> 1) + (g & 1), r2 = 2 * p.r;
  const auto fetch_b = [&] {
    if (fs.ct < ct1 && list) {
      const int i = __ffs(fs.todo) - 1;
      const int rank = __shfl_sync(0xffffffffu, my_rank, i);
      const int64_t of = __shfl_sync(0xffffffffu, b_of, i);
      const int k = 32 * fs.ch + 8 * q, n = fs.ct * kCols + c_lane;
      const uint16_t* src = p.B + of + (static_cast<int64_t>(n) * p.r + k);
      uint4* dst = bq + f_at * (4 * 256);
      const bool in = k < rank;
      if ((fs.ct + 1) * kCols <= p.N) {
#pragma unroll
        for (int t = 0; t < 4; ++t) copy16(dst + t * 256, in ? src + t * r2 : p.B, in);
      } else {
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const bool on = in && n + 2 * t < p.N;
          copy16(dst + t * 256, on ? src + t * r2 : p.B, on);
        }
      }
      next_step(fs);
      f_at = f_at + 1 == kBQueue ? 0 : f_at + 1;
    }
  };
  // N not a multiple of 8: rows begin anywhere, so a lane takes one column of each row; its base is on its
  // way during the products, which come to the rows through shared memory (the base queue's place).  With
  // eight columns a lane, in single elements, 494 rows of 11655 columns took 1.4 times as long (25.1 us now, K
  // 4096, rank 32).
  const bool vec = p.N % 8 == 0;
  float* stage = reinterpret_cast<float*>(expand_smem + sizeof(uint4) * kBQueue * 4 * 256) + warp * (16 * kStageLd);
  const uint32_t adapted = __ballot_sync(0xffffffffu, mine >= 0);
  const bool own[2] = {((own_rows >> g) & 1u) != 0, ((own_rows >> (g + 8)) & 1u) != 0};
  const auto fetch_base = [&](int ct, int at) {
    if (!vec) return;                          // the place is the staged rows'
    const int n = ct * kCols + 8 * q;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int m = m0 + 8 * h + g;
      const bool on = own[h] && ct < ct1 && m < p.M && n < p.N;
      copy16(baseq + (at * 2 + h) * 256, on ? p.base + static_cast<int64_t>(m) * p.N + n : p.base, on);
    }
  };
  // Groups of copies, by number: 0 .. Q - 2 the first steps' B, on its way while the shrink finishes;
  // Q - 1 the first tiles' bases; Q + s, at step s, the B of step s + Q - 1 and, at a tile's first
  // step, the base of the tile Q - 1 tiles on.
#pragma unroll
  for (int i = 0; i < kBQueue - 1; ++i) {
    fetch_b();
    copy_commit();
  }
  pdl_wait();
#pragma unroll
  for (int i = 0; i < kBaseQueue - 1; ++i) fetch_base(ct0 + i, i);
  copy_commit();
  const int id[2] = {__shfl_sync(0xffffffffu, mine, g), __shfl_sync(0xffffffffu, mine, g + 8)};
  const int ranks[2] = {__shfl_sync(0xffffffffu, my_rank, g), __shfl_sync(0xffffffffu, my_rank, g + 8)};
  float half_up[2][CH == 4 ? 2 : 1];
  if constexpr (F16) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int c = 0; c < (CH == 4 ? 2 : 1); ++c)
        half_up[h][c] = own[h] && id[h] >= 0 ? __ldcg(powers(p, V) + static_cast<int64_t>(c) * p.M + m0 + 8 * h + g) : 1.f;
  }
  uint4 v[CH][2], vl[LO ? CH : 1][2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int ch = 0; ch < CH; ++ch) {
      v[ch][h] = make_uint4(0, 0, 0, 0);
      if constexpr (LO) vl[ch][h] = v[ch][h];
      if (own[h] && 32 * ch + 8 * q < ranks[h]) {
        const uint16_t* from = V + static_cast<int64_t>(m0 + 8 * h + g) * (p.r + p.lo) + 32 * ch + 8 * q;
        v[ch][h] = __ldcg(reinterpret_cast<const uint4*>(from));
        if constexpr (LO) vl[ch][h] = __ldcg(reinterpret_cast<const uint4*>(from + p.lo));
      }
    }
  // fp16: the power of two that the row's sums are multiplied by; halves of its ranks that were divided by
  // different ones are brought to the larger
  float up[2] = {1.f, 1.f};
  if constexpr (F16) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      up[h] = CH == 4 ? fmaxf(half_up[h][0], half_up[h][CH / 4]) : half_up[h][0];
      if constexpr (CH == 4) {
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) {
          const float down = half_up[h][ch / 2] * inverse_power(up[h]);
          if (down == 1.f) continue;
          scale_f16(v[ch][h], down);
          if constexpr (LO) scale_f16(vl[ch][h], down);
        }
      }
    }
  }
  const int steps = max(1, __popc(list) * CH);   // a tile
  int b_at = 0, base_at = 0;
#pragma unroll 1
  for (int ct = ct0; ct < ct1; ++ct) {
    fetch_base(ct + kBaseQueue - 1, base_at == 0 ? kBaseQueue - 1 : base_at - 1);
    float acc[4][4];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][e] = 0.f;
    const int col = ct * kCols + lane;
    const int64_t first_at = static_cast<int64_t>(m0) * p.N + col;
    uint16_t single[16];
    if (!vec) {
#pragma unroll
      for (int r = 0; r < 16; ++r)
        single[r] = ((own_rows >> r) & 1u) && m0 + r < p.M && col < p.N ? p.base[first_at + static_cast<int64_t>(r) * p.N] : 0;
    }
    // An adapter's product runs for all 16 rows, and its own rows take it, so that an infinity or a NaN in its B
    // reaches no other's.  They take it when the next adapter's B is there: at once, the products' latency showed
    // (64 rows of 48 adapters, whole call: 23.5 us instead of 22.6).
    float prod[4][4];
    int of = -2;                               // no row's adapter
    const auto take = [&] {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[t][e] = id[e >> 1] == of ? prod[t][e] : acc[t][e];
    };
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) prod[t][e] = 0.f;
#pragma unroll 1
    for (uint32_t todo = list; todo; todo &= todo - 1) {
#pragma unroll
      for (int ch = 0; ch < CH; ++ch) {
        fetch_b();
        copy_commit();
        copy_wait<kBQueue - 1>();              // groups up to s + 1: the B of step s among them
        if (ch == 0) {
          take();
          of = __shfl_sync(0xffffffffu, mine, __ffs(todo) - 1);
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) prod[t][e] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < 4; ++t) mma_k32<F16>(prod[t], v[ch][0], v[ch][1], bq[(b_at * 4 + t) * 256]);
        if constexpr (LO) {
#pragma unroll
          for (int t = 0; t < 4; ++t) mma_k32<F16>(prod[t], vl[ch][0], vl[ch][1], bq[(b_at * 4 + t) * 256]);
        }
        b_at = b_at + 1 == kBQueue ? 0 : b_at + 1;
      }
    }
    take();
    if (!list) {
      copy_commit();
      copy_wait<kBQueue - 1>();
    }
    // This tile's base: tile i, of T steps a tile, has group Q + (i - Q + 1) T at most, and groups up
    // to (i + 1) T are here; only the first tiles' group Q - 1 may be later.
    if ((ct - ct0 + 1) * steps < kBQueue - 1) copy_wait<1>();
    if (vec) {
      const int n = ct * kCols + 8 * q;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int m = m0 + 8 * h + g;
        if (m >= p.M || !own[h] || n >= p.N) continue;
        const uint4 y = baseq[(base_at * 2 + h) * 256];
        uint32_t w[4] = {y.x, y.y, y.z, y.w};
        if (id[h] >= 0) {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const float2 f = unpack2<F16>(w[t]);
            if constexpr (F16) w[t] = pack2<F16>(fmaf(acc[t][2 * h], up[h], f.x), fmaf(acc[t][2 * h + 1], up[h], f.y));
            else w[t] = pack2<F16>(f.x + acc[t][2 * h], f.y + acc[t][2 * h + 1]);
          }
        }
        *reinterpret_cast<uint4*>(p.Y + static_cast<int64_t>(m) * p.N + n) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int e = 0; e < 2; ++e) stage[(8 * h + g) * kStageLd + 8 * q + 2 * t + e] = acc[t][2 * h + e] * up[h];
      __syncwarp();
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (((own_rows >> r) & 1u) && m0 + r < p.M && col < p.N)
          p.Y[first_at + static_cast<int64_t>(r) * p.N] =
              (adapted >> r) & 1u ? round1<F16>(unpack2<F16>(single[r]).x + stage[r * kStageLd + lane]) : single[r];
      __syncwarp();
    }
    base_at = base_at + 1 == kBaseQueue ? 0 : base_at + 1;
  }
  copy_wait<0>();
}
constexpr size_t kExpandSmem = static_cast<size_t>(kBQueue * 4 + kBaseQueue * 2) * 256 * 16;

// The expand of many rows: a CTA has 128 rows and walks over `span` tiles of 64 columns on the tensor
// cores.  acc = V [128 rows, r] B^T [r, 64 columns], one accumulator in tensor memory for each adapter that
// occurs in the rows; base comes by TMA, is added to in its place in shared memory and
// leaves from there by TMA.  Two groups of four warps (a row a thread) take the tiles in turn, each with
// two accumulators of its own; the other warps move base and Y, issue the products, and copy B.  Two CTAs
// an SM (one with more than 64 ranks or V in two parts).  26 us by itself at 4001 rows, N 8192, rank 64: 131 MB, 5.1 TB/s; with one
// group, which held a tile's sums in registers until base was there, the whole call took 50 us instead of 47.
// A multiple of the groups: a slot of base is then always the same group's, which sees each of its phases.
constexpr int kExCols = 64, kExBase = 4, kExB = 3;
static_assert(kExBase % 2 == 0, "a wait by parity may not leave out a phase");
constexpr int kExThreads = 352, kExWBase = 8, kExWMma = 9;   // warps 0 .. 7 add; 10: B
template <int CR, bool LO>                     // chunks of 64 ranks; V in two parts
struct ExpandSmem {
  uint8_t base[kExBase][kTileRows * 128];
  uint8_t v[LO ? 2 : 1][CR][kTileRows * 128];
  uint8_t b[kExB][CR][kExCols * 128];
  uint64_t base_full[kExBase], added[kExBase], b_full[kExB], b_empty[kExB], v_full, acc_full[2][2], acc_empty[2][2], drain;
  Found who;
  int place[kTileRows];                        // of each row's adapter in `who`
  uint32_t tmem_base;
};

template <bool F16, int CR, bool LO>
__global__ void __launch_bounds__(kExThreads, CR == 1 && !LO ? 2 : 1)
    k_lora_expand_tile(const __grid_constant__ CUtensorMap tbase, const __grid_constant__ CUtensorMap ty,
                       const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tvl,
                       const __grid_constant__ CUtensorMap tb, const LoraArgs p, const uint16_t* V, int span, int base_ready) {
  using S = ExpandSmem<CR, LO>;
  constexpr int kParts = LO ? 2 : 1;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw + smem_align_pad(smem_raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kExBase; ++i) mbar_init(&sm.base_full[i], 1), mbar_init(&sm.added[i], 4);
    for (int i = 0; i < kExB; ++i) mbar_init(&sm.b_full[i], 1), mbar_init(&sm.b_empty[i], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&sm.acc_full[i >> 1][i & 1], 1), mbar_init(&sm.acc_empty[i >> 1][i & 1], 4);
    mbar_init(&sm.v_full, 1), mbar_init(&sm.drain, 1);
    fence_barrier_init();
  }
  if (warp == kExWMma) {
    tmem_alloc(&sm.tmem_base, 256);            // two accumulators of 64 columns a group
    tmem_relinquish();
  }
  pdl_launch_dependents();
  const int m0 = blockIdx.y * kTileRows, row = threadIdx.x & (kTileRows - 1);
  const int ct0 = blockIdx.x * span, tiles = min(span, (p.N + kExCols - 1) / kExCols - ct0);
  // adapter and ranks are the caller's: the shrink, this kernel's predecessor, has waited for them
  const int mine = warp < 4 ? row_adapter(p, m0 + row) : -1;
  int place = find_adapters(sm.who, warp < 4 ? warp : -1, mine);
  if (warp < 4) sm.place[row] = place;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int found = sm.who.count();
  const uint32_t tmem = sm.tmem_base;
  bool ok = true;
  const auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t code) {
    return __all_sync(0xffffffffu, mbar_wait_short(bar, parity, &g_lora_err, code));
  };
  if (warp == kExWBase) {
    // -------------------------------------------------------------------- base in, Y out
    if (!base_ready) pdl_wait();
    const uint64_t normal = l2_policy_evict_normal();
    const auto load = [&](int i) {
      mbar_arrive_expect_tx(&sm.base_full[i % kExBase], kTileRows * 128);
      tma_load_2d(sm.base[i % kExBase], &tbase, (ct0 + i) * kExCols, m0, &sm.base_full[i % kExBase], normal);
    };
    int issued = min(tiles, kExBase);
    if (elect_one())
      for (int i = 0; i < issued; ++i) load(i);
    __syncwarp();
    for (int i = 0; i < tiles; ++i) {
      if (!wait(&sm.added[i % kExBase], (i / kExBase) & 1, kErrWaitFull)) break;
      if (elect_one()) {
        tma_store_2d(&ty, sm.base[i % kExBase], (ct0 + i) * kExCols, m0);
        bulk_commit();
        bulk_wait_read<0>();                   // the tile has left its slot
        if (issued < tiles) load(issued);
      }
      __syncwarp();
      issued = min(issued + 1, tiles);
    }
    if (elect_one()) bulk_wait<0>();
    // every copy has landed before the memory goes
    for (int i = max(issued - kExBase, 0); i < issued; ++i) wait(&sm.base_full[i % kExBase], (i / kExBase) & 1, kErrDrain);
  } else if (warp == kExWMma) {
    // -------------------------------------------------------------------- V, products
    pdl_wait();
    if (found) {
      if (elect_one()) {
        mbar_arrive_expect_tx(&sm.v_full, kParts * CR * kTileRows * 128);
#pragma unroll
        for (int part = 0; part < kParts; ++part)
#pragma unroll
          for (int c = 0; c < CR; ++c)
            tma_load_2d(sm.v[part][c], part ? &tvl : &tv, 64 * c, m0, &sm.v_full, l2_policy_evict_first());
      }
      __syncwarp();
      float half_up[4][2];                     // of rows lane, lane + 32, ...
      if constexpr (F16 && CR == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            half_up[i][c] = sm.place[32 * i + lane] >= 0 ? __ldcg(powers(p, V) + static_cast<int64_t>(c) * p.M + m0 + 32 * i + lane) : 1.f;
      }
      ok = wait(&sm.v_full, 0, kErrWaitFull);
      if constexpr (F16 && CR == 2) {          // halves of a row's ranks that were divided by different powers
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float down = inverse_power(fmaxf(half_up[i][0], half_up[i][1]));
          if (!ok || half_up[i][0] == half_up[i][1]) continue;
          const int c = half_up[i][0] < half_up[i][1] ? 0 : 1;
          for (int k = 0; k < kParts * 8; ++k)
            scale_f16(*reinterpret_cast<uint4*>(sm.v[k >> 3][c] + (32 * i + lane) * 128 + 16 * (k & 7)), half_up[i][c] * down);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
    }
    constexpr uint32_t fmt = F16 ? 0u : 1u;
    constexpr uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((kExCols >> 3) << 17) | ((kTileRows >> 4) << 24);
    const int steps = (p.r + 15) / 16;         // past r both operands are filled with zeros
    uint32_t ord = 0;
    for (int i = 0; i < tiles && ok; ++i)
      for (int d = 0; d < found; ++d, ++ord) {
        const int s = ord % kExB, grp = i & 1;
        const uint32_t use = static_cast<uint32_t>(i >> 1) * found + d, buf = use & 1;   // of this group's
        ok = wait(&sm.acc_empty[grp][buf], ((use >> 1) & 1) ^ 1, kErrWaitAccum) && wait(&sm.b_full[s], (ord / kExB) & 1, kErrWaitFull);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int part = 0; part < kParts; ++part)
            for (int k = 0; k < steps; ++k)
              tc_mma_ss_f16(tmem + 128 * grp + 64 * buf, smem_desc_sw128(smem_u32(sm.v[part][k >> 2])) + 2 * (k & 3),
                            smem_desc_sw128(smem_u32(sm.b[s][k >> 2])) + 2 * (k & 3), idesc, (part || k) ? 1u : 0u);
          tc_commit(&sm.b_empty[s]);
          tc_commit(&sm.acc_full[grp][buf]);
        }
        __syncwarp();
      }
    if (elect_one()) tc_commit(&sm.drain);     // nothing under way any more, whatever happened
    wait(&sm.drain, 0, kErrDrain);
  } else if (warp > kExWMma) {
    // -------------------------------------------------------------------- B
    const uint64_t keep = l2_policy_evict_last();
    int ord = 0;
    for (int i = 0; i < tiles && ok; ++i)
      for (int d = 0; d < found; ++d, ++ord) {
        const int s = ord % kExB;
        ok = wait(&sm.b_empty[s], ((ord / kExB) & 1) ^ 1, kErrWaitEmpty);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&sm.b_full[s], CR * kExCols * 128);
#pragma unroll
          for (int c = 0; c < CR; ++c)
            tma_load_4d(sm.b[s][c], &tb, 64 * c, (ct0 + i) * kExCols, sm.who.id[d], 0, &sm.b_full[s], keep);
        }
        __syncwarp();
      }
    for (int i = max(ord - kExB, 0); i < ord; ++i) wait(&sm.b_full[i % kExB], (i / kExB) & 1, kErrDrain);
  } else {
    // -------------------------------------------------------------------- base + acc, a row a thread
    const int group = warp >> 2;
    place = sm.place[row];
    float up = 1.f;
    if constexpr (F16) {
      pdl_wait();
      if (place >= 0) up = row_power(p, V, m0 + row);
    }
    uint32_t use = 0;
    for (int i = group; i < tiles && ok; i += 2) {
      const int s = i % kExBase;
      ok = wait(&sm.base_full[s], (i / kExBase) & 1, kErrWaitFull);
      for (int d = 0; d < found; ++d, ++use) {
        const uint32_t buf = use & 1;
        ok = wait(&sm.acc_full[group][buf], (use >> 1) & 1, kErrWaitAccum);
        if (!ok) break;
        tc_fence_after();
        const bool own = place == d;
        if (__any_sync(0xffffffffu, own)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t v[32];
            tmem_ld32(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 128 * group + 64 * buf + 32 * h, v);
            tc_wait_ld();
            if (own) {                         // rows without an adapter keep their base, bit for bit
              uint8_t* at = sm.base[s] + row * 128;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                uint4* q = reinterpret_cast<uint4*>(at + (((4 * h + c) ^ (row & 7)) << 4));
                const uint4 y = *q;
                uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                  const float2 f = unpack2<F16>(w[t]);
                  const float a0 = __uint_as_float(v[8 * c + 2 * t]), a1 = __uint_as_float(v[8 * c + 2 * t + 1]);
                  w[t] = F16 ? pack2<F16>(fmaf(a0, up, f.x), fmaf(a1, up, f.y)) : pack2<F16>(f.x + a0, f.y + a1);
                }
                *q = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.acc_empty[group][buf]);
      }
      if (!ok) break;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.added[s]);
    }
  }
  __syncwarp();
  __syncthreads();
  if (warp == kExWMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
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

// The kernels on tcgen05, by 128 rows, or those on mma.sync, by the adapters that lead in each 16 rows.  The
// former cost a product and a pass over the rows for each adapter that occurs in 128 of them, which only the
// device knows; at 32 rows an adapter or more, on average over all, it is few where requests' rows are
// neighbours.  (Beyond kMostRows the grid of the latter's shrink would end.)  K 4096, in us,
// mma.sync / tcgen05:
//   shrink (with the expand that fits), N 4096: 8 adapters, 257 rows of rank 32 11.5 / 18.6, 512 rows of rank 16 13.3 /
//     15.3, 1024 rows 22.2 / 18.7, 1024 rows of rank 64 28.6 / 19.7, 2048 rows 48.6 / 22.1; 1024 rows that take 64
//     adapters in turn 90 / 137
//   expand (with the shrink that fits), N 8192: 8 adapters, 256 rows of rank 16 11.0 / 13.2, 512 rows 16.3 / 16.9, 1024
//     rows 23.1 / 21.9, 2048 rows of rank 64 46.4 / 28.3, 4001 rows 64.9 / 41.1; 64 adapters in turn, 1024 rows 113 /
//     263, 2048 rows 209 / 317
constexpr int kFewRows = 512, kRowsAdapter = 32, kMostRows = 16384;
template <bool F16, int NT>
cudaError_t launch_rows(const LoraArgs& a, uint16_t* V, cudaStream_t stream) {
  // At least four steps of 32 a warp, up to 8 CTAs.  One CTA / this many (4), K 4096, in us: 3 rows
  // 7.6 / 5.9, 16 rows of 16 adapters 8.3 / 7.3, 64 rows of 48 25.8 / 22.4 (N 28672), 200 rows 34.9 / 39.9.
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
  // A small X leaves the tiles' clusters too little to share.  By 16 rows / by 128 rows, 8 adapters of rank 40, in
  // us: 965 x 896 12.5 / 13.6, 1024 x 512 10.9 / 12.6, 1024 x 1024 12.7 / 12.9, 2048 x 1024 16.5 / 14.5, 4096 x 512
  // 20.5 / 14.8, 1024 x 2048 16.0 / 14.2.
  const bool small = static_cast<int64_t>(a.M) * a.K < (1 << 20);
  if (!lora_many_rows(a.M, a.L) || (small && a.M <= kMostRows)) {
    if (a.r <= 32) return launch_rows<F16, 4>(a, V, stream);
    if (a.r <= 64) return launch_rows<F16, 8>(a, V, stream);
    return launch_rows<F16, 16>(a, V, stream);
  }
  const int tiles = (a.M + kTileRows - 1) / kTileRows, steps = (a.K + 63) / 64;
  // Two CTAs an SM, at least two steps of 64 each (at least four: 4096 x 512 16.2 us instead of 14.8).  One CTA /
  // this many (8), whole calls, K 4096, N 8192, in us: 1024 rows 49.8 / 21.9, 2048 rows of rank 64 46.0 / 28.3, 4001
  // rows 58.5 / 41.2.
  unsigned c = 1;
  while (c < 8 && static_cast<int>(tiles * c) < 2 * device_sm_count() && steps >= static_cast<int>(2 * c) * 2) c *= 2;
  const int box_ranks = std::min(64, (a.r + 15) / 16 * 16);
  const CUtensorMapDataType dt = F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap tx, ta;
  cudaError_t e = make_tmap_2d(&tx, dt, a.X, a.K, a.M, static_cast<uint64_t>(a.K) * 2, 64, kTileRows, CU_TENSOR_MAP_SWIZZLE_128B,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
  if (e == cudaSuccess)
    e = make_tmap_2d(&ta, dt, a.A, a.K, static_cast<uint64_t>(a.L) * a.r, static_cast<uint64_t>(a.K) * 2, 64, box_ranks,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
  constexpr size_t smem = sizeof(TileSmem) + 1024;
  if (e == cudaSuccess) e = set_smem_attr_once(reinterpret_cast<const void*>(k_lora_shrink_tile<F16>), smem);
  if (e != cudaSuccess) return e;
  return launch_cluster(k_lora_shrink_tile<F16>, dim3(c, tiles, (a.r + 63) / 64), 192, smem, c, stream, tx, ta, a, V, box_ranks);
}

template <bool F16>
cudaError_t expand_t(const LoraArgs& a, const uint16_t* V, bool base_ready, cudaStream_t stream) {
  const int64_t blocks = (a.M + 15) / 16, cols = (a.N + kCols - 1) / kCols;
  const int sms = device_sm_count();
  int ls = 0, lr = 0;
  int64_t span = 1;
  if (lora_many_rows(a.M, a.L) && a.N % 8 == 0) {
    // one wave: two CTAs an SM, with more than 64 ranks or V in two parts one
    const int64_t row_ctas = (a.M + kTileRows - 1) / kTileRows, tiles = (a.N + kExCols - 1) / kExCols;
    const int64_t across = std::max<int64_t>(1, (a.r <= 64 && !a.lo ? 2 : 1) * sms / row_ctas);
    span = (tiles + across - 1) / across;
    const dim3 grid(static_cast<unsigned>((tiles + span - 1) / span), static_cast<unsigned>(row_ctas));
    const CUtensorMapDataType dt = F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const uint64_t n = a.N, r = a.r;
    CUtensorMap tbase, ty, tv, tvl, tb;
    const uint64_t v_stride = static_cast<uint64_t>(a.r + a.lo) * 2;
    cudaError_t e = make_tmap_2d(&tbase, dt, a.base, n, a.M, n * 2, kExCols, kTileRows, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
    if (e == cudaSuccess) e = make_tmap_2d(&ty, dt, a.Y, n, a.M, n * 2, kExCols, kTileRows, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE);
    if (e == cudaSuccess) e = make_tmap_2d(&tvl, dt, V + a.lo, r, a.M, v_stride, 64, kTileRows, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
    if (e == cudaSuccess) e = make_tmap_2d(&tv, dt, V, r, a.M, v_stride, 64, kTileRows, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
    const uint64_t bd[4] = {r, n, static_cast<uint64_t>(a.L), 1}, bs[3] = {r * 2, n * r * 2, n * r * 2 * a.L};
    const uint32_t bb[4] = {64, kExCols, 1, 1};
    if (e == cudaSuccess) e = make_tmap_4d(&tb, dt, a.B, bd, bs, bb, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
    if (e != cudaSuccess) return e;
    const auto launch = [&](auto kern, size_t smem) {
      const cudaError_t se = set_smem_attr_once(reinterpret_cast<const void*>(kern), smem);
      if (se != cudaSuccess) return se;
      return launch_pdl(kern, grid, kExThreads, smem, stream, tbase, ty, tv, tvl, tb, a, V, static_cast<int>(span), base_ready ? 1 : 0);
    };
    if (a.lo) {
      if (a.r <= 64) return launch(k_lora_expand_tile<F16, 1, true>, sizeof(ExpandSmem<1, true>) + 1024);
      return launch(k_lora_expand_tile<F16, 2, true>, sizeof(ExpandSmem<2, true>) + 1024);
    }
    if (a.r <= 64) return launch(k_lora_expand_tile<F16, 1, false>, sizeof(ExpandSmem<1, false>) + 1024);
    return launch(k_lora_expand_tile<F16, 2, false>, sizeof(ExpandSmem<2, false>) + 1024);
  }
  // Subsets of the adapters, up to those that a block can hold, while there are few warps for the
  // SMs.  Row blocks: as many as there are.  8 warps a CTA, and column tiles enough for one wave of two
  // CTAs an SM.  No subsets / this rule / always all, K 4096, in us: 16 rows of 16 adapters, N 4096 10.2 / 7.3 /
  // 7.3, N 28672 14.4 / 11.8 / 11.8; 64 rows of 48, N 4096 14.7 / 11.3 / 11.3, N 28672 24.5 / 22.4 / 33.9; 200 rows,
  // N 14336 39.8 / 39.9 / 52.8.  One column tile a warp / this rule: 64 rows, N 28672 26.9 / 22.4.
  const int most = std::min(std::min(a.M, 16), a.L);
  while (ls < 3 && (1 << ls) < most && (blocks * cols << ls) < 24ll * sms) ++ls;
  while (lr + ls < 3 && (1 << lr) < blocks) ++lr;
  span = std::min<int64_t>(8, std::max<int64_t>(1, ((blocks * cols << ls) + 16 * sms - 1) / (16 * sms)));
  const int64_t per = (8 >> (lr + ls)) * span;
  const dim3 grid(static_cast<unsigned>((cols + per - 1) / per), static_cast<unsigned>((blocks + (1 << lr) - 1) >> lr));
  const auto launch = [&](void (*kern)(LoraArgs, const uint16_t*, int, int, int)) {
    const cudaError_t e = set_smem_attr_once(reinterpret_cast<const void*>(kern), kExpandSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, grid, 256, kExpandSmem, stream, a, V, lr, ls, static_cast<int>(span));
  };
  if (a.r <= 32) return launch(a.lo ? k_lora_expand<F16, 1, true> : k_lora_expand<F16, 1, false>);
  if (a.r <= 64) return launch(a.lo ? k_lora_expand<F16, 2, true> : k_lora_expand<F16, 2, false>);
  return launch(a.lo ? k_lora_expand<F16, 4, true> : k_lora_expand<F16, 4, false>);
}

}  // namespace

bool lora_many_rows(int64_t M, int64_t L) { return M > kFewRows && (M / kRowsAdapter >= L || M > kMostRows); }

// V, then the rows' powers of two (fp16).
size_t lora_scratch_bytes(int64_t M, int64_t v_width) {
  return (static_cast<size_t>(M) * v_width * sizeof(uint16_t) + 16 + static_cast<size_t>(M) * 2 * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_lora_shrink(int dtype, const LoraArgs& a, void* scratch, cudaStream_t stream) {
  uint16_t* V = static_cast<uint16_t*>(scratch);
  return dtype == kF16 ? shrink_t<true>(a, V, stream) : shrink_t<false>(a, V, stream);
}

cudaError_t launch_lora_expand(int dtype, const LoraArgs& a, void* scratch, bool base_ready, cudaStream_t stream) {
  const uint16_t* V = static_cast<const uint16_t*>(scratch);
  return dtype == kF16 ? expand_t<true>(a, V, base_ready, stream) : expand_t<false>(a, V, base_ready, stream);
}

}  // namespace wq

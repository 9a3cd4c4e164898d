// Norm of every query and key head, rotation by the token's position, and the write of keys and
// values to their places in a cache kept in pages -- one pass between the QKV projection and
// attention.
//
//   x' = x / sqrt(mean(x^2) + eps) * w        per head of d elements (w given; else x' = x)
//   pair (a, b) of the first `rot` elements -> (a c - b s, b c + a s), c and s from the row of
//   the table at the token's position; the rest of the head unrotated.
//
// Bandwidth-bound: every element is read once and written once.  A thread holds two 16-byte pieces
// of a head, chosen so that both elements of each pair are its own (half-split pairs: pieces j and
// j + rot/16; adjacent pairs: any, j and j + d/16), and d / 16 neighbouring lanes hold a head, so
// only the sum of squares takes shuffles.  With one piece a thread and the partners by shuffles the
// instructions, not the bytes, set the time (8192 tokens of 80 heads of 128: 88 us instead of 61).  Sums, norm and
// rotation are float32; each output is rounded once.  8192 tokens, 80 heads, with cache: 60.6 us, 5.6 TB/s of 340 MB;
// 2047 tokens, 40 heads, no cache: 9.4 us, 4.6 TB/s; one token: 2.0 us, a launch and two dependent loads (all in a
// graph, inputs not in L2).
#include "elem16.cuh"
#include "internal.h"

namespace wq {

__device__ uint32_t g_rope_err;

uint32_t rope_read_and_clear_error() {
  uint32_t v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_rope_err, sizeof(v));
  cudaMemcpyToSymbol(g_rope_err, &z, sizeof(z));
  return v;
}

namespace {

constexpr int kRopeThreads = 128;

// Source of element 8 c of a row (query heads, key heads, then value heads) of token t.
template <int D>
__device__ __forceinline__ const uint16_t* row_source(const RopeArgs& a, int64_t t, int row) {
  if (row < a.Hq) return a.Q + t * a.q_stride + static_cast<int64_t>(row) * D;
  if (row < a.Hq + a.Hkv) return a.K + t * a.k_stride + static_cast<int64_t>(row - a.Hq) * D;
  return a.V + t * a.v_stride + static_cast<int64_t>(row - a.Hq - a.Hkv) * D;
}

// Position of token t, forced into the table; slot, or -1 where nothing is written.
__device__ __forceinline__ int token_position(const RopeArgs& a, int64_t t) {
  int pos = __ldg(a.positions + t);
  if (static_cast<uint32_t>(pos) >= static_cast<uint32_t>(a.max_pos)) {
    atomicOr(&g_rope_err, kErrIndex);
    pos = min(max(pos, 0), a.max_pos - 1);
  }
  return pos;
}
__device__ __forceinline__ int token_slot(const RopeArgs& a, int64_t t) {
  if (!a.slots) return 0;
  const int slot = __ldg(a.slots + t);
  if (static_cast<int64_t>(slot) >= a.pages * a.page_size) {
    atomicOr(&g_rope_err, kErrIndex);
    return -1;
  }
  return slot;
}

// A thread's pieces of a head (in units of 8 elements), and whether they are turned.  Neighbouring
// threads have neighbouring pieces.
struct Pieces {
  int a, b;
  bool turn_a, turn_b;
};
template <int D>
__device__ __forceinline__ Pieces pieces(const RopeArgs& p, int j) {
  const int n = p.rot >> 4;                    // threads with half-split pairs
  if (p.interleaved) return {j, j + D / 16, 8 * j < p.rot, 8 * j + D / 2 < p.rot};
  if (j < n) return {j, j + n, true, true};
  return {j + n, j + D / 16, false, false};    // past rot: the first half of the rest, and the second
}

// cos / sin of a thread's 8 pairs.
struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ void load_turn(Turn& u, const RopeArgs& a, int pos, const Pieces& pc) {
  const float* row = a.cos_sin + static_cast<int64_t>(pos) * a.rot;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    if (!(q ? pc.turn_b : pc.turn_a)) continue;
    const int i = a.interleaved ? 4 * (q ? pc.b : pc.a) : 8 * pc.a + 4 * q;
    const float4 cv = __ldg(reinterpret_cast<const float4*>(row + i));
    const float4 sv = __ldg(reinterpret_cast<const float4*>(row + (a.rot >> 1) + i));
    u.c[4 * q] = cv.x, u.c[4 * q + 1] = cv.y, u.c[4 * q + 2] = cv.z, u.c[4 * q + 3] = cv.w;
    u.s[4 * q] = sv.x, u.s[4 * q + 1] = sv.y, u.s[4 * q + 2] = sv.z, u.s[4 * q + 3] = sv.w;
  }
}

template <bool F16>
__device__ __forceinline__ void unpack_piece(uint64_t (&f)[4], const uint4& x) {
  f[0] = unpack_pair<F16>(x.x), f[1] = unpack_pair<F16>(x.y), f[2] = unpack_pair<F16>(x.z), f[3] = unpack_pair<F16>(x.w);
}
template <bool F16>
__device__ __forceinline__ uint4 pack_piece(const uint64_t (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float2 v = unpair(f[q]);
    w[q] = pack2<F16>(v.x, v.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Two pieces of a head: norm, rotation, rounding.  All lanes of the warp take part.
template <bool F16, int D>
__device__ __forceinline__ void turn_pieces(const RopeArgs& a, uint4& xa, uint4& xb, const Turn& u, const uint16_t* weight,
                                            const Pieces& pc, bool is_v) {
  uint64_t fa[4], fb[4];
  unpack_piece<F16>(fa, xa);
  unpack_piece<F16>(fb, xb);
  if (a.q_weight || a.k_weight) {              // the same for the whole grid
    uint64_t sq = mul_pair(fa[0], fa[0]), sq2 = mul_pair(fb[0], fb[0]);
#pragma unroll
    for (int q = 1; q < 4; ++q) sq = fma_pair(fa[q], fa[q], sq), sq2 = fma_pair(fb[q], fb[q], sq2);
    const float2 s2 = unpair(add_pair(sq, sq2));
    float sum = s2.x + s2.y;
#pragma unroll
    for (int o = D / 32; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (weight && !is_v) {
      const float inv = rsqrtf(sum * (1.f / D) + a.eps);
      const uint64_t i2 = pair_f(inv, inv);
      uint64_t wa[4], wb[4];
      unpack_piece<F16>(wa, __ldg(reinterpret_cast<const uint4*>(weight) + pc.a));
      unpack_piece<F16>(wb, __ldg(reinterpret_cast<const uint4*>(weight) + pc.b));
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        fa[q] = mul_pair(fa[q], mul_pair(wa[q], i2));
        fb[q] = mul_pair(fb[q], mul_pair(wb[q], i2));
      }
    }
  }
  if (is_v) return;
  if (a.interleaved) {
    if (pc.turn_a) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 x = unpair(fa[q]);
        fa[q] = pair_f(fmaf(-x.y, u.s[q], x.x * u.c[q]), fmaf(x.x, u.s[q], x.y * u.c[q]));
      }
    }
    if (pc.turn_b) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 x = unpair(fb[q]);
        fb[q] = pair_f(fmaf(-x.y, u.s[4 + q], x.x * u.c[4 + q]), fmaf(x.x, u.s[4 + q], x.y * u.c[4 + q]));
      }
    }
  } else if (pc.turn_a) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint64_t c = pair_f(u.c[2 * q], u.c[2 * q + 1]), s = pair_f(u.s[2 * q], u.s[2 * q + 1]);
      const uint64_t n = pair_f(-u.s[2 * q], -u.s[2 * q + 1]), x = fa[q];
      fa[q] = fma_pair(fb[q], n, mul_pair(x, c));
      fb[q] = fma_pair(x, s, mul_pair(fb[q], c));
    }
  }
  xa = pack_piece<F16>(fa);
  xb = pack_piece<F16>(fb);
}

// Where a row goes; null where it is not written.
template <int D>
__device__ __forceinline__ uint16_t* row_target(const RopeArgs& a, int64_t t, int row, int slot) {
  if (row < a.Hq) return a.Qo + (t * a.Hq + row) * D;
  const bool is_v = row >= a.Hq + a.Hkv;
  const int h = is_v ? row - a.Hq - a.Hkv : row - a.Hq;
  if (!a.slots) return a.Ko + (t * a.Hkv + h) * D;
  if (slot < 0) return nullptr;
  const int64_t page = slot >> a.log_page;
  const int at = slot & (a.page_size - 1);
  return (is_v ? a.v_cache : a.k_cache) + (((page * a.Hkv + h) << a.log_page) + at) * D;
}

// Few tokens: one head a thread, nothing kept; the call is over in one round of loads.
template <bool F16, int D>
__global__ void __launch_bounds__(kRopeThreads) k_qk_norm_rope(const RopeArgs a) {
  constexpr int TPH = D / 16;                  // threads per head
  pdl_launch_dependents();
  pdl_wait();
  const int t = blockIdx.x, j = threadIdx.x % TPH;
  const Pieces pc = pieces<D>(a, j);
  const int rows = a.Hq + (a.slots ? 2 : 1) * a.Hkv, row = blockIdx.y * (kRopeThreads / TPH) + threadIdx.x / TPH;
  uint4 xa = make_uint4(0, 0, 0, 0), xb = xa;
  if (row < rows) {
    const uint4* src = reinterpret_cast<const uint4*>(row_source<D>(a, t, row));
    xa = src[pc.a], xb = src[pc.b];
  }
  const int slot = token_slot(a, t), pos = token_position(a, t);
  Turn u;
  load_turn(u, a, pos, pc);
  turn_pieces<F16, D>(a, xa, xb, u, row < a.Hq ? a.q_weight : a.k_weight, pc, row >= a.Hq + a.Hkv);
  uint4* dst = row < rows ? reinterpret_cast<uint4*>(row_target<D>(a, t, row, slot)) : nullptr;
  if (dst) dst[pc.a] = xa, dst[pc.b] = xb;
}

// Many tokens: a grid that fills the SMs once divides the (token, pass of heads) units evenly; the rows
// of the next units come through a queue in shared memory (each thread its own places: no barrier),
// the next token's cos / sin are in registers.  With a block for each token's share, 8 blocks an SM
// waited for two dependent rounds of loads each: 3.9 TB/s at 8192 tokens of 80 heads.
constexpr int kWalkThreads = 128, kWalkQueue = 8, kWalkCtas = 6;     // CTAs an SM
template <bool F16, int D>
__global__ void __launch_bounds__(kWalkThreads, kWalkCtas) k_qk_norm_rope_walk(const RopeArgs a, int passes) {
  constexpr int TPH = D / 16, HPB = kWalkThreads / TPH;
  __shared__ uint4 queue[kWalkQueue][2][kWalkThreads];
  pdl_launch_dependents();
  pdl_wait();
  const int j = threadIdx.x % TPH, r0 = threadIdx.x / TPH;
  const Pieces pc = pieces<D>(a, j);
  const int rows = a.Hq + (a.slots ? 2 : 1) * a.Hkv;
  // this CTA's share of all (token, pass) units
  const int64_t units = static_cast<int64_t>(a.T) * passes;
  const int64_t lo = units * blockIdx.x / gridDim.x;
  int left = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x - lo);
  int t = static_cast<int>(lo / passes), pass = static_cast<int>(lo - static_cast<int64_t>(t) * passes);
  int ft = t, fpass = pass, fleft = left, f_at = 0;      // the next unit to fetch
  const auto fetch = [&] {
    if (fleft > 0) {
      const int row = fpass * HPB + r0;
      const bool on = row < rows;
      const uint16_t* src = on ? row_source<D>(a, ft, row) : a.Q;
      copy16(&queue[f_at][0][threadIdx.x], on ? src + 8 * pc.a : src, on);
      copy16(&queue[f_at][1][threadIdx.x], on ? src + 8 * pc.b : src, on);
      --fleft;
      if (++fpass == passes) fpass = 0, ++ft;
      f_at = (f_at + 1) % kWalkQueue;
    }
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < kWalkQueue - 1; ++i) fetch();
  Turn now, next;
  int slot = token_slot(a, t);
  load_turn(now, a, token_position(a, t), pc);
  int pos_next = t + 1 < a.T ? token_position(a, t + 1) : 0;
  int at = 0;
#pragma unroll 1
  for (; left > 0; ++t, pass = 0) {
    int slot_next = 0;
    if (t + 1 < a.T) {
      load_turn(next, a, pos_next, pc);
      slot_next = token_slot(a, t + 1);
      if (t + 2 < a.T) pos_next = token_position(a, t + 2);
    }
#pragma unroll 1
    for (; pass < passes && left > 0; ++pass, --left) {
      const int row = pass * HPB + r0;
      fetch();
      copy_wait<kWalkQueue - 1>();
      uint4 xa = queue[at][0][threadIdx.x], xb = queue[at][1][threadIdx.x];
      turn_pieces<F16, D>(a, xa, xb, now, row < a.Hq ? a.q_weight : a.k_weight, pc, row >= a.Hq + a.Hkv);
      uint4* dst = row < rows ? reinterpret_cast<uint4*>(row_target<D>(a, t, row, slot)) : nullptr;
      if (dst) dst[pc.a] = xa, dst[pc.b] = xb;
      at = (at + 1) % kWalkQueue;
    }
    now = next, slot = slot_next;
  }
  copy_wait<0>();
}

template <bool F16, int D>
cudaError_t launch_rope_t(const RopeArgs& a, cudaStream_t stream) {
  constexpr int TPH = D / 16, HPB = kRopeThreads / TPH;
  static_assert(kRopeThreads == kWalkThreads, "both take the same heads a pass");
  const int rows = a.Hq + (a.slots ? 2 : 1) * a.Hkv, passes = (rows + HPB - 1) / HPB;
  const int fill = kWalkCtas * device_sm_count();
  // From eight units a CTA on the walk's set-up pays.  Without / with it, in us, keys and values into the cache
  // (measured as above): 32 + 8 heads of 128, 1024 tokens (3 units a CTA) 6.0 / 7.2, 2047 (7) 12.6 / 13.3, 4096 (13)
  // 24.5 / 22.2; 64 + 8 heads, 1024 tokens (6) 9.6 / 9.8, 2047 (11) 19.4 / 18.2, 4096 (22) 38.0 / 33.4; 16 + 16 heads
  // of 64, 2047 tokens (4) 7.0 / 7.8, 4096 (9) 15.7 / 14.9.  2047 tokens, 32 + 8 heads, no cache (6) 9.6 / 10.2.
  if (static_cast<int64_t>(a.T) * passes < 8ll * fill) return launch_pdl(k_qk_norm_rope<F16, D>, dim3(a.T, passes), kRopeThreads, 0, stream, a);
  return launch_pdl(k_qk_norm_rope_walk<F16, D>, dim3(fill), kWalkThreads, 0, stream, a, passes);
}

template <bool F16>
cudaError_t launch_rope_d(const RopeArgs& a, cudaStream_t stream) {
  if (a.d == 64) return launch_rope_t<F16, 64>(a, stream);
  if (a.d == 128) return launch_rope_t<F16, 128>(a, stream);
  return launch_rope_t<F16, 256>(a, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(int dtype, const RopeArgs& args, cudaStream_t stream) {
  RopeArgs a = args;
  a.log_page = 0;
  while (a.slots && (1 << a.log_page) < a.page_size) ++a.log_page;
  return dtype == kF16 ? launch_rope_d<true>(a, stream) : launch_rope_d<false>(a, stream);
}

}  // namespace wq

// Norm of every query and key head, rotation by the token's position, and the write of keys and
// values to their places in a cache kept in pages -- one pass between the QKV projection and
// attention.
//
//   x' = x / sqrt(mean(x^2) + eps) * w        per head of d elements (w given; else x' = x)
//   pair (a, b) of the first `rot` elements -> (a c - b s, b c + a s), c and s from the row of
//   the table at the token's position; the rest of the head unrotated.
//
// Bandwidth-bound: every element is read once and written once.  A thread holds 8 consecutive
// elements (one 16-byte access) and d / 8 neighbouring lanes hold a head, so the sum of squares
// and the partner of a half-split pair come by shuffles.  A thread keeps its place in the head
// and walks over heads of one token, so that its cos / sin values (64 bytes a thread, four times
// its data) are loaded once per token and not once per head.
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

// D: head elements.  HPT: heads a thread takes (all of one token).
template <bool F16, int D, int HPT>
__global__ void __launch_bounds__(kRopeThreads) k_qk_norm_rope(const RopeArgs a) {
  constexpr int TPH = D / 8;                     // threads per head
  constexpr int HPB = kRopeThreads / TPH;        // heads per pass of a block
  pdl_launch_dependents();
  pdl_wait();
  const int t = blockIdx.x;
  const int c = threadIdx.x % TPH;               // this thread's 8 elements: 8c .. 8c + 7
  const int rows = a.Hq + (a.slots ? 2 : 1) * a.Hkv;   // Q heads, K heads, then V heads
  const int row0 = blockIdx.y * (HPB * HPT) + threadIdx.x / TPH;

  int slot = 0;
  if (a.slots) {
    slot = __ldg(a.slots + t);
    if (static_cast<int64_t>(slot) >= a.pages * a.page_size) {
      if (threadIdx.x == 0) atomicOr(&g_rope_err, kErrIndex);
      slot = -1;
    }
  }
  uint4 x[HPT];
#pragma unroll
  for (int i = 0; i < HPT; ++i) {
    const int row = row0 + i * HPB;
    x[i] = make_uint4(0, 0, 0, 0);
    if (row < rows) {
      const uint16_t* src;
      if (row < a.Hq) src = a.Q + t * a.q_stride + static_cast<int64_t>(row) * D;
      else if (row < a.Hq + a.Hkv) src = a.K + t * a.k_stride + static_cast<int64_t>(row - a.Hq) * D;
      else src = a.V + t * a.v_stride + static_cast<int64_t>(row - a.Hq - a.Hkv) * D;
      x[i] = *reinterpret_cast<const uint4*>(src + 8 * c);
    }
  }
  int pos = __ldg(a.positions + t);
  if (static_cast<uint32_t>(pos) >= static_cast<uint32_t>(a.max_pos)) {
    if (threadIdx.x == 0) atomicOr(&g_rope_err, kErrIndex);
    pos = min(max(pos, 0), a.max_pos - 1);
  }
  // cos / sin of this thread's elements.  Half-split pairs (i, i + rot/2): element e uses index
  // e mod rot/2.  Adjacent pairs (2i, 2i + 1): element e uses index e / 2.
  const int half = a.rot >> 1;
  const bool turned = 8 * c < a.rot;             // rot is a multiple of 16
  float cs[8], sn[8];
  if (turned) {
    const float* row = a.cos_sin + static_cast<int64_t>(pos) * a.rot;
    if (a.interleaved) {
      const float4 cv = __ldg(reinterpret_cast<const float4*>(row + 4 * c));
      const float4 sv = __ldg(reinterpret_cast<const float4*>(row + half + 4 * c));
      const float cc[4] = {cv.x, cv.y, cv.z, cv.w}, ss[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        cs[2 * e] = cs[2 * e + 1] = cc[e];
        sn[2 * e] = sn[2 * e + 1] = ss[e];
      }
    } else {
      const int i0 = 8 * c < half ? 8 * c : 8 * c - half;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 cv = __ldg(reinterpret_cast<const float4*>(row + i0) + q);
        const float4 sv = __ldg(reinterpret_cast<const float4*>(row + half + i0) + q);
        cs[4 * q] = cv.x, cs[4 * q + 1] = cv.y, cs[4 * q + 2] = cv.z, cs[4 * q + 3] = cv.w;
        sn[4 * q] = sv.x, sn[4 * q + 1] = sv.y, sn[4 * q + 2] = sv.z, sn[4 * q + 3] = sv.w;
      }
      if (8 * c < half) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sn[e] = -sn[e];   // first of the pair: a c - b s
      }
    }
  }
  // lane holding the other half of a half-split pair (rot/2 is a multiple of 8)
  const int lane = threadIdx.x & 31;
  const int mate = a.interleaved || !turned ? lane : (8 * c < half ? lane + half / 8 : lane - half / 8);

#pragma unroll
  for (int i = 0; i < HPT; ++i) {
    const int row = row0 + i * HPB;
    const bool is_q = row < a.Hq, is_v = row >= a.Hq + a.Hkv;
    float f[8];
    {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 v = unpack2<F16>(w[q]);
        f[2 * q] = v.x;
        f[2 * q + 1] = v.y;
      }
    }
    const uint16_t* weight = is_q ? a.q_weight : a.k_weight;
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(f[e], f[e], sum);
#pragma unroll
    for (int o = TPH / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (weight && row < rows && !is_v) {
      const float inv = rsqrtf(sum * (1.f / D) + a.eps);
      const uint4 wv = __ldg(reinterpret_cast<const uint4*>(weight + 8 * c));
      const uint32_t w[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 v = unpack2<F16>(w[q]);
        f[2 * q] *= inv * v.x;
        f[2 * q + 1] *= inv * v.y;
      }
    }
    float g[8];
    if (a.interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        g[2 * e] = -f[2 * e + 1];
        g[2 * e + 1] = f[2 * e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] = __shfl_sync(0xffffffffu, f[e], mate);
    }
    if (turned && !is_v) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = fmaf(g[e], sn[e], f[e] * cs[e]);
    }
    if (row >= rows) continue;
    const uint4 y = is_v ? x[i] : make_uint4(pack2<F16>(f[0], f[1]), pack2<F16>(f[2], f[3]), pack2<F16>(f[4], f[5]),
                                              pack2<F16>(f[6], f[7]));
    uint16_t* dst;
    if (is_q) {
      dst = a.Qo + (static_cast<int64_t>(t) * a.Hq + row) * D;
    } else {
      const int h = is_v ? row - a.Hq - a.Hkv : row - a.Hq;
      if (a.slots) {
        if (slot < 0) continue;
        const int page = slot / a.page_size, at = slot % a.page_size;
        dst = (is_v ? a.v_cache : a.k_cache) + ((static_cast<int64_t>(page) * a.Hkv + h) * a.page_size + at) * D;
      } else {
        dst = a.Ko + (static_cast<int64_t>(t) * a.Hkv + h) * D;
      }
    }
    *reinterpret_cast<uint4*>(dst + 8 * c) = y;
  }
}

template <bool F16, int D>
cudaError_t launch_rope_t(const RopeArgs& a, cudaStream_t stream) {
  constexpr int HPB = kRopeThreads / (D / 8);
  const int rows = a.Hq + (a.slots ? 2 : 1) * a.Hkv;
  const auto grid = [&](int hpt) { return dim3(a.T, (rows + HPB * hpt - 1) / (HPB * hpt)); };
  if (a.T < 512) return launch_pdl(k_qk_norm_rope<F16, D, 1>, grid(1), kRopeThreads, 0, stream, a);
  return launch_pdl(k_qk_norm_rope<F16, D, 4>, grid(4), kRopeThreads, 0, stream, a);
}

template <bool F16>
cudaError_t launch_rope_d(const RopeArgs& a, cudaStream_t stream) {
  if (a.d == 64) return launch_rope_t<F16, 64>(a, stream);
  if (a.d == 128) return launch_rope_t<F16, 128>(a, stream);
  return launch_rope_t<F16, 256>(a, stream);
}

}  // namespace

cudaError_t launch_qk_norm_rope(int dtype, const RopeArgs& a, cudaStream_t stream) {
  return dtype == kF16 ? launch_rope_d<true>(a, stream) : launch_rope_d<false>(a, stream);
}

}  // namespace wq

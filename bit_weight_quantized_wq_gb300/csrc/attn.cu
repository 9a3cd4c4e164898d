// Attention of a batch whose requests share a long prefix, over a cache kept in pages.
//   o = softmax(scale q [Kp; Ks]^T) [Vp; Vs],  lse = log sum exp(scale q [Kp; Ks]^T)
// Kp, Vp: the shared prefix; Ks, Vs: the request's own keys, causal among its new tokens (the
// last of its own keys).
#include "elem16.cuh"
#include "internal.h"

namespace wq {

__device__ uint32_t g_attn_err;

uint32_t attn_read_and_clear_error() {
  uint32_t v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_attn_err, sizeof(v));
  cudaMemcpyToSymbol(g_attn_err, &z, sizeof(z));
  return v;
}

namespace {

// One warp per (request, new token, query head); lanes hold D / 32 elements each.
template <bool F16, int D>
__global__ void __launch_bounds__(256) k_attn_rows(const AttnArgs p) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int E = D / 32;
  const int r = blockIdx.x;
  const int h = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (h >= p.Hq) return;
  const int first = p.q_start ? p.q_start[r] : r;
  int n_new = p.q_start ? p.q_start[r + 1] - first : 1;
  if (n_new < 0 || n_new > p.max_new || first < 0 || first + n_new > p.T) {
    if (lane == 0) atomicOr(&g_attn_err, kErrIndex);
    return;
  }
  int len = p.max_blocks ? p.suffix_lens[r] : 0;
  if (len < 0 || len > p.max_blocks * p.page_size) {
    if (lane == 0) atomicOr(&g_attn_err, kErrIndex);
    len = min(max(len, 0), p.max_blocks * p.page_size);
  }
  const int kvh = h / (p.Hq / p.Hkv);
  for (int i = blockIdx.z; i < n_new; i += gridDim.z) {
    const int t = first + i;
    float q[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      q[e] = load1<F16>(p.Q + t * p.q_stride + static_cast<int64_t>(h) * D + E * lane + e) * p.scale;
      o[e] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    const int seen = max(0, len - n_new + i + 1);
    for (int j = 0; j < p.prefix_len + seen; ++j) {
      const int jj = j < p.prefix_len ? j : j - p.prefix_len;
      const int page = j < p.prefix_len ? p.prefix_pages[jj / p.page_size]
                                        : p.block_table[static_cast<int64_t>(r) * p.max_blocks + jj / p.page_size];
      if (page < 0 || page >= p.pages) {
        if (lane == 0) atomicOr(&g_attn_err, kErrIndex);
        continue;
      }
      const int64_t at = ((static_cast<int64_t>(page) * p.Hkv + kvh) * p.page_size + jj % p.page_size) * D + E * lane;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(q[e], load1<F16>(p.k_cache + at + e), s);
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
      const float m2 = fmaxf(m, s);
      const float base = m2 == -INFINITY ? 0.f : m2;
      const float keep = __expf(m - base), e1 = __expf(s - base);
      m = m2;
      l = l * keep + e1;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = o[e] * keep + e1 * load1<F16>(p.v_cache + at + e);
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
    for (int e = 0; e < E; ++e)
      p.O[(static_cast<int64_t>(t) * p.Hq + h) * D + E * lane + e] = round1<F16>(o[e] * inv);
    if (lane == 0 && p.lse) p.lse[static_cast<int64_t>(t) * p.Hq + h] = (m == -INFINITY ? 0.f : m) + logf(l);
  }
}

}  // namespace

size_t attn_workspace_bytes(int64_t T, int64_t R, int64_t Hq, int64_t Hkv, int64_t d, int64_t max_new) {
  (void)T, (void)R, (void)Hq, (void)Hkv, (void)d, (void)max_new;
  return kWsHeaderBytes;
}

cudaError_t launch_attn_shared_prefix(int dtype, const AttnArgs& a, void* ws, cudaStream_t stream) {
  (void)ws;
  const dim3 grid(a.R, (a.Hq + 7) / 8, a.max_new < 64 ? a.max_new : 64);
  if (dtype == kF16)
    return launch_pdl(a.d == 64 ? k_attn_rows<true, 64> : k_attn_rows<true, 128>, grid, 256, 0, stream, a);
  return launch_pdl(a.d == 64 ? k_attn_rows<false, 64> : k_attn_rows<false, 128>, grid, 256, 0, stream, a);
}

}  // namespace wq

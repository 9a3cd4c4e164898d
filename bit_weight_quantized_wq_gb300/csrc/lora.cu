// Low-rank adapters of many requests beside a shared projection:
//   Y[m] = base[m] + s[a] (X[m] A[a]^T) B[a]^T,   a = adapter[m];  a = -1: Y[m] = base[m].
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

// Adapter of row m and its rank rounded up to 8 (0: no adapter).
__device__ __forceinline__ int row_adapter(const LoraArgs& p, int m, int& rank) {
  const int a = __ldg(p.adapter + m);
  rank = 0;
  if (a < 0 || a >= p.L) {
    if (a != -1) atomicOr(&g_lora_err, kErrIndex);
    return -1;
  }
  rank = p.ranks ? __ldg(p.ranks + a) : p.r;
  if (rank < 0 || rank > p.r) {
    atomicOr(&g_lora_err, kErrIndex);
    rank = min(max(rank, 0), p.r);
  }
  rank = (rank + 7) & ~7;
  return a;
}

// V[m, j] = s X[m] . A[a, j], one CTA per row, one warp per j.
template <bool F16>
__global__ void __launch_bounds__(256) k_lora_shrink(const LoraArgs p, float* V) {
  pdl_launch_dependents();
  pdl_wait();
  const int m = blockIdx.x;
  int rank;
  const int a = row_adapter(p, m, rank);
  const int lane = threadIdx.x & 31;
  const uint4* x = reinterpret_cast<const uint4*>(p.X + static_cast<int64_t>(m) * p.K);
  for (int j = threadIdx.x >> 5; j < rank; j += 8) {
    const uint4* w = reinterpret_cast<const uint4*>(p.A + (static_cast<int64_t>(a) * p.r + j) * p.K);
    float sum = 0.f;
    for (int v = lane; v < p.K / 8; v += 32) {
      const uint4 xv = x[v], wv = w[v];
      const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w}, ws[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 f = unpack2<F16>(xs[q]), g = unpack2<F16>(ws[q]);
        sum = fmaf(f.x, g.x, fmaf(f.y, g.y, sum));
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) V[static_cast<int64_t>(m) * p.r + j] = sum * __ldg(p.scales + a);
  }
}

template <bool F16>
__global__ void __launch_bounds__(256) k_lora_expand(const LoraArgs p, const float* V) {
  pdl_launch_dependents();
  pdl_wait();
  const int m = blockIdx.x;
  const int n = blockIdx.y * 256 + threadIdx.x;
  if (n >= p.N) return;
  int rank;
  const int a = row_adapter(p, m, rank);
  float y = load1<F16>(p.base + static_cast<int64_t>(m) * p.N + n);
  if (rank > 0) {
    const uint4* b = reinterpret_cast<const uint4*>(p.B + (static_cast<int64_t>(a) * p.N + n) * p.r);
    const float* v = V + static_cast<int64_t>(m) * p.r;
    float sum = 0.f;
    for (int j = 0; j < rank / 8; ++j) {
      const uint4 bv = b[j];
      const uint32_t bs[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 g = unpack2<F16>(bs[q]);
        sum = fmaf(v[8 * j + 2 * q], g.x, fmaf(v[8 * j + 2 * q + 1], g.y, sum));
      }
    }
    y += sum;
  }
  if (a >= 0) p.Y[static_cast<int64_t>(m) * p.N + n] = round1<F16>(y);
  else p.Y[static_cast<int64_t>(m) * p.N + n] = p.base[static_cast<int64_t>(m) * p.N + n];
}

}  // namespace

size_t lora_scratch_bytes(int64_t M, int64_t K, int64_t N, int64_t r) {
  (void)K;
  (void)N;
  return (static_cast<size_t>(M) * r * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_lora_shrink(int dtype, const LoraArgs& a, void* scratch, cudaStream_t stream) {
  return launch_pdl(dtype == kF16 ? k_lora_shrink<true> : k_lora_shrink<false>, dim3(a.M), 256, 0, stream, a,
                    static_cast<float*>(scratch));
}

cudaError_t launch_lora_expand(int dtype, const LoraArgs& a, void* scratch, cudaStream_t stream) {
  return launch_pdl(dtype == kF16 ? k_lora_expand<true> : k_lora_expand<false>, dim3(a.M, (a.N + 255) / 256), 256, 0,
                    stream, a, static_cast<const float*>(scratch));
}

}  // namespace wq

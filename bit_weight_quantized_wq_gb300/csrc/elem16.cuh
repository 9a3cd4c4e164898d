// The two 16-bit element types of the attention-block operators (rope.cu, attn.cu, lora.cu) and
// the small helpers those kernels share.
#pragma once

#include "common.cuh"

namespace wq {

// Two packed 16-bit elements <-> two floats.  bf16 -> float is a shift, exact; the way back
// rounds to nearest even, once.
template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (F16) {
    const __half2 h = *reinterpret_cast<const __half2*>(&v);
    return __half22float2(h);
  } else {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <bool F16>
__device__ __forceinline__ float load1(const uint16_t* p) {
  if constexpr (F16) return __half2float(__ushort_as_half(*p));
  else return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}
template <bool F16>
__device__ __forceinline__ uint16_t round1(float v) {
  if constexpr (F16) return __half_as_ushort(__float2half_rn(v));
  else return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Launch with programmatic stream serialization: the CTAs may start while the previous kernel
// of the stream drains; the kernel reads and writes global memory only after pdl_wait().
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kern)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace wq

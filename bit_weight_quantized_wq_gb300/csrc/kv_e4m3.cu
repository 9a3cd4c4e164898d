// The cache of keys and values in 8 bits: new tokens quantized as they are written to their pages, and
// tokens read back in 16 bits.
//
//   e' = max(e, lowest exponent with amax <= 448 * 2^e')     per page and head; keys and values apart
//   code = E4M3(x * 2^-e')                                   nearest, ties to even
//
// amax is over the call's tokens of the page; e counts where the page holds tokens before them, and when
// e' > e those are re-encoded, code -> E4M3(code * 2^(e - e')).  With a power of two as the scale that is
// a shift of exponents: it loses what falls below the lowest steps of E4M3 and nothing else, so a page
// written token by token holds what one written at once holds, but for those steps.  (A free float32
// scale rounds every code again at each growth.)
#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "kv_e4m3.cuh"

namespace wq {

__device__ uint32_t g_kv_err;

uint32_t kv_read_and_clear_error() {
  uint32_t v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_kv_err, sizeof(v));
  cudaMemcpyToSymbol(g_kv_err, &z, sizeof(z));
  return v;
}

namespace {

// How many of key(0), .., key(n - 1), which ascend, are at most x; all THREADS threads of the CTA.  A round has them look at
// as many places, so that thousands of requests take two or three rounds.  (Where the keys do not ascend: some number.)
template <int THREADS, class Key>
__device__ __forceinline__ int count_up_to(int n, int x, const Key& key) {
  int lo = 0, hi = n;                          // the number lies in lo .. hi
  while (lo < hi) {
    const int step = (hi - lo + THREADS - 1) / THREADS, at = lo + step * static_cast<int>(threadIdx.x) + step - 1;
    const int in = __syncthreads_count(at < hi && key(at) <= x);
    lo += in * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

constexpr int kAppendThreads = 128;

// A page that the call writes: request r's block, its new tokens' rows and places.
struct Touched {
  int row, count;        // first of the call's rows, number of rows
  int place;             // of the first in the page; 0: the page starts afresh
  int page;              // -1: none
};

// Pages that request r's new tokens lie in; `first` and `n`: its rows.
__device__ __forceinline__ int touched_pages(const KvAppendArgs& a, int r, int& first, int& n, int& len, bool& bad) {
  first = a.q_start ? __ldg(a.q_start + r) : r;
  const int end = a.q_start ? __ldg(a.q_start + r + 1) : r + 1;
  len = __ldg(a.lens + r);
  n = end - first;
  bad = first < 0 || end < first || end > a.T || n > a.max_new || len < 0 || len > a.max_blocks << a.log_page;
  bad |= !bad && len > 0 && len < n;
  if (bad || n == 0 || len == 0) return 0;     // length 0: a row that pads a batch
  return ((len - 1) >> a.log_page) - ((len - n) >> a.log_page) + 1;
}

// Request r's index-th page of those that the call writes.
__device__ __forceinline__ Touched touched_page(const KvAppendArgs& a, int r, int first, int n, int len, int index) {
  Touched u;
  const int start = len - n, block = (start >> a.log_page) + index, lo = max(start, block << a.log_page);
  u.row = first + lo - start;
  u.count = min(len, (block + 1) << a.log_page) - lo;
  u.place = lo & (a.page_size - 1);
  u.page = __ldg(a.block_table + static_cast<int64_t>(r) * a.max_blocks + block);
  if (static_cast<uint32_t>(u.page) >= static_cast<uint32_t>(a.pages)) {
    atomicOr(&g_kv_err, kErrIndex);
    u.page = -1;
  }
  return u;
}

// How a CTA finds its page: each request has as many places (one, or two) whether it has pages for them or not; requests of
// up to a CTA's threads have their pages counted; more have places that begin at first_place, and the CTA searches.
enum class Find { kEach, kCount, kSearch };

// Where request r's places begin: n tokens lie in at most n / page_size + 2 pages, and in at most n.
__device__ __forceinline__ int first_place(const KvAppendArgs& a, int r, bool by_token) {
  const int row = __ldg(a.q_start + r);
  return by_token ? row : (row >> a.log_page) + 2 * r;
}

// The page of place `index`, if there is one; `places`: of each request (kEach), or 1: places by tokens (kSearch).
template <Find HOW>
__device__ __forceinline__ Touched find_touched(const KvAppendArgs& a, int index, int places) {
  int first = 0, n = 0, len = 0;
  bool bad = false;
  if constexpr (HOW == Find::kEach) {
    const int r = places == 1 ? index : index / places, j = index - r * places;
    const int c = touched_pages(a, r, first, n, len, bad);
    if (bad) atomicOr(&g_kv_err, kErrIndex);
    return j < c ? touched_page(a, r, first, n, len, j) : Touched{0, 0, 0, -1};
  } else if constexpr (HOW == Find::kSearch) {
    if (blockIdx.y == 0)                       // each CTA checks some of the requests
      for (int r = blockIdx.x * kAppendThreads + threadIdx.x; r < a.R; r += gridDim.x * kAppendThreads) {
        touched_pages(a, r, first, n, len, bad);
        if (bad) atomicOr(&g_kv_err, kErrIndex);
      }
    const int r = count_up_to<kAppendThreads>(a.R, index, [&](int i) { return first_place(a, i, places); }) - 1;
    if (r < 0) return Touched{0, 0, 0, -1};
    const int j = index - first_place(a, r, places), c = touched_pages(a, r, first, n, len, bad);
    return 0 <= j && j < c ? touched_page(a, r, first, n, len, j) : Touched{0, 0, 0, -1};
  } else {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = threadIdx.x;
    __shared__ int sums[kAppendThreads / 32];
    __shared__ Touched out;
    if (threadIdx.x == 0) out.page = -1;
    int c = 0;
    if (r < a.R) {
      c = touched_pages(a, r, first, n, len, bad);
      if (bad && blockIdx.x == 0 && blockIdx.y == 0) atomicOr(&g_kv_err, kErrIndex);
    }
    int in = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += v;
    }
    if (lane == 31) sums[warp] = in;
    __syncthreads();
    int at = in - c;
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w)
      if (w < warp) at += sums[w];
    if (at <= index && index < at + c) out = touched_page(a, r, first, n, len, index - at);
    __syncthreads();
    return out;
  }
}

// The lowest exponent with amax <= 448 * 2^e = 1.75 * 2^(e + 8), kept in the range.
__device__ __forceinline__ int scale_exponent(float amax) {
  if (amax <= 448.f * 5.421010862427522e-20f) return kScaleLow;     // 448 * 2^-64
  const uint32_t bits = __float_as_uint(amax);
  return min(static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0), kScaleHigh);
}

// N threads (a warp or the CTA) have a page of one head's keys or values: P pieces of 8 elements each.
// Large calls of prompts come near the bytes (2 read, 1 written an element): 31850 tokens of 8 heads of 128 in pages of 64 35.7
// us, 5.5 TB/s.  11006 tokens are two waves of CTAs, each of which loads a page, waits for its maximum, stores and ends: 18.8
// us, 3.6 TB/s, and some 12 where the tokens are in L2 still (there 256 threads a page and head took 13.6, 512 20.8: fewer
// bytes under way before a page's maximum is known).  Decoding is bound by launch and dependent loads (starts and
// lengths, then the page and the tokens): one token 2.1 us.
template <bool F16, int D, int N, int P, Find HOW>
__global__ void __launch_bounds__(kAppendThreads) k_kv_append(const KvAppendArgs a, int places) {
  constexpr int kRow = D / 8;                  // pieces a token
  constexpr uint32_t kInf = F16 ? 0x7c00u : 0x7f80u;
  __shared__ uint32_t tops[kAppendThreads / 32];
  pdl_launch_dependents();
  pdl_wait();
  const Touched u = find_touched<HOW>(a, blockIdx.x, places);
  if (u.page < 0) return;
  const int unit = blockIdx.y * (kAppendThreads / N) + threadIdx.x / N, j = threadIdx.x % N;
  const bool on = unit < 2 * a.Hkv;            // with N = 128 always
  const int head = on ? unit >> 1 : 0, is_v = unit & 1;
  uint8_t* scale_at = (is_v ? a.v_scales : a.k_scales) + static_cast<int64_t>(u.page) * a.Hkv + head;
  uint8_t* dst = (is_v ? a.v_cache : a.k_cache) + ((static_cast<int64_t>(u.page) * a.Hkv + head) << a.log_page) * D;
  const uint16_t* src = (is_v ? a.V : a.K) + u.row * (is_v ? a.v_stride : a.k_stride) + head * D;
  const int64_t stride = is_v ? a.v_stride : a.k_stride;
  const int pieces = on ? u.count * kRow : 0;
  const uint32_t old_byte = *scale_at;
  uint4 x[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int q = p * N + j;
    x[p] = q < pieces ? __ldg(reinterpret_cast<const uint4*>(src + (q / kRow) * stride + (q % kRow) * 8)) : make_uint4(0, 0, 0, 0);
  }
  uint32_t top2 = 0;                           // two magnitudes as 16-bit patterns, which order as the values do
#pragma unroll
  for (int p = 0; p < P; ++p)
    top2 = __vmaxu2(__vmaxu2(top2, __vmaxu2(x[p].x & 0x7fff7fffu, x[p].y & 0x7fff7fffu)),
                    __vmaxu2(x[p].z & 0x7fff7fffu, x[p].w & 0x7fff7fffu));
  const bool odd = max(top2 & 0xffffu, top2 >> 16) >= kInf;      // an infinity or a NaN among them
  uint32_t top = max(top2 & 0xffffu, top2 >> 16);
  if (odd) {                                   // the largest finite one instead
    top = 0;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        const uint32_t word = (&x[p].x)[w >> 1], m = (word >> (16 * (w & 1))) & 0x7fffu;
        if (m < kInf) top = max(top, m);
      }
  }
  top = __reduce_max_sync(0xffffffffu, top);
  if (N > 32) {
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kAppendThreads / 32; ++w) top = max(top, tops[w]);
  }
  const float amax = unpack2<F16>(top).x;
  int e = scale_exponent(amax);
  const int old = min(max(static_cast<int>(old_byte) - kScaleBias, kScaleLow), kScaleHigh);
  if (u.place > 0) e = max(e, old);
  if (!on) return;
  __syncwarp();                                // every lane has read the old scale (N = 128: the barrier above)
  if (j == 0) *scale_at = static_cast<uint8_t>(e + kScaleBias);
  const float down = pow2_normal(-e);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int q = p * N + j;
    if (q >= pieces) break;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f = unpack2<F16>((&x[p].x)[i]);
      f.x *= down, f.y *= down;
      if (odd) {                               // infinities are kept as NaN, not as large numbers
        if (isinf(f.x)) f.x = __uint_as_float(0x7fffffffu);
        if (isinf(f.y)) f.y = __uint_as_float(0x7fffffffu);
      }
      w[i] = f32_to_e4m3x2(f.x, f.y);
    }
    *reinterpret_cast<uint2*>(dst + u.place * D + q * 8) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
  }
  if (u.place > 0 && e > old) {                // the page's scale has grown: tokens held already
    const float shift = pow2_normal(max(old - e, -126));
    for (int q = j; q < u.place * (D / 16); q += N) {
      uint4* at = reinterpret_cast<uint4*>(dst) + q;
      uint4 c = *at;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t& w = (&c.x)[i];
        const float2 lo = unpack2<true>(e4m3_low(w)), hi = unpack2<true>(e4m3_high(w));
        w = f32_to_e4m3x2(lo.x * shift, lo.y * shift) | (f32_to_e4m3x2(hi.x * shift, hi.y * shift) << 16);
      }
      *at = c;
    }
  }
}

template <bool F16, int D, Find HOW>
cudaError_t launch_append_t(const KvAppendArgs& a, unsigned pages, int places, cudaStream_t stream) {
  const int pieces = std::min(a.page_size, a.max_new) * D / 8;
  if (pieces <= 4 * 32)
    return launch_pdl(k_kv_append<F16, D, 32, 4, HOW>, dim3(pages, (2 * a.Hkv + 3) / 4), kAppendThreads, 0, stream, a, places);
  const dim3 grid(pages, 2 * a.Hkv);
  if (pieces <= 8 * 128) return launch_pdl(k_kv_append<F16, D, 128, 8, HOW>, grid, kAppendThreads, 0, stream, a, places);
  return launch_pdl(k_kv_append<F16, D, 128, 16, HOW>, grid, kAppendThreads, 0, stream, a, places);
}

// Where no request can have more than two pages, as many places each: 512 requests of one token 8.3 us counted, 6.0 so.
// Counting, which every CTA does for itself, is a load less than a search while it is one round of a CTA's threads (7
// prompts in L2 12.3 / 12.8 us); 512 requests with two pieces of 512 tokens among them 38 / 25 us, 4096 677 / 136.
template <bool F16, int D>
cudaError_t launch_append_t(const KvAppendArgs& a, cudaStream_t stream) {
  const int each = 1 + (a.max_new + a.page_size - 2) / a.page_size;      // pages that max_new tokens of a request lie in
  if (each <= 2) return launch_append_t<F16, D, Find::kEach>(a, static_cast<unsigned>(a.R) * each, each, stream);
  const int64_t by_pages = a.T / a.page_size + 2ll * a.R;
  const unsigned pages = static_cast<unsigned>(std::min<int64_t>(a.T, by_pages));
  if (a.R <= kAppendThreads) return launch_append_t<F16, D, Find::kCount>(a, pages, 0, stream);
  return launch_append_t<F16, D, Find::kSearch>(a, pages, a.T <= by_pages, stream);
}

// ------------------------------------------------------------------------------- reading back
constexpr int kReadThreads = 256;

// Codes at scale byte `byte` as two packed elements of the output's type.  Most scales are exact in fp16 and reach no
// infinity (2^-14 .. 2^7): one product there.
template <bool F16>
__device__ __forceinline__ uint32_t scaled_pair(uint32_t f16x2, uint32_t byte, bool plain) {
  if (F16 && plain) {
    const __half2 s = __half2half2(__ushort_as_half(static_cast<uint16_t>((byte - kScaleBias + 15) << 10)));
    const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&f16x2), s);
    return *reinterpret_cast<const uint32_t*>(&y);
  }
  const float s = scale_value(byte);
  float2 f = unpack2<true>(f16x2);
  f.x *= s, f.y *= s;
  if (F16) {                                   // past the type's largest value: that value (NaN stays NaN)
    if (fabsf(f.x) > 65504.f) f.x = copysignf(65504.f, f.x);
    if (fabsf(f.y) > 65504.f) f.y = copysignf(65504.f, f.y);
  }
  return pack2<F16>(f.x, f.y);
}

// A CTA has TOK rows of the output, K or V; a thread 16 elements at a time (16 bytes in, 32 out).  Bound by reads and writes
// of HBM mixed once its instructions are few: with divisions for every unit, and fp16 by way of float32 and a clamp, the
// ALU was at 65%, and with a thread looking up its request's pages one after the other: 24 requests of up to 8191 tokens took
// 118 us, now 94 (6.4 TB/s of reads and writes).
template <bool F16, int D, int TOK, int kReadAhead>
__global__ void __launch_bounds__(kReadThreads) k_kv_read(const KvReadArgs a) {
  constexpr int kPieces = D / 16;
  __shared__ int64_t where[TOK];               // of each row: its token of head 0, counted in tokens of the cache; -1: none
  __shared__ int pages[TOK], requests[TOK], places[TOK];
  pdl_launch_dependents();
  pdl_wait();
  const int t0 = blockIdx.x * TOK, count = min(TOK, a.T - t0);
  if (threadIdx.x < TOK) requests[threadIdx.x] = -1;
  // The requests of its rows: a CTA looks at all of them, a thread one, or where there are more, for the first (that each CTA
  // went through all of them, 65536 requests of 4 tokens took 861 us, so 58; 16384 168, so 72; 4096 of one 14, so 9.5).
  const bool many = a.R > kReadThreads;
  int from = 0;
  if (many) from = max(0, count_up_to<kReadThreads>(a.R, t0, [&](int r) { return __ldg(a.starts + r); }) - 1);
  __syncthreads();
  for (int base = from; base < a.R; base += kReadThreads) {
    if (many && base > from && __ldg(a.starts + base) >= t0 + count) break;
    const int r = base + threadIdx.x;
    if (r >= a.R) continue;
    const int lo = __ldg(a.starts + r), hi = __ldg(a.starts + r + 1);
    if (lo < 0 || hi < lo || hi > a.T) {
      if (blockIdx.x == 0) atomicOr(&g_kv_err, kErrIndex);
      continue;
    }
    for (int t = max(lo, t0); t < min(hi, t0 + count); ++t) requests[t - t0] = r, places[t - t0] = t - lo;
  }
  if (many && blockIdx.y == 0)                 // each CTA checks some of them
    for (int r = blockIdx.x * kReadThreads + threadIdx.x; r < a.R; r += gridDim.x * kReadThreads) {
      const int lo = __ldg(a.starts + r), hi = __ldg(a.starts + r + 1);
      if (lo < 0 || hi < lo || hi > a.T) atomicOr(&g_kv_err, kErrIndex);
    }
  __syncthreads();
  if (threadIdx.x < TOK) {
    const int r = requests[threadIdx.x], pos = places[threadIdx.x], block = pos >> a.log_page;
    int64_t at = -1;
    if (r >= 0) {
      const int page = block < a.max_blocks ? __ldg(a.block_table + static_cast<int64_t>(r) * a.max_blocks + block) : -1;
      if (static_cast<uint32_t>(page) < static_cast<uint32_t>(a.pages)) {
        at = ((static_cast<int64_t>(page) * a.Hkv) << a.log_page) + (pos & (a.page_size - 1));
        pages[threadIdx.x] = page;
      } else {
        atomicOr(&g_kv_err, kErrIndex);
      }
    }
    where[threadIdx.x] = at;
  }
  __syncthreads();
  const uint8_t* cache = blockIdx.y ? a.v_cache : a.k_cache;
  const uint8_t* scales = blockIdx.y ? a.v_scales : a.k_scales;
  uint16_t* out = (blockIdx.y ? a.Vo : a.Ko) + static_cast<int64_t>(t0) * a.Hkv * D;
  const int per_token = a.Hkv * kPieces, units = count * per_token;
  const int step_t = kReadThreads / per_token, step_u = kReadThreads - step_t * per_token;
  int t = threadIdx.x / per_token, u = threadIdx.x - t * per_token;      // the unit's token, and its place among the token's
  for (int base = threadIdx.x; base < units; base += kReadThreads * kReadAhead) {
    uint4 c[kReadAhead];
    uint32_t byte[kReadAhead];
    bool on[kReadAhead];
#pragma unroll
    for (int i = 0; i < kReadAhead; ++i) {
      const int h = u / kPieces;
      const int64_t at = base + i * kReadThreads < units ? where[t] : -1;
      on[i] = at >= 0;
      c[i] = make_uint4(0, 0, 0, 0), byte[i] = kScaleBias;
      if (on[i]) {
        c[i] = __ldg(reinterpret_cast<const uint4*>(cache + (at + (static_cast<int64_t>(h) << a.log_page)) * D) + u % kPieces);
        byte[i] = __ldg(scales + static_cast<int64_t>(pages[t]) * a.Hkv + h);
      }
      t += step_t, u += step_u;
      if (u >= per_token) u -= per_token, ++t;
    }
#pragma unroll
    for (int i = 0; i < kReadAhead; ++i) {
      if (!on[i]) continue;
      const bool plain = byte[i] - (kScaleBias - 14) <= 14 + 7;
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t word = (&c[i].x)[k >> 1];
        w[k] = scaled_pair<F16>(k & 1 ? e4m3_high(word) : e4m3_low(word), byte[i], plain);
      }
      uint4* dst = reinterpret_cast<uint4*>(out) + 2ll * (base + i * kReadThreads);
      dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
      dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

template <bool F16, int D>
cudaError_t launch_read_t(const KvReadArgs& a, cudaStream_t stream) {
  // A CTA's threads have a unit each, so that a call is over in one round of loads, until there are enough CTAs for the
  // chain of loads before it to matter: 16 rows a CTA from 700000 units on.  4 / 16 / 32 rows, 8 heads of 128 (64 units a
  // row), in us: 700 rows 3.1 / 3.8 / 5.2, 6000 9.1 / 11.3 / 13.5, 12000 15.0 / 14.9 / 21, 30000 37 / 35 / 37, 98000 118 /
  // 94 / 97; 2 heads of 64 (8 units), 9000 rows 7.5 / 3.6 / 3.9, 18000 12.5 / 5.8 / 4.8, 45000 28 / 10.8 / 8.7.
  const int per_row = a.Hkv * D / 16;
  const auto read = [&](auto rows, auto ahead) {
    constexpr int n = decltype(rows)::value;
    return launch_pdl(k_kv_read<F16, D, n, decltype(ahead)::value>, dim3((a.T + n - 1) / n, 2), kReadThreads, 0, stream, a);
  };
  using One = std::integral_constant<int, 1>;
  if (per_row <= 12) return read(std::integral_constant<int, 32>(), One());
  if (static_cast<int64_t>(a.T) * per_row >= 700000) return read(std::integral_constant<int, 16>(), std::integral_constant<int, 2>());
  return read(std::integral_constant<int, 4>(), One());
}

int log2_of(int page_size) {
  int l = 0;
  while ((1 << l) < page_size) ++l;
  return l;
}

}  // namespace

cudaError_t launch_kv_append(int dtype, const KvAppendArgs& args, cudaStream_t stream) {
  KvAppendArgs a = args;
  a.log_page = log2_of(a.page_size);
  if (dtype == kF16) return a.d == 64 ? launch_append_t<true, 64>(a, stream) : launch_append_t<true, 128>(a, stream);
  return a.d == 64 ? launch_append_t<false, 64>(a, stream) : launch_append_t<false, 128>(a, stream);
}

cudaError_t launch_kv_read(int dtype, const KvReadArgs& args, cudaStream_t stream) {
  KvReadArgs a = args;
  a.log_page = log2_of(a.page_size);
  if (dtype == kF16) return a.d == 64 ? launch_read_t<true, 64>(a, stream) : launch_read_t<true, 128>(a, stream);
  return a.d == 64 ? launch_read_t<false, 64>(a, stream) : launch_read_t<false, 128>(a, stream);
}

}  // namespace wq

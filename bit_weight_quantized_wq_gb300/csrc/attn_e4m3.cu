// Attention over a cache of keys and values held in 8 bits: E4M3 codes in pages, a power-of-two scale
// for each page and head.
//   o = softmax(scale q K^T) V,  lse = log sum exp(scale q K^T),  causal among a request's new tokens
// With K = 2^ek Kc, V = 2^ev Vc (codes Kc, Vc; exponents of the key's page), c = scale log2(e):
//   x_j = c 2^ek (q . Kc_j) + ev,  w_j = 2^(x_j - m),  o = sum w_j Vc_j / sum w_j 2^-ev
// so a page's scales cost one multiply-add a score, and the weights w of the second product are largest
// where their products with the codes are, whatever the scales are: m follows the largest x, not the
// largest score.  Codes are exact in fp16.  A bf16 query is too, behind a power of two a row; w is rounded
// to fp16 (11 bits) for the second product, its sum kept in float32 unrounded.
//
// Work.  An item is up to 64 query rows of one request and key/value head (row = new token * G + query
// head of the group, G = Hq / Hkv) against the keys that its last row sees, in tiles of 64.  All items'
// tiles lie on one line, with a weight a tile and a constant an item; the line is cut into equal shares,
// one for each CTA.  A CTA's run of tiles may begin and end inside items: what it computes of such an
// item (a segment) goes to the workspace, unnormalised, and the last CTA that is done with the item
// joins its segments in line order.  A CTA has two such segments at most, its first and its last.
//
// The kernel: a warp has 16 rows and takes 16 keys at a time straight from global memory
// into the registers that mma.sync wants them in: for S = Q K^T a thread's 4 bytes along d are one
// fragment (Q is loaded in the same order of d), for O += P V the bytes of two keys are interleaved as
// they are widened, so V needs no transposition, and the scores' registers are P's.  4 warps: the row
// tiles of the item (1, 2 or 4), and the 16-key steps shared out among the warps of a row tile.
#include <algorithm>

#include "internal.h"
#include "kv_e4m3.cuh"

namespace wq {

__device__ uint32_t g_attn8_err;

uint32_t attn_e4m3_read_and_clear_error() {
  uint32_t v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_attn8_err, sizeof(v));
  cudaMemcpyToSymbol(g_attn8_err, &z, sizeof(z));
  return v;
}

namespace {

constexpr int kTile = 64;              // keys a tile of the line
constexpr int kStep = 16;              // keys a warp takes at a time (a page holds whole steps)
constexpr int kFewRows = 64;           // rows an item
constexpr int kFewThreads = 128, kFewWarps = 4, kFewCtas = 3;     // CTAs an SM
constexpr float kLazy = 8.f;           // the running maximum follows when it grew by more than 2^8 ...
constexpr float kUp = 7.f;             // ... and weights stand 2^7 higher, up to 2^15: fp16 reaches 2^-31 of the largest

struct Params {
  AttnE4m3Args a;
  int G, log_page;
  float c;                   // scale * log2(e)
  int* count;                // segments of the item that begins in a CTA which are done [ctas]
  float *po;                 // partials [cta][2][64][d], largest exponents and sums [cta][2][64][2]
  float2 *ml;
};

// One request's new tokens and keys, forced into range.
struct Request {
  int first, n, len;
  bool bad;
};
__device__ __forceinline__ Request request(const AttnE4m3Args& a, int r) {
  Request q;
  q.first = a.q_start ? __ldg(a.q_start + r) : r;
  const int end = a.q_start ? __ldg(a.q_start + r + 1) : r + 1;
  q.len = __ldg(a.lens + r);
  q.n = end - q.first;
  const int cap = a.max_blocks * a.page_size;
  q.bad = q.first < 0 || end < q.first || end > a.T || q.n > a.max_new || q.len < 0 || q.len > cap;
  if (q.first < 0 || end < q.first || end > a.T || q.n > a.max_new) q.n = 0, q.first = 0;
  q.len = min(max(q.len, 0), cap);
  return q;
}
// Keys that row `row` of the request sees.
__device__ __forceinline__ int keys_seen(const Request& q, int token) { return min(max(q.len - q.n + token + 1, 0), q.len); }

// The items of one request and head: row tiles, their key tiles and line lengths.
struct Shape {
  int rows, tiles, weight;
};
constexpr int kWItem = 12;
__device__ __forceinline__ int tile_weight(int rows) { return rows <= 16 ? 8 : rows <= 32 ? 12 : 20; }
__device__ __forceinline__ Shape shape(const Params& p, const Request& q, int rt) {
  Shape s;
  s.rows = min(kFewRows, q.n * p.G - rt * kFewRows);
  s.tiles = max(1, (keys_seen(q, (rt * kFewRows + s.rows - 1) / p.G) + kTile - 1) / kTile);
  s.weight = tile_weight(s.rows);
  return s;
}
__device__ __forceinline__ int row_tiles(const Params& p, const Request& q) { return (q.n * p.G + kFewRows - 1) / kFewRows; }
__device__ __forceinline__ long long head_cost(const Params& p, const Request& q) {
  long long c = 0;
  for (int rt = 0; rt < row_tiles(p, q); ++rt) {
    const Shape s = shape(p, q, rt);
    c += static_cast<long long>(s.tiles) * s.weight + kWItem;
  }
  return c;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16 bytes of the cache, read once.
__device__ __forceinline__ uint4 load_codes(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 load_codes8(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// The line's length and the request in which position b0 lies; all threads of the CTA.
struct Place {
  long long share, b0, at;   // line units a CTA; where this CTA's begins; where request r begins
  int r;                     // -1: nothing for this CTA
};
__device__ __forceinline__ Place find_place(const Params& p) {
  __shared__ long long sums[kFewWarps];
  __shared__ long long found_at;
  __shared__ int found_r;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long mine = 0, first_cost = 0;
  for (int r = threadIdx.x; r < p.a.R; r += kFewThreads) {
    const Request q = request(p.a, r);
    if (q.bad && blockIdx.x == 0) atomicOr(&g_attn8_err, kErrIndex);
    const long long c = p.a.Hkv * head_cost(p, q);
    if (r < kFewThreads) first_cost = c;
    mine += c;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) sums[warp] = mine;
  if (threadIdx.x == 0) found_r = -1, found_at = 0;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kFewWarps; ++w) total += sums[w];
  Place s;
  s.share = max(static_cast<long long>(tile_weight(kFewRows)), (total + gridDim.x - 1) / gridDim.x);
  s.b0 = blockIdx.x * s.share;
  long long before = 0;
  for (int base = 0; base < p.a.R && before <= s.b0 && s.b0 < total; base += kFewThreads) {
    const int r = base + threadIdx.x;
    const long long c = base == 0 ? first_cost : r < p.a.R ? p.a.Hkv * head_cost(p, request(p.a, r)) : 0;
    long long in = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += v;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = in;
    __syncthreads();
    long long at = before + in - c;
#pragma unroll
    for (int w = 0; w < kFewWarps; ++w) {
      if (w < warp) at += sums[w];
      before += sums[w];
    }
    if (at <= s.b0 && s.b0 < at + c) found_r = r, found_at = at;
  }
  __syncthreads();
  s.r = found_r, s.at = found_at;
  return s;
}

// First tile of an item (line start s, tiles n of weight w) that starts at or after position b.
__device__ __forceinline__ int tile_at(long long b, long long s, int n, int w) {
  if (b <= s) return 0;
  const long long d = b - s;
  return d >= static_cast<long long>(n) * w ? n : (static_cast<int>(d) + w - 1) / w;
}

template <int D>
struct FewSmem {
  // a warp's outputs: [row][D / 32 quarters of 32 columns], padded so that stores of 16 bytes fall on all banks
  static constexpr int kQuarter = D / 4 + 4, kRow = 4 * kQuarter;
  float o[kFewWarps][16][kRow];
  float2 ml[kFewWarps][16];
  int last;
};

template <bool F16, int D>
__global__ void __launch_bounds__(kFewThreads, kFewCtas) k_attn_e4m3(const __grid_constant__ Params p) {
  constexpr int KS = D / 16;                   // 16-wide steps of d
  constexpr int NT = D / 8;                    // 8-wide tiles of d
  __shared__ FewSmem<D> sm;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const Place place = find_place(p);
  if (place.r < 0) return;
  const long long b0 = place.b0, b1 = b0 + place.share;
  long long line = place.at;
  int r = place.r, kvh = 0, rt = 0;
  Request q = request(p.a, r);
  {                                            // heads before the share
    const long long head = head_cost(p, q);
    kvh = static_cast<int>((b0 - line) / head);
    line += kvh * head;
  }
#pragma unroll 1
  while (line < b1) {
    if (rt == row_tiles(p, q)) {               // on to the next item
      rt = 0;
      if (q.n == 0 || ++kvh == p.a.Hkv) {
        kvh = 0;
        if (++r == p.a.R) break;
        q = request(p.a, r);
      }
      continue;
    }
    const Shape it = shape(p, q, rt);
    const long long start = line;
    const int row0 = rt * kFewRows;
    line += static_cast<long long>(it.tiles) * it.weight + kWItem;
    ++rt;
    const int lo = tile_at(b0, start, it.tiles, it.weight), hi = tile_at(b1, start, it.tiles, it.weight);
    if (lo >= hi) continue;

    // ------------------------------------------------------------------ this warp's rows
    const int mt = it.rows <= 16 ? 1 : it.rows <= 32 ? 2 : 4, wk = kFewWarps / mt;
    const int m_tile = warp & (mt - 1), phase = warp / mt;
    const int row_base = m_tile * 16;          // within the item
    int lim[2];                                // keys that rows g and g + 8 see
    float crow[2];                             // c, times the power of two taken from the row's query
    uint32_t qf[KS][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = row_base + g + 8 * h;
      const bool valid = row < it.rows;
      const int tok = (row0 + row) / p.G, head = kvh * p.G + (row0 + row) - tok * p.G;
      lim[h] = valid ? keys_seen(q, tok) : 0;
      uint4 x[D / 32];
      const uint16_t* src = p.a.Q + (q.first + tok) * p.a.q_stride + head * D;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)         // 16 elements at 16 t, and for d = 128 at 64 + 16 t
        x[i] = valid ? __ldg(reinterpret_cast<const uint4*>(src + 64 * (i >> 1) + 16 * t) + (i & 1)) : make_uint4(0, 0, 0, 0);
      crow[h] = p.c;
      if (!F16) {
        uint32_t mx = 0;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu), __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu)));
        mx = max(mx & 0xffffu, mx >> 16);
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int k = bf16_to_f16_exponent(mx);
        const float down = pow2_normal(-k);
        crow[h] *= pow2_normal(k);
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const float2 f = unpack2<false>((&x[i].x)[w]);
            (&x[i].x)[w] = pack2<true>(f.x * down, f.y * down);
          }
      }
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        qf[s][h] = (&x[s >> 1].x)[2 * (s & 1)];
        qf[s][2 + h] = (&x[s >> 1].x)[2 * (s & 1) + 1];
      }
    }
    const int lim_top = __reduce_max_sync(0xffffffffu, max(lim[0], lim[1]));
    // lowest limit among the rows that exist
    const int lim_low = __reduce_min_sync(0xffffffffu, min(row_base + g < it.rows ? lim[0] : 0x7fffffff,
                                                           row_base + g + 8 < it.rows ? lim[1] : 0x7fffffff));

    // ------------------------------------------------------------------ its keys: steps of 16
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
    const int s0 = lo * (kTile / kStep) + phase, s1 = min(hi * (kTile / kStep), (lim_top + kStep - 1) / kStep);
    const int steps = s1 > s0 ? (s1 - s0 + wk - 1) / wk : 0;
    const int32_t* table = p.a.block_table + static_cast<int64_t>(r) * p.a.max_blocks;
    const int steps_log = p.log_page - 4;      // steps a page, log2

    // Lane i looks up step i of a window of 32: its page and the page's scales.
    int page_i = 0;
    uint32_t scale_i = 0;
    const auto look_up = [&](int base) {
      page_i = 0;
      if (base + lane < steps) {
        page_i = __ldg(table + ((s0 + (base + lane) * wk) >> steps_log));
        if (static_cast<uint32_t>(page_i) >= static_cast<uint32_t>(p.a.pages)) {
          atomicOr(&g_attn8_err, kErrIndex);
          page_i = 0;
        }
      }
      const int64_t at = static_cast<int64_t>(page_i) * p.a.Hkv + kvh;
      scale_i = __ldg(p.a.k_scales + at) | (static_cast<uint32_t>(__ldg(p.a.v_scales + at)) << 8);
    };
    // Bytes of a step's first key within the caches.
    const auto offset = [&](int j) {
      const int64_t page = __shfl_sync(0xffffffffu, page_i, j & 31);
      return (((page * p.a.Hkv + kvh) << p.log_page) + (((s0 + j * wk) << 4) & (p.a.page_size - 1))) * D;
    };
    uint4 kc[2][D / 64];                       // keys 4 (g / 2) + g % 2 and + 2; bytes 16 t and, for d = 128, 64 + 16 t
    uint32_t vc[4][D / 32];                    // keys 4 t .. 4 t + 3; bytes (D / 8) g ..
    const auto load_k = [&](int64_t at) {
      const uint8_t* src = p.a.k_cache + at + (4 * (g >> 1) + (g & 1)) * D + 16 * t;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < D / 64; ++i) kc[n][i] = load_codes(src + 2 * n * D + 64 * i);
    };
    const auto load_v = [&](int64_t at) {
      const uint8_t* src = p.a.v_cache + at + 4 * t * D + (D / 8) * g;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (D == 128) {
          const uint4 v = load_codes(src + i * D);
          vc[i][0] = v.x, vc[i][1] = v.y, vc[i][2] = v.z, vc[i][3] = v.w;
        } else {
          const uint2 v = load_codes8(src + i * D);
          vc[i][0] = v.x, vc[i][1] = v.y;
        }
      }
    };
    int64_t at = 0, at_next = 0;
    uint32_t scales = 0;
    if (steps > 0) {
      look_up(0);
      at = offset(0);
      scales = __shfl_sync(0xffffffffu, scale_i, 0);
      load_k(at);
      load_v(at);
    }
#pragma unroll 1
    for (int j = 0; j < steps; ++j) {
      const int key0 = (s0 + j * wk) << 4;
      // S = Q K^T: c[n][0..1] row g, keys 4 t + 2 n, + 1; c[n][2..3] row g + 8
      float s[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const uint32_t w = (&kc[n][k >> 2].x)[k & 3];
          mma16816(s[n], qf[k], e4m3_low(w), e4m3_high(w));
        }
      uint32_t scales_next = 0;
      if (j + 1 < steps) {
        if (((j + 1) & 31) == 0) look_up(j + 1);
        at_next = offset(j + 1);
        scales_next = __shfl_sync(0xffffffffu, scale_i, (j + 1) & 31);
        load_k(at_next);
      }
      const float k_scale = scale_value(scales & 0xffu), ev = static_cast<float>(static_cast<int>(scales >> 8) - kScaleBias);
      const float inv_v = scale_value(2 * kScaleBias - (scales >> 8));
      float x[2][4];                           // [row][key of the thread's four]
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float ck = crow[h] * k_scale;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[h][i] = fmaf(s[i >> 1][2 * h + (i & 1)], ck, ev);
      }
      if (key0 + kStep > lim_low) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (key0 + 4 * t + i >= lim[h]) x[h][i] = -INFINITY;
        if (key0 + kStep > q.len) {            // places behind the request's tokens hold anything
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (key0 + 4 * t + i >= q.len) {
#pragma unroll
              for (int w = 0; w < D / 32; ++w) vc[i][w] = 0;
            }
        }
      }
      const float top0 = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[0][2], x[0][3]));
      const float top1 = fmaxf(fmaxf(x[1][0], x[1][1]), fmaxf(x[1][2], x[1][3]));
      if (__any_sync(0xffffffffu, top0 > m[0] + kLazy || top1 > m[1] + kLazy)) {
        float keep[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float top = h ? top1 : top0;
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const bool grow = top > m[h] + kLazy;
          keep[h] = grow ? exp2_approx(m[h] - top) : 1.f;
          if (grow) m[h] = top;
          sum[h] *= keep[h];
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[n][0] *= keep[0], acc[n][1] *= keep[0], acc[n][2] *= keep[1], acc[n][3] *= keep[1];
      }
      uint32_t pf[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float base = kUp - (m[h] == -INFINITY ? 0.f : m[h]);
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = exp2_approx(x[h][i] + base);
        sum[h] = fmaf((w[0] + w[1]) + (w[2] + w[3]), inv_v, sum[h]);
        pf[h] = pack2<true>(w[0], w[1]);
        pf[2 + h] = pack2<true>(w[2], w[3]);
      }
      // O += P V: tile n has the thread's byte n, d = (D / 8) g + n of the fragment's column g
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t sel = half ? 0x7362u : 0x5140u;
          const uint32_t a = __byte_perm(vc[0][w], vc[1][w], sel), b = __byte_perm(vc[2][w], vc[3][w], sel);
          mma16816(acc[4 * w + 2 * half], pf, e4m3_low(a), e4m3_low(b));
          mma16816(acc[4 * w + 2 * half + 1], pf, e4m3_high(a), e4m3_high(b));
        }
      }
      if (j + 1 < steps) {
        load_v(at_next);
        scales = scales_next;
      }
    }

    // ------------------------------------------------------------------ the warps of a row tile
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
      sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
      if (t == 0) sm.ml[warp][g + 8 * h] = make_float2(m[h], sum[h]);
      // columns (D / 4) t .. + D / 4 of the row: acc[n][2 h] at n, acc[n][2 h + 1] at D / 8 + n
      float4* dst = reinterpret_cast<float4*>(&sm.o[warp][g + 8 * h][t * FewSmem<D>::kQuarter]);
#pragma unroll
      for (int n = 0; n < NT; n += 4) {
        dst[n / 4] = make_float4(acc[n][2 * h], acc[n + 1][2 * h], acc[n + 2][2 * h], acc[n + 3][2 * h]);
        dst[(NT + n) / 4] = make_float4(acc[n][2 * h + 1], acc[n + 1][2 * h + 1], acc[n + 2][2 * h + 1], acc[n + 3][2 * h + 1]);
      }
    }
    __syncthreads();
    const int c0 = static_cast<int>(start / place.share), c1 = static_cast<int>((start + static_cast<long long>(it.tiles - 1) * it.weight) / place.share);
    const bool whole = c0 == c1;
    const int cta = blockIdx.x;
    const auto finish = [&](int row, int col, const float4& o, float top, float total) {
      const float inv = total == 0.f ? 0.f : 1.f / total;
      const int tok = (row0 + row) / p.G, head = kvh * p.G + (row0 + row) - tok * p.G;
      const int64_t at_row = static_cast<int64_t>(q.first + tok) * p.a.Hq + head;
      *reinterpret_cast<uint2*>(p.a.O + at_row * D + col) =
          make_uint2(pack2<F16>(o.x * inv, o.y * inv), pack2<F16>(o.z * inv, o.w * inv));
      if (col == 0 && p.a.lse)
        p.a.lse[at_row] = total == 0.f ? -INFINITY : ((top == -INFINITY ? 0.f : top) - kUp + log2f(total)) * 0.6931471805599453f;
    };
    const int units = it.rows * (D / 4);       // four columns of a row
#pragma unroll 1
    for (int u = threadIdx.x; u < units; u += kFewThreads) {
      const int row = u / (D / 4), col = 4 * (u % (D / 4)), tile = row >> 4, in = row & 15;
      float top = -INFINITY, total = 0.f;
      for (int w = tile; w < kFewWarps; w += mt) top = fmaxf(top, sm.ml[w][in].x);
      const float ref = top == -INFINITY ? 0.f : top;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = tile; w < kFewWarps; w += mt) {
        const float2 ml = sm.ml[w][in];
        const float f = exp2_approx(ml.x - ref);
        total = fmaf(ml.y, f, total);
        const float4 v = *reinterpret_cast<const float4*>(&sm.o[w][in][(col / (D / 4)) * FewSmem<D>::kQuarter + col % (D / 4)]);
        o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
      }
      if (whole) {
        finish(row, col, o, top, total);
      } else {
        const int64_t at_row = (2ll * cta + (cta == c0 ? 1 : 0)) * kFewRows + row;
        *reinterpret_cast<float4*>(p.po + at_row * D + col) = o;
        if (col == 0) p.ml[at_row] = make_float2(top, total);
      }
    }
    if (!whole) {
      // the last CTA that is done with the item joins what all of them left, in line order
      __syncthreads();
      if (threadIdx.x == 0) {
        __threadfence();
        const int done = atomicAdd(p.count + c0, 1);
        sm.last = done == c1 - c0;
        if (sm.last) p.count[c0] = 0;
        __threadfence();
      }
      __syncthreads();
      if (sm.last) {
#pragma unroll 1
        for (int u = threadIdx.x; u < units; u += kFewThreads) {
          const int row = u / (D / 4), col = 4 * (u % (D / 4));
          const auto slot = [&](int c) { return (2ll * c + (c == c0 ? 1 : 0)) * kFewRows + row; };
          float top = -INFINITY, total = 0.f;
          for (int c = c0; c <= c1; ++c) top = fmaxf(top, __ldcg(&p.ml[slot(c)].x));
          const float ref = top == -INFINITY ? 0.f : top;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int c = c0; c <= c1; ++c) {
            const float2 ml = __ldcg(p.ml + slot(c));
            const float4 v = __ldcg(reinterpret_cast<const float4*>(p.po + slot(c) * D + col));
            const float f = exp2_approx(ml.x - ref);
            total = fmaf(ml.y, f, total);
            o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
          }
          finish(row, col, o, top, total);
        }
      }
    }
    __syncthreads();                           // shared memory is free again
  }
}

struct Layout {
  int ctas;
  size_t po, ml, bytes;
};

Layout layout(int64_t d) {
  Layout l{};
  l.ctas = kFewCtas * device_sm_count();
  size_t off = kWsHeaderBytes;
  const auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  const size_t rows = static_cast<size_t>(l.ctas) * 2 * kFewRows;
  l.po = take(rows * d * sizeof(float));
  l.ml = take(rows * sizeof(float2));
  l.bytes = off;
  return l;
}

template <bool F16, int D>
cudaError_t launch_t(const AttnE4m3Args& a, uint8_t* ws, cudaStream_t stream) {
  const Layout l = layout(D);
  Params p{};
  p.a = a;
  p.G = a.Hq / a.Hkv;
  p.log_page = 4;
  while ((1 << p.log_page) < a.page_size) ++p.log_page;
  p.c = a.scale * 1.4426950408889634f;
  p.count = reinterpret_cast<int*>(ws);        // the header's counters: zero, and left so
  p.po = reinterpret_cast<float*>(ws + l.po), p.ml = reinterpret_cast<float2*>(ws + l.ml);
  return launch_pdl(k_attn_e4m3<F16, D>, dim3(l.ctas), kFewThreads, 0, stream, p);
}

}  // namespace

size_t attn_e4m3_workspace_bytes(int64_t d) { return layout(d).bytes; }

cudaError_t launch_attn_e4m3(int dtype, const AttnE4m3Args& a, void* ws, cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  if (dtype == kF16) return a.d == 64 ? launch_t<true, 64>(a, w, stream) : launch_t<true, 128>(a, w, stream);
  return a.d == 64 ? launch_t<false, 64>(a, w, stream) : launch_t<false, 128>(a, w, stream);
}

}  // namespace wq

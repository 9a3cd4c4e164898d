// Attention over a cache of keys and values held in 8 bits: E4M3 codes in pages, a power-of-two scale
// for each page and head.
//   o = softmax(scale q K^T) V,  lse = log sum exp(scale q K^T),  causal among a request's new tokens
// With K = 2^ek Kc, V = 2^ev Vc (codes Kc, Vc; exponents of the key's page), c = scale log2(e):
//   x_j = c 2^ek (q . Kc_j) + ev,  w_j = 2^(x_j - m),  o = sum w_j Vc_j / sum w_j 2^-ev
// so a page's scales cost one multiply-add a score, and the weights w of the second product are largest
// where their products with the codes are, whatever the scales are: m follows the largest x, not the
// largest score.  Codes are exact in fp16.  A bf16 query is too, behind a power of two a row; w is rounded
// to fp16 for the second product, to 11 bits down to 2^-21 of the row's largest w and to steps of 2^-31 of that below: tensor
// cores take 16 bits, and float32 weights in two parts would double a product that prompts are bound by.  It shows where
// all that an element's result comes from has a w so small: pages of scales 2^21 below that of a page with zeros there.
// The sum of the w stays in float32, unrounded.  (Float32 ends 2^-133 below the largest w, so with exponents ev 100 apart
// what the sum loses of a key is below 2^-33 of the whole.)
//
// Work.  An item is a tile of query rows of one request and key/value head (row = new token * G + query
// head of the group, G = Hq / Hkv) against the keys that its last row sees, in tiles of 64.  All items'
// tiles lie on one line, with a weight a tile and a constant an item; the line is cut into equal shares,
// one for each CTA.  A CTA's run of tiles may begin and end inside items: what it computes of such an
// item (a segment) goes to the workspace, unnormalised, and the last CTA that is done with the item
// joins its segments in line order.  A CTA has two such segments at most, its first and its last.
// Two kernels share a call's requests, each with a line of its own: up to 32 rows a head (64 with heads of 64), and more.
//
// Few rows (k_attn_e4m3): a warp has 8 NR rows of the item (its row tile, one of two at most), and the warps of a
// row tile take the steps of 16 keys (32 where d is 64) in turn, copied by the warp itself with cp.async two steps
// ahead: 512 contiguous bytes a copy, kept in that order but for a swizzle of the 16-byte chunks.  (With each thread
// copying what it will read, in the fragments' order, a copy of 512 bytes took 26 passes of the shared memory instead
// of 4.)  Products are transposed, S^T = K Q^T and O^T = V^T P^T, so that eight rows fill a fragment of mma.sync: for
// the first a thread's 4 bytes along d are a fragment of K (Q is loaded in the same order of d), for the second the
// bytes of two keys are interleaved as they are widened, so V needs no transposition, and an 8 x 8 transposition in
// registers turns the scores into the fragment of P.  Bound by the bytes where requests are long: 64 requests over up to
// 16384 keys, 64 heads on 8, 174 us, 6.2 TB/s; a short call by its chain of loads, barriers and the join: one request
// over 500 keys 6.8 us, one over 131071 54 us.
#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "kv_e4m3.cuh"
#include "line.cuh"
#include "tcgen05.cuh"

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
constexpr float kLazy = 8.f;           // the running maximum follows when it grew by more than 2^8 ...
constexpr float kUp = 7.f;             // ... and weights stand 2^7 higher, up to 2^15: fp16 reaches 2^-31 of the largest

// n / d for 0 <= n < 2^31 by a multiplication: q = (hi(n mul) + n) >> shift with mul = 2^32 (2^shift - d) / d + 1.
struct Divisor {
  uint32_t mul, shift;
  Divisor(uint32_t d = 1) : shift(0) {
    while ((1u << shift) < d) ++shift;
    mul = static_cast<uint32_t>((static_cast<uint64_t>((1u << shift) - d) << 32) / d + 1);
    if (d == 1) mul = 0;
  }
  __device__ int of(int n) const { return static_cast<int>((__umulhi(n, mul) + static_cast<uint32_t>(n)) >> shift); }
};

struct Params {
  AttnE4m3Args a;
  int G, log_page;
  Divisor by_G;
  int few;                   // requests of up to so many rows are the first kernel's
  float c;                   // scale * log2(e)
  int* count;                // segments (or groups) that are done of the item, and of the group, that begins in a CTA [2][ctas]
  float *po;                 // partials [cta][2][rows of an item][d], largest exponents and sums [cta][2][rows][2]
  float2 *ml;
  bool beside;               // the kernel for few rows: behind the other one of the same call
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

// The lines: rows of an item, the weight of a tile (by the item's rows) and the constant of an item, which stands for
// its set-up, its output and its part of a join.  Measured: first line, 20 / 60 / 120 / 240, 48 requests of up to 4 new
// tokens 57.8 / 45.2 / 46.3 / 47.1 us and 64 single tokens over long caches 174.5 / 173.8 / 175.0 / 181.4; second line,
// 60 / 80 / 100 / 130 / 160, pieces of 3 prompts 405 / 399 / 402 / 405 / 408 us, prompts beside single tokens 72.8 / 73.3 /
// 73.5 / 74.1 / 74.6, 48 requests of up to 8 new tokens 85 / 87 / 89 / 92 / 96, 100 items of 1024 keys 44 / 39 / 37 / 38 / 38.
constexpr int kFewWarps = 4;           // of a CTA of the kernel for few rows
constexpr int few_most_rows(int d) { return d == 64 ? 64 : 32; }       // of a request's head in it
template <int NR>
struct FewLine {
  __device__ static bool takes(const Params& p, int rows) { return rows <= p.few; }
  // eight rows a warp: one row tile; sixteen: one or two, each with half of the warps, and items of up to 32 rows
  static constexpr int kThreads = 32 * kFewWarps, kRows = NR == 1 ? 8 : 32, kItem = 60, kMost = NR == 1 ? 8 : 12;
  __device__ static int weight(int rows) { return rows <= 8 * NR ? 8 : kMost; }
};

constexpr int kManyThreads = 512, kManyRows = 256;
struct ManyLine {
  __device__ static bool takes(const Params& p, int rows) { return rows > p.few; }
  static constexpr int kThreads = kManyThreads, kRows = kManyRows, kItem = 80, kMost = 10;
  __device__ static int weight(int rows) { return rows <= kManyRows / 2 ? 5 : kMost; }
};

// One item: row tile rt of a request and head.
struct Shape {
  int rows, tiles, weight;
};
template <class L>
__device__ __forceinline__ int row_tiles(const Params& p, const Request& q) {
  const int rows = q.n * p.G;
  return L::takes(p, rows) ? (rows + L::kRows - 1) / L::kRows : 0;
}
template <class L>
__device__ __forceinline__ Shape shape(const Params& p, const Request& q, int rt) {
  Shape s;
  s.rows = min(L::kRows, q.n * p.G - rt * L::kRows);
  s.tiles = max(1, (keys_seen(q, p.by_G.of(rt * L::kRows + s.rows - 1)) + kTile - 1) / kTile);
  s.weight = L::weight(s.rows);
  return s;
}
// Line length of row tile rt.
template <class L>
__device__ __forceinline__ long long item_cost(const Params& p, const Request& q, int rt) {
  const Shape s = shape<L>(p, q, rt);
  return static_cast<long long>(s.tiles) * s.weight + L::kItem;
}
// Line length of all row tiles of a head, by a thread.
template <class L>
__device__ __forceinline__ long long head_cost(const Params& p, const Request& q) {
  long long c = 0;
  for (int rt = 0; rt < row_tiles<L>(p, q); ++rt) c += item_cost<L>(p, q, rt);
  return c;
}
// The same where every lane of a warp has a request: those of many row tiles are added up by all lanes, one after the other.
template <class L>
__device__ __forceinline__ long long head_costs(const Params& p, const Request& q) {
  constexpr int kAlone = 4;
  const int rts = row_tiles<L>(p, q);
  long long c = rts <= kAlone ? head_cost<L>(p, q) : 0;
  for (uint32_t left = __ballot_sync(0xffffffffu, rts > kAlone); left; left &= left - 1) {
    const int from = __ffs(left) - 1, n = __shfl_sync(0xffffffffu, rts, from), lane = threadIdx.x & 31;
    Request x;
    x.n = __shfl_sync(0xffffffffu, q.n, from), x.len = __shfl_sync(0xffffffffu, q.len, from);
    long long sum = 0;
    for (int rt = lane; rt < n; rt += 32) sum += item_cost<L>(p, x, rt);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == from) c = sum;
  }
  return c;
}
__device__ __forceinline__ long long warp_scan(long long c) {      // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, c, o);
    if (lane >= o) c += v;
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

// The 8 x 8 transpose of a matrix of 16-bit elements held two a thread.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Byte offset of the 16 bytes `c` of key `key` in a stage as TMA's 128-byte swizzle leaves them: rows of 128 bytes
// (two keys where d is 64), the 8 chunks of a row exchanged by the row's number.
template <int D>
__device__ __forceinline__ int chunk_at(int key, int c) {
  const int row = key / (128 / D), chunk = D == 128 ? c : 4 * (key & 1) + c;
  return 128 * row + 16 * (chunk ^ (row & 7));
}
// The key of fragment row m among a piece's 16, chosen so that eight lanes' reads of K (keys of rows g) and of V
// (keys of rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9) fall on all banks.
template <int D>
__device__ __forceinline__ int key_of_row(int m) {
  return D == 128 ? m : 4 * ((m & 7) >> 1) + 2 * (m >> 3) + (m & 1);
}

// `bytes` (a multiple of 16) from a 16-byte aligned address on their way to L2.
__device__ __forceinline__ void prefetch_l2(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// The scales of keys behind a request's tokens, K | V << 8: 1.  (A page that is not the request's holds any bytes, and
// 0 and 255 times a weight of 0 are not 0.)
constexpr uint32_t kNoScale = kScaleBias | (kScaleBias << 8);

// 0xff in the bytes of four codes that are NaN.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); }

// Four codes of a key's values from element `col` on; 0 where its page is out of range.
__device__ __forceinline__ uint32_t value_codes(const Params& p, const int32_t* table, int head, int key, int d, int col) {
  const int page = __ldg(table + (key >> p.log_page));
  if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.a.pages)) return 0;
  const int64_t at = ((static_cast<int64_t>(page) * p.a.Hkv + head) << p.log_page) + (key & (p.a.page_size - 1));
  return __ldg(reinterpret_cast<const uint32_t*>(p.a.v_cache + at * d + col));
}

// A wait of a whole warp on a barrier in a ring, bounded as mbar_wait_short is; once one has run out, all others give up too.  `sleep_ns`: of
// a warp that is far ahead, so that it leaves the issue slots to others.
__device__ __forceinline__ bool stage_wait(uint64_t* bar, uint32_t parity, volatile int* failed, uint32_t code, uint32_t sleep_ns = 0) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const long long t0 = clock64();
  while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
    if (sleep_ns) __nanosleep(sleep_ns);
    if (__any_sync(0xffffffffu, *failed != 0)) return false;
    if (__any_sync(0xffffffffu, clock64() - t0 > 4000000000ll)) {
      atomicOr(&g_attn8_err, code);
      *failed = 1;
      return false;
    }
  }
  return true;
}

// The line's length and the request in which position b0 lies; all threads of the CTA.
struct Place {
  long long share, b0, b1;   // line units a CTA; where this CTA's begin and end
  long long at;              // where request r begins
  long long head;            // line length of a head of it
  int r;                     // -1: nothing for this CTA
};
template <class L>
__device__ __forceinline__ Place find_place(const Params& p) {
  constexpr int kWarps = L::kThreads / 32;
  __shared__ long long sums[kWarps];
  __shared__ long long found_at, found_head;
  __shared__ int found_r;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // Shares rounded up exactly for many rows, or cuts drift into items that fit the CTAs: 152 items of 512 keys 37 us, exactly
  // 23.  (For few rows that took 0.2 us and gave none.)
  const auto take = [&](Place& s, long long total) {
    s.share = line_share(total, gridDim.x, L::kMost, L::kRows == kManyRows);
    s.b0 = blockIdx.x * s.share, s.b1 = min(s.b0 + s.share, total);
  };
  // line length of a head of request r (none past the last); all lanes of the warp
  const auto cost_of = [&](int r) {
    Request q{0, 0, 0, false};
    if (r < p.a.R) q = request(p.a, r);
    if (q.bad && blockIdx.x == 0) atomicOr(&g_attn8_err, kErrIndex);
    return head_costs<L>(p, q);
  };
  Place s;
  if (p.a.R <= 32) {                           // every warp by itself
    const long long h = cost_of(lane), c = p.a.Hkv * h, in = warp_scan(c);
    take(s, __shfl_sync(0xffffffffu, in, 31));
    const uint32_t here = __ballot_sync(0xffffffffu, in - c <= s.b0 && s.b0 < in);
    s.r = here ? __ffs(here) - 1 : -1;
    s.at = __shfl_sync(0xffffffffu, in - c, max(s.r, 0));
    s.head = __shfl_sync(0xffffffffu, h, max(s.r, 0));
    return s;
  }
  long long mine = 0, first = 0;
  for (int base = 0; base < p.a.R; base += L::kThreads) {
    const long long h = cost_of(base + threadIdx.x);
    if (base == 0) first = h;
    mine += p.a.Hkv * h;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) sums[warp] = mine;
  if (threadIdx.x == 0) found_r = -1, found_at = 0, found_head = 0;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += sums[w];
  take(s, total);
  long long before = 0;
  for (int base = 0; base < p.a.R && before <= s.b0 && s.b0 < total; base += L::kThreads) {
    const int r = base + threadIdx.x;
    const long long h = base == 0 ? first : cost_of(r), c = p.a.Hkv * h, in = warp_scan(c);
    __syncthreads();
    if (lane == 31) sums[warp] = in;
    __syncthreads();
    long long at = before + in - c;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += sums[w];
      before += sums[w];
    }
    if (at <= s.b0 && s.b0 < at + c) found_r = r, found_at = at, found_head = h;
  }
  __syncthreads();
  s.r = found_r, s.at = found_at, s.head = found_head;
  return s;
}

// Counts this CTA's part of one step of a join; true in the CTA that is the last of n, which sees what the others have
// written, and leaves the counter at 0.  After a barrier of the CTA's writers, by one thread.
__device__ __forceinline__ bool last_part(int* count, int n) {
  int done;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(done) : "l"(count) : "memory");
  if (done + 1 < n) return false;
  *count = 0;
  return true;
}

// A segment: what one CTA has of an item.
struct Segment {
  Request q;
  int r, head, tile;               // request, key/value head, row tile
  Shape it;
  int lo, hi;                      // key tiles
  long long start;                 // the item's place on the line

  __device__ bool whole() const { return lo == 0 && hi == it.tiles; }
  // The CTAs that have the item's first and last tile.
  __device__ void ctas(long long share, int& c0, int& c1) const {
    c0 = quotient(start, share), c1 = quotient(start + static_cast<long long>(it.tiles - 1) * it.weight, share);
  }
  // Its stages of KEYS keys, up to the last key that the item's last row sees.
  template <class L, int KEYS>
  __device__ int stages(const Params& p, int& first) const {
    const int seen = keys_seen(q, p.by_G.of(tile * L::kRows + it.rows - 1));
    first = lo * (kTile / KEYS);
    return max(0, min(hi * (kTile / KEYS), (seen + KEYS - 1) / KEYS) - first);
  }
};

// Walks over the segments of one CTA's share of the line.  All lanes of a warp.
template <class L>
struct Walk {
  const Params& p;
  long long b0, b1, line;          // the share, and where the next item begins
  int r, kvh, rt, rts;             // the next item; row tiles of its request
  Request q;

  __device__ Walk(const Params& p_, const Place& s) : p(p_), b0(s.b0), b1(s.b1), line(s.at), r(s.r), kvh(0), rt(0) {
    q = request(p.a, r);
    rts = row_tiles<L>(p, q);
    kvh = quotient(b0 - line, s.head);               // heads before the share, and row tiles
    line += kvh * s.head;
    for (bool found = rts == 1; !found && rt < rts; rt += found ? 0 : 32) {
      const int lane = threadIdx.x & 31;
      const long long c = rt + lane < rts ? item_cost<L>(p, q, rt + lane) : 0, in = warp_scan(c);
      const uint32_t past = __ballot_sync(0xffffffffu, line + in > b0);
      found = past != 0;
      const int at = found ? __ffs(past) - 1 : 31;
      line += __shfl_sync(0xffffffffu, found ? in - c : in, at);
      if (found) rt += at;
    }
  }
  // To the first request from r on that has rows on this line, 32 at a time: a thousand of the other line lie between two
  // prompts of a batch (one at a time, prompts at both ends of 1024 decoding requests took 278 us, so 107).
  __device__ bool to_request() {
    for (; r < p.a.R; r += 32) {
      Request x{0, 0, 0, false};
      const int lane = threadIdx.x & 31;
      if (r + lane < p.a.R) x = request(p.a, r + lane);
      const uint32_t here = __ballot_sync(0xffffffffu, row_tiles<L>(p, x) > 0);
      if (here) {
        const int at = __ffs(here) - 1;
        r += at;
        q.first = __shfl_sync(0xffffffffu, x.first, at), q.n = __shfl_sync(0xffffffffu, x.n, at);
        q.len = __shfl_sync(0xffffffffu, x.len, at);
        rts = row_tiles<L>(p, q);
        return true;
      }
    }
    return false;
  }
  __device__ bool next(Segment& x) {
    while (line < b1) {
      if (rt == rts) {
        rt = 0;
        if (++kvh == p.a.Hkv) {
          kvh = 0, ++r;
          if (!to_request()) return false;
        }
      }
      const Shape it = shape<L>(p, q, rt);
      const long long start = line;
      line += static_cast<long long>(it.tiles) * it.weight + L::kItem;
      ++rt;
      x.lo = tile_at(b0, start, it.tiles, it.weight), x.hi = tile_at(b1, start, it.tiles, it.weight);
      if (x.lo < x.hi) {
        x.q = q, x.r = r, x.head = kvh, x.tile = rt - 1, x.it = it, x.start = start;
        return true;
      }
    }
    return false;
  }
};

// The warp that copies: stages of KEYS keys and values of all the CTA's items into a ring of N places (ring(i): where
// stage i's keys go, its values follow), and the scales of the stage's boxes to scales(i).  A box is what one copy
// takes: a page's run of up to KEYS keys.
template <class L, int D, int KEYS, int N, class Next, class Done, class Ring, class Scales>
__device__ __forceinline__ void copy_items(const Params& p, const CUtensorMap& tk, const CUtensorMap& tv, const Next& next, const Done& done,
                                           const Ring& ring, uint64_t* full, uint64_t* empty, const Scales& scales, int* failed) {
  const int lane = threadIdx.x & 31;
  uint32_t stage = 0;                          // of all items so far
  const uint64_t once = l2_policy_evict_first();
  const int box = min(p.a.page_size, KEYS), boxes = KEYS / box, log_box = 31 - __clz(box);
  bool ok = true;
  while (const Segment* seg = ok ? next() : nullptr) {
    const Segment& x = *seg;
    int first;
    const int n = x.template stages<L, KEYS>(p, first), len = x.q.len;
    const int32_t* table = p.a.block_table + static_cast<int64_t>(x.r) * p.a.max_blocks;
    // lane i has box base + i of the item; the table of the 32 after it is on its way
    const auto key_of = [&](int base) { return first * KEYS + ((base + lane) << log_box); };
    const auto held = [&](int base) { return base + lane < n * boxes && key_of(base) < len; };
    const auto table_at = [&](int base) { return held(base) ? __ldg(table + (key_of(base) >> p.log_page)) : 0; };
    int row = 0, ahead = table_at(0);
    uint32_t scale = 0;
#pragma unroll 1
    for (int j = 0; j < n; ++j, ++stage) {
      const int b0 = j * boxes;
      if ((b0 & 31) == 0) {
        int page = ahead;
        if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.a.pages)) {
          atomicOr(&g_attn8_err, kErrIndex);
          page = 0;
        }
        row = page * p.a.Hkv + x.head;
        scale = kNoScale;
        if (held(b0)) scale = __ldg(p.a.k_scales + row) | (static_cast<uint32_t>(__ldg(p.a.v_scales + row)) << 8);
        ahead = table_at(b0 + 32);
      }
      const int s = stage % N;
      ok = stage_wait(&empty[s], ((stage / N) & 1) ^ 1, failed, kErrWaitEmpty);
      if (!ok) break;
      const int mine = lane - (b0 & 31);
      if (mine >= 0 && mine < boxes) scales(stage)[mine] = static_cast<uint16_t>(scale);
      int rows[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) rows[i] = __shfl_sync(0xffffffffu, row, (b0 + i) & 31);
      // boxes with a key of the request
      const int count = min(boxes, (len - (first + j) * KEYS + box - 1) >> log_box);
      __syncwarp();
      if (elect_one()) {
        mbar_arrive_expect_tx(&full[s], 2 * count * box * D);
        uint8_t* dst = ring(stage);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < count) {
            const int in_page = (((first + j) * KEYS + (i << log_box)) & (p.a.page_size - 1)) * D / 128;
            tma_load_4d(dst + i * box * D, &tk, 0, in_page, 0, rows[i], &full[s], once);
            tma_load_4d(dst + KEYS * D + i * box * D, &tv, 0, in_page, 0, rows[i], &full[s], once);
          }
      }
      __syncwarp();
    }
    if (ok) done();
  }
  // the last fill of each place has landed before the CTA's memory goes
  for (uint32_t i = stage > N ? stage - N : 0; i < stage; ++i)
    mbar_wait_short(&full[i % N], (i / N) & 1, &g_attn8_err, kErrDrain);
}

constexpr int kStages = 3;             // steps of a warp in shared memory, two of them under way
constexpr int kStepBytes = 2048;       // of K, and of V
template <int D, int NR>
struct FewSmem {
  static constexpr int kRow = D + 4;
  union {
    uint8_t ring[kFewWarps][kStages][2][kStepBytes];   // K, V
    float o[kFewWarps][8 * NR][kRow];                  // the warps' outputs, once their steps are done
  };
  float2 ml[kFewWarps][8 * NR];
  int last;
};

// Codes global -> shared memory.
__device__ __forceinline__ void copy_codes(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// CTAs an SM: as many as there are registers for (with 12 warps of 168 registers for eight rows, 64 requests over up to
// 16384 keys took 204 us instead of 174: the kernel is bound by what its warps wait for).
constexpr int few_ctas(int nr) { return nr == 1 ? 4 : 3; }

template <bool F16, int D, int NR>
__global__ void __launch_bounds__(FewLine<NR>::kThreads, few_ctas(NR)) k_attn_e4m3(const __grid_constant__ Params p) {
  using L = FewLine<NR>;
  using S = FewSmem<D, NR>;
  constexpr int kKeys = kStepBytes / D;        // of a step
  constexpr int kPieces = kKeys / 16;
  constexpr int KS = D / 16;                   // 16-wide steps of d, and 16-row tiles of V^T
  constexpr int R2 = 2 * NR;                   // rows that a thread has scores of: 2 t, 2 t + 1 (and 8 more each)
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  pdl_launch_dependents();
  // Behind the kernel for many rows this one need not wait: that one lets it start after its own wait, and the two share
  // nothing.  It does not end before that one, so that what waits for this call waits for both.
  if (!p.beside) pdl_wait();
  // where this lane's copies go: chunk 32 i + lane of a step is chunk lane % 8 of row 4 i + lane / 8 of 128 bytes
  const uint32_t ring = smem_u32(sm.ring[warp][0][0]);
  const uint32_t to_even = 128 * (lane >> 3) + 16 * ((lane & 7) ^ (lane >> 3)), to_odd = to_even ^ 64;
  const uint8_t *k_lane = p.a.k_cache + 16 * lane, *v_lane = p.a.v_cache + 16 * lane;
  const Place place = find_place<L>(p);
  if (place.r < 0) {
    pdl_wait();
    return;
  }
  Walk<L> walk(p, place);
  Segment seg;
#pragma unroll 1
  while (walk.next(seg)) {
    const Request& q = seg.q;
    const Shape& it = seg.it;
    const int kvh = seg.head;
    // ------------------------------------------------------------------ this warp's rows
    const int mt = NR > 1 && it.rows > 8 * NR ? 2 : 1, wk = kFewWarps / mt;
    // the item's first row (below, rows are counted from it); 0 where one item has all
    const int row0 = NR > 1 && few_most_rows(D) > L::kRows ? seg.tile * L::kRows : 0;
    const int row_base = (warp & (mt - 1)) * 8 * NR, phase = warp / mt;
    // the most keys that a row of the warp sees, and the fewest
    const int lim_top = keys_seen(q, p.by_G.of(row0 + min(it.rows, row_base + 8 * NR) - 1)), lim_low = keys_seen(q, p.by_G.of(row0 + row_base));
    uint4 raw[NR][D / 32];                     // elements (D / 4) t .. of rows g and g + 8
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const int row = row_base + 8 * n + g, tok = p.by_G.of(row0 + row), head = kvh * p.G + row0 + row - tok * p.G;
      const uint16_t* src = p.a.Q + (q.first + tok) * p.a.q_stride + head * D + (D / 4) * t;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) raw[n][i] = row < it.rows ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0, 0, 0, 0);
    }
    int first;
    const int n_steps = seg.template stages<L, kKeys>(p, first);
    const int s0 = first + phase, s1 = min(first + n_steps, (lim_top + kKeys - 1) / kKeys);
    const int steps = s1 > s0 ? (s1 - s0 + wk - 1) / wk : 0;
    const int32_t* table = p.a.block_table + static_cast<int64_t>(seg.r) * p.a.max_blocks;

    // Lane i looks up piece i (16 keys) of a window of 32: its page, as the piece's place in the caches (16 D bytes
    // each: as many as memory can hold fit 32 bits), and the page's scales; the table of the window after it is on its
    // way, the scales of the one before it are kept for the steps that the copies are ahead.
    const auto key_of = [&](int piece) { return (s0 + (piece / kPieces) * wk) * kKeys + 16 * (piece % kPieces); };
    const auto held = [&](int base) { return base + lane < steps * kPieces && key_of(base + lane) < q.len; };
    const auto table_at = [&](int base) { return held(base) ? __ldg(table + (key_of(base + lane) >> p.log_page)) : 0; };
    int page_next = table_at(0);
    uint32_t piece_i = 0, scale_i = 0, scale_before = 0;
    const auto look_up = [&](int base) {
      int page = page_next;
      if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.a.pages)) {
        atomicOr(&g_attn8_err, kErrIndex);
        page = 0;
      }
      const uint32_t at = static_cast<uint32_t>(page) * p.a.Hkv + kvh;
      piece_i = (at << (p.log_page - 4)) + ((key_of(base + lane) & (p.a.page_size - 1)) >> 4);
      scale_before = scale_i;
      scale_i = kNoScale;
      if (held(base)) scale_i = __ldg(p.a.k_scales + at) | (static_cast<uint32_t>(__ldg(p.a.v_scales + at)) << 8);
      page_next = table_at(base + 32);
    };
    const auto issue = [&](int j) {
      if (j < steps) {
        if (((j * kPieces) & 31) == 0) look_up(j * kPieces);
        const uint32_t slot = ring + (j % kStages) * (2 * kStepBytes);
#pragma unroll
        for (int h = 0; h < kPieces; ++h) {
          const uint32_t piece = __shfl_sync(0xffffffffu, piece_i, (j * kPieces + h) & 31);
          const uint8_t *k = k_lane + static_cast<uint64_t>(piece) * (16 * D), *v = v_lane + static_cast<uint64_t>(piece) * (16 * D);
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {   // 16 keys are D contiguous chunks
            const uint32_t dst = slot + (i & 1 ? to_odd : to_even) + 16 * D * h + 512 * i;
            copy_codes(dst, k + 512 * i);
            copy_codes(dst + kStepBytes, v + 512 * i);
          }
        }
      }
      copy_commit();
    };
#pragma unroll
    for (int j = 0; j < kStages - 1; ++j) issue(j);
    uint32_t qf[KS][NR][2];
    float crow[R2];                            // c, times the power of two taken from the row's query
    int lim[R2];                               // keys that the row sees
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      uint4(&x)[D / 32] = raw[n];
      float c = p.c;
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
        c *= pow2_normal(k);
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
        qf[s][n][0] = (&x[s >> 1].x)[2 * (s & 1)];
        qf[s][n][1] = (&x[s >> 1].x)[2 * (s & 1) + 1];
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        crow[2 * n + i] = F16 ? p.c : __shfl_sync(0xffffffffu, c, 4 * (2 * t + i));
        const int mine = row_base + 8 * n + 2 * t + i;
        lim[2 * n + i] = mine < it.rows ? keys_seen(q, p.by_G.of(row0 + mine)) : 0;
      }
    }

    // ------------------------------------------------------------------ its steps
    float acc[KS][NR][4];
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int n = 0; n < NR; ++n) acc[j][n][0] = acc[j][n][1] = acc[j][n][2] = acc[j][n][3] = 0.f;
    float m[R2], sum[R2];
#pragma unroll
    for (int i = 0; i < R2; ++i) m[i] = -INFINITY, sum[i] = 0.f;
    uint32_t odd = 0;                          // NaN that were taken out of values
#pragma unroll 1
    for (int j = 0; j < steps; ++j) {
      // the scales of step j: the look-ups may be a window ahead
      uint32_t scales[kPieces];
#pragma unroll
      for (int h = 0; h < kPieces; ++h) {
        const int piece = j * kPieces + h, ahead = min(j + kStages - 2, steps - 1) * kPieces;
        scales[h] = __shfl_sync(0xffffffffu, (piece >> 5) == (ahead >> 5) ? scale_i : scale_before, piece & 31);
      }
      __syncwarp();                            // all lanes have read the step before
      issue(j + kStages - 1);
      copy_wait<kStages - 1>();
      __syncwarp();                            // all lanes' copies are there
      const uint8_t *k_at = sm.ring[warp][j % kStages][0], *v_at = sm.ring[warp][j % kStages][1];
      const int key0 = (s0 + j * wk) * kKeys;
      // S^T = K Q^T: s[h][n][0 .. 1] the key of row g, query rows 2 t, 2 t + 1; s[h][n][2 .. 3] that of row g + 8
      float s[kPieces][NR][4];
#pragma unroll
      for (int h = 0; h < kPieces; ++h) {
        uint4 k[2][D / 64];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int w = 0; w < D / 64; ++w)
            k[i][w] = *reinterpret_cast<const uint4*>(k_at + 16 * D * h + chunk_at<D>(key_of_row<D>(g + 8 * i), (D / 64) * t + w));
        float odd[NR][4];                    // two sums, so that products need not wait for one another
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[h][n][i] = odd[n][i] = 0.f;
#pragma unroll
        for (int c = 0; c < KS; ++c) {
          const uint32_t w0 = (&k[0][c >> 2].x)[c & 3], w1 = (&k[1][c >> 2].x)[c & 3];
          const uint32_t a[4] = {e4m3_low(w0), e4m3_low(w1), e4m3_high(w0), e4m3_high(w1)};
#pragma unroll
          for (int n = 0; n < NR; ++n) mma16816(NR == 1 && (c & 1) ? odd[n] : s[h][n], a, qf[c][n][0], qf[c][n][1]);
        }
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (NR == 1) s[h][n][i] += odd[n][i];
      }
      float x[kPieces][R2][2];               // [row][key of row g, g + 8]
      const bool edge = key0 + 16 * kPieces > lim_low;
#pragma unroll
      for (int h = 0; h < kPieces; ++h) {
        const float k_scale = scale_value(scales[h] & 0xffu), ev = static_cast<float>(static_cast<int>(scales[h] >> 8) - kScaleBias);
#pragma unroll
        for (int i = 0; i < R2; ++i) {
          const float ck = crow[i] * k_scale;
#pragma unroll
          for (int e = 0; e < 2; ++e) x[h][i][e] = fmaf(s[h][i >> 1][2 * e + (i & 1)], ck, ev);
        }
      }
      if (edge) {
#pragma unroll
        for (int h = 0; h < kPieces; ++h)
#pragma unroll
          for (int i = 0; i < R2; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (key0 + 16 * h + key_of_row<D>(g + 8 * e) >= lim[i]) x[h][i][e] = -INFINITY;
      }
      float top[R2];
      bool grows = false;
#pragma unroll
      for (int i = 0; i < R2; ++i) {
        top[i] = fmaxf(x[0][i][0], x[0][i][1]);
        if (kPieces == 2) top[i] = fmaxf(top[i], fmaxf(x[kPieces - 1][i][0], x[kPieces - 1][i][1]));
        grows |= top[i] > m[i] + kLazy;
      }
      if (__any_sync(0xffffffffu, grows)) {
        float keep[R2];
#pragma unroll
        for (int i = 0; i < R2; ++i) {
          float all = top[i];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
          const bool grow = all > m[i] + kLazy;
          keep[i] = grow ? exp2_approx(m[i] - all) : 1.f;
          if (grow) m[i] = all;
          sum[i] *= keep[i];
        }
#pragma unroll
        for (int c = 0; c < KS; ++c)
#pragma unroll
          for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[c][n][i] *= keep[2 * n + (i & 1)];
      }
#pragma unroll
      for (int h = 0; h < kPieces; ++h) {
        const float inv_v = scale_value(2 * kScaleBias - (scales[h] >> 8));
        uint32_t pf[NR][2];
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          float w[2][2];                     // [key][row]
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float base = kUp - (m[2 * n + i] == -INFINITY ? 0.f : m[2 * n + i]);
#pragma unroll
            for (int e = 0; e < 2; ++e) w[e][i] = exp2_approx(x[h][2 * n + i][e] + base);
            sum[2 * n + i] = fmaf(w[0][i] + w[1][i], inv_v, sum[2 * n + i]);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) pf[n][e] = transposed(pack2<true>(w[e][0], w[e][1]));
        }
        uint32_t v[4][D / 32];               // keys of rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9; bytes (D / 8) g ..
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = key_of_row<D>(2 * t + 8 * (i >> 1) + (i & 1));
          const uint8_t* src = v_at + 16 * D * h + chunk_at<D>(key, D == 128 ? g : g >> 1);
          if constexpr (D == 128) {
            const uint4 c = *reinterpret_cast<const uint4*>(src);
            v[i][0] = c.x, v[i][1] = c.y, v[i][2] = c.z, v[i][3] = c.w;
          } else {
            const uint2 c = reinterpret_cast<const uint2*>(src)[g & 1];
            v[i][0] = c.x, v[i][1] = c.y;
          }
        }
        if (edge && key0 + 16 * h + 16 > q.len) {      // places behind the request's tokens hold anything
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (key0 + 16 * h + key_of_row<D>(2 * t + 8 * (i >> 1) + (i & 1)) >= q.len) {
#pragma unroll
              for (int w = 0; w < D / 32; ++w) v[i][w] = 0;
            }
        }
        // A NaN among values that not all rows see would reach those rows too, as 0 times it: it is taken out, and put into
        // the rows that see it with their output.
        if (edge && lim_low < lim_top) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
              const uint32_t nan = nan_codes(v[i][w]);
              v[i][w] &= ~nan, odd |= nan;
            }
        }
        // O^T += V^T P^T: tile c has bytes 2 c and 2 c + 1 of the threads' runs of d
#pragma unroll
        for (int c = 0; c < KS; ++c) {
          const uint32_t sel = c & 1 ? 0x7362u : 0x5140u;
          const uint32_t w0 = __byte_perm(v[0][c >> 1], v[1][c >> 1], sel), w1 = __byte_perm(v[2][c >> 1], v[3][c >> 1], sel);
          const uint32_t a[4] = {e4m3_low(w0), e4m3_high(w0), e4m3_low(w1), e4m3_high(w1)};
#pragma unroll
          for (int n = 0; n < NR; ++n) mma16816(acc[c][n], a, pf[n][0], pf[n][1]);
        }
      }
    }
    copy_wait<0>();

    // ------------------------------------------------------------------ the warps' outputs
    __syncthreads();                           // the ring becomes the outputs' place
#pragma unroll
    for (int i = 0; i < R2; ++i) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
      const int row = 8 * (i >> 1) + 2 * t + (i & 1);
      if (g == 0) sm.ml[warp][row] = make_float2(m[i], sum[i]);
      float4* dst = reinterpret_cast<float4*>(&sm.o[warp][row][(D / 8) * g]);
#pragma unroll
      for (int c = 0; c < KS; c += 2) {
        const float(&a)[4] = acc[c][i >> 1], (&b)[4] = acc[c + 1][i >> 1];
        dst[c / 2] = make_float4(a[i & 1], a[2 + (i & 1)], b[i & 1], b[2 + (i & 1)]);
      }
    }
    const bool put_nan = __syncthreads_or(odd != 0);
    const bool whole = seg.whole();
    const int cta = blockIdx.x;
    int c0, c1;
    seg.ctas(place.share, c0, c1);
    const auto finish = [&](int row, int col, const float4& o, float top, float total) {
      const float inv = total == 0.f ? 0.f : 1.f / total;
      const int tok = p.by_G.of(row0 + row), head = kvh * p.G + row0 + row - tok * p.G;
      const int64_t at_row = static_cast<int64_t>(q.first + tok) * p.a.Hq + head;
      *reinterpret_cast<uint2*>(p.a.O + at_row * D + col) =
          make_uint2(pack2<F16>(o.x * inv, o.y * inv), pack2<F16>(o.z * inv, o.w * inv));
      if (col == 0 && p.a.lse)
        p.a.lse[at_row] = total == 0.f ? -INFINITY : ((top == -INFINITY ? 0.f : top) - kUp + log2f(total)) * 0.6931471805599453f;
    };
    const int units = it.rows * (D / 4);       // four columns of a row
#pragma unroll 1
    for (int u = threadIdx.x; u < units; u += L::kThreads) {
      const int row = u / (D / 4), col = 4 * (u % (D / 4)), tile = row / (8 * NR), in = row % (8 * NR);
      float top = -INFINITY, total = 0.f;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w)
        if ((w & (mt - 1)) == tile) top = fmaxf(top, sm.ml[w][in].x);
      const float ref = top == -INFINITY ? 0.f : top;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) {
        if ((w & (mt - 1)) != tile) continue;
        const float2 ml = sm.ml[w][in];
        const float f = exp2_approx(ml.x - ref);
        total = fmaf(ml.y, f, total);
        const float4 v = *reinterpret_cast<const float4*>(&sm.o[w][in][col]);
        o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
      }
      if (__builtin_expect(put_nan, 0)) {      // the segment's keys that the row sees, of the steps that not all rows see
        const int from = max(first, keys_seen(q, p.by_G.of(row0)) / kKeys);
        const int end = min(keys_seen(q, p.by_G.of(row0 + row)), (first + n_steps) * kKeys);
#pragma unroll 1
        for (int key = from * kKeys; key < end; ++key) {
          const uint32_t nan = nan_codes(value_codes(p, table, kvh, key, D, col));
          if (nan & 0xffu) o.x = NAN;
          if (nan & 0xff00u) o.y = NAN;
          if (nan & 0xff0000u) o.z = NAN;
          if (nan & 0xff000000u) o.w = NAN;
        }
      }
      if (whole) {
        finish(row, col, o, top, total);
      } else {
        const int64_t at_row = (2ll * cta + (cta == c0 ? 1 : 0)) * L::kRows + row;
        *reinterpret_cast<float4*>(p.po + at_row * D + col) = o;
        if (col == 0) p.ml[at_row] = make_float2(top, total);
      }
    }
    if (!whole) {
      const auto last = [&](const Join& j) {
        __syncthreads();
        if (threadIdx.x == 0) sm.last = last_part(p.count + j.counter, j.n);
        __syncthreads();
        return sm.last != 0;
      };
      Join round = first_join(c0, c1, cta, gridDim.x);
      while (last(round)) {
        const int first = round.first, step = round.step, n = round.n;
        // Few loads wait for others: neighbouring threads (`parts` of them) take a unit's segments in turn, or a thread has
        // two units where there are more than threads, eight segments at a time.  (One unit after the other: 8 requests of 4
        // new tokens over up to 8192 keys, 32 heads on 8, 25.6 us, so 22.0; two also where there is one: one request over 500
        // keys 6.7, so 7.1.)
        const int parts = units * 8 <= L::kThreads ? 8 : units * 4 <= L::kThreads ? 4 : units * 2 <= L::kThreads ? 2 : 1;
        const int part = threadIdx.x & (parts - 1);
        const auto join = [&](auto each) {
          constexpr int U = decltype(each)::value, kApart = L::kThreads / (D / 4);      // rows from a thread's unit to its next
#pragma unroll 1
          for (int u0 = 0; u0 < units * parts; u0 += U * L::kThreads) {
            const int u = min((u0 + static_cast<int>(threadIdx.x)) / parts, units - 1), row = u / (D / 4), col = 4 * (u % (D / 4));
            const bool two = U == 2 && row + kApart < it.rows;
            const auto slot = [&](int i) {
              const int c = first + i * step;
              return (2ll * c + (c == c0 ? 1 : 0)) * L::kRows + row;
            };
            float top[U], total[U];
            float4 o[U];
#pragma unroll
            for (int k = 0; k < U; ++k) top[k] = -INFINITY, total[k] = 0.f, o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int base = part; base < n; base += 8 * parts) {
              float2 ml[U][8];
              float4 v[U][8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int k = 0; k < U; ++k) {
                  ml[k][i] = make_float2(-INFINITY, 0.f), v[k][i] = make_float4(0.f, 0.f, 0.f, 0.f);
                  if (base + i * parts < n && (k == 0 || two)) {
                    const long long at = slot(base + i * parts) + k * kApart;
                    ml[k][i] = __ldcg(p.ml + at);
                    v[k][i] = __ldcg(reinterpret_cast<const float4*>(p.po + at * D + col));
                  }
                }
#pragma unroll
              for (int k = 0; k < U; ++k) {
                float now = top[k];
#pragma unroll
                for (int i = 0; i < 8; ++i) now = fmaxf(now, ml[k][i].x);
                const float ref = now == -INFINITY ? 0.f : now, keep = exp2_approx(top[k] - ref);
                total[k] *= keep, o[k].x *= keep, o[k].y *= keep, o[k].z *= keep, o[k].w *= keep;
                top[k] = now;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const float f = exp2_approx(ml[k][i].x - ref);
                  const float4& x = v[k][i];
                  total[k] = fmaf(ml[k][i].y, f, total[k]);
                  o[k].x = fmaf(x.x, f, o[k].x), o[k].y = fmaf(x.y, f, o[k].y), o[k].z = fmaf(x.z, f, o[k].z), o[k].w = fmaf(x.w, f, o[k].w);
                }
              }
            }
            if (U == 1)
              for (int d = 1; d < parts; d <<= 1) {
                const float other = __shfl_xor_sync(0xffffffffu, top[0], d), now = fmaxf(top[0], other), ref = now == -INFINITY ? 0.f : now;
                const float f = exp2_approx(top[0] - ref);
                top[0] = now;
                total[0] *= f, o[0].x *= f, o[0].y *= f, o[0].z *= f, o[0].w *= f;
                total[0] += __shfl_xor_sync(0xffffffffu, total[0], d);
                o[0].x += __shfl_xor_sync(0xffffffffu, o[0].x, d), o[0].y += __shfl_xor_sync(0xffffffffu, o[0].y, d);
                o[0].z += __shfl_xor_sync(0xffffffffu, o[0].z, d), o[0].w += __shfl_xor_sync(0xffffffffu, o[0].w, d);
              }
            if (part == 0 && u0 + static_cast<int>(threadIdx.x) < units * parts) {
#pragma unroll
              for (int k = 0; k < U; ++k) {
                if (k == 1 && !two) break;
                const int r = row + k * kApart;
                if (round.final) {
                  finish(r, col, o[k], top[k], total[k]);
                } else {
                  *reinterpret_cast<float4*>(p.po + (slot(0) + k * kApart) * D + col) = o[k];
                  if (col == 0) sm.ml[r / (8 * NR)][r % (8 * NR)] = make_float2(top[k], total[k]);
                }
              }
            }
          }
        };
        if (units <= L::kThreads) join(std::integral_constant<int, 1>());
        else join(std::integral_constant<int, 2>());
        if (round.final) break;
        __syncthreads();                       // all have read what the group's first CTA left
        for (int row = threadIdx.x; row < it.rows; row += L::kThreads)
          p.ml[(2ll * first + (first == c0 ? 1 : 0)) * L::kRows + row] = sm.ml[row / (8 * NR)][row % (8 * NR)];
        round = final_join(c0, c1);
      }
    }
    __syncthreads();                           // and the ring again
  }
  pdl_wait();
}

// ------------------------------------------------------------------------------- many rows
// Items of up to 256 rows on the tensor cores (tcgen05).  Two lanes of 128 rows, each with its own output and two
// buffers of scores in tensor memory, its own warp that issues the products and its own four softmax warps, a row a
// thread.  With more than 128 rows in the item both lanes see every key tile; with up to 128 both have the same rows and
// take the tiles in turn, and the first adds up the outputs (in one lane of tensor memory a row has both).  A tile's
// codes come by TMA (128-byte swizzle), two warps widen K and two V to fp16 tiles, which serve both lanes:
//   S = Q K^T       both operands from shared memory; the softmax warps put Q there, in fp16
//   W = 2^(x - m)   written over S in tensor memory, fp16
//   O += W V        W from tensor memory, V from shared memory, d contiguous (transposed operand)
// The products of a tile run while the softmax of the lane's tile before it, and of the other lane's, runs.  A warp walks
// over the segments ahead of the others.  Bound by the products: a tile of 256 rows takes some 1820 cycles, and the
// tensor core's part of them is 1760 (S has to read Q from shared memory for every 64 keys, as attn.cu says).  Pieces of
// 3 prompts, 5119 new tokens over up to 10007 keys, 32 heads on 8: 338 to 413 us by how deep each lies, 1128 to 1165 TFLOP/s of
// what the rows see.
constexpr int kRawStages = 3;          // tiles of codes, K and V
constexpr int kWideStages = 3;         // tiles of fp16, of K and of V
constexpr int kScaleRing = 16;         // tiles' scales: more than the copies are ahead of the softmax warps
constexpr int kSegments = 4;           // segments that the walk is ahead of the other warps
constexpr int kWWiden = 8, kWMma = 12, kWCopy = 14, kWWalk = 15;       // first warps of a role; warps 0 .. 7: softmax
constexpr int kManyRegs = 168, kManyRegsOther = 88;    // of 128 a thread at launch
constexpr int kTmemCols = 512, kColO = 256;            // two S of 64 columns a lane, then O of 128 a lane
static_assert(8 * kManyRegs + 8 * kManyRegsOther == 128 * 16, "registers are those of the launch");

template <int D>
struct ManySmem {
  uint8_t raw[kRawStages][2][kTile * D];       // codes of K, V
  uint8_t wide[2][kWideStages][kTile * D * 2]; // fp16 K, V: [D / 64][64 keys][128 bytes], swizzled
  uint8_t q[2][128 * D * 2];                   // [D / 64][128 rows][128 bytes], swizzled
  uint64_t raw_full[kRawStages], raw_empty[kRawStages];
  uint64_t full[2][kWideStages], empty[2][kWideStages];
  uint64_t q_full[2], q_empty[2], s_full[2][2], p_full[2][2], pv_done[2], o_full[2], o_empty[2], drain[2];
  float2 ml[128];                              // the second lane's statistics, where it has the first one's rows
  uint64_t seg_full[kSegments], seg_empty[kSegments], meet;
  Segment seg[kSegments];
  int odd[kSegments];                          // NaN were taken out of a segment's values
  uint16_t scales[kScaleRing][4];
  int last, failed;
  uint32_t tmem_base;
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 32 bytes to an address that is a multiple of 32.
__device__ __forceinline__ void store32(void* to, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
               "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// The first key of the key tiles of an item of many rows that not all its rows see whole.
__device__ __forceinline__ int seen_by_all(const Params& p, const Segment& x) {
  return keys_seen(x.q, p.by_G.of(x.tile * kManyRows)) / kTile * kTile;
}

// The key tiles of an item of n tiles that lane l takes.
struct Turns {
  int first, step, n;
  __device__ Turns(int rows, int n_, int l) : first(rows > 128 ? 0 : l), step(rows > 128 ? 1 : 2), n(n_) {}
  __device__ bool mine(int j) const { return step == 1 || ((j ^ first) & 1) == 0; }
  __device__ bool any() const { return first < n; }
};

template <bool F16, int D>
__global__ void __launch_bounds__(kManyThreads, 1)
    k_attn_e4m3_many(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const __grid_constant__ Params p) {
  using L = ManyLine;
  using S = ManySmem<D>;
  constexpr int CH = D / 64;
  constexpr uint32_t kQChunk = 128 * 128, kKvChunk = kTile * 128;       // bytes of 64 elements of all rows / keys
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw + smem_align_pad(smem_raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRawStages; ++i) mbar_init(&sm.raw_full[i], 1), mbar_init(&sm.raw_empty[i], 4);
    for (int i = 0; i < 2; ++i) {
      for (int s = 0; s < kWideStages; ++s) mbar_init(&sm.full[i][s], 2), mbar_init(&sm.empty[i][s], 2);
      mbar_init(&sm.q_full[i], 4), mbar_init(&sm.q_empty[i], 1);
      for (int b = 0; b < 2; ++b) mbar_init(&sm.s_full[i][b], 1), mbar_init(&sm.p_full[i][b], 4);
      mbar_init(&sm.pv_done[i], 1), mbar_init(&sm.o_full[i], 1), mbar_init(&sm.o_empty[i], 4), mbar_init(&sm.drain[i], 1);
    }
    for (int i = 0; i < kSegments; ++i) mbar_init(&sm.seg_full[i], 1), mbar_init(&sm.seg_empty[i], kWWalk);
    mbar_init(&sm.meet, kWWiden);
    sm.failed = 0;
    fence_barrier_init();
  }
  if (threadIdx.x == 32 * kWCopy) tma_prefetch_desc(&tk), tma_prefetch_desc(&tv);
  pdl_wait();
  pdl_launch_dependents();                     // not before: the kernel for few rows reads what this one waited for
  const Place place = find_place<L>(p);
  if (place.r < 0) return;
  if (warp == kWMma) {
    tmem_alloc(&sm.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  bool ok = true;
  // The segment in its place in the ring, or null at the end or after a wait that ran out; given back when the warp is
  // done with it.  `ahead`: the one after it.
  uint32_t n_seg = 0;
  const auto segment = [&](uint32_t ahead) -> const Segment* {
    const uint32_t i = n_seg + ahead;
    ok = ok && stage_wait(&sm.seg_full[i % kSegments], (i / kSegments) & 1, &sm.failed, kErrWaitFull);
    return ok && sm.seg[i % kSegments].hi > 0 ? &sm.seg[i % kSegments] : nullptr;
  };
  const auto segment_done = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.seg_empty[n_seg % kSegments]);
    ++n_seg;
  };

  if (warp >= kWWiden) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kManyRegsOther));
    if (warp == kWWalk) {
      // ------------------------------------------------------------------ the walk
      Walk<L> walk(p, place);
      bool more = true;
      for (uint32_t i = 0; more && ok; ++i) {
        Segment x;
        more = walk.next(x);
        if (!more) x.hi = 0;
        ok = stage_wait(&sm.seg_empty[i % kSegments], ((i / kSegments) & 1) ^ 1, &sm.failed, kErrWaitEmpty, 500);
        if (lane == 0 && ok) {
          sm.seg[i % kSegments] = x, sm.odd[i % kSegments] = 0;
          mbar_arrive(&sm.seg_full[i % kSegments]);
        }
        if (more && i > 0) {                    // its queries on their way to L2; the first ones are asked for right away
          const int row0 = x.tile * kManyRows, t0 = p.by_G.of(row0), tokens = p.by_G.of(row0 + x.it.rows - 1) - t0 + 1;
          const uint32_t bytes = p.G * D * 2;
          for (int t = lane; t < tokens; t += 32)
            prefetch_l2(p.a.Q + (x.q.first + t0 + t) * p.a.q_stride + static_cast<int64_t>(x.head) * p.G * D, bytes);
        }
      }
    } else if (warp == kWCopy) {
      // ------------------------------------------------------------------ codes and scales
      copy_items<L, D, kTile, kRawStages>(
          p, tk, tv, [&] { return segment(0); }, segment_done, [&](uint32_t i) { return sm.raw[i % kRawStages][0]; }, sm.raw_full,
          sm.raw_empty, [&](uint32_t i) { return sm.scales[i % kScaleRing]; }, &sm.failed);
    } else if (warp < kWMma) {
      // ------------------------------------------------------------------ codes -> fp16
      // Two warps widen K, two V, so that neither waits for the other's barriers.  A thread widens 16 codes at a time, of
      // keys 16 apart.  Eight lanes have four chunks each of two keys, chosen (k and k ^ 5, or k ^ 1 where d is 64) so
      // that what they read and what they write falls on all banks.
      const int v = (warp - kWWiden) >> 1, u = threadIdx.x & 63, chunk = u & 3;
      const int key = (2 * (u >> 3)) ^ (((u >> 2) & 1) * (D == 128 ? 5 : 1));    // 0 .. 15
      const uint32_t from = chunk_at<D>(key, chunk), to = 128 * key + 16 * ((2 * chunk) ^ (key & 7));
      uint32_t tile = 0;
      while (const Segment* x = segment(0)) {
        int first;
        const int n = x->stages<L, kTile>(p, first), len = x->q.len, all_see = seen_by_all(p, *x);
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j, ++tile) {
          const uint32_t rs = tile % kRawStages, ws = tile % kWideStages;
          ok = stage_wait(&sm.raw_full[rs], (tile / kRawStages) & 1, &sm.failed, kErrWaitFull);
          ok = ok && stage_wait(&sm.empty[v][ws], ((tile / kWideStages) & 1) ^ 1, &sm.failed, kErrWaitEmpty);
          if (!ok) break;
          const uint8_t* src = sm.raw[rs][v];
          uint8_t* dst = sm.wide[v][ws];
          const int left = len - (first + j) * kTile;
          const bool tail = v && left < kTile;          // V's places behind the tokens hold anything: zeros
          // A NaN among values that not all rows see would reach those rows too, as 0 times it: it is taken out, and put into
          // the rows that see it with their output.
          const bool edge = v && (first + j) * kTile >= all_see;
          uint32_t odd = 0;
#pragma unroll
          for (int plane = 0; plane < CH; ++plane) {
            uint4 c[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = *reinterpret_cast<const uint4*>(src + (from ^ (64 * plane)) + 16 * D * i);
            if (__builtin_expect(tail, 0)) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (key + 16 * i >= left) c[i] = make_uint4(0, 0, 0, 0);
            }
            if (__builtin_expect(edge, 0)) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  uint32_t& w = (&c[i].x)[e];
                  const uint32_t nan = nan_codes(w);
                  w &= ~nan, odd |= nan;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint8_t* at = dst + plane * kKvChunk + 2048 * i;
              *reinterpret_cast<uint4*>(at + to) = make_uint4(e4m3_low(c[i].x), e4m3_high(c[i].x), e4m3_low(c[i].y), e4m3_high(c[i].y));
              *reinterpret_cast<uint4*>(at + (to ^ 16)) = make_uint4(e4m3_low(c[i].z), e4m3_high(c[i].z), e4m3_low(c[i].w), e4m3_high(c[i].w));
            }
          }
          if (odd) sm.odd[n_seg % kSegments] = 1;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.full[v][ws]), mbar_arrive(&sm.raw_empty[rs]);
        }
        if (!ok) break;
        segment_done();
      }
    } else if (warp < kWCopy) {
      // ------------------------------------------------------------------ products of lane l
      const int l = warp - kWMma;
      constexpr uint32_t id_qk = (1u << 4) | ((kTile >> 3) << 17) | ((128u >> 4) << 24);
      constexpr uint32_t id_wv = (1u << 4) | (1u << 16) | ((D >> 3) << 17) | ((128u >> 4) << 24);
      const uint32_t t_s = tmem + 128 * l, t_o = tmem + kColO + 128 * l;
      const uint64_t k0 = smem_desc_sw128(smem_u32(sm.wide[0][0])), v0 = smem_desc_sw128_mn(smem_u32(sm.wide[1][0]), kKvChunk);
      const uint64_t qd = smem_desc_sw128(smem_u32(sm.q[l]));
      constexpr uint32_t kWideBytes = kTile * D * 2;
      uint32_t k_tile = 0, v_tile = 0, items = 0;       // tiles and items of this lane's own alike for all
      uint32_t s_cnt = 0, p_cnt = 0;            // tiles of this lane whose S was issued / whose W was taken
      while (const Segment* x = segment(0)) {
        int first;
        const int n = x->stages<L, kTile>(p, first);
        // Every place of the rings is waited for and given back by both lanes, also where only the other one uses it: a
        // wait by parity is only sound if no phase is left out.
        const Turns turns(x->it.rows, n, l);
        // S runs ahead by two tiles of the lane's own: the next two, or two of the next three
        const int ahead = turns.step == 1 ? 2 : 3;
        if (turns.any()) ok = stage_wait(&sm.q_full[l], items & 1, &sm.failed, kErrWaitFull);
        const auto qk = [&](int j) {
          const uint32_t sl = k_tile % kWideStages;
          ok = stage_wait(&sm.full[0][sl], (k_tile / kWideStages) & 1, &sm.failed, kErrWaitFull);
          if (!ok) return;
          ++k_tile;
          if (!turns.mine(j)) {
            if (lane == 0) mbar_arrive(&sm.empty[0][sl]);
            __syncwarp();
            return;
          }
          const uint64_t kd = k0 + sl * (kWideBytes >> 4);
          const uint32_t b = s_cnt & 1, t = t_s + 64 * b;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4 * CH; ++k)
              tc_mma_ss_f16(t, qd + (((k >> 2) * kQChunk + 32 * (k & 3)) >> 4), kd + (((k >> 2) * kKvChunk + 32 * (k & 3)) >> 4),
                            id_qk, k ? 1u : 0u);
            tc_commit(&sm.s_full[l][b]);
            tc_commit(&sm.empty[0][sl]);
            if (j + turns.step >= n) tc_commit(&sm.q_empty[l]);
          }
          __syncwarp();
          ++s_cnt;
        };
        const auto wv = [&](int j) {
          const uint32_t sl = v_tile % kWideStages;
          ok = stage_wait(&sm.full[1][sl], (v_tile / kWideStages) & 1, &sm.failed, kErrWaitFull);
          if (!ok) return;
          ++v_tile;
          if (!turns.mine(j)) {
            if (lane == 0) mbar_arrive(&sm.empty[1][sl]);
            __syncwarp();
            return;
          }
          // first: the lane's previous item has left the output columns
          const bool begins = j == turns.first;
          if (begins) ok = stage_wait(&sm.o_empty[l], (items & 1) ^ 1, &sm.failed, kErrWaitAccum);
          const uint32_t b = p_cnt & 1, t = t_s + 64 * b;
          ok = ok && stage_wait(&sm.p_full[l][b], (p_cnt >> 1) & 1, &sm.failed, kErrWaitFull);
          if (!ok) return;
          const uint64_t vd = v0 + sl * (kWideBytes >> 4);
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k) tc_mma_ts(t_o, t + 8 * k, vd + ((k * 2048) >> 4), id_wv, (begins && k == 0) ? 0u : 1u);
            tc_commit(&sm.pv_done[l]);
            if (j + turns.step >= n) tc_commit(&sm.o_full[l]);
            tc_commit(&sm.empty[1][sl]);
          }
          __syncwarp();
          ++p_cnt;
        };
#pragma unroll 1
        for (int j = 0; j < n + ahead && ok; ++j) {
          if (j >= ahead) wv(j - ahead);
          if (ok && j < n) qk(j);
        }
        if (!ok) break;
        if (turns.any()) ++items;
        segment_done();
      }
      // every product and commit of this warp (elect.sync names the same lane each time) has completed before tensor memory and barriers go
      if (elect_one()) tc_commit(&sm.drain[l]);
      mbar_wait_short(&sm.drain[l], 0, &g_attn8_err, kErrDrain);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
    // -------------------------------------------------------------------- softmax, one row a thread
    const int l = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_o = tmem + lane_base + kColO + 128 * l;
    const int log_box = 31 - __clz(min(p.a.page_size, kTile));
    uint32_t cnt = 0, items = 0, tile = 0;      // tiles and items of this lane; tiles of all items
    uint32_t q_items = 0;                       // items of this lane whose Q is on its way
    // What this thread's row of a segment needs.
    struct Row {
      bool both, valid;                         // both lanes have the same rows; this row is one
      int tok, head, n, first;
      float c;                                  // scale * log2(e), times the power of two taken from the query
    };
    const auto row_of = [&](const Segment& x) {
      Row w;
      w.both = x.it.rows <= 128;
      const int row_item = w.both ? row : 128 * l + row, row_all = x.tile * kManyRows + row_item;
      w.valid = row_item < x.it.rows;
      w.tok = p.by_G.of(row_all), w.head = x.head * p.G + row_all - w.tok * p.G;
      w.n = x.template stages<L, kTile>(p, w.first);
      w.c = p.c;
      return w;
    };
    // Q to shared memory, and there to fp16, behind a power of two of the row where it is bf16.  Loops that stay
    // loops: code that runs once an item comes from L2, and unrolled it took 4 us an item.
    const auto put_q = [&](const Segment& x, Row& w) {
      if (!Turns(x.it.rows, w.n, l).any()) return;
      constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;      // lanes a row, rows a copy of the warp
      uint8_t* const q = sm.q[l] + (warp & 3) * 32 * 128;       // the warp's 32 rows
      const auto place_of = [&](int to, int unit) { return (unit >> 3) * kQChunk + to * 128 + 16 * ((unit & 7) ^ (to & 7)); };
      const int64_t row_at = (x.q.first + w.tok) * p.a.q_stride + static_cast<int64_t>(w.head) * D;
      const uint32_t rows = __ballot_sync(0xffffffffu, w.valid);
      ok = ok && stage_wait(&sm.q_empty[l], (q_items & 1) ^ 1, &sm.failed, kErrWaitEmpty);
#pragma unroll 4
      for (int i = 0; i < kLanes; ++i) {
        const int to = i * kAtOnce + lane / kLanes;
        const int64_t at = __shfl_sync(0xffffffffu, row_at, to);
        const bool on = (rows >> to) & 1;      // rows that do not exist: zeros
        copy16(q + place_of(to, lane % kLanes), on ? p.a.Q + at + 8 * (lane % kLanes) : p.a.Q, on);
      }
      copy_commit();
      copy_wait<0>();
      __syncwarp();
      if (!F16) {
        uint32_t mx = 0;
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
          const uint4 v = *reinterpret_cast<const uint4*>(q + place_of(lane, i));
          mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
        }
        const int k = bf16_to_f16_exponent(max(mx & 0xffffu, mx >> 16));
        const float down = pow2_normal(-k);
        w.c *= pow2_normal(k);
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
          uint4* at = reinterpret_cast<uint4*>(q + place_of(lane, i));
          uint4 v = *at;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 f = unpack2<false>((&v.x)[e]);
            (&v.x)[e] = pack2<true>(f.x * down, f.y * down);
          }
          *at = v;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.q_full[l]);
      ++q_items;
    };
    // All softmax warps meet, by a wait that is bounded as the others are: one that gave up leaves none behind.
    uint32_t meets = 0;
    const auto meet = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.meet);
      ok = stage_wait(&sm.meet, meets++ & 1, &sm.failed, kErrWaitReduce) && ok;
    };
    const Segment* seg = segment(0);
    Row w{};
    if (seg) w = row_of(*seg), put_q(*seg, w);
#pragma unroll 1
    while (seg) {
      const Segment& x = *seg;
      const int n = ok ? w.n : 0, first = w.first;
      const bool valid = w.valid, active = __any_sync(0xffffffffu, valid);
      const Turns turns(x.it.rows, n, l);
      const int lim = valid ? keys_seen(x.q, w.tok) : 0;
      const float c = w.c;
      float m = -INFINITY, sum = 0.f;           // m: the largest x, in units of log2
#pragma unroll 1
      for (int j = turns.first; j < n && ok; j += turns.step, ++cnt) {
        const int key0 = (first + j) * kTile;
        const uint32_t b = cnt & 1, t_s = tmem + lane_base + 128 * l + 64 * b, at = tile + j;
        ok = stage_wait(&sm.s_full[l][b], (cnt >> 1) & 1, &sm.failed, kErrWaitAccum);
        // the tile's V is there, and with it the scales; its place is not filled again before this tile's product
        ok = ok && stage_wait(&sm.full[1][at % kWideStages], (at / kWideStages) & 1, &sm.failed, kErrWaitFull);
        if (!ok) break;
        tc_fence_after();
        if (active) {
          uint32_t v[2][32];
          tmem_ld32(t_s, v[0]);
          tmem_ld32(t_s + 32, v[1]);
          float ck[4], ev[4], inv[4];           // of each 16 keys
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t sc = sm.scales[at % kScaleRing][(16 * q) >> log_box];
            // not 0, which the masked scores' infinities turn into NaN; what this changes of x is below 2^-94
            ck[q] = fmaxf(c * scale_value(sc & 0xffu), 1.17549435e-38f), ev[q] = static_cast<float>(static_cast<int>(sc >> 8) - kScaleBias);
            inv[q] = scale_value(2 * kScaleBias - (sc >> 8));
          }
          tc_wait_ld();
          if (__builtin_expect(__any_sync(0xffffffffu, valid && key0 + kTile > lim), 0)) {
            const int left = lim - key0;
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (32 * q + e >= left) v[q][e] = 0xff800000u;
          }
          float top = -INFINITY;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t* w = &v[q >> 1][16 * (q & 1)];
            float mq = fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1]));
#pragma unroll
            for (int e = 2; e < 16; e += 2) mq = max3(mq, __uint_as_float(w[e]), __uint_as_float(w[e + 1]));
            top = fmaxf(top, fmaf(mq, ck[q], ev[q]));
          }
          const bool grow = valid && top > m + kLazy;
          if (__builtin_expect(__any_sync(0xffffffffu, grow), 0)) {
            const float keep = grow ? exp2_approx(m - top) : 1.f;
            if (grow) m = top;
            sum *= keep;
            if (j != turns.first) {
              // the lane's last product has left the output (one phase at most is outstanding: this tile's S was
              // issued after the product before that one)
              ok = stage_wait(&sm.pv_done[l], (cnt - 1) & 1, &sm.failed, kErrWaitAccum);
              if (!ok) break;
              tc_fence_after();
              const uint64_t keep2 = pair_f(keep, keep);
#pragma unroll 1
              for (int q = 0; q < D / 32; ++q) {
                uint32_t o[32];
                tmem_ld32(t_o + 32 * q, o);
                tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                  const float2 f = unpair(mul_pair(pair(o[e], o[e + 1]), keep2));
                  o[e] = __float_as_uint(f.x), o[e + 1] = __float_as_uint(f.y);
                }
                tmem_st32(t_o + 32 * q, o);
              }
            }
          }
          const float base = kUp - (m == -INFINITY ? 0.f : m);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint64_t c2 = pair_f(ck[q], ck[q]), b2 = pair_f(base + ev[q], base + ev[q]);
            uint64_t part = 0;
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t* s = &v[q >> 1][16 * (q & 1) + 2 * e];
              const float2 y = unpair(fma_pair(pair(s[0], s[1]), c2, b2));
              const float a = exp2_approx(y.x), d = exp2_approx(y.y);
              part = add_pair(part, pair_f(a, d));
              w[e] = pack2<true>(a, d);
            }
            tmem_st8(t_s + 8 * q, w);
            const float2 s2 = unpair(part);
            sum = fmaf(s2.x + s2.y, inv[q], sum);
          }
          tc_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[l][b]);
      }
      tile += n;
      // the next segment's Q is put in place before this one's output is taken, so that its first products run beside that
      const Segment* next = segment(1);
      const Row done = w;
      if (next) w = row_of(*next), put_q(*next, w);
      // ------------------------------------------------------------------ the segment's output
      bool out = valid;                         // this thread has a row's output
      const int row_item = done.both ? row : 128 * l + row;
      const bool had = turns.any() && ok;
      if (had) {
        ok = stage_wait(&sm.o_full[l], items & 1, &sm.failed, kErrWaitAccum);
        tc_fence_after();
        ++items;
      }
      float f0 = 1.f, f1 = 0.f;                 // of this lane's output, and of the second lane's
      if (done.both) {                          // the first lane adds up both
        if (l == 1) sm.ml[row] = make_float2(m, sum);
        tc_fence_before();
        meet();
        tc_fence_after();
        out = valid && l == 0;
        if (l == 0) {
          const float2 other = sm.ml[row];
          const float top = fmaxf(m, other.x), ref = top == -INFINITY ? 0.f : top;
          f0 = exp2_approx(m - ref), f1 = exp2_approx(other.x - ref);
          sum = fmaf(other.y, f1, sum * f0), m = top;
        }
      }
      const int64_t at_row = static_cast<int64_t>(x.q.first + done.tok) * p.a.Hq + done.head;
      const bool wide_rows = (reinterpret_cast<uintptr_t>(p.a.O) & 31) == 0;
      // 32 columns of the row, given as the sums' bits
      const auto finish = [&](int q, const uint32_t (&o)[32], float inv) {
        uint32_t h[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) h[i] = pack2<F16>(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
        uint16_t* dst = p.a.O + at_row * D + 32 * q;
        if (wide_rows) {                        // whole sectors: 304 items of 512 keys 39.4 -> 37.7 us
          store32(dst, &h[0]), store32(dst + 16, &h[8]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) reinterpret_cast<uint4*>(dst)[i] = make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
        }
      };
      const auto finish_lse = [&](float top, float total) {
        if (p.a.lse)
          p.a.lse[at_row] = total == 0.f ? -INFINITY : ((top == -INFINITY ? 0.f : top) - kUp + log2f(total)) * 0.6931471805599453f;
      };
      int c0, c1;
      x.ctas(place.share, c0, c1);
      // partials [cta][2][d / 4][256 rows][4]: a warp writes and reads whole lines
      const auto slot = [&](int at) { return 2ll * at + (at == c0 ? 1 : 0); };
      const auto part = [&](int at) { return reinterpret_cast<float4*>(p.po) + slot(at) * (D / 4) * kManyRows + row_item; };
      const auto put_part = [&](int at, int q, const uint32_t (&o)[32]) {
        float4* po = part(at) + 8 * q * kManyRows;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          po[e * kManyRows] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]), __uint_as_float(o[4 * e + 2]),
                                          __uint_as_float(o[4 * e + 3]));
      };
      const bool whole = x.whole();
      if (__any_sync(0xffffffffu, out)) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          if (n > 0) tmem_ld32(t_o + 32 * q, o);
          if (done.both && n > 1) {
            uint32_t o1[32];
            tmem_ld32(t_o + 128 + 32 * q, o1);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(fmaf(__uint_as_float(o1[e]), f1, __uint_as_float(o[e]) * f0));
          } else if (n > 0) {
            tc_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0;
          }
          if (out) {
            if (whole) finish(q, o, inv);
            else put_part(blockIdx.x, q, o);
          }
        }
        if (out) {
          if (whole) finish_lse(m, sum);
          else p.ml[slot(blockIdx.x) * kManyRows + row_item] = make_float2(m, sum);
        }
        // NaN that were taken out of the values: over the row's elements, of the keys that it sees of those that not all rows do
        if (__builtin_expect(sm.odd[n_seg % kSegments] != 0 && out, 0)) {
          const int32_t* table = p.a.block_table + static_cast<int64_t>(x.r) * p.a.max_blocks;
          const int from = max(first * kTile, seen_by_all(p, x)), end = min(lim, (first + n) * kTile);
#pragma unroll 1
          for (int key = from; key < end; ++key) {
#pragma unroll 1
            for (int col = 0; col < D; col += 4) {
              uint32_t nan = nan_codes(value_codes(p, table, x.head, key, D, col));
#pragma unroll 1
              for (int e = 0; nan != 0; ++e, nan >>= 8) {
                if (!(nan & 1)) continue;
                if (whole) p.a.O[at_row * D + col + e] = 0x7fff;         // a NaN in both types
                else reinterpret_cast<float*>(part(blockIdx.x) + (col / 4) * kManyRows)[e] = NAN;
              }
            }
          }
        }
      }
      tc_fence_before();
      if (done.both) meet();                    // the first lane has read the second one's
      else __syncwarp();
      if (had && lane == 0) mbar_arrive(&sm.o_empty[l]);
      if (!whole) {
        const auto last = [&](const Join& j) {
          meet();
          if (threadIdx.x == 0) sm.last = last_part(p.count + j.counter, j.n);
          meet();
          return sm.last != 0;
        };
        Join round = first_join(c0, c1, blockIdx.x, gridDim.x);
        while (last(round)) {
          const int first = round.first, step = round.step, n_parts = round.n;
          if (out) {                           // a row's partials are read and written by its thread alone
            float top = -INFINITY, total = 0.f;
#pragma unroll 4
            for (int i = 0; i < n_parts; ++i) top = fmaxf(top, __ldcg(&p.ml[slot(first + i * step) * kManyRows + row_item].x));
            const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll 4
            for (int i = 0; i < n_parts; ++i) {
              const float2 ml = __ldcg(p.ml + slot(first + i * step) * kManyRows + row_item);
              total = fmaf(ml.y, exp2_approx(ml.x - ref), total);
            }
            const float inv = total == 0.f ? 0.f : 1.f / total;
            // 32 columns at a time, two segments' loads under way
#pragma unroll 1
            for (int q = 0; q < D / 32; ++q) {
              uint32_t sums[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) sums[e] = 0;
#pragma unroll 1
              for (int i0 = 0; i0 < n_parts; i0 += 2) {
                float4 v[2][8];
                float f[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const int at = first + min(i0 + i, n_parts - 1) * step;
                  f[i] = __ldcg(&p.ml[slot(at) * kManyRows + row_item].x);
#pragma unroll
                  for (int e = 0; e < 8; ++e) v[i][e] = __ldcg(part(at) + (8 * q + e) * kManyRows);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  if (i0 + i >= n_parts) break;
                  const float scale = exp2_approx(f[i] - ref);
#pragma unroll
                  for (int e = 0; e < 8; ++e) {
                    uint32_t* a = &sums[4 * e];
                    const float4& x4 = v[i][e];
                    a[0] = __float_as_uint(fmaf(x4.x, scale, __uint_as_float(a[0])));
                    a[1] = __float_as_uint(fmaf(x4.y, scale, __uint_as_float(a[1])));
                    a[2] = __float_as_uint(fmaf(x4.z, scale, __uint_as_float(a[2])));
                    a[3] = __float_as_uint(fmaf(x4.w, scale, __uint_as_float(a[3])));
                  }
                }
              }
              if (round.final) {
                finish(q, sums, inv);
              } else {
                put_part(first, q, sums);
              }
            }
            if (round.final) finish_lse(top, total);
            else p.ml[slot(first) * kManyRows + row_item] = make_float2(top, total);
          }
          if (round.final) break;
          round = final_join(c0, c1);
        }
      }
      segment_done();
      seg = next;
    }
  }
  __syncwarp();
  __syncthreads();
  if (warp == kWMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Of each kernel: counters, two segments of each CTA.
struct Layout {
  int sms;
  size_t count[2], po[2], ml[2], bytes;
  void give(Params& p, int i, uint8_t* ws) const {
    p.count = reinterpret_cast<int*>(ws + count[i]);       // in the header: zero, and left so
    p.po = reinterpret_cast<float*>(ws + po[i]), p.ml = reinterpret_cast<float2*>(ws + ml[i]);
  }
};
constexpr int kMany = 0, kFew = 1;

Layout layout(int64_t d) {
  Layout l{};
  l.sms = device_sm_count();
  size_t off = kWsHeaderBytes;
  const auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  const size_t rows[2] = {kManyRows, static_cast<size_t>(std::max(few_ctas(1) * FewLine<1>::kRows, few_ctas(2) * FewLine<2>::kRows))};
  l.count[kMany] = 0, l.count[kFew] = 2 * l.sms * sizeof(int);
  for (int i : {kMany, kFew}) {
    l.po[i] = take(2 * l.sms * rows[i] * d * sizeof(float));
    l.ml[i] = take(2 * l.sms * rows[i] * sizeof(float2));
  }
  l.bytes = off;
  return l;
}

// The cache as rows of 128 bytes: a box is a page's run of up to `keys` keys.
cudaError_t cache_map(CUtensorMap* map, const uint8_t* cache, const AttnE4m3Args& a, int keys) {
  const uint64_t rows = static_cast<uint64_t>(a.page_size) * a.d / 128;
  const uint64_t dims[4] = {128, rows, 1, static_cast<uint64_t>(a.pages) * a.Hkv};
  const uint64_t strides[3] = {128, rows * 128, rows * 128};
  const uint32_t box[4] = {128, static_cast<uint32_t>(std::min(a.page_size, keys) * a.d / 128), 1, 1};
  return make_tmap_4d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, cache, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

template <bool F16, int D, int NR>
cudaError_t launch_few(Params p, const Layout& l, uint8_t* ws, cudaStream_t stream) {
  constexpr size_t smem = sizeof(FewSmem<D, NR>);
  constexpr int ctas = few_ctas(NR);
  static_assert(ctas * (smem + 1024 + 1024) <= 227 * 1024, "CTAs of the kernel for few rows do not fit an SM");
  const cudaError_t e = set_smem_attr_once(reinterpret_cast<const void*>(k_attn_e4m3<F16, D, NR>), smem);
  if (e != cudaSuccess) return e;
  l.give(p, kFew, ws);
  return launch_pdl(k_attn_e4m3<F16, D, NR>, dim3(l.sms * ctas), FewLine<NR>::kThreads, smem, stream, p);
}

template <bool F16, int D>
cudaError_t launch_many(Params p, const Layout& l, uint8_t* ws, cudaStream_t stream) {
  constexpr size_t smem = sizeof(ManySmem<D>) + 1024;
  static_assert(smem <= 227 * 1024, "shared memory of the kernel for many rows over the per-CTA limit");
  CUtensorMap tk, tv;
  cudaError_t e = cache_map(&tk, p.a.k_cache, p.a, kTile);
  if (e == cudaSuccess) e = cache_map(&tv, p.a.v_cache, p.a, kTile);
  if (e == cudaSuccess) e = set_smem_attr_once(reinterpret_cast<const void*>(k_attn_e4m3_many<F16, D>), smem);
  if (e != cudaSuccess) return e;
  l.give(p, kMany, ws);
  return launch_pdl(k_attn_e4m3_many<F16, D>, dim3(l.sms), kManyThreads, smem, stream, tk, tv, p);
}

template <bool F16, int D>
cudaError_t launch_t(const AttnE4m3Args& a, uint8_t* ws, cudaStream_t stream) {
  Params p{};
  p.a = a;
  p.G = a.Hq / a.Hkv;
  p.by_G = Divisor(p.G);
  const int64_t rows = static_cast<int64_t>(a.max_new) * p.G;
  const Layout l = layout(D);
  p.log_page = 4;
  while ((1 << p.log_page) < a.page_size) ++p.log_page;
  p.c = a.scale * 1.4426950408889634f;
  // Requests of up to 32 rows a head (64 with heads of 64), or of up to 8 where a call also has longer ones and a single
  // token's rows are no more (the decoding requests beside prompts), go to the first kernel.  First / second kernel with
  // 24, 32, 40, 48, 64, 96 rows (8 heads a key head), in us: 4 requests over up to 40000 keys 50 / 71, 53 / 72, 72 / 72,
  // 72 / 73, 80 / 71, 114 / 73; 48 over up to 4096 63 / 88, 68 / 88, 89 / 89, 94 / 89, 110 / 88, 154 / 90; heads of 64: the
  // latter 38 / 80, 41 / 79, 52 / 81, 55 / 81, 65 / 81, 89 / 85.
  constexpr int kMost = few_most_rows(D);
  p.few = rows <= kMost || p.G > 8 ? kMost : 8;
  p.beside = rows > kMost;
  if (p.beside) {
    const cudaError_t e = launch_many<F16, D>(p, l, ws, stream);
    if (e != cudaSuccess) return e;
  }
  return std::min<int64_t>(rows, p.few) <= 8 ? launch_few<F16, D, 1>(p, l, ws, stream) : launch_few<F16, D, 2>(p, l, ws, stream);
}

}  // namespace

size_t attn_e4m3_workspace_bytes(int64_t d) { return layout(d).bytes; }

cudaError_t launch_attn_e4m3(int dtype, const AttnE4m3Args& a, void* ws, cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  if (dtype == kF16) return a.d == 64 ? launch_t<true, 64>(a, w, stream) : launch_t<true, 128>(a, w, stream);
  return a.d == 64 ? launch_t<false, 64>(a, w, stream) : launch_t<false, 128>(a, w, stream);
}

}  // namespace wq

// Attention of a batch whose requests share a long prefix, over a cache kept in pages.
//   o = softmax(scale q [Kp; Ks]^T) [Vp; Vs],  lse = log sum exp(scale q [Kp; Ks]^T)
// Kp, Vp: the shared prefix; Ks, Vs: the request's own keys, causal among its new tokens (the
// last of its own keys).
//
// Work.  An item is a set of query rows against one run of keys of one key/value head:
//   prefix items: all T tokens' rows of the head (row = token * G + query head of the group,
//     G = Hq / Hkv), in tiles of up to 2 * tb tokens (tb = 128 / G), against the prefix;
//   suffix items: one request's rows, tiled alike, against its own keys.
// Keys are taken in tiles of 64.  All items' tiles lie on one line (with a weight a tile and a
// constant an item); the line is cut into equal shares, one for each CTA (one per SM), so a CTA
// works through a run of tiles that may begin and end inside items, whatever the lengths are.
// What a CTA computes of an item (a segment: unnormalised output, running maximum and sum) goes
// to the workspace in float32, and a second kernel joins the segments of each row in line order.
//
// A CTA runs two lanes, each a 128-row tensor-core tile with its own output and two buffers of
// scores in tensor memory, its own warp that issues the products, and its own four softmax warps
// (one row a thread):
//   rows mode (more than tb tokens in the item): the lanes hold different rows and both see every
//     key tile, so K and V are read once for 256 rows;
//   keys mode (up to tb tokens): both lanes hold the same rows and take the key tiles in turn (every
//     other item the second lane begins, so that items of one tile keep both lanes busy).
// The products of one tile run while the softmax of the lane's tile before it, and of the other
// lane's tiles, runs:
//   S = Q K^T       both operands from shared memory (TMA, 128-byte swizzle)
//   P = 2^(c S - m) written back over S in tensor memory, 16 bits
//   O += P V        P from tensor memory, V from shared memory, d contiguous (transposed operand)
// Tiles of 64 keys: two buffers of scores a lane then fit beside the outputs (4 x 64 + 2 x 128 =
// 512 columns).  With tiles of 128 keys and one buffer a lane's softmax and its products took
// turns, and the tensor core idled.
// The running maximum is only followed when it grows by more than 2^8 (the output in tensor memory
// is then rescaled); until then P is at most 2^8, which float32 sums and 16-bit P carry as well.
// S has one product of N = 64 a K16 step, which takes the time that reading Q from shared memory takes
// (some 70 cycles), not the tensor core's 32: the tensor pipe bounds rows mode at about two thirds of its
// rate.  2048 rows on 8 heads over 32768 keys: 234 us, 1174 TFLOP/s.  N = 128 (two key tiles) halves that time,
// but needs both score buffers of a lane at once, and the lane then waits for its own products: 284 us;
// with the pair's second P in shared memory, so that the wait ends when the scores are in registers, 298 us
// (P V with both operands in shared memory and V transposed takes some 150 cycles a step).
// Keys mode is bound by the bytes: 262144 keys, 8 rows on 8 heads, 164 us, 6.6 TB/s; 64 requests over up to
// 16384 keys of their own (half of that on average), 64 heads on 8, 325 us, 6.6 TB/s.  Short calls are bound by the chain of dependent loads, waits and launches:
// 2 requests over 500 + 40 keys 11.7 us, of which the second kernel some 3.
// P is rounded to the cache's type for the second product (the tensor core takes both operands in
// one type); the sum of P is kept unrounded in float32.
#include <algorithm>
#include <type_traits>

#include "elem16.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace wq {

__device__ uint32_t g_attn_err;

uint32_t attn_read_and_clear_error() {
  uint32_t v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_attn_err, sizeof(v));
  cudaMemcpyToSymbol(g_attn_err, &z, sizeof(z));
  return v;
}

namespace {

constexpr int kRows = 128;            // rows per lane
constexpr int kTile = 64;             // keys per tile
constexpr int kThreads = 512;         // 2 lanes x 4 softmax warps; K, V and Q copies, a product warp a lane, scheduler
constexpr int kWarps = kThreads / 32;
constexpr int kWTma = 8, kWMma = 10, kWSched = 12, kWQ = 13;   // the last two warps only take part in the set-up
// Registers a thread: 128 at launch; the softmax warps take what the other eight give up.
constexpr int kRegsSoftmax = 168, kRegsOther = 88;
constexpr int kItems = 4;             // items the scheduler is ahead of the other warps
constexpr int kTmemCols = 512;        // two S of 64 columns a lane, then O of 128 a lane
constexpr int kColO = 256;
// Weights on the line, in units of about 200 SM cycles: a key tile in rows mode, in keys mode with
// more than 32 rows (all softmax warps at work) and with up to 32; an item's own cost, alike.  With all tiles
// alike and items free: 128 requests, 64 heads, over 8192 + up to 2048 keys 142 us instead of 112; 48 requests
// of up to 4 new tokens, heads of 64, 43 instead of 31; one weight up or down by 1 moves these by 1 to 5%
// either way.
constexpr int kWRows = 10, kWKeys = 8, kWFew = 5, kWItemRows = 20, kWItem = 16;
constexpr long long kMaxLine = 1ll << 30;
constexpr float kLazy = 8.f;          // rescale when the maximum grew by more than 2^8

// A segment of an item: what one CTA computes of it.
struct __align__(16) Item {
  int lo, hi;        // key tiles; hi = 0: no more
  int len;           // keys of the run
  int kvh;
  int tok0, ntok;    // first token (row of Q) and tokens of the item
  int seg;           // partial slot
  int lim0;          // suffix: keys token 0 of the item sees (token i sees i more)
  int r;             // request, or -1: the prefix
  int pad[3];
};

template <int D>
struct Smem {
  static constexpr int kTileBytes = kTile * D * 2;      // a K or V tile: [D / 64][64 keys][128 B]
  static constexpr int kQBytes = kRows * D * 2;         // a Q tile: [D / 64][128 rows][128 B]
  static constexpr int kStages = D == 128 ? 5 : 8;      // K tiles, and V tiles, in flight
  uint8_t kv[2][kStages][kTileBytes];                   // rings of K and of V tiles
  uint8_t q[2][kQBytes];
  uint64_t full[2][kStages], empty[2][kStages];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2][2], p_full[2][2];                  // [lane][buffer]
  uint64_t pv_done[2], o_full[2], o_empty[2], drain[2];
  uint64_t item_full[kItems], item_empty[kItems];
  Item items[kItems];
  long long scan[kWarps], scan_rest[kWarps];
  int scan_items[kWarps];
  int r0, r0_line, r0_item;
  uint32_t tmem_base;
};

// Where the second kernel finds a token's own-key segments.
struct __align__(16) TokenRecord {
  int line, item;       // of its request's first item
  int len, n;           // own keys and new tokens of the request
  int i, pad[3];        // the token's place among them
};

struct Params {
  AttnArgs a;
  int G, tb;                 // query heads per key/value head; tokens per lane tile (kRows / G)
  int log_page;              // log2 of the page size
  int p_rts, p_full, p_head; // prefix: row tiles of a head, line length of a full one, of a head
  int prefix_tiles;
  int q_rows_suffix;         // rows a suffix lane tile can have (its partial's row capacity)
  int ctas;
  TokenRecord* token;        // [T]
  int* share;                // line units a CTA; 0: nothing to join
  // Prefix partials: [segment][lane][128 / 8][D / 4][8][4] and [segment][lane][128][2]; suffix
  // partials with q_rows_suffix (a multiple of 8) for 128.  Rows go in eights, four columns at a
  // time, so that a warp with a row a thread writes whole 128-byte lines, and so does one that
  // reads eight rows.
  float *po_p, *ml_p;
  float *po_s, *ml_s;
};

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// One request's new tokens and own keys, forced into range.
struct Request {
  int first, n, len;
  bool bad_n, bad_len;
};
__device__ __forceinline__ Request checked(const AttnArgs& a, int r, int first, int end, int len) {
  Request q;
  q.first = first, q.len = len;
  q.n = end - q.first;
  // requests cover the tokens from 0 to T without gaps
  q.bad_n = q.first < 0 || end < q.first || end > a.T || q.n > a.max_new || (r == 0 && q.first != 0) ||
            (r == a.R - 1 && end != a.T);
  if (q.bad_n) q.n = 0, q.first = 0;
  const int cap = a.max_blocks * a.page_size;
  q.bad_len = q.len < 0 || q.len > cap;
  q.len = min(max(q.len, 0), cap);
  return q;
}
__device__ __forceinline__ Request request(const AttnArgs& a, int r) {
  return checked(a, r, a.q_start ? __ldg(a.q_start + r) : r, a.q_start ? __ldg(a.q_start + r + 1) : r + 1,
                 a.max_blocks ? __ldg(a.suffix_lens + r) : 0);
}

// Items of ntok tokens: row tiles, and the tokens of tile rt.
__device__ __forceinline__ int row_tiles(const Params& p, int ntok) {
  return ntok <= 2 * p.tb ? (ntok > 0 ? 1 : 0) : ceil_div(ntok, 2 * p.tb);
}
__device__ __forceinline__ int tile_tokens(const Params& p, int ntok, int rt) { return min(2 * p.tb, ntok - rt * 2 * p.tb); }
// Rows mode or keys mode of an item of so many tokens.  More rows than a lane holds would read K and V
// twice in keys mode.  Rows mode for one lane's rows leaves the other lane idle; rows / keys mode, heads
// of 128, in us: 1 token of 32 heads on 8 over 32768 keys 39.0 / 33.7, 16 tokens of 64 heads 45.0 / 40.0, 32
// requests over 8192 + up to 700 35.0 / 28.5, 64 requests over up to 4096 of their own 115.2 / 93.0.
__host__ __device__ inline bool rows_mode(int tb, int tokens) { return tokens > tb; }
__host__ __device__ inline int tile_weight(int tb, int G, int tokens) {
  return rows_mode(tb, tokens) ? kWRows : (tokens * G > 32 ? kWKeys : kWFew);
}
__host__ __device__ inline int item_weight(int tb, int tokens) { return rows_mode(tb, tokens) ? kWItemRows : kWItem; }
// Line length of an item in rows mode.
__device__ __forceinline__ int full_cost(int tiles) { return tiles * kWRows + kWItemRows; }
// Line length of all row tiles of one head (T is int or, where it may be too long, long long).
template <typename L>
__device__ __forceinline__ L head_cost(const Params& p, int ntok, int tiles) {
  const int rts = row_tiles(p, ntok);
  if (rts == 0 || tiles == 0) return 0;
  const int last = tile_tokens(p, ntok, rts - 1);
  return static_cast<L>(rts - 1) * (static_cast<L>(tiles) * kWRows + kWItemRows) +
         static_cast<L>(tiles) * tile_weight(p.tb, p.G, last) + item_weight(p.tb, last);
}
// First tile of an item (line start s, tiles n of weight w) that starts at or after position b.
// Tile t therefore belongs to the CTA whose share holds position s + t w.
__device__ __forceinline__ int tile_at(int b, int s, int n, int w) {
  const uint32_t x = static_cast<uint32_t>(b - s + w - 1);
  return b <= s ? 0 : min(n, static_cast<int>(w == kWRows ? x / kWRows : (w == kWKeys ? x / kWKeys : x / kWFew)));
}

// Walks over the items of one CTA's share (the scheduler warp).
struct Walk {
  const Params& p;
  int cta, b0, b1;
  int h, t, pline, pitem; // next prefix item and its line position
  int r, kvh, rt, item;   // next suffix item
  int line;               // its line position
  Request q;              // request r
  int raw[3];             // of request r + 1, read ahead: where it ends, the next one's end, own keys

  __device__ Walk(const Params& p_, int share, int prefix_cost, int r0, int r0_line, int r0_item)
      : p(p_), cta(blockIdx.x) {
    b0 = cta * share;
    b1 = b0 + share;
    h = p.a.Hkv, t = 0, pline = 0, pitem = 0;
    if (b0 < prefix_cost) {
      h = b0 / p.p_head;
      t = p.p_rts == 1 ? 0 : min((b0 - h * p.p_head) / p.p_full, p.p_rts - 1);
      pline = h * p.p_head + t * p.p_full;
      pitem = h * p.p_rts + t;
    }
    r = r0, line = r0_line, item = r0_item, kvh = 0, rt = 0;
    if (h == p.a.Hkv && r < p.a.R) {
      q = request(p.a, r);
      read_ahead();
    }
  }

  __device__ void read_ahead() {
    if (r + 1 < p.a.R) {
      raw[0] = p.a.q_start ? __ldg(p.a.q_start + r + 1) : r + 1;
      raw[1] = p.a.q_start ? __ldg(p.a.q_start + r + 2) : r + 2;
      raw[2] = p.a.max_blocks ? __ldg(p.a.suffix_lens + r + 1) : 0;
    }
  }

  __device__ bool next(Item& it) {
    while (h < p.a.Hkv) {
      if (pline >= b1) return false;
      it.ntok = tile_tokens(p, p.a.T, t);
      const int w = tile_weight(p.tb, p.G, it.ntok);
      it.kvh = h, it.r = -1;
      it.lo = tile_at(b0, pline, p.prefix_tiles, w), it.hi = tile_at(b1, pline, p.prefix_tiles, w);
      it.len = p.a.prefix_len;
      it.tok0 = t * 2 * p.tb;
      it.lim0 = p.a.prefix_len;
      it.seg = cta + pitem;
      pline += p.prefix_tiles * w + item_weight(p.tb, it.ntok);
      ++pitem;
      if (it.tok0 + 2 * p.tb >= p.a.T) t = 0, ++h;
      else ++t;
      if (h == p.a.Hkv && r < p.a.R) {         // on to the requests
        q = request(p.a, r);
        read_ahead();
      }
      if (it.lo < it.hi) return true;
    }
    while (r < p.a.R) {
      const int tiles = ceil_div(q.len, kTile), rts = row_tiles(p, q.n);
      if (tiles == 0 || rts == 0 || kvh == p.a.Hkv) {
        ++r, kvh = 0, rt = 0;
        if (r < p.a.R) q = checked(p.a, r, raw[0], raw[1], raw[2]);
        read_ahead();
        continue;
      }
      if (line >= b1) return false;
      it.ntok = tile_tokens(p, q.n, rt);
      const int w = tile_weight(p.tb, p.G, it.ntok);
      it.kvh = kvh, it.r = r;
      it.lo = tile_at(b0, line, tiles, w), it.hi = tile_at(b1, line, tiles, w);
      it.len = q.len;
      it.tok0 = q.first + rt * 2 * p.tb;
      it.lim0 = q.len - q.n + rt * 2 * p.tb + 1;
      it.seg = cta + item;
      line += tiles * w + item_weight(p.tb, it.ntok);
      ++item;
      if (++rt == rts) rt = 0, ++kvh;
      if (it.lo < it.hi) return true;
    }
    return false;
  }
};

// Tiles by which a lane's S = Q K^T runs ahead of its O += P V: two tiles of its own, which are in
// rows mode the next two, in keys mode two of the next four.
__device__ __forceinline__ int k_ahead(bool rows) { return rows ? 2 : 4; }

// A wait of a whole warp: every lane waits (bounded as mbar_wait_short is), and all of them go on or
// none.  The vote is the branch: a barrier that has completed costs half of what a wait by lane and
// a vote on its result does (some 40 cycles instead of 80).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t code) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const long long t0 = clock64();
  while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
    if (__any_sync(0xffffffffu, clock64() - t0 > 4000000000ll)) {
      atomicOr(&g_attn_err, code);
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

template <bool F16, int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn(const __grid_constant__ CUtensorMap tq_p, const __grid_constant__ CUtensorMap tq_s,
           const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const __grid_constant__ Params p) {
  using S = Smem<D>;
  constexpr int NS = S::kStages;
  constexpr int CH = D / 64;
  constexpr uint32_t kQChunk = kRows * 128, kKvChunk = kTile * 128;   // bytes of 64 elements of all rows / keys
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw + smem_align_pad(smem_raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    // K, V and Q tiles are given back by both lanes' product warps
    for (int i = 0; i < 2; ++i) {
      for (int s = 0; s < NS; ++s) mbar_init(&sm.full[i][s], 1), mbar_init(&sm.empty[i][s], 2);
      mbar_init(&sm.q_full[i], 1), mbar_init(&sm.q_empty[i], 2);
      for (int b = 0; b < 2; ++b) mbar_init(&sm.s_full[i][b], 1), mbar_init(&sm.p_full[i][b], 4);
      mbar_init(&sm.pv_done[i], 1), mbar_init(&sm.o_full[i], 1), mbar_init(&sm.o_empty[i], 4);
      mbar_init(&sm.drain[i], 1);
    }
    for (int i = 0; i < kItems; ++i) mbar_init(&sm.item_full[i], 1), mbar_init(&sm.item_empty[i], 13);
    fence_barrier_init();
  }
  if (warp == kWMma) {
    tmem_alloc(&sm.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  if (warp == kWQ && lane == 0) {
    tma_prefetch_desc(&tq_p), tma_prefetch_desc(&tq_s), tma_prefetch_desc(&tk), tma_prefetch_desc(&tv);
  }
  pdl_launch_dependents();
  pdl_wait();

  // ---------------------------------------------------------------- the line: its length, and
  // the request in which this CTA's share begins.  A thread has a request; more requests than
  // threads go in further rounds, their total first.
  const long long prefix_long = static_cast<long long>(p.a.Hkv) * p.p_head;
  Request q0{0, 0, 0, false, false};
  bool bad = false;
  long long c0 = 0, rest = 0;
  int n0 = 0;
  for (int r = threadIdx.x; r < p.a.R; r += kThreads) {
    const Request q = request(p.a, r);
    const int tiles = ceil_div(q.len, kTile);
    const long long c = p.a.Hkv * head_cost<long long>(p, q.n, tiles);
    bad |= q.bad_n;
    if (blockIdx.x == 0 && (q.bad_n || q.bad_len)) atomicOr(&g_attn_err, kErrIndex);
    if (r == threadIdx.x) q0 = q, c0 = c, n0 = tiles ? p.a.Hkv * row_tiles(p, q.n) : 0;
    else rest += c;
  }
  long long ic = c0;                      // inclusive scans over the warp
  int in = n0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long uc = __shfl_up_sync(0xffffffffu, ic, o);
    const int un = __shfl_up_sync(0xffffffffu, in, o);
    if (lane >= o) ic += uc, in += un;
  }
  if (p.a.R > kThreads) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, o);
  }
  if (lane == 31) sm.scan[warp] = ic, sm.scan_items[warp] = in, sm.scan_rest[warp] = rest;
  if (threadIdx.x == 0) sm.r0 = p.a.R, sm.r0_line = 0, sm.r0_item = 0;
  bad = __syncthreads_or(bad);
  long long total = prefix_long, at_long = prefix_long, run_long = prefix_long;
  int item = 0, run_items = 0;
  const int with_requests = min(kWarps, (p.a.R + 31) / 32);
#pragma unroll 4
  for (int w = 0; w < with_requests; ++w) {
    const long long wc = sm.scan[w];
    total += wc + (p.a.R > kThreads ? sm.scan_rest[w] : 0);
    run_long += wc, run_items += sm.scan_items[w];
    if (w < warp) at_long += wc, item += sm.scan_items[w];
  }
  if (total > kMaxLine) {                 // too long for the line's 32 bits: reported
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_attn_err, kErrIndex);
    bad = true;
  }
  // Nothing is computed then, nor where a q_start does not cover the tokens once each: the workspace's
  // partials are counted for requests whose new tokens add up to T.
  if (bad) total = 0;
  const bool work = total > 0;
  const int prefix_cost = static_cast<int>(prefix_long > kMaxLine ? 0 : prefix_long);
  // at least a tile for each lane
  const int share = max(2 * kWRows, static_cast<int>((static_cast<uint32_t>(total) + p.ctas - 1) / static_cast<uint32_t>(p.ctas)));
  const int b0 = blockIdx.x * share;
  const auto place = [&](int r, const Request& q, int at, int c, int first_item) {
    if (blockIdx.x == 0)
      for (int i = 0; i < q.n; ++i) p.token[q.first + i] = TokenRecord{at, first_item, q.len, q.n, i, {0, 0, 0}};
    // the first request whose items reach past b0
    if ((at <= b0 && b0 < at + c) || (r == 0 && b0 < prefix_cost)) sm.r0 = r, sm.r0_line = at, sm.r0_item = first_item;
  };
  if (work) {
    if (static_cast<int>(threadIdx.x) < p.a.R)
      place(threadIdx.x, q0, static_cast<int>(at_long + ic - c0), static_cast<int>(c0), item + in - n0);
    int run = static_cast<int>(run_long);
    for (int base = kThreads; base < p.a.R; base += kThreads) {
      const int r = base + threadIdx.x;
      int c = 0, n = 0;
      Request q{0, 0, 0, false, false};
      if (r < p.a.R) {
        q = request(p.a, r);
        const int tiles = ceil_div(q.len, kTile);
        c = p.a.Hkv * head_cost<int>(p, q.n, tiles);
        n = tiles ? p.a.Hkv * row_tiles(p, q.n) : 0;
      }
      int sc = c, sn = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int uc = __shfl_up_sync(0xffffffffu, sc, o), un = __shfl_up_sync(0xffffffffu, sn, o);
        if (lane >= o) sc += uc, sn += un;
      }
      __syncthreads();
      if (lane == 31) sm.scan[warp] = sc, sm.scan_items[warp] = sn;
      __syncthreads();
      int at = run + sc - c, first_item = run_items + sn - n;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const int wc = static_cast<int>(sm.scan[w]), wi = sm.scan_items[w];
        if (w < warp) at += wc, first_item += wi;
        run += wc, run_items += wi;
      }
      if (r < p.a.R) place(r, q, at, c, first_item);
    }
  } else if (!bad && blockIdx.x == 0) {
    // nobody sees any key: the join still writes every row's 0 and -inf
    for (int t = threadIdx.x; t < p.a.T; t += kThreads) p.token[t] = TokenRecord{0, 0, 0, 1, 0, {0, 0, 0}};
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.share = bad ? 0 : share;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  // The next segment, in its place in the ring, or null at the end or after a wait that ran out;
  // given back when the warp is done with it.
  uint32_t n_items = 0;
  bool ok = true;
  const auto next_item = [&]() -> const Item* {
    ok = warp_wait(&sm.item_full[n_items % kItems], (n_items / kItems) & 1, kErrWaitFull);
    const Item* it = &sm.items[n_items % kItems];
    return ok && it->hi > 0 ? it : nullptr;
  };
  // The one after it, without leaving it (waits for the scheduler, which is up to kItems ahead).
  const auto peek_item = [&]() -> const Item* {
    const uint32_t i = n_items + 1;
    ok = warp_wait(&sm.item_full[i % kItems], (i / kItems) & 1, kErrWaitFull);
    const Item* it = &sm.items[i % kItems];
    return ok && it->hi > 0 ? it : nullptr;
  };
  const auto item_done = [&] {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.item_empty[n_items % kItems]);
    ++n_items;
  };

  if (warp >= kWTma) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
  if (warp == kWTma || warp == kWTma + 1) {
    // -------------------------------------------------------------------- TMA producers: K, V
    // With pages of 16 tokens a tile is eight copies, and each takes some 40 cycles to issue, so K
    // and V (and Q) have a warp each.  One elected lane issues; the page numbers come to it by
    // shuffles.
    const CUtensorMap* map = warp == kWTma ? &tk : &tv;
    const int ring = warp - kWTma;
    const uint64_t pol_keep = l2_policy_evict_last(), pol_once = l2_policy_evict_first();
    // boxes of 2^lb rows, 2^lt of them a tile, 2^lp of them a page
    const int lb = min(p.log_page, 6), lt = 6 - lb, lp = p.log_page - lb;
    uint32_t ord = 0;
    // Page numbers: lane i holds that of box base + i of the segment, read 32 boxes ahead and, for the
    // first 32 boxes, while the segment before is being loaded.
    const auto boxes_of = [&](const Item* it) {
      return min(((it->len + (1 << lb) - 1) >> lb) - (it->lo << lt), (it->hi - it->lo) << lt);
    };
    const auto page_ids = [&](const Item* it, int n_boxes, int base) {
      const int32_t* list = it->r < 0 ? p.a.prefix_pages : p.a.block_table + static_cast<int64_t>(it->r) * p.a.max_blocks;
      return base + lane < n_boxes ? __ldg(list + (((it->lo << lt) + base + lane) >> lp)) : 0;
    };
    // their rows of the tensor map, page * Hkv + head; -1: zero fill
    const auto map_row = [&](int id, int kvh) {
      if (static_cast<uint32_t>(id) < static_cast<uint32_t>(p.a.pages)) return id * p.a.Hkv + kvh;
      atomicOr(&g_attn_err, kErrIndex);
      return -1;
    };
    const Item* it = next_item();
    int raw = it ? page_ids(it, boxes_of(it), 0) : 0;
    while (it) {
      const int first = it->lo << lt, n = it->hi - it->lo, kvh = it->kvh, n_boxes = boxes_of(it);
      const uint64_t pol = it->r < 0 ? pol_keep : pol_once;
      int row = map_row(raw, kvh), raw_next = n_boxes > 32 ? page_ids(it, n_boxes, 32) : 0;
      const Item* after = peek_item();
      if (!ok) break;
      raw = after ? page_ids(after, boxes_of(after), 0) : 0;
#pragma unroll 1
      for (int j = 0; j < n; ++j, ++ord) {
        const int s = ord % NS, b0 = j << lt, here = min(1 << lt, n_boxes - b0);
        const int in_page = ((first + b0) & ((1 << lp) - 1)) << lb;    // pages of 128: one box a tile, half a page
        int rows[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) rows[i] = __shfl_sync(0xffffffffu, row, (b0 + i) & 31);
        ok = warp_wait(&sm.empty[ring][s], ((ord / NS) & 1) ^ 1, kErrWaitEmpty);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&sm.full[ring][s], (here << lb) * 128 * CH);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < here) {
#pragma unroll
              for (int c = 0; c < CH; ++c)
                tma_load_4d(&sm.kv[ring][s][c * kKvChunk + ((i << lb) * 128)], map, 0, in_page, c, rows[i], &sm.full[ring][s],
                            pol);
            }
        }
        __syncwarp();
        if (((b0 + (1 << lt)) & 31) == 0 && j + 1 < n) {
          row = map_row(raw_next, kvh);
          raw_next = page_ids(it, n_boxes, b0 + (1 << lt) + 32);
        }
      }
      if (!ok) break;
      item_done();
      it = after;
    }
    // drain: the last fill of each slot has landed before the CTA's memory goes
    for (uint32_t i = ord > NS ? ord - NS : 0; i < ord; ++i)
      mbar_wait_short(&sm.full[ring][i % NS], (i / NS) & 1, &g_attn_err, kErrDrain);
  } else if (warp == kWQ) {
    // -------------------------------------------------------------------- TMA producer: Q
    const uint64_t pol_keep = l2_policy_evict_last();
    uint32_t qord = 0;
    while (const Item* it = next_item()) {   // one 128-row tile, or one per lane
      const bool prefix = it->r < 0;
      const int box_tok = prefix ? p.tb : min(p.tb, p.a.max_new);
      for (int i = 0; i < (rows_mode(p.tb, it->ntok) ? 2 : 1); ++i, ++qord) {
        const int s = qord & 1;
        ok = warp_wait(&sm.q_empty[s], ((qord >> 1) & 1) ^ 1, kErrWaitEmpty);
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&sm.q_full[s], box_tok * p.G * 128 * CH);
#pragma unroll
          for (int c = 0; c < CH; ++c)
            tma_load_4d(&sm.q[s][c * kQChunk], prefix ? &tq_p : &tq_s, 0, c, it->kvh * p.G, it->tok0 + i * p.tb, &sm.q_full[s],
                        pol_keep);
        }
        __syncwarp();
      }
      if (!ok) break;
      item_done();
    }
    for (uint32_t i = qord > 2 ? qord - 2 : 0; i < qord; ++i)
      mbar_wait_short(&sm.q_full[i & 1], (i >> 1) & 1, &g_attn_err, kErrDrain);
  } else if (warp == kWSched) {
    // -------------------------------------------------------------------- scheduler
    if (lane == 0) {
      Walk walk(p, share, work ? prefix_cost : 0, work ? sm.r0 : p.a.R, sm.r0_line, sm.r0_item);
      bool more = true;
      for (uint32_t i = 0; more; ++i) {
        Item x{};
        more = walk.next(x);
        if (!more) x.hi = 0;
        if (!mbar_wait_short(&sm.item_empty[i % kItems], ((i / kItems) & 1) ^ 1, &g_attn_err, kErrWaitEmpty)) break;
        sm.items[i % kItems] = x;
        mbar_arrive(&sm.item_full[i % kItems]);
      }
    }
  } else if (warp == kWMma || warp == kWMma + 1) {
    // -------------------------------------------------------------------- products of lane l
    const int l = warp - kWMma;
    constexpr uint32_t fmt = F16 ? 0u : 1u;
    constexpr uint32_t id_qk = (1u << 4) | (fmt << 7) | (fmt << 10) | ((kTile >> 3) << 17) | ((kRows >> 4) << 24);
    constexpr uint32_t id_pv = (1u << 4) | (fmt << 7) | (fmt << 10) | (1u << 16) | ((D >> 3) << 17) | ((kRows >> 4) << 24);
    const uint32_t t_s = tmem + 128 * l, t_o = tmem + kColO + 128 * l;
    const uint64_t k0 = smem_desc_sw128(smem_u32(&sm.kv[0][0][0])), v0 = smem_desc_sw128_mn(smem_u32(&sm.kv[1][0][0]), kKvChunk);
    const uint64_t q0 = smem_desc_sw128(smem_u32(&sm.q[0][0]));
    uint32_t k_ord = 0, v_ord = 0, qord = 0, o_cnt = 0;
    uint32_t s_cnt = 0, p_cnt = 0;            // tiles of this lane whose S was issued / whose P was taken
    // Every slot of the rings is waited for and given back once by each lane, also where only the
    // other lane uses it: a wait by parity is only sound if no phase of the slot is left out.
    while (const Item* it = next_item()) {
      const int n = it->hi - it->lo;
      const bool rows = rows_mode(p.tb, it->ntok);
      const int nq = rows ? 2 : 1, ahead = k_ahead(rows), flip = n_items & 1;
      const uint64_t qd = q0 + ((qord + (rows ? l : 0)) & 1) * (S::kQBytes >> 4);
      for (int i = 0; i < nq && ok; ++i) ok = warp_wait(&sm.q_full[(qord + i) & 1], ((qord + i) >> 1) & 1, kErrWaitFull);
      if (!ok) break;
      const auto qk = [&](int j) {              // S = Q K(j)^T
        const uint32_t sl = k_ord % NS;
        ok = warp_wait(&sm.full[0][sl], (k_ord / NS) & 1, kErrWaitFull);
        if (!ok) return;
        ++k_ord;
        if (!rows && ((j ^ flip) & 1) != l) {   // a tile of the other lane
          if (elect_one()) mbar_arrive(&sm.empty[0][sl]);
          __syncwarp();
          return;
        }
        const uint64_t kd = k0 + sl * (S::kTileBytes >> 4);
        const uint32_t b = s_cnt & 1, t = t_s + 64 * b;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4 * CH; ++k)
            tc_mma_ss_f16(t, qd + (((k >> 2) * kQChunk + 32 * (k & 3)) >> 4), kd + (((k >> 2) * kKvChunk + 32 * (k & 3)) >> 4),
                          id_qk, k ? 1u : 0u);
          tc_commit(&sm.s_full[l][b]);
          tc_commit(&sm.empty[0][sl]);
        }
        __syncwarp();
        ++s_cnt;
      };
      const auto pv = [&](int j) {              // O += P(j) V(j)
        const uint32_t sl = v_ord % NS;
        ok = warp_wait(&sm.full[1][sl], (v_ord / NS) & 1, kErrWaitFull);
        if (!ok) return;
        ++v_ord;
        if (!rows && ((j ^ flip) & 1) != l) {
          if (elect_one()) mbar_arrive(&sm.empty[1][sl]);
          __syncwarp();
          return;
        }
        const bool first = rows ? j == 0 : j < 2, last = j + (rows ? 1 : 2) >= n;
        // first: the lane's previous item has left the output columns
        if (first) ok = warp_wait(&sm.o_empty[l], (o_cnt++ & 1) ^ 1, kErrWaitAccum);
        const uint32_t b = p_cnt & 1, t = t_s + 64 * b;
        ok = ok && warp_wait(&sm.p_full[l][b], (p_cnt >> 1) & 1, kErrWaitFull);
        if (!ok) return;
        const uint64_t vd = v0 + sl * (S::kTileBytes >> 4);
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kTile / 16; ++k)
            tc_mma_ts(t_o, t + 8 * k, vd + ((k * 2048) >> 4), id_pv, (first && k == 0) ? 0u : 1u);
          tc_commit(&sm.pv_done[l]);
          if (last) tc_commit(&sm.o_full[l]);
          tc_commit(&sm.empty[1][sl]);
        }
        __syncwarp();
        ++p_cnt;
      };
#pragma unroll 1
      for (int j = 0; j < n + ahead && ok; ++j) {
        if (j >= ahead) pv(j - ahead);
        if (ok && j < n) qk(j);
      }
      if (!ok) break;
      if (elect_one())
        for (int i = 0; i < nq; ++i) tc_commit(&sm.q_empty[(qord + i) & 1]);
      qord += nq;
      item_done();
    }
    // every product and commit of this warp (elect.sync names the same lane each time) has completed before tensor memory and barriers go
    if (elect_one()) tc_commit(&sm.drain[l]);
    mbar_wait_short(&sm.drain[l], 0, &g_attn_err, kErrDrain);
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // -------------------------------------------------------------------- softmax, one row a thread
    const int l = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_o = tmem + lane_base + kColO + 128 * l;
    const float c = p.a.scale * 1.4426950408889634f;
    const uint64_t c2 = pair(__float_as_uint(c), __float_as_uint(c));
    const int tok = row / p.G;
    uint32_t cnt = 0, o_cnt = 0, v_end = 0;     // tiles of this lane so far; V tiles of all items so far
    while (const Item* it = next_item()) {
      const int lo = it->lo, n = it->hi - lo, len = it->len;
      const bool prefix = it->r < 0, rows = rows_mode(p.tb, it->ntok);
      const int tok_item = tok + (rows && l ? p.tb : 0);
      const bool valid = tok < p.tb && tok_item < it->ntok;
      const bool active = __any_sync(0xffffffffu, valid);
      // keys this row sees
      const int lim = !valid ? 0 : (prefix ? len : min(max(it->lim0 + tok_item, 0), len));
      float m = -INFINITY, sum = 0.f;           // m in units of log2, already times c
      v_end += n;
      const int j0 = rows ? 0 : l ^ static_cast<int>(n_items & 1), step = rows ? 1 : 2;
#pragma unroll 1
      for (int j = j0; j < n; j += step, ++cnt) {
        const int key0 = (lo + j) * kTile;
        const uint32_t b = cnt & 1, t_s = tmem + lane_base + 128 * l + 64 * b;
        ok = warp_wait(&sm.s_full[l][b], (cnt >> 1) & 1, kErrWaitAccum);
        if (!ok) break;
        tc_fence_after();
        if (active) {
          uint32_t v[2][32];
          tmem_ld32(t_s, v[0]);
          tmem_ld32(t_s + 32, v[1]);
          tc_wait_ld();
          if (__builtin_expect(__any_sync(0xffffffffu, valid && key0 + kTile > lim), 0)) {
            const int left = lim - key0;
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (32 * q + e >= left) v[q][e] = 0xff800000u;
          }
          float mq[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t* w = &v[q >> 1][16 * (q & 1)];
            mq[q] = fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1]));
#pragma unroll
            for (int e = 2; e < 16; e += 2) mq[q] = max3(mq[q], __uint_as_float(w[e]), __uint_as_float(w[e + 1]));
          }
          const float mc = fmaxf(max3(mq[0], mq[1], mq[2]), mq[3]) * c;
          const bool grow = valid && mc > m + kLazy;
          if (__builtin_expect(__any_sync(0xffffffffu, grow), 0)) {
            const float keep = grow ? exp2_approx(m - mc) : 1.f;
            if (grow) m = mc;
            sum *= keep;
            if (j != j0) {
              // the lane's last product has left the output (one phase at most is outstanding: this
              // tile's S was issued after the product before that one)
              ok = warp_wait(&sm.pv_done[l], (cnt - 1) & 1, kErrWaitAccum);
              if (!ok) break;
              tc_fence_after();
              const uint64_t keep2 = pair(__float_as_uint(keep), __float_as_uint(keep));
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
          const uint32_t base = __float_as_uint(m == -INFINITY ? 0.f : -m);
          const uint64_t base2 = pair(base, base);
          uint64_t sums[2] = {0, 0};
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 x = unpair(fma_pair(pair(v[q][2 * e], v[q][2 * e + 1]), c2, base2));
              const float a = exp2_approx(x.x), d = exp2_approx(x.y);
              sums[e & 1] = add_pair(sums[e & 1], pair(__float_as_uint(a), __float_as_uint(d)));
              w[e] = pack2<F16>(a, d);
            }
            tmem_st16(t_s + 16 * q, w);
          }
          const float2 s2 = unpair(add_pair(sums[0], sums[1]));
          sum += s2.x + s2.y;
          tc_wait_st();
        }
        // V rows past the run's end hold whatever the page or the slot held: zero them, since
        // their weight 0 times a NaN would not be 0 (in rows mode both lanes write the same zeros,
        // each before its own product).  Only an item's last tile has such rows.
        if (__builtin_expect(key0 + kTile > len, 0)) {
          const uint32_t vo = v_end - 1;
          ok = warp_wait(&sm.full[1][vo % NS], (vo / NS) & 1, kErrWaitFull);
          if (!ok) break;
          if ((row & 63) >= len - key0 && (row >> 6) < CH) {
            uint4* z = reinterpret_cast<uint4*>(&sm.kv[1][vo % NS][(row >> 6) * kKvChunk + (row & 63) * 128]);
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[l][b]);
      }
      if (!ok) break;
      // ---------------------------------------------------------------- the segment's partial
      const int cap = prefix ? kRows : p.q_rows_suffix;
      const long long slot = 2ll * it->seg + l;
      if (j0 < n) {
        ok = warp_wait(&sm.o_full[l], o_cnt++ & 1, kErrWaitAccum);
        if (!ok) break;
        tc_fence_after();
        if (active) {
          float4* po = reinterpret_cast<float4*>(prefix ? p.po_p : p.po_s) + (slot * (cap >> 3) + (row >> 3)) * (2 * D) + (row & 7);
          uint32_t o[D / 32][32];
#pragma unroll
          for (int q = 0; q < D / 32; ++q) tmem_ld32(t_o + 32 * q, o[q]);
          tc_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.o_empty[l]);
          if (valid) {
#pragma unroll
            for (int q = 0; q < D / 32; ++q)
#pragma unroll
              for (int e = 0; e < 8; ++e)
                po[8 * (8 * q + e)] = make_float4(__uint_as_float(o[q][4 * e]), __uint_as_float(o[q][4 * e + 1]),
                                            __uint_as_float(o[q][4 * e + 2]), __uint_as_float(o[q][4 * e + 3]));
          }
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.o_empty[l]);
        }
      }
      if (valid) reinterpret_cast<float2*>(prefix ? p.ml_p : p.ml_s)[slot * cap + row] = make_float2(m, sum);
      item_done();
    }
  }
  __syncwarp();
  __syncthreads();
  if (warp == kWMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the segments of each row.  A warp has eight consecutive rows of one key/value head (row =
// token * G + query head of the group) and a C-th of their columns: lane 8c + i has row i and a
// quarter (c) of those columns.  W warps take the rows' segments in turn, and the first of them adds
// up what they found.
constexpr int kJoinWarps = 8;
template <bool F16, int D, int W, int C>
__global__ void __launch_bounds__(kJoinWarps * 32) k_attn_join(const __grid_constant__ Params p) {
  constexpr int E = D / 4 / C;                          // columns of a lane
  extern __shared__ float part[];                       // [E + 2][warp][32]
  __shared__ float weights[kJoinWarps][32][8];
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w0 = warp % W;
  const int row_all = (blockIdx.x * (kJoinWarps / W) + warp / W) * 8 + (lane & 7), kvh = blockIdx.y;
  const int t = row_all / p.G, g = row_all - t * p.G, col = (blockIdx.z * 4 + (lane >> 3)) * (E / 4);   // first group of four columns
  const bool here = t < p.a.T;
  pdl_wait();
  const int share = __ldcg(p.share);
  const int4 rec = here ? __ldcg(reinterpret_cast<const int4*>(p.token + t)) : make_int4(0, 0, 0, 1);
  const int i_tok = here ? __ldcg(&p.token[t].i) : 0;
  if (share == 0) return;                               // the requests do not cover the tokens

  // The segments of one run of keys that hold the row: slots first, first + step, ...
  struct Run {
    int first, count, step, row;
  };
  const auto find = [&](int tok, int ntok_all, int tiles, int line, int head, int ordinal) {
    Run r{0, 0, 1, 0};
    if (tiles == 0) return r;
    const int span = 2 * p.tb, rt = ntok_all <= span ? 0 : tok / span, ntok = tile_tokens(p, ntok_all, rt);
    const bool rows = rows_mode(p.tb, ntok);
    const int w = tile_weight(p.tb, p.G, ntok);
    const int s = line + kvh * head + (rt ? rt * full_cost(tiles) : 0);
    const int c0 = s / share, c1 = (s + (tiles - 1) * w) / share;
    const int in_tile = tok - rt * span, half = in_tile >= p.tb ? 1 : 0;
    r.row = (in_tile - half * p.tb) * p.G + g;
    r.first = 2 * (c0 + ordinal + kvh * row_tiles(p, ntok_all) + rt) + (rows ? half : 0);
    r.count = (c1 - c0 + 1) * (rows ? 1 : 2);
    r.step = rows ? 2 : 1;                              // keys mode: both lanes' slots hold the row
    return r;
  };
  const int tiles_s = ceil_div(rec.z, kTile);
  const Run run_p = find(t, p.a.T, here ? p.prefix_tiles : 0, 0, p.p_head, 0);
  const Run run_s = find(i_tok, rec.w, here ? tiles_s : 0, rec.x, head_cost<int>(p, rec.w, tiles_s), rec.y);
  const int n = run_p.count + run_s.count;
  const auto slot = [&](int i, bool& in_p) {
    in_p = i < run_p.count;
    return in_p ? run_p.first + i * run_p.step : run_s.first + (i - run_p.count) * run_s.step;
  };
  // Rounds of 32 segments: their statistics first (eight loads a lane, all under way at once), the
  // weights into shared memory, then the outputs, whose loads wait for nothing.
  float(*wt)[8] = weights[warp];
  float top = -INFINITY, total = 0.f;
  float4 o[E / 4];
#pragma unroll
  for (int e = 0; e < E / 4; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int most = __reduce_max_sync(0xffffffffu, n);
  const auto source = [&](int i) {                      // a lane's columns of segment i
    bool in_p;
    const long long s = slot(i, in_p);
    const int cap8 = in_p ? kRows / 8 : p.q_rows_suffix >> 3, row = in_p ? run_p.row : run_s.row;
    return reinterpret_cast<const float4*>(in_p ? p.po_p : p.po_s) + (s * cap8 + (row >> 3)) * (2 * D) + (row & 7) + col * 8;
  };
  // The first segments' outputs come beside the statistics, whether they will count or not: four where
  // the warps are few (C = 4: 1 request over 500 keys 12.4 -> 11.6 us, 2 over 8192 17.9 -> 16.4, 16 over 8192 + up to
  // 700 23.9 -> 21.9), else half as many (48 requests of up to 4 new tokens: 31.5 us with none, 31.0 with two, 32.4
  // with four).
  constexpr int kAhead = C == 4 ? 4 : E <= 16 ? 16 / E : 1;
  float4 first[kAhead][E / 4];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const float4* src = w0 + k * W < n ? source(w0 + k * W) : reinterpret_cast<const float4*>(p.po_s);
#pragma unroll
    for (int e = 0; e < E / 4; ++e) first[k][e] = __ldcg(src + 8 * e);
  }
  for (int base = w0; base < most; base += 32 * W) {
    float2 ml[8];
    float m2 = top;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = base + (4 * k + (lane >> 3)) * W;
      bool in_p;
      const long long s = slot(i, in_p);
      ml[k] = i < n ? __ldcg(reinterpret_cast<const float2*>(in_p ? p.ml_p : p.ml_s) +
                             s * (in_p ? kRows : p.q_rows_suffix) + (in_p ? run_p.row : run_s.row))
                    : make_float2(-INFINITY, 0.f);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) m2 = fmaxf(m2, ml[k].x);
    m2 = fmaxf(m2, __shfl_xor_sync(0xffffffffu, m2, 8));
    m2 = fmaxf(m2, __shfl_xor_sync(0xffffffffu, m2, 16));
    const float ref = m2 == -INFINITY ? 0.f : m2, keep = exp2_approx(top - ref);
    float add = 0.f;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      // No tile, or nothing seen: maybe no output either, so not read; the sign of its weight -0 says so.  A weight
      // that is too small for float32 is 0 and read, since 0 times an infinity or a NaN is NaN.  A sum that is NaN
      // counts whatever the weight: NaN scores raise no maximum, which may be -inf, or far below the row's.
      const float f = ml[k].y == 0.f ? -0.f : ml[k].y != ml[k].y ? __uint_as_float(0x7fffffffu) : exp2_approx(ml[k].x - ref);
      add = fmaf(ml[k].y, f, add);
      wt[4 * k + (lane >> 3)][lane & 7] = f;
    }
    __syncwarp();
    add += __shfl_xor_sync(0xffffffffu, add, 8);
    add += __shfl_xor_sync(0xffffffffu, add, 16);
    top = m2;
    total = fmaf(total, keep, add);
    if (base != w0) {
#pragma unroll
      for (int e = 0; e < E / 4; ++e) o[e].x *= keep, o[e].y *= keep, o[e].z *= keep, o[e].w *= keep;
    }
    const int here_n = min(32, (most - base + W - 1) / W);
    const auto add_part = [&](const float4 (&v)[E / 4], float f) {
      const bool live = __float_as_int(f) >= 0;
#pragma unroll
      for (int e = 0; e < E / 4; ++e) {
        o[e].x = fmaf(live ? v[e].x : 0.f, f, o[e].x), o[e].y = fmaf(live ? v[e].y : 0.f, f, o[e].y);
        o[e].z = fmaf(live ? v[e].z : 0.f, f, o[e].z), o[e].w = fmaf(live ? v[e].w : 0.f, f, o[e].w);
      }
    };
    int k0 = 0;
    if (base == w0) {
      k0 = kAhead;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) add_part(first[k], wt[k][lane & 7]);
    }
#pragma unroll(E >= 16 ? 2 : 8)
    for (int k = k0; k < here_n; ++k) {
      const float f = wt[k][lane & 7];
      // without a branch, so that several segments' loads are under way: a row without this segment
      // loads some line of the workspace and drops it
      const float4* src = __float_as_int(f) >= 0 ? source(base + k * W) : reinterpret_cast<const float4*>(p.po_s);
      float4 v[E / 4];
#pragma unroll
      for (int e = 0; e < E / 4; ++e) v[e] = __ldcg(src + 8 * e);
      add_part(v, f);
    }
  }
  if constexpr (W > 1) {
    const auto at = [&](int k, int w) -> float& { return part[(k * kJoinWarps + w) * 32 + lane]; };
    at(0, warp) = top, at(1, warp) = total;
#pragma unroll
    for (int e = 0; e < E / 4; ++e)
      at(2 + 4 * e, warp) = o[e].x, at(3 + 4 * e, warp) = o[e].y, at(4 + 4 * e, warp) = o[e].z, at(5 + 4 * e, warp) = o[e].w;
    __syncthreads();
    if (w0 != 0) return;
#pragma unroll
    for (int w = 1; w < W; ++w) top = fmaxf(top, at(0, warp + w));
    const float all = top == -INFINITY ? 0.f : top;
    total = 0.f;
#pragma unroll
    for (int e = 0; e < E / 4; ++e) o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int w = 0; w < W; ++w) {
      const float f = exp2_approx(at(0, warp + w) - all);
      total = fmaf(at(1, warp + w), f, total);
#pragma unroll
      for (int e = 0; e < E / 4; ++e) {
        o[e].x = fmaf(at(2 + 4 * e, warp + w), f, o[e].x), o[e].y = fmaf(at(3 + 4 * e, warp + w), f, o[e].y);
        o[e].z = fmaf(at(4 + 4 * e, warp + w), f, o[e].z), o[e].w = fmaf(at(5 + 4 * e, warp + w), f, o[e].w);
      }
    }
  }
  if (!here) return;
  const float inv = total == 0.f ? 0.f : 1.f / total;
  const long long row_out = static_cast<long long>(t) * p.a.Hq + kvh * p.G + g;
  uint2* dst = reinterpret_cast<uint2*>(p.a.O + row_out * D + 4 * col);
#pragma unroll
  for (int e = 0; e < E / 4; ++e)
    dst[e] = make_uint2(pack2<F16>(o[e].x * inv, o[e].y * inv), pack2<F16>(o[e].z * inv, o[e].w * inv));
  if (lane < 8 && blockIdx.z == 0 && p.a.lse)
    p.a.lse[row_out] = total == 0.f ? -INFINITY : ((top == -INFINITY ? 0.f : top) + log2f(total)) * 0.6931471805599453f;
}
template <int D>
constexpr size_t kJoinSmem = static_cast<size_t>(D / 4 + 2) * kJoinWarps * 32 * 4;   // C = 1

struct Layout {
  int G, tb, n_prefix, rows_s, ctas;
  size_t token, share, po_p, ml_p, po_s, ml_s, bytes;
};

Layout layout(int64_t T, int64_t R, int64_t Hq, int64_t Hkv, int64_t d, int64_t max_new) {
  Layout l{};
  l.G = static_cast<int>(Hq / Hkv);
  l.tb = kRows / l.G;
  l.ctas = device_sm_count();
  const int64_t span = 2 * l.tb;
  l.n_prefix = static_cast<int>(Hkv * ((T + span - 1) / span));
  // requests' row tiles: no more than one each and one more for every full tile of tokens
  const int64_t tiles_each = (max_new + span - 1) / span;
  const int64_t n_suffix = Hkv * std::min(R * tiles_each, R + T / span);
  l.rows_s = static_cast<int>(std::min<int64_t>(kRows, (max_new * l.G + 7) / 8 * 8));
  size_t off = kWsHeaderBytes;
  const auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  l.token = take(T * sizeof(TokenRecord));
  l.share = take(sizeof(int));
  const size_t sp = 2 * static_cast<size_t>(l.ctas + l.n_prefix), ss = 2 * static_cast<size_t>(l.ctas + n_suffix);
  l.po_p = take(sp * kRows * d * sizeof(float));
  l.ml_p = take(sp * kRows * 2 * sizeof(float));
  l.po_s = take(ss * l.rows_s * d * sizeof(float));
  l.ml_s = take(ss * l.rows_s * 2 * sizeof(float));
  l.bytes = off;
  return l;
}

// The prefix's items on the line: row tiles of a head, the length of a full one and of all of them.
struct PrefixLine {
  int row_tiles;
  long long full, head;
  PrefixLine(int64_t T, int64_t prefix_len, int tb, int G) {
    const int64_t tiles = (prefix_len + kTile - 1) / kTile, span = 2 * tb;
    row_tiles = static_cast<int>((T + span - 1) / span);
    const int last = static_cast<int>(T - (row_tiles - 1) * span);
    full = tiles * kWRows + kWItemRows;
    head = tiles ? (row_tiles - 1) * full + tiles * tile_weight(tb, G, last) + item_weight(tb, last) : 0;
  }
};

template <bool F16, int D>
cudaError_t launch_t(const AttnArgs& a, uint8_t* ws, cudaStream_t stream) {
  const Layout l = layout(a.T, a.R, a.Hq, a.Hkv, D, a.max_new);
  Params p{};
  p.a = a;
  p.G = l.G, p.tb = l.tb;
  p.log_page = 4;
  while ((1 << p.log_page) < a.page_size) ++p.log_page;
  p.prefix_tiles = (a.prefix_len + kTile - 1) / kTile;
  const PrefixLine line(a.T, a.prefix_len, p.tb, p.G);
  p.p_rts = line.row_tiles, p.p_full = static_cast<int>(line.full), p.p_head = static_cast<int>(line.head);
  p.q_rows_suffix = l.rows_s;
  p.ctas = l.ctas;
  p.token = reinterpret_cast<TokenRecord*>(ws + l.token);
  p.share = reinterpret_cast<int*>(ws + l.share);
  p.po_p = reinterpret_cast<float*>(ws + l.po_p), p.ml_p = reinterpret_cast<float*>(ws + l.ml_p);
  p.po_s = reinterpret_cast<float*>(ws + l.po_s), p.ml_s = reinterpret_cast<float*>(ws + l.ml_s);

  const CUtensorMapDataType dt = F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  CUtensorMap tq_p, tq_s, tk, tv;
  const uint64_t qd[4] = {64, D / 64, static_cast<uint64_t>(a.Hq), static_cast<uint64_t>(a.T)};
  const uint64_t qs[3] = {128, D * 2, static_cast<uint64_t>(a.q_stride) * 2};
  const uint32_t bp[4] = {64, 1, static_cast<uint32_t>(p.G), static_cast<uint32_t>(p.tb)};
  const uint32_t bs[4] = {64, 1, static_cast<uint32_t>(p.G), static_cast<uint32_t>(std::min(p.tb, a.max_new))};
  const uint64_t cd[4] = {64, static_cast<uint64_t>(a.page_size), D / 64, static_cast<uint64_t>(a.pages) * a.Hkv};
  const uint64_t cs[3] = {D * 2, 128, static_cast<uint64_t>(a.page_size) * D * 2};
  const uint32_t cb[4] = {64, static_cast<uint32_t>(std::min(a.page_size, kTile)), 1, 1};
  cudaError_t e = make_tmap_4d(&tq_p, dt, a.Q, qd, qs, bp, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
  if (e == cudaSuccess) e = make_tmap_4d(&tq_s, dt, a.Q, qd, qs, bs, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B);
  if (e == cudaSuccess) e = make_tmap_4d(&tk, dt, a.k_cache, cd, cs, cb, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
  if (e == cudaSuccess) e = make_tmap_4d(&tv, dt, a.v_cache, cd, cs, cb, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
  if (e != cudaSuccess) return e;
  constexpr size_t smem = sizeof(Smem<D>) + 1024;
  static_assert(smem <= 227 * 1024, "attention kernel shared memory over the per-CTA limit");
  e = set_smem_attr_once(reinterpret_cast<const void*>(k_attn<F16, D>), smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k_attn<F16, D>, dim3(l.ctas), kThreads, smem, stream, tq_p, tq_s, tk, tv, p);
  if (e != cudaSuccess) return e;
  // Few rows have many segments each (the prefix is spread over all SMs): more warps a row.
  const int blocks = (a.T * p.G + 7) / 8;               // of eight rows of a head
  const auto join = [&](void (*kern)(Params), int w, int c) {
    const int per = kJoinWarps / w;
    return launch_pdl(kern, dim3((blocks + per - 1) / per, a.Hkv, c), kJoinWarps * 32, w > 1 ? kJoinSmem<D> : 0, stream, p);
  };
  // W C warps for each eight rows of a head, as long as they fit the SMs at once (32 an SM).  One warp / this
  // rule / always 8 C, in us: 2 requests over 8192 keys 30 / 16 / 16, 32 requests over 8192 + up to 700 43 / 28 /
  // 28, 128 requests 62 / 58 / 70, 256 requests of 64 heads over 32768 + up to 1024 291 / 293 / 349.
  const long long warps = static_cast<long long>(blocks) * a.Hkv, fit = 32ll * l.ctas;
  constexpr int C = D == 128 ? 4 : 2;
  if (warps * 8 * C <= fit) return join(k_attn_join<F16, D, 8, C>, 8, C);
  if (warps * 8 * 2 <= fit) return join(k_attn_join<F16, D, 8, 2>, 8, 2);
  if (warps * 4 * 2 <= fit) return join(k_attn_join<F16, D, 4, 2>, 4, 2);
  if (warps * 2 * 2 <= fit) return join(k_attn_join<F16, D, 2, 2>, 2, 2);
  if (warps * 2 <= fit) return join(k_attn_join<F16, D, 1, 2>, 1, 2);
  return join(k_attn_join<F16, D, 1, 1>, 1, 1);
}

}  // namespace

size_t attn_workspace_bytes(int64_t T, int64_t R, int64_t Hq, int64_t Hkv, int64_t d, int64_t max_new) {
  return layout(T, R, Hq, Hkv, d, max_new).bytes;
}

bool attn_prefix_fits(int64_t T, int64_t Hq, int64_t Hkv, int64_t prefix_len) {
  const int G = static_cast<int>(Hq / Hkv);
  return PrefixLine(T, prefix_len, kRows / G, G).head <= kMaxLine / Hkv;
}

cudaError_t launch_attn_shared_prefix(int dtype, const AttnArgs& a, void* ws, cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  if (dtype == kF16) return a.d == 64 ? launch_t<true, 64>(a, w, stream) : launch_t<true, 128>(a, w, stream);
  return a.d == 64 ? launch_t<false, 64>(a, w, stream) : launch_t<false, 128>(a, w, stream);
}

}  // namespace wq

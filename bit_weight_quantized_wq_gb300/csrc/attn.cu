// Attention of a batch whose requests share a long prefix, over a cache kept in pages.
//   o = softmax(scale q [Kp; Ks]^T) [Vp; Vs],  lse = log sum exp(scale q [Kp; Ks]^T)
// Kp, Vp: the shared prefix; Ks, Vs: the request's own keys, causal among its new tokens (the
// last of its own keys).
//
// Work.  An item is a set of query rows against one run of keys of one key/value head:
//   prefix items: all T tokens' rows of the head (row = token * G + query head of the group,
//     G = Hq / Hkv), in tiles of up to 2 * tb tokens (tb = 128 / G), against the prefix;
//   suffix items: one request's rows, tiled alike, against its own keys.
// Keys are taken in tiles of 128.  All items' tiles lie on one line (with a weight a tile and a
// constant an item); the line is cut into equal shares, one for each CTA (one per SM), so a CTA
// works through a run of tiles that may begin and end inside items, whatever the lengths are.
// What a CTA computes of an item (a segment: unnormalised output, running maximum and sum) goes
// to the workspace in float32, and a second kernel joins the segments of each row in line order.
//
// A CTA runs two lanes, each a 128-row tensor-core tile with its own scores and output in tensor
// memory and its own four softmax warps (one row a thread):
//   rows mode (more than tb tokens in the item): the lanes hold different rows and both see every
//     key tile, so K and V are read once for 256 rows;
//   keys mode (up to tb tokens): both lanes hold the same rows and take the key tiles in turn.
// The tensor core works on one lane's products while the other lane's softmax runs:
//   S = Q K^T       both operands from shared memory (TMA, 128-byte swizzle)
//   P = 2^(c S - m) written back over S in tensor memory, 16 bits
//   O += P V        P from tensor memory, V from shared memory, d contiguous (transposed operand)
// The running maximum is only followed when it grows by more than 2^8 (the output in tensor memory
// is then rescaled); until then P is at most 2^8, which float32 sums and 16-bit P carry as well.
// P is rounded to the cache's type for the second product (the tensor core takes both operands in
// one type); the sum of P is kept unrounded in float32.
#include <algorithm>

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

constexpr int kTile = 128;            // keys per tile, rows per lane
constexpr int kThreads = 320;         // 2 x 4 softmax warps, TMA warp, MMA warp
constexpr int kWTma = 8, kWMma = 9;
constexpr int kTmemCols = 512;        // S of both lanes, O of both lanes: 4 x 128 columns
constexpr int kColO = 256;
// Weights on the line: a key tile in either mode, and an item's own cost.
constexpr int kWRows = 4, kWKeys = 4, kWItem = 4;
constexpr float kLazy = 8.f;          // rescale when the maximum grew by more than 2^8

template <int D>
struct Smem {
  static constexpr int kBytes = kTile * D * 2;          // a Q, K or V tile: [D / 64][128 rows][128 B]
  static constexpr int kStages = D == 128 ? 5 : 10;     // K and V tiles in flight
  uint8_t kv[kStages][kBytes];
  uint8_t q[2][kBytes];
  uint64_t full[kStages], empty[kStages];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2], o_full[2], o_empty[2];
  long long scan[kThreads / 32 + 2];
  int scan_items[kThreads / 32 + 2];
  long long total;
  long long r0_line;
  int r0, r0_item;
  uint32_t tmem_base;
};

struct Params {
  AttnArgs a;
  int G, tb;                 // query heads per key/value head; tokens per lane tile
  int n_prefix;              // prefix items
  int prefix_tiles;
  int q_rows_suffix;         // rows a suffix lane tile can have (its partial's row capacity)
  int ctas;
  long long* start;          // [R] line position of each request's first item
  int* item0;                // [R] ordinal of it
  int* owner;                // [T] request of each token
  long long* share;          // [1]
  float *po_p, *ml_p;        // prefix partials: [segment][lane][D / 4][128][4], [segment][lane][128][2]
  float *po_s, *ml_s;        // suffix partials, with q_rows_suffix rows
};

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// One request's new tokens and own keys, forced into range.
struct Request {
  int first, n, len;
  bool bad;
};
__device__ __forceinline__ Request request(const AttnArgs& a, int r) {
  Request q;
  q.first = a.q_start ? __ldg(a.q_start + r) : r;
  const int end = a.q_start ? __ldg(a.q_start + r + 1) : r + 1;
  q.len = a.max_blocks ? __ldg(a.suffix_lens + r) : 0;
  q.n = end - q.first;
  q.bad = false;
  if (q.first < 0 || end < q.first || end > a.T || q.n > a.max_new) q.bad = true, q.n = 0, q.first = 0;
  const int cap = a.max_blocks * a.page_size;
  if (q.len < 0 || q.len > cap) q.bad = true, q.len = min(max(q.len, 0), cap);
  return q;
}

// Items of ntok tokens: row tiles, and the mode of tile rt.
__device__ __forceinline__ int row_tiles(const Params& p, int ntok) { return ceil_div(ntok, 2 * p.tb); }
__device__ __forceinline__ int tile_tokens(const Params& p, int ntok, int rt) { return min(2 * p.tb, ntok - rt * 2 * p.tb); }
__device__ __forceinline__ int weight(const Params& p, int tokens) { return tokens > p.tb ? kWRows : kWKeys; }
// Line length of all row tiles of one head.
__device__ __forceinline__ long long head_cost(const Params& p, int ntok, int tiles) {
  const int rts = row_tiles(p, ntok);
  if (rts == 0 || tiles == 0) return 0;
  return static_cast<long long>(rts - 1) * (static_cast<long long>(tiles) * kWRows + kWItem) +
         static_cast<long long>(tiles) * weight(p, tile_tokens(p, ntok, rts - 1)) + kWItem;
}
// First tile of an item (line start s, tiles n of weight w) at or after line position b.
__device__ __forceinline__ int tile_at(long long b, long long s, int n, int w) {
  if (b <= s) return 0;
  const long long t = (b - s + w - 1) / w;
  return t > n ? n : static_cast<int>(t);
}

struct Item {
  bool prefix, rows;
  int kvh, r;
  int lo, hi;        // key tiles
  int len;           // keys of the run
  int tok0, ntok;    // first token (row of Q) and tokens of the item
  int lim0;          // keys token 0 of the item sees (suffix: token i sees i more)
  int seg;           // partial slot
};

// Walks over the items of one CTA's share; every role of the CTA walks the same way.
struct Walk {
  const Params& p;
  long long b0, b1;
  int cta;
  int ip;                 // next prefix item
  int r, kvh, rt, item;   // next suffix item
  long long line;         // its line position
  Request q, nq;          // request r and, read ahead, r + 1

  __device__ Walk(const Params& p_, int cta_, long long share, long long prefix_cost, int r0, long long r0_line, int r0_item)
      : p(p_), cta(cta_) {
    b0 = static_cast<long long>(cta) * share;
    b1 = b0 + share;
    ip = p.n_prefix;
    if (b0 < prefix_cost) {
      const long long hc = prefix_cost / p.a.Hkv;
      const int rts = row_tiles(p, p.a.T);
      const long long full = static_cast<long long>(p.prefix_tiles) * kWRows + kWItem;
      const long long k = (b0 % hc) / full;
      ip = static_cast<int>(b0 / hc) * rts + static_cast<int>(k < rts ? k : rts - 1);
    }
    r = r0, line = r0_line, item = r0_item, kvh = 0, rt = 0;
    if (r < p.a.R) q = request(p.a, r);
    if (r + 1 < p.a.R) nq = request(p.a, r + 1);
  }

  __device__ bool next(Item& it) {
    while (ip < p.n_prefix) {
      const int rts = p.n_prefix / p.a.Hkv;
      const int h = ip / rts, t = ip % rts;
      const long long s = h * head_cost(p, p.a.T, p.prefix_tiles) +
                          t * (static_cast<long long>(p.prefix_tiles) * kWRows + kWItem);
      if (s >= b1) return false;
      it.ntok = tile_tokens(p, p.a.T, t);
      const int w = weight(p, it.ntok);
      it.prefix = true;
      it.kvh = h, it.r = 0;
      it.rows = it.ntok > p.tb;
      it.lo = tile_at(b0, s, p.prefix_tiles, w), it.hi = tile_at(b1, s, p.prefix_tiles, w);
      it.len = p.a.prefix_len;
      it.tok0 = t * 2 * p.tb;
      it.lim0 = p.a.prefix_len;
      it.seg = cta + ip;
      ++ip;
      if (it.lo < it.hi) return true;
    }
    while (r < p.a.R) {
      const int tiles = ceil_div(q.len, kTile), rts = row_tiles(p, q.n);
      if (tiles == 0 || rts == 0 || kvh == p.a.Hkv) {
        ++r, kvh = 0, rt = 0;
        q = nq;
        if (r + 1 < p.a.R) nq = request(p.a, r + 1);
        continue;
      }
      if (line >= b1) return false;
      it.ntok = tile_tokens(p, q.n, rt);
      const int w = weight(p, it.ntok);
      it.prefix = false;
      it.kvh = kvh, it.r = r;
      it.rows = it.ntok > p.tb;
      it.lo = tile_at(b0, line, tiles, w), it.hi = tile_at(b1, line, tiles, w);
      it.len = q.len;
      it.tok0 = q.first + rt * 2 * p.tb;
      it.lim0 = q.len - q.n + rt * 2 * p.tb + 1;
      it.seg = cta + item;
      line += static_cast<long long>(tiles) * w + kWItem;
      ++item;
      if (++rt == rts) rt = 0, ++kvh;
      if (it.lo < it.hi) return true;
    }
    return false;
  }
};

// Order in which an item's n key tiles reach shared memory: K0, K1, V0, K2, V1, ..., V(n-1).
__device__ __forceinline__ uint32_t ord_k(int j) { return j == 0 ? 0u : 2u * j - 1; }
__device__ __forceinline__ uint32_t ord_v(int j, int n) { return j == n - 1 ? 2u * n - 1 : 2u * j + 2; }

// A wait of a whole warp: every lane waits (bounded), and all of them go on or none.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t code) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, &g_attn_err, code));
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool F16, int D>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn(const __grid_constant__ CUtensorMap tq_p, const __grid_constant__ CUtensorMap tq_s,
           const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const __grid_constant__ Params p) {
  using S = Smem<D>;
  constexpr int NS = S::kStages;
  constexpr int CH = D / 64;
  constexpr uint32_t kChunk = kTile * 128;     // bytes of one 64-element chunk of a tile
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  S& sm = *reinterpret_cast<S*>(smem_raw + smem_align_pad(smem_raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) mbar_init(&sm.full[s], 1), mbar_init(&sm.empty[s], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 1), mbar_init(&sm.q_empty[i], 1);
      mbar_init(&sm.s_full[i], 1), mbar_init(&sm.p_full[i], 128);
      mbar_init(&sm.o_full[i], 1), mbar_init(&sm.o_empty[i], 128);
    }
    fence_barrier_init();
  }
  if (warp == kWMma) {
    tmem_alloc(&sm.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  if (warp == kWTma && lane == 0) {
    tma_prefetch_desc(&tq_p), tma_prefetch_desc(&tq_s), tma_prefetch_desc(&tk), tma_prefetch_desc(&tv);
  }
  pdl_launch_dependents();
  pdl_wait();

  // ---------------------------------------------------------------- the line: its length, and
  // the request in which this CTA's share begins
  const long long prefix_cost = p.a.Hkv * head_cost(p, p.a.T, p.prefix_tiles);
  long long mine = 0;
  for (int r = threadIdx.x; r < p.a.R; r += kThreads) {
    const Request q = request(p.a, r);
    mine += p.a.Hkv * head_cost(p, q.n, ceil_div(q.len, kTile));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) sm.scan[warp] = mine;
  if (threadIdx.x == 0) sm.r0 = p.a.R, sm.r0_line = 0, sm.r0_item = 0;
  __syncthreads();
  long long total = prefix_cost;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) total += sm.scan[w];
  long long share = (total + p.ctas - 1) / p.ctas;
  if (share < kWKeys) share = kWKeys;
  const long long b0 = blockIdx.x * share;
  {
    long long run = prefix_cost;
    int run_items = 0;
    for (int base = 0; base < p.a.R; base += kThreads) {
      const int r = base + threadIdx.x;
      long long c = 0;
      int n = 0;
      if (r < p.a.R) {
        const Request q = request(p.a, r);
        const int tiles = ceil_div(q.len, kTile);
        c = p.a.Hkv * head_cost(p, q.n, tiles);
        n = tiles ? p.a.Hkv * row_tiles(p, q.n) : 0;
        if (blockIdx.x == 0) {
          if (q.bad) atomicOr(&g_attn_err, kErrIndex);
          for (int i = 0; i < q.n; ++i) p.owner[q.first + i] = r;
        }
      }
      long long ic = c;
      int in = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long uc = __shfl_up_sync(0xffffffffu, ic, o);
        const int un = __shfl_up_sync(0xffffffffu, in, o);
        if (lane >= o) ic += uc, in += un;
      }
      __syncthreads();
      if (lane == 31) sm.scan[warp] = ic, sm.scan_items[warp] = in;
      __syncthreads();
      long long before = run;
      int before_items = run_items;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += sm.scan[w], before_items += sm.scan_items[w];
        run += sm.scan[w], run_items += sm.scan_items[w];
      }
      const long long at = before + ic - c;
      const int item = before_items + in - n;
      if (r < p.a.R) {
        if (blockIdx.x == 0) p.start[r] = at, p.item0[r] = item;
        // the first request whose items reach past b0
        if ((at <= b0 && b0 < at + c) || (r == 0 && b0 < prefix_cost)) sm.r0 = r, sm.r0_line = at, sm.r0_item = item;
      }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.share = share;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  Item it;

  if (warp == kWTma) {
    // -------------------------------------------------------------------- TMA producer
    Walk walk(p, blockIdx.x, share, prefix_cost, sm.r0, sm.r0_line, sm.r0_item);
    const uint64_t pol_keep = l2_policy_evict_last(), pol_once = l2_policy_evict_first();
    const int page = p.a.page_size, ppt = kTile / page;
    uint32_t ord = 0, qord = 0;
    bool ok = true;
    while (ok && walk.next(it)) {
      const int n = it.hi - it.lo;
      // Q: one 128-row tile per lane that has rows of its own
      const int nq = it.rows ? 2 : 1;
      const int box_tok = it.prefix ? p.tb : min(p.tb, p.a.max_new);
      for (int i = 0; i < nq; ++i, ++qord) {
        const int s = qord & 1;
        ok = warp_wait(&sm.q_empty[s], ((qord >> 1) & 1) ^ 1, kErrWaitEmpty);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sm.q_full[s], box_tok * p.G * 128 * CH);
          for (int c = 0; c < CH; ++c)
            tma_load_4d(&sm.q[s][c * kChunk], it.prefix ? &tq_p : &tq_s, 0, c, it.kvh * p.G, it.tok0 + i * p.tb,
                        &sm.q_full[s], pol_keep);
        }
        __syncwarp();
      }
      if (!ok) break;
      const int32_t* list = it.prefix ? p.a.prefix_pages : p.a.block_table + static_cast<int64_t>(it.r) * p.a.max_blocks;
      const uint64_t pol = it.prefix ? pol_keep : pol_once;
      // lane l < ppt * CH loads page l % ppt of chunk l / ppt of each tile; page numbers are read
      // one tile ahead
      const int my_page = lane % ppt, my_chunk = lane / ppt;
      const int n_pages = ceil_div(it.len, page);
      const auto page_id = [&](int j) {     // row of the tensor map: page * Hkv + head, or -1 (zero fill)
        const int i = (it.lo + j) * ppt + my_page;
        if (j >= n || i >= n_pages) return -1;
        const int id = __ldg(list + i);
        if (id < 0 || id >= p.a.pages) {
          atomicOr(&g_attn_err, kErrIndex);
          return -1;
        }
        return id * p.a.Hkv + it.kvh;
      };
      const auto load = [&](const CUtensorMap* map, int j, int id) {
        const int s = ord % NS;
        if (!warp_wait(&sm.empty[s], ((ord / NS) & 1) ^ 1, kErrWaitEmpty)) return false;
        const int pages_here = min(ppt, n_pages - (it.lo + j) * ppt);
        if (lane == 0) mbar_arrive_expect_tx(&sm.full[s], pages_here * page * 128 * CH);
        __syncwarp();
        if (my_chunk < CH && my_page < pages_here)
          tma_load_4d(&sm.kv[s][my_chunk * kChunk + my_page * page * 128], map, 0, 0, my_chunk, id, &sm.full[s], pol);
        ++ord;
        return true;
      };
      int id0 = page_id(0), id1 = page_id(1);
      ok = load(&tk, 0, id0);
      for (int j = 0; ok && j < n; ++j) {
        const int id2 = page_id(j + 2);
        if (j + 1 < n) ok = load(&tk, j + 1, id1);
        if (ok) ok = load(&tv, j, id0);
        id0 = id1, id1 = id2;
      }
    }
    // drain: the last fill of each slot has landed before the CTA's memory goes
    for (uint32_t i = ord > NS ? ord - NS : 0; i < ord; ++i)
      mbar_wait(&sm.full[i % NS], (i / NS) & 1, &g_attn_err, kErrDrain);
    for (uint32_t i = qord > 2 ? qord - 2 : 0; i < qord; ++i)
      mbar_wait(&sm.q_full[i & 1], (i >> 1) & 1, &g_attn_err, kErrDrain);
  } else if (warp == kWMma) {
    // -------------------------------------------------------------------- MMA issuer
    if (lane == 0) {
      Walk walk(p, blockIdx.x, share, prefix_cost, sm.r0, sm.r0_line, sm.r0_item);
      constexpr uint32_t fmt = F16 ? 0u : 1u;
      constexpr uint32_t id_qk = (1u << 4) | (fmt << 7) | (fmt << 10) | ((kTile >> 3) << 17) | ((kTile >> 4) << 24);
      constexpr uint32_t id_pv = (1u << 4) | (fmt << 7) | (fmt << 10) | (1u << 16) | ((D >> 3) << 17) | ((kTile >> 4) << 24);
      uint32_t ord = 0, qord = 0, p_cnt[2] = {0, 0}, o_cnt[2] = {0, 0};
      bool ok = true;
      const auto wait_kv = [&](uint32_t o) { return mbar_wait(&sm.full[o % NS], (o / NS) & 1, &g_attn_err, kErrWaitFull); };
      const auto qk = [&](int l, uint32_t qs, uint32_t ko) {
        const uint64_t a = smem_desc_sw128(smem_u32(&sm.q[qs][0])), b = smem_desc_sw128(smem_u32(&sm.kv[ko % NS][0]));
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_ss_f16(tmem + 128 * l, a + static_cast<uint64_t>((c * kChunk + 32 * kk) >> 4),
                          b + static_cast<uint64_t>((c * kChunk + 32 * kk) >> 4), id_qk, (c | kk) ? 1u : 0u);
        tc_commit(&sm.s_full[l]);
      };
      const auto pv = [&](int l, uint32_t vo, bool first) {
        const uint64_t b = smem_desc_sw128_mn(smem_u32(&sm.kv[vo % NS][0]), kChunk);
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kTile / 16; ++kk)
          tc_mma_ts(tmem + kColO + 128 * l, tmem + 128 * l + 8 * kk, b + static_cast<uint64_t>((kk * 2048) >> 4), id_pv,
                    (!first || kk) ? 1u : 0u);
      };
      const auto wait_p = [&](int l, bool first) {
        if (first) {   // the lane's previous item has left the output columns
          if (!mbar_wait(&sm.o_empty[l], (o_cnt[l] & 1) ^ 1, &g_attn_err, kErrWaitAccum)) return false;
          ++o_cnt[l];
        }
        const bool r = mbar_wait(&sm.p_full[l], p_cnt[l] & 1, &g_attn_err, kErrWaitFull);
        ++p_cnt[l];
        return r;
      };
      while (ok && walk.next(it)) {
        const int n = it.hi - it.lo;
        uint32_t qs[2];
        for (int i = 0; i < (it.rows ? 2 : 1) && ok; ++i, ++qord) {
          qs[i] = qord & 1;
          ok = mbar_wait(&sm.q_full[qs[i]], (qord >> 1) & 1, &g_attn_err, kErrWaitFull);
        }
        if (!it.rows) qs[1] = qs[0];
        if (!ok || !(ok = wait_kv(ord))) break;
        if (it.rows) {
          qk(0, qs[0], ord), qk(1, qs[1], ord);
          tc_commit(&sm.empty[ord % NS]);
          for (int j = 0; j < n; ++j) {
            const uint32_t vo = ord + ord_v(j, n), ko = ord + ord_k(j + 1);
            const bool more = j + 1 < n;
            if (!(ok = wait_kv(vo))) break;
            for (int l = 0; l < 2; ++l) {
              if (!(ok = wait_p(l, j == 0))) break;
              pv(l, vo, j == 0);
              if (more) {
                if (l == 0 && !(ok = wait_kv(ko))) break;
                qk(l, qs[l], ko);
              } else {
                tc_commit(&sm.o_full[l]);
              }
            }
            if (!ok) break;
            if (more) tc_commit(&sm.empty[ko % NS]);
            tc_commit(&sm.empty[vo % NS]);
          }
        } else {
          for (int j = 0; j < min(n, 2); ++j) {
            const uint32_t ko = ord + ord_k(j);
            if (j && !(ok = wait_kv(ko))) break;
            qk(j, qs[0], ko);
            tc_commit(&sm.empty[ko % NS]);
          }
          for (int j = 0; j < n && ok; ++j) {
            const int l = j & 1;
            const uint32_t vo = ord + ord_v(j, n);
            if (!(ok = wait_kv(vo)) || !(ok = wait_p(l, j < 2))) break;
            pv(l, vo, j < 2);
            if (j + 2 < n) {
              const uint32_t ko = ord + ord_k(j + 2);
              if (!(ok = wait_kv(ko))) break;
              qk(l, qs[0], ko);
              tc_commit(&sm.empty[ko % NS]);
            } else {
              tc_commit(&sm.o_full[l]);
            }
            tc_commit(&sm.empty[vo % NS]);
          }
        }
        if (!ok) break;
        for (int i = 0; i < (it.rows ? 2 : 1); ++i) tc_commit(&sm.q_empty[qs[i]]);
        ord += 2 * n;
      }
      // the last commit has landed before the CTA's barriers go
      if (ok && qord > 0) mbar_wait(&sm.q_empty[(qord - 1) & 1], ((qord - 1) >> 1) & 1, &g_attn_err, kErrDrain);
      if (!ok) {   // a wait ran out: the tensor memory must be idle before it is given back
        tc_commit(&sm.o_full[0]);
        mbar_wait(&sm.o_full[0], 0, &g_attn_err, kErrDrain);
        mbar_wait(&sm.o_full[0], 1, &g_attn_err, kErrDrain);
      }
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------------- softmax, one row a thread
    Walk walk(p, blockIdx.x, share, prefix_cost, sm.r0, sm.r0_line, sm.r0_item);
    const int l = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lane_base + 128 * l, t_o = tmem + lane_base + kColO + 128 * l;
    const float c = p.a.scale * 1.4426950408889634f;
    const int tok = row / p.G;
    uint32_t s_cnt = 0, o_cnt = 0, ord = 0;
    bool ok = true;
    while (ok && walk.next(it)) {
      const int n = it.hi - it.lo;
      const int nl = it.rows ? n : (n + 1 - l) / 2;      // tiles of this lane
      const int ntok = it.rows ? (l == 0 ? p.tb : it.ntok - p.tb) : it.ntok;
      const int tok_item = tok + (it.rows && l ? p.tb : 0);
      const bool valid = tok < ntok && tok < p.tb;
      const bool active = __any_sync(0xffffffffu, valid);
      const int lim = it.prefix ? it.len : min(max(it.lim0 + tok_item, 0), it.len);
      float m = -INFINITY, sum = 0.f;                    // m in units of log2, already times c
      for (int jj = 0; jj < nl; ++jj) {
        const int j = it.rows ? jj : 2 * jj + l;
        const int key0 = (it.lo + j) * kTile;
        ok = warp_wait(&sm.s_full[l], s_cnt & 1, kErrWaitAccum);
        if (!ok) break;
        ++s_cnt;
        tc_fence_after();
        if (active) {
          uint32_t v[4][32];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld32(t_s + 32 * q, v[q]);
          tc_wait_ld();
          if (__any_sync(0xffffffffu, valid && key0 + kTile > lim)) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (key0 + 32 * q + e >= lim) v[q][e] = 0xff800000u;
          }
          float mx = -INFINITY;
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 32; ++e) mx = fmaxf(mx, __uint_as_float(v[q][e]));
          const float mc = mx * c;
          const bool grow = valid && mc > m + kLazy;
          if (__any_sync(0xffffffffu, grow)) {
            const float keep = grow ? exp2_approx(m - mc) : 1.f;
            if (grow) m = mc;
            sum *= keep;
            if (jj > 0) {
#pragma unroll
              for (int q = 0; q < D / 32; ++q) {
                uint32_t o[32];
                tmem_ld32(t_o + 32 * q, o);
                tc_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                tmem_st32(t_o + 32 * q, o);
              }
            }
          }
          const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const float a = exp2_approx(fmaf(__uint_as_float(v[2 * q + e / 16][2 * (e % 16)]), c, -base));
              const float b = exp2_approx(fmaf(__uint_as_float(v[2 * q + e / 16][2 * (e % 16) + 1]), c, -base));
              sum += a + b;
              w[e] = pack2<F16>(a, b);
            }
            tmem_st32(t_s + 32 * q, w);
          }
          tc_wait_st();
        }
        // V rows past the run's end hold whatever the page or the slot held: zero them, since
        // their weight 0 times a NaN would not be 0
        if (key0 + kTile > it.len) {
          const uint32_t vo = ord + ord_v(j, n);
          ok = warp_wait(&sm.full[vo % NS], (vo / NS) & 1, kErrWaitFull);
          if (!ok) break;
          if (row >= it.len - key0) {
#pragma unroll
            for (int ch = 0; ch < CH; ++ch) {
              uint4* z = reinterpret_cast<uint4*>(&sm.kv[vo % NS][ch * kChunk + row * 128]);
#pragma unroll
              for (int e = 0; e < 8; ++e) z[e] = make_uint4(0, 0, 0, 0);
            }
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        mbar_arrive(&sm.p_full[l]);
      }
      if (!ok) break;
      ord += 2 * n;
      // ---------------------------------------------------------------- the segment's partial
      const int cap = it.prefix ? kTile : p.q_rows_suffix;
      const long long slot = 2ll * it.seg + l;
      float2* ml = reinterpret_cast<float2*>(it.prefix ? p.ml_p : p.ml_s) + slot * cap + row;
      if (nl > 0) {
        ok = warp_wait(&sm.o_full[l], o_cnt & 1, kErrWaitAccum);
        if (!ok) break;
        ++o_cnt;
        tc_fence_after();
        if (active) {
          float4* po = reinterpret_cast<float4*>(it.prefix ? p.po_p : p.po_s) + slot * (D / 4) * cap + row;
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld32(t_o + 32 * q, o);
            tc_wait_ld();
            if (valid) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                po[(8 * q + e) * cap] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                    __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
            }
          }
        }
        tc_fence_before();
        mbar_arrive(&sm.o_empty[l]);
      }
      if (valid) *ml = make_float2(m, sum);
    }
  }
  __syncwarp();
  __syncthreads();
  if (warp == kWMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the segments of each row: one CTA per token, threads over (key/value head, 4 output
// columns, query head of the group).
template <bool F16, int D>
__global__ void __launch_bounds__(256) k_attn_join(const __grid_constant__ Params p) {
  pdl_launch_dependents();
  pdl_wait();
  const int t = blockIdx.x;
  const int r = __ldcg(p.owner + t);
  if (r < 0 || r >= p.a.R) return;                      // a token of no request
  const Request q = request(p.a, r);
  const int i_tok = t - q.first;
  if (i_tok < 0 || i_tok >= q.n) return;
  const long long share = __ldcg(p.share);
  const long long line_r = __ldcg(p.start + r);
  const int item_r = __ldcg(p.item0 + r);
  const int tiles_s = ceil_div(q.len, kTile);
  const int span = 2 * p.tb;
  const long long hc_p = head_cost(p, p.a.T, p.prefix_tiles), hc_s = head_cost(p, q.n, tiles_s);

  for (int x = threadIdx.x; x < p.a.Hq * (D / 4); x += blockDim.x) {
    const int g = x % p.G, cg = (x / p.G) % (D / 4), kvh = x / (p.G * (D / 4));
    float top = -INFINITY, total = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    // the run's partials in line order, the sums rescaled where the maximum grows
    const auto take = [&](const float* ml, const float* po, long long slot, int cap, int row) {
      const float2 s = __ldcg(reinterpret_cast<const float2*>(ml) + slot * cap + row);
      if (s.y == 0.f) return;
      const float m2 = fmaxf(top, s.x);
      const float base = m2 == -INFINITY ? 0.f : m2;
      const float a = exp2_approx(top - base), b = exp2_approx(s.x - base);
      const float4 v = __ldcg(reinterpret_cast<const float4*>(po) + (slot * (D / 4) + cg) * cap + row);
      top = m2;
      total = total * a + s.y * b;
      o.x = o.x * a + v.x * b, o.y = o.y * a + v.y * b, o.z = o.z * a + v.z * b, o.w = o.w * a + v.w * b;
    };
    const auto run = [&](int tok, int ntok_all, int tiles, long long line, int ordinal, const float* ml, const float* po, int cap) {
      const int rt = tok / span, rts = row_tiles(p, ntok_all);
      const int ntok = tile_tokens(p, ntok_all, rt);
      const bool rows = ntok > p.tb;
      const int w = rows ? kWRows : kWKeys;
      const long long s = line + rt * (static_cast<long long>(tiles) * kWRows + kWItem);
      const int item = ordinal + kvh * rts + rt;
      const int row = (tok % p.tb) * p.G + g, half = (tok / p.tb) & 1;
      const int last = static_cast<int>((s + static_cast<long long>(tiles) * w - 1) / share);
      for (int cta = static_cast<int>(s / share); cta <= last; ++cta) {
        if (tile_at(cta * share, s, tiles, w) >= tile_at((cta + 1) * share, s, tiles, w)) continue;
        const long long slot = 2ll * (cta + item);
        if (rows) {
          take(ml, po, slot + half, cap, row);
        } else {
          take(ml, po, slot, cap, row);
          take(ml, po, slot + 1, cap, row);
        }
      }
    };
    if (p.prefix_tiles) run(t, p.a.T, p.prefix_tiles, kvh * hc_p, 0, p.ml_p, p.po_p, kTile);
    if (tiles_s) run(i_tok, q.n, tiles_s, line_r + kvh * hc_s, item_r, p.ml_s, p.po_s, p.q_rows_suffix);
    const float inv = total == 0.f ? 0.f : 1.f / total;
    const int h = kvh * p.G + g;
    const long long row = static_cast<long long>(t) * p.a.Hq + h;
    *reinterpret_cast<uint2*>(p.a.O + row * D + 4 * cg) = make_uint2(pack2<F16>(o.x * inv, o.y * inv), pack2<F16>(o.z * inv, o.w * inv));
    if (cg == 0 && p.a.lse)
      p.a.lse[row] = total == 0.f ? -INFINITY : ((top == -INFINITY ? 0.f : top) + log2f(total)) * 0.6931471805599453f;
  }
}

struct Layout {
  int G, tb, n_prefix, rows_s, ctas;
  size_t start, item0, owner, share, po_p, ml_p, po_s, ml_s, bytes;
};

Layout layout(int64_t T, int64_t R, int64_t Hq, int64_t Hkv, int64_t d, int64_t max_new) {
  Layout l{};
  l.G = static_cast<int>(Hq / Hkv);
  l.tb = kTile / l.G;
  l.ctas = device_sm_count();
  const int64_t span = 2 * l.tb;
  l.n_prefix = static_cast<int>(Hkv * ((T + span - 1) / span));
  // requests' row tiles: no more than one each and one more for every full tile of tokens
  const int64_t tiles_each = (max_new + span - 1) / span;
  const int64_t n_suffix = Hkv * std::min(R * tiles_each, R + T / span);
  l.rows_s = static_cast<int>(std::min<int64_t>(kTile, max_new * l.G));
  size_t off = kWsHeaderBytes;
  const auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) / 256 * 256;
    return at;
  };
  l.start = take(R * sizeof(long long));
  l.item0 = take(R * sizeof(int));
  l.owner = take(T * sizeof(int));
  l.share = take(sizeof(long long));
  const size_t sp = 2 * static_cast<size_t>(l.ctas + l.n_prefix), ss = 2 * static_cast<size_t>(l.ctas + n_suffix);
  l.po_p = take(sp * kTile * d * sizeof(float));
  l.ml_p = take(sp * kTile * 2 * sizeof(float));
  l.po_s = take(ss * l.rows_s * d * sizeof(float));
  l.ml_s = take(ss * l.rows_s * 2 * sizeof(float));
  l.bytes = off;
  return l;
}

template <bool F16, int D>
cudaError_t launch_t(const AttnArgs& a, uint8_t* ws, cudaStream_t stream) {
  const Layout l = layout(a.T, a.R, a.Hq, a.Hkv, D, a.max_new);
  Params p{};
  p.a = a;
  p.G = l.G, p.tb = l.tb;
  p.prefix_tiles = (a.prefix_len + kTile - 1) / kTile;
  p.n_prefix = p.prefix_tiles ? l.n_prefix : 0;
  p.q_rows_suffix = l.rows_s;
  p.ctas = l.ctas;
  p.start = reinterpret_cast<long long*>(ws + l.start);
  p.item0 = reinterpret_cast<int*>(ws + l.item0);
  p.owner = reinterpret_cast<int*>(ws + l.owner);
  p.share = reinterpret_cast<long long*>(ws + l.share);
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
  const uint32_t cb[4] = {64, static_cast<uint32_t>(a.page_size), 1, 1};
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
  return launch_pdl(k_attn_join<F16, D>, dim3(a.T), 256, 0, stream, p);
}

}  // namespace

size_t attn_workspace_bytes(int64_t T, int64_t R, int64_t Hq, int64_t Hkv, int64_t d, int64_t max_new) {
  return layout(T, R, Hq, Hkv, d, max_new).bytes;
}

cudaError_t launch_attn_shared_prefix(int dtype, const AttnArgs& a, void* ws, cudaStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  if (dtype == kF16) return a.d == 64 ? launch_t<true, 64>(a, w, stream) : launch_t<true, 128>(a, w, stream);
  return a.d == 64 ? launch_t<false, 64>(a, w, stream) : launch_t<false, 128>(a, w, stream);
}

}  // namespace wq

// The line of work of attention over the 8-bit cache: how it is cut into shares, and how an item that is cut is
// joined again.  Shared by both kernels of attn_e4m3.cu; plain C++ too, so that a test runs these very rules on the CPU.
#pragma once

#if defined(__CUDACC__)
#define WQ_LINE_FN __host__ __device__ __forceinline__
#else
#define WQ_LINE_FN inline
#endif

namespace wq {

// a / b in float32, to some units in the last place.
WQ_LINE_FN float line_ratio(long long a, long long b) {
#if defined(__CUDA_ARCH__)
  return __fdividef(static_cast<float>(a), static_cast<float>(b));
#else
  return static_cast<float>(a) / static_cast<float>(b);
#endif
}

// a / b of positions on a line, exact where it is below 2^20 (a 64-bit division takes some hundred instructions).
WQ_LINE_FN int quotient(long long a, long long b) {
  int q = static_cast<int>(line_ratio(a, b));
  if (q * b > a) --q;
  else if ((q + 1) * b <= a) ++q;
  return q;
}

// An equal share of the line for each CTA, rounded up so that the shares cover it, and no shorter than the heaviest
// tile, so that every CTA between an item's first and last has a tile of it.  `exactly`: rounded up by no more than has
// to be.
WQ_LINE_FN long long line_share(long long total, long long ctas, int heaviest, bool exactly) {
  long long share = static_cast<long long>(line_ratio(total, ctas) * 1.000001f) + 1;
  if (share < heaviest) share = heaviest;
  if (exactly)
    while (share > heaviest && (share - 1) * ctas >= total) --share;
  return share;
}

// First tile of an item (line start s, tiles n of weight w) that starts at or after position b.
WQ_LINE_FN int tile_at(long long b, long long s, int n, int w) {
  if (b <= s) return 0;
  const long long d = b - s;
  return d >= static_cast<long long>(n) * w ? n : (static_cast<int>(d) + w - 1) / w;
}

// An item's segments, one in each of the CTAs c0 .. c1, are joined in line order by the last CTA that is done with it, or,
// where there are more of them than kGroup, in two steps: groups of kGroup neighbours, each joined in the place of its
// first, then the groups.
constexpr int kGroup = 8;

// One step of a join: the last of the n CTAs that count it joins what CTAs first, first + step, .. (n of them) have left.
struct Join {
  int counter;               // its place among the counters, [2][ctas]
  int first, step, n;
  bool final;                // the join of the item; else of a group, after which comes the final one
};

// The item's own counter, by the CTA that it begins in: of the items that begin in a CTA only the last is cut.
WQ_LINE_FN Join final_join(int c0, int c1) {
  const int segments = c1 - c0 + 1;
  if (segments <= kGroup) return {c0, c0, 1, segments, true};
  return {c0, c0, kGroup, (segments + kGroup - 1) / kGroup, true};
}

// What the CTA counts first.  A group's counter goes by the group's first CTA.  That CTA lies between the item's ends, and so
// is no other item's, or it is c0, where no other item's group of two or more can begin: of an item that ends there, only a
// group of that CTA alone.  So a group of one is not counted at all: its segment stands in its place already.  (Counted,
// it took the arrivals of the next item's first group with it, whose rows then were not written.)
WQ_LINE_FN Join first_join(int c0, int c1, int cta, int ctas) {
  if (c1 - c0 + 1 <= kGroup) return final_join(c0, c1);
  const int first = c0 + (cta - c0) / kGroup * kGroup, n = c1 - first + 1 < kGroup ? c1 - first + 1 : kGroup;
  if (n == 1) return final_join(c0, c1);
  return {ctas + first, first, 1, n, false};
}

}  // namespace wq

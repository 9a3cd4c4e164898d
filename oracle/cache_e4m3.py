"""Float64 oracle of the 8-bit cache: new tokens quantized into pages, tokens read back, attention over
the pages.  Plain loops over requests, pages and heads, written from the definitions; shares no code
with the CUDA path.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

Format: E4M3 codes [pages, Hkv, page_size, d] (``oracle.fp8``; the pages name FP8 for the cache,
推理优化与量化算子深度技术调研 §1.6), one E8M0 byte a page and head: element = E4M3(code) 2^(byte - 127).
"""
import math

import numpy as np

from oracle import fp8

LOW, HIGH, BIAS = -64, 64, 127
VALUES = fp8.e4m3_values()


def need(x):
    """The lowest exponent e in [-64, 64] with max |x| <= 448 2^e over the finite elements of x."""
    a = np.abs(x[np.isfinite(x)])
    top = float(a.max()) if a.size else 0.0
    e = LOW
    while e < HIGH and top > math.ldexp(448.0, e):
        e += 1
    return e


def encode(x, e):
    """Codes of x 2^-e (exact in float64; infinities become NaN)."""
    y = np.ldexp(np.asarray(x, np.float64), -e)
    codes = _round(np.clip(np.where(np.isfinite(y), y, 0.0), -448.0, 448.0))
    return np.where(np.isfinite(y), codes, 0x7F).astype(np.uint8)


def _round(y):
    """Nearest codes of float64 y in +-448, ties to the even code, the sign kept on a zero."""
    mag = VALUES[:127]
    a = np.abs(y)
    hi = np.clip(np.searchsorted(mag, a, side="left"), 1, 126)
    lo = hi - 1
    dl, dh = a - mag[lo], mag[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return np.where(np.signbit(y), code | 0x80, code)


def append(K, V, k_cache, v_cache, k_scales, v_scales, table, lens, q_start):
    """Updates the cache arrays in place with the new tokens K, V [T, Hkv, d]."""
    page = k_cache.shape[2]
    for r in range(len(q_start) - 1):
        n, total = q_start[r + 1] - q_start[r], int(lens[r])
        first = total - n
        if n == 0 or first < 0:
            continue
        for block in range(first // page, (total - 1) // page + 1):
            lo, hi, p = max(first, block * page), min(total, (block + 1) * page), table[r][block]
            held = lo - block * page
            rows = slice(q_start[r] + lo - first, q_start[r] + hi - first)
            for x, cache, scales in ((K, k_cache, k_scales), (V, v_cache, v_scales)):
                for h in range(cache.shape[1]):
                    e = need(x[rows, h])
                    if held:
                        was = int(scales[p, h]) - BIAS
                        e = max(e, was)
                        cache[p, h, :held] = encode(np.ldexp(VALUES[cache[p, h, :held]], was), e)
                    cache[p, h, held:held + hi - lo] = encode(x[rows, h], e)
                    scales[p, h] = e + BIAS


def tokens(cache, scales, pages, n):
    """The first n tokens [n, Hkv, d] along a page list, float64."""
    page = cache.shape[2]
    p = np.asarray(pages[:-(-n // page)], int)
    x = np.ldexp(VALUES[cache[p]], scales[p].astype(int)[..., None, None] - BIAS)      # [blocks, Hkv, page, d]
    return x.transpose(0, 2, 1, 3).reshape(-1, cache.shape[1], cache.shape[3])[:n]


def attend(q, k_cache, v_cache, k_scales, v_scales, table, lens, q_start, scale):
    """-> (o [T, Hq, d], lse [T, Hq], oabs [T, Hq, d] = sum p |v|, reach [T, Hq] = max_j scale sum |q| |k|);
    rows that see no key, or belong to no request: o = 0, lse = -inf."""
    T, Hq, d = q.shape
    group = Hq // k_cache.shape[1]
    o, oabs = np.zeros((T, Hq, d)), np.zeros((T, Hq, d))
    lse, reach = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for r in range(len(q_start) - 1):
        n_new, n = q_start[r + 1] - q_start[r], int(lens[r])
        k, v = tokens(k_cache, k_scales, table[r], n), tokens(v_cache, v_scales, table[r], n)
        for h in range(Hq):
            kh, vh = k[:, h // group], v[:, h // group]
            for i in range(n_new):
                seen, t = max(0, n - n_new + i + 1), q_start[r] + i
                if seen == 0:
                    continue
                score = scale * (kh[:seen] @ q[t, h])
                reach[t, h] = scale * (np.abs(kh[:seen]) @ np.abs(q[t, h])).max()
                top = score.max()
                e = np.exp(score - top)
                lse[t, h] = top + np.log(e.sum())
                p = e / e.sum()
                o[t, h], oabs[t, h] = p @ vh[:seen], p @ np.abs(vh[:seen])
    return o, lse, oabs, reach

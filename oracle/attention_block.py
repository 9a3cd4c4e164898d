"""Float64 oracle of the attention-block operators: adapters beside a projection, head norm with
rotation, attention over a shared prefix.  Plain loops over tokens and heads, written from the
formulas; shares no code with the CUDA path.  Each function also returns what the callers'
tolerances are made of (sums of absolute values)."""
import numpy as np


def norm_rotate(x, weight, eps, cos_sin, positions, interleaved):
    """x [T, H, d] -> x' : per head x / sqrt(mean x^2 + eps) * weight (weight None: x), then pairs
    turned by the angle whose cosine and sine are the position's row of cos_sin [P, rot]."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    rot = cos_sin.shape[1]
    half = rot // 2
    for t in range(x.shape[0]):
        c = np.asarray(cos_sin[positions[t], :half], np.float64)
        s = np.asarray(cos_sin[positions[t], half:], np.float64)
        for h in range(x.shape[1]):
            v = x[t, h].copy()
            if weight is not None:
                v = v / np.sqrt(np.sum(v * v) / v.size + eps) * np.asarray(weight, np.float64)
            out = v.copy()
            for i in range(half):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
                out[a] = v[a] * c[i] - v[b] * s[i]
                out[b] = v[a] * s[i] + v[b] * c[i]
            y[t, h] = out
    return y


def cache_rows(cache, pages, n):
    """The first n tokens' rows [n, Hkv, d] of a cache [pages, Hkv, page_size, d] along a page list."""
    page_size = cache.shape[2]
    return np.array([cache[pages[j // page_size], :, j % page_size] for j in range(n)],
                    np.float64).reshape(n, cache.shape[1], cache.shape[3])


def attend(q, k_cache, v_cache, prefix_pages, prefix_len, block_table, suffix_lens, q_start, scale):
    """-> (o [T, Hq, d], lse [T, Hq], oabs [T, Hq, d] = sum_j p_j |v_j|); a row without keys gives
    o = 0 and lse = -inf."""
    q = np.asarray(q, np.float64)
    T, Hq, d = q.shape
    Hkv = k_cache.shape[1]
    group = Hq // Hkv
    o, oabs = np.zeros((T, Hq, d)), np.zeros((T, Hq, d))
    lse = np.full((T, Hq), -np.inf)
    kp, vp = cache_rows(k_cache, prefix_pages, prefix_len), cache_rows(v_cache, prefix_pages, prefix_len)
    for r in range(len(q_start) - 1):
        n_new = q_start[r + 1] - q_start[r]
        n = 0 if block_table is None else int(suffix_lens[r])
        ks = cache_rows(k_cache, [] if n == 0 else block_table[r], n)
        vs = cache_rows(v_cache, [] if n == 0 else block_table[r], n)
        for i in range(n_new):
            seen = max(0, n - n_new + i + 1)
            k = np.concatenate((kp, ks[:seen]))
            v = np.concatenate((vp, vs[:seen]))
            if k.shape[0] == 0:
                continue
            t = q_start[r] + i
            for h in range(Hq):
                score = scale * (k[:, h // group] @ q[t, h])
                top = score.max()
                e = np.exp(score - top)
                lse[t, h] = top + np.log(e.sum())
                p = e / e.sum()
                o[t, h] = p @ v[:, h // group]
                oabs[t, h] = p @ np.abs(v[:, h // group])
    return o, lse, oabs


def adapters(x, a, b, adapter, scales, ranks=None):
    """-> (delta [M, N], dabs [M, N]): scales[a] (x A^T) B^T and scales[a] sum_j |v_j| |b_j|, per row
    of its adapter; zero rows for adapter -1."""
    x = np.asarray(x, np.float64)
    delta = np.zeros((x.shape[0], b.shape[1]))
    dabs = np.zeros_like(delta)
    for m in range(x.shape[0]):
        i = int(adapter[m])
        if i < 0:
            continue
        r = a.shape[1] if ranks is None else int(ranks[i])
        v = np.asarray(a[i, :r], np.float64) @ x[m]
        w = np.asarray(b[i, :, :r], np.float64)
        s = float(scales[i])
        delta[m] = s * (w @ v)
        dabs[m] = abs(s) * (np.abs(w) @ np.abs(v))
    return delta, dabs

"""CPU checks of the 8-bit cache: the float64 oracle against closed forms and invariants, and the
library's refusals (nothing is launched)."""
import ctypes

import numpy as np
import pytest

from bit_weight_quantized_wq_gb300 import binding
from bit_weight_quantized_wq_gb300 import build as wqbuild
from oracle import attention_block as ab
from oracle import cache_e4m3 as c8
from oracle import fp8


# ------------------------------------------------------------------------------ the oracle
def test_need_is_the_lowest_power_of_two_that_holds_the_values():
    for top, e in ((448.0, 0), (448.0001, 1), (449.0, 1), (224.0, -1), (224.01, 0), (1.75, -8), (0.0, -64), (1e-30, -64), (1e38, 64),
                   (448.0 * 2.0 ** -64, -64), (448.0 * 2.0 ** -63, -63)):
        assert c8.need(np.array([0.0, -top, top / 2])) == e, top
    assert c8.need(np.array([np.nan, np.inf, 3.5])) == c8.need(np.array([3.5]))
    assert c8.need(np.array([np.nan])) == -64


def test_encode_agrees_with_the_fp8_oracle_and_rounds_once():
    rng = np.random.default_rng(0)
    x = np.float32(rng.standard_normal(2000) * 100).clip(-448, 448)
    assert np.array_equal(c8.encode(x, 0), fp8.e4m3_round(x))
    assert np.array_equal(c8.encode(x, -3), c8.encode(x * 8.0, 0)) and c8.encode(np.array([500.0]), 0)[0] == 0x7E
    y = c8.VALUES[c8.encode(x, 0)]
    assert np.all(np.abs(y - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10))
    assert c8.encode(np.array([np.inf, -np.inf, np.nan]), 2).tolist() == [0x7F] * 3
    assert np.array_equal(c8.encode(c8.VALUES[:127], 0), np.arange(127))


def _empty(pages, hkv, page, d):
    rng = np.random.default_rng(5)
    caches = [rng.integers(0, 127, (pages, hkv, page, d)).astype(np.uint8) for _ in range(2)]
    return caches + [rng.integers(100, 140, (pages, hkv)).astype(np.uint8) for _ in range(2)]


def test_token_by_token_holds_what_one_call_holds_but_for_the_lowest_steps():
    rng = np.random.default_rng(1)
    K, V = (rng.standard_normal((37, 2, 8)) * np.exp(rng.standard_normal((37, 1, 1))) for _ in range(2))
    table = [[3, 0, 2]]
    one, each = _empty(4, 2, 16, 8), _empty(4, 2, 16, 8)
    c8.append(K, V, *one, table, [37], [0, 37])
    for t in range(37):
        c8.append(K[t:t + 1], V[t:t + 1], *each, table, [t + 1], [0, 1])
    for i, x in ((0, K), (1, V)):
        a, b = (c8.tokens(c[i], c[i + 2], table[0], 37) for c in (one, each))
        assert all(np.array_equal(one[i + 2][p], each[i + 2][p]) for p in table[0])
        lowest = np.ldexp(2.0 ** -9, one[i + 2][table[0]].astype(int) - 127).max()
        assert np.abs(a - b).max() <= lowest
        assert np.all(np.abs(a - x) <= 2.0 ** -4 * np.abs(x) + lowest)
    assert np.array_equal(one[0][1], _empty(4, 2, 16, 8)[0][1])            # a page that is not the request's


def test_a_page_starts_afresh_and_its_scale_grows():
    caches = _empty(2, 1, 16, 8)
    caches[2][:] = 191
    big, small = np.full((1, 1, 8), 7.0), np.full((1, 1, 8), 7e-3)
    c8.append(small, small, *caches, [[1]], [1], [0, 1])
    low = int(caches[2][1, 0])
    c8.append(big, big, *caches, [[1]], [2], [0, 1])
    assert low == 127 + c8.need(small) and int(caches[2][1, 0]) == 127 + c8.need(big) and int(caches[2][0, 0]) == 191
    c8.append(small, small, *caches, [[1]], [3], [0, 1])                   # grows, never shrinks
    assert int(caches[2][1, 0]) == 127 + c8.need(big)
    c8.append(small, small, *caches, [[1]], [1], [0, 1])
    assert int(caches[2][1, 0]) == low


def test_attend_is_the_16_bit_caches_attention_of_the_values_read_back():
    rng = np.random.default_rng(2)
    caches = _empty(6, 2, 16, 8)
    K, V, q = rng.standard_normal((33, 2, 8)), rng.standard_normal((33, 2, 8)), rng.standard_normal((6, 4, 8))
    table = [[4, 1, 5], [0, 3, -1]]
    c8.append(K[:20], V[:20], *caches, table, [20, 0], [0, 20, 20])
    c8.append(K[20:], V[20:], *caches, table, [20, 13], [0, 0, 13])
    got = c8.attend(q, *caches, table, [20, 13], [0, 2, 6], 0.3)
    wide = [np.ldexp(c8.VALUES[caches[i]], caches[i + 2].astype(int)[..., None, None] - 127) for i in (0, 1)]
    want = ab.attend(q, *wide, [], 0, table, [20, 13], [0, 2, 6], 0.3)
    assert all(np.allclose(a, b, rtol=1e-12, atol=1e-12) for a, b in zip(got, want))
    o, lse, _, _ = c8.attend(q[:2], *caches, table, [0, 1], [0, 1, 2], 0.3)
    assert np.all(o[0] == 0) and np.all(np.isneginf(lse[0])) and np.allclose(o[1], wide[1][0, :, 0].repeat(2, 0))


# ------------------------------------------------------------------------------ the refusals
@pytest.fixture(scope="module")
def lib():
    import os
    newest = max(os.path.getmtime(os.path.join(wqbuild.CSRC, f)) for f in os.listdir(wqbuild.CSRC))
    if not os.path.exists(binding.LIB_PATH) or os.path.getmtime(binding.LIB_PATH) < newest:
        wqbuild.build()
    return binding.load_library()


def _p(i, odd=0):
    """Distinct, far apart, aligned addresses that are never dereferenced."""
    return ctypes.c_void_p(0x100000000 * (i + 1) + odd)


CACHE = dict(kc=_p(10), vc=_p(11), ks=_p(12, 1), vs=_p(13, 3), pages=9, page=16, table=_p(14), blocks=4)


def _append(lib, **kw):
    a = dict(CACHE, dtype=0, K=_p(0), kst=256, V=_p(1), vst=256, T=4, R=2, Hkv=2, d=128, lens=_p(2), qs=_p(3), new=4)
    a.update(kw)
    return lib.wq_kv_append_e4m3(a["dtype"], a["K"], a["kst"], a["V"], a["vst"], a["T"], a["R"], a["Hkv"], a["d"], a["kc"], a["vc"],
                                 a["ks"], a["vs"], a["pages"], a["page"], a["table"], a["blocks"], a["lens"], a["qs"], a["new"], None)


def _read(lib, **kw):
    a = dict(CACHE, dtype=0, Hkv=2, d=128, starts=_p(2), R=2, T=4, K=_p(0), V=_p(1))
    a.update(kw)
    return lib.wq_kv_read_e4m3(a["dtype"], a["kc"], a["vc"], a["ks"], a["vs"], a["pages"], a["page"], a["Hkv"], a["d"], a["table"],
                               a["blocks"], a["starts"], a["R"], a["T"], a["K"], a["V"], None)


def _attend(lib, **kw):
    a = dict(CACHE, dtype=0, Q=_p(0), qst=1024, T=4, R=2, Hq=8, Hkv=2, d=128, lens=_p(2), qs=_p(3), new=4, scale=0.1, O=_p(4),
             lse=_p(5), ws=_p(6), wsb=None)
    a.update(kw)
    if a["wsb"] is None:
        a["wsb"] = lib.wq_attn_e4m3_workspace_bytes(a["T"], a["R"], a["Hq"], a["Hkv"], a["d"], a["new"])
    return lib.wq_attn_e4m3(a["dtype"], a["Q"], a["qst"], a["T"], a["R"], a["Hq"], a["Hkv"], a["d"], a["kc"], a["vc"], a["ks"], a["vs"],
                            a["pages"], a["page"], a["table"], a["blocks"], a["lens"], a["qs"], a["new"], a["scale"], a["O"], a["lse"],
                            a["ws"], a["wsb"], None)


@pytest.mark.parametrize("call,arrays", [(_append, ("K", "V", "lens")), (_read, ("K", "V", "starts")), (_attend, ("Q", "O", "lens"))])
def test_refusals_that_the_three_share(lib, call, arrays):
    assert call(lib, dtype=2) == 7
    for name in arrays + ("kc", "vc", "ks", "vs", "table"):
        assert call(lib, **{name: None}) == 1, name
    for bad in (dict(T=0), dict(T=(1 << 24) + 1), dict(R=0), dict(R=(1 << 24) + 1), dict(d=96), dict(d=256), dict(page=8), dict(page=48),
                dict(page=256), dict(pages=0), dict(pages=1 << 31), dict(blocks=0), dict(blocks=(1 << 26) + 1), dict(Hkv=0)):
        assert call(lib, **bad) == 2, bad
    for name in ("kc", "vc") + arrays[:2]:
        assert call(lib, **{name: _p(30, 8)}) == 3, name
    for name in ("table", arrays[2]):
        assert call(lib, **{name: _p(30, 2)}) == 3, name


def test_append_refusals(lib):
    for bad in (dict(kst=248), dict(vst=260), dict(kst=1 << 41), dict(new=0), dict(qs=None), dict(Hkv=1025, kst=1 << 20, vst=1 << 20)):
        assert _append(lib, **bad) == 2, bad
    assert _append(lib, qs=_p(3, 1)) == 3
    for a, b in (("kc", "vc"), ("K", "kc"), ("V", "vc"), ("ks", "vs"), ("ks", "kc"), ("vs", "kc"), ("ks", "vc"), ("vs", "vc"), ("K", "vs")):
        base = dict(K=_p(0), V=_p(1), **CACHE)
        assert _append(lib, **{a: base[b] if base[b].value % 16 == 0 else ctypes.c_void_p(base[b].value // 16 * 16)}) == 7, (a, b)


def test_read_refusals(lib):
    assert _read(lib, K=_p(1)) == 7 and _read(lib, K=_p(10)) == 7 and _read(lib, V=_p(11)) == 7 and _read(lib, V=_p(12)) == 7


def test_attend_refusals(lib):
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert _attend(lib, scale=scale) == 7
    for bad in (dict(Hq=7), dict(Hq=512, Hkv=2, qst=65536), dict(Hq=1025, Hkv=1025, qst=1 << 20), dict(qst=1016), dict(qst=1028),
                dict(new=0), dict(qs=None), dict(T=1 << 24, Hq=128, Hkv=1, qst=16384)):
        assert _attend(lib, **bad) == 2, bad
    assert _attend(lib, ws=None) == 4 and _attend(lib, wsb=1 << 20) == 4 and _attend(lib, ws=_p(6, 8)) == 3
    assert _attend(lib, lse=_p(5, 2)) == 3 and _attend(lib, qs=_p(3, 2)) == 3
    assert _attend(lib, O=_p(0)) == 7 and _attend(lib, O=_p(0, 1024)) == 7 and _attend(lib, O=_p(10)) == 7 and _attend(lib, O=_p(12)) == 7
    assert lib.wq_attn_e4m3_workspace_bytes(4, 2, 7, 2, 128, 1) == 0 and lib.wq_attn_e4m3_workspace_bytes(4, 2, 8, 2, 96, 1) == 0


def test_attend_refuses_outputs_that_overlap(lib):
    """lse is stored while other CTAs still read queries and codes: it shares no byte with them, nor with O."""
    stats, last = 4 * 8 * 4, 3 * 1024 * 2 + 8 * 128 * 2                   # bytes of lse, and of Q from its first to its last element
    for name, at in (("Q", 0), ("O", 4), ("k_cache", 10), ("v_cache", 11), ("k_scales", 12), ("v_scales", 13)):
        assert _attend(lib, lse=_p(at)) == 7, name
        assert _attend(lib, lse=ctypes.c_void_p(_p(at).value - stats + 4)) == 7, name
    assert _attend(lib, lse=_p(0, last - 4)) == 7 and _attend(lib, lse=_p(4, 4 * 8 * 128 * 2 - 4)) == 7

"""CPU checks of the attention-block operators: the float64 oracle against closed forms and
invariants, and the library's refusals (nothing is launched)."""
import ctypes

import numpy as np
import pytest

from oracle import attention_block as ab
from bit_weight_quantized_wq_gb300 import binding
from bit_weight_quantized_wq_gb300 import build as wqbuild


# ------------------------------------------------------------------------------ the oracle
def _table(n, rot):
    ang = np.arange(n)[:, None] * (1e4 ** (-np.arange(0, rot, 2) / rot))
    return np.concatenate((np.cos(ang), np.sin(ang)), 1)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_depends_on_distance_only(interleaved):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((4, 2, 64))
    tab = _table(50, 32)
    y = ab.norm_rotate(x, None, 0.0, tab, [0, 3, 7, 49], interleaved)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-12)
    assert np.allclose(y[0], x[0])                          # position 0: no turn
    assert np.array_equal(y[:, :, 32:], x[:, :, 32:])       # past rot: untouched
    q, k = x[:1, :1], x[1:2, :1]
    at = lambda i, j: float((ab.norm_rotate(q, None, 0, tab, [i], interleaved)
                             * ab.norm_rotate(k, None, 0, tab, [j], interleaved)).sum())
    assert abs(at(5, 2) - at(40, 37)) < 1e-10 and abs(at(5, 2) - at(5, 3)) > 1e-3


def test_norm_gives_unit_mean_square_times_weight():
    x = np.random.default_rng(2).standard_normal((3, 2, 64)) * 7
    y = ab.norm_rotate(x, np.full(64, 2.0), 0.0, np.concatenate((np.ones((1, 8)), np.zeros((1, 8))), 1), [0, 0, 0], False)
    assert np.allclose((y * y).mean(-1), 4.0)


def test_attend_against_one_dense_softmax_and_empty_rows():
    rng = np.random.default_rng(3)
    kc, vc = rng.standard_normal((6, 2, 16, 64)), rng.standard_normal((6, 2, 16, 64))
    q = rng.standard_normal((3, 4, 64))
    o, lse, oabs = ab.attend(q, kc, vc, [4, 1], 20, [[0, 3], [2, 5]], [18, 0], [0, 2, 3], 0.125)
    k = np.concatenate((kc[4], kc[1][:, :4], kc[0], kc[3][:, :2]), 1)     # [Hkv, 38, d]
    v = np.concatenate((vc[4], vc[1][:, :4], vc[0], vc[3][:, :2]), 1)
    for i, n in ((0, 37), (1, 38)):
        for h in range(4):
            s = np.exp(0.125 * k[h // 2, :n] @ q[i, h])
            assert np.allclose(o[i, h], s @ v[h // 2, :n] / s.sum())
            assert np.isclose(lse[i, h], np.log(s.sum()))
    s = np.exp(0.125 * k[1, :20] @ q[2, 3])                               # a request without own keys
    assert np.allclose(o[2, 3], s @ v[1, :20] / s.sum())
    o, lse, _ = ab.attend(q[:1], kc, vc, [], 0, None, None, [0, 1], 0.125)
    assert np.all(o == 0) and np.all(np.isneginf(lse))
    assert np.all(oabs >= 0)


def test_adapters_is_a_low_rank_weight():
    rng = np.random.default_rng(4)
    x, a, b = rng.standard_normal((3, 16)), rng.standard_normal((2, 8, 16)), rng.standard_normal((2, 10, 8))
    d, dabs = ab.adapters(x, a, b, [1, -1, 0], [0.5, 2.0])
    assert np.allclose(d[0], 2.0 * x[0] @ (b[1] @ a[1]).T)
    assert np.allclose(d[2], 0.5 * x[2] @ (b[0] @ a[0]).T)
    assert np.all(d[1] == 0) and np.all(dabs >= np.abs(d) - 1e-9)


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


def _rope(lib, **kw):
    a = dict(dtype=0, T=4, Hq=8, Hkv=2, d=128, Q=_p(0), qs=1024, K=_p(1), ks=256, wq=None, wk=None, eps=1e-6, tab=_p(2),
             n=64, rot=128, il=0, pos=_p(3), Qo=_p(4), Ko=_p(5))
    a.update(kw)
    return lib.wq_qk_norm_rope(a["dtype"], a["T"], a["Hq"], a["Hkv"], a["d"], a["Q"], a["qs"], a["K"], a["ks"], a["wq"],
                               a["wk"], a["eps"], a["tab"], a["n"], a["rot"], a["il"], a["pos"], a["Qo"], a["Ko"], None)


def test_rope_refusals(lib):
    assert _rope(lib, dtype=2) == 7 and _rope(lib, il=2) == 7
    assert _rope(lib, eps=-1.0) == 7 and _rope(lib, eps=float("nan")) == 7
    for name in ("Q", "K", "tab", "pos", "Qo", "Ko"):
        assert _rope(lib, **{name: None}) == 1, name
    assert _rope(lib, T=0) == 2 and _rope(lib, d=96) == 2 and _rope(lib, rot=24) == 2 and _rope(lib, rot=0) == 2
    assert _rope(lib, rot=256) == 2 and _rope(lib, n=0) == 2
    assert _rope(lib, qs=1016) == 2 and _rope(lib, ks=260) == 2
    assert _rope(lib, Q=_p(0, 8)) == 3 and _rope(lib, Ko=_p(5, 2)) == 3
    assert _rope(lib, Qo=_p(0), qs=2048) == 7           # in place only without a stride
    assert _rope(lib, Qo=_p(0, 1024)) == 7              # partly over its input
    assert _rope(lib, Ko=_p(0)) == 7 and _rope(lib, Ko=_p(4)) == 7 and _rope(lib, Qo=_p(1)) == 7


def _rope_cache(lib, **kw):
    a = dict(T=4, Hq=8, Hkv=2, d=128, Q=_p(0), V=_p(1), vs=256, kc=_p(2), vc=_p(3), pages=4, page=16, slots=_p(4), Qo=_p(5))
    a.update(kw)
    return lib.wq_qk_norm_rope_cache(0, a["T"], a["Hq"], a["Hkv"], a["d"], a["Q"], 1024, _p(6), 256, a["V"], a["vs"], None,
                                     None, 1e-6, _p(7), 64, 128, 0, _p(8), a["Qo"], a["kc"], a["vc"], a["pages"], a["page"],
                                     a["slots"], None)


def test_rope_cache_refusals(lib):
    for name in ("V", "kc", "vc", "slots"):
        assert _rope_cache(lib, **{name: None}) == 1, name
    assert _rope_cache(lib, page=48) == 2 and _rope_cache(lib, pages=0) == 2 and _rope_cache(lib, pages=1 << 30) == 2
    assert _rope_cache(lib, vs=128) == 2 and _rope_cache(lib, kc=_p(2, 4)) == 3
    assert _rope_cache(lib, vc=_p(2)) == 7 and _rope_cache(lib, kc=_p(0)) == 7 and _rope_cache(lib, vc=_p(5)) == 7


def _attn(lib, **kw):
    a = dict(dtype=0, Q=_p(0), qs=1024, T=4, R=4, Hq=8, Hkv=2, d=128, kc=_p(1), vc=_p(2), pages=9, page=16, pp=_p(3), P=40,
             bt=_p(4), nb=3, sl=_p(5), q0=None, new=1, scale=0.1, O=_p(6), lse=_p(7), ws=_p(8), wsb=1 << 40)
    a.update(kw)
    return lib.wq_attn_shared_prefix(a["dtype"], a["Q"], a["qs"], a["T"], a["R"], a["Hq"], a["Hkv"], a["d"], a["kc"], a["vc"],
                                     a["pages"], a["page"], a["pp"], a["P"], a["bt"], a["nb"], a["sl"], a["q0"], a["new"],
                                     a["scale"], a["O"], a["lse"], a["ws"], a["wsb"], None)


def test_attn_refusals(lib):
    assert _attn(lib, dtype=-1) == 7
    for s in (0.0, -1.0, float("inf"), float("nan")):
        assert _attn(lib, scale=s) == 7
    for name in ("Q", "kc", "vc", "pp", "bt", "sl", "O"):
        assert _attn(lib, **{name: None}) == 1, name
    assert _attn(lib, T=0) == 2 and _attn(lib, R=0) == 2 and _attn(lib, Hq=9) == 2 and _attn(lib, d=256) == 2
    assert _attn(lib, page=8) == 2 and _attn(lib, P=-1) == 2 and _attn(lib, nb=-1) == 2 and _attn(lib, qs=512) == 2
    assert _attn(lib, T=5) == 2 and _attn(lib, new=2) == 2 and _attn(lib, q0=_p(9), new=0) == 2
    assert _attn(lib, Q=_p(0, 8)) == 3 and _attn(lib, lse=_p(7, 2)) == 3 and _attn(lib, q0=_p(9, 1)) == 3
    assert _attn(lib, O=_p(0)) == 7
    assert _attn(lib, ws=None) == 4 and _attn(lib, wsb=16) == 4 and _attn(lib, ws=_p(8, 8)) == 3
    assert lib.wq_attn_workspace_bytes(4, 4, 8, 2, 128, 1) > 0
    assert lib.wq_attn_workspace_bytes(4, 4, 8, 3, 128, 1) == 0


def test_attn_refuses_more_prefix_work_than_one_call_holds(lib):
    """Hq = Hkv = 8: row tiles of 256 tokens.  8 * ceil(T / 256) * (10 ceil(P / 64) + 20) <= 2^30."""
    T = 256 * 16
    most = 64 * (((1 << 30) // 8 // 16 - 20) // 10)
    assert _attn(lib, Hq=8, Hkv=8, qs=8 * 128, T=T, q0=_p(9), P=most + 64, pages=64) == 2
    assert _attn(lib, Hq=8, Hkv=8, qs=8 * 128, T=T, q0=_p(9), P=most, pages=64) != 2


def _lora(lib, **kw):
    a = dict(dtype=0, base=_p(0), X=_p(1), M=4, K=128, N=64, A=_p(2), B=_p(3), L=2, r=16, ranks=None, ad=_p(4), s=_p(5),
             Y=_p(6), ws=_p(7), wsb=1 << 40)
    a.update(kw)
    return lib.wq_lora_add(a["dtype"], a["base"], a["X"], a["M"], a["K"], a["N"], a["A"], a["B"], a["L"], a["r"], a["ranks"],
                           a["ad"], a["s"], a["Y"], a["ws"], a["wsb"], None)


def test_lora_refusals(lib):
    assert _lora(lib, dtype=2) == 7
    for name in ("base", "X", "A", "B", "ad", "s", "Y"):
        assert _lora(lib, **{name: None}) == 1, name
    for kw in (dict(M=0), dict(N=0), dict(K=12), dict(K=0), dict(r=4), dict(r=136), dict(r=0), dict(L=0)):
        assert _lora(lib, **kw) == 2, kw
    assert _lora(lib, X=_p(1, 8)) == 3 and _lora(lib, ranks=_p(9, 2)) == 3
    assert _lora(lib, Y=_p(0, 16)) == 7 and _lora(lib, Y=_p(1)) == 7
    assert _lora(lib, ws=None) == 4 and _lora(lib, wsb=16) == 4
    assert lib.wq_lora_workspace_bytes(4, 128, 64, 12) == 0 and lib.wq_lora_workspace_bytes(4, 128, 64, 16) > 0
    w4 = lambda fmt=0, z=_p(9), ws=_p(7), wsb=1 << 40, K=128, r=16: lib.wq_gemm_w4a16_lora(
        fmt, _p(1), 4, K, 64, _p(8), _p(10), z, _p(2), _p(3), 2, r, None, _p(4), _p(5), _p(6), ws, wsb, None)
    assert w4(fmt=3) == 7 and w4(z=None) == 1 and w4(K=64) == 2 and w4(r=4) == 2 and w4(ws=None) == 4 and w4(wsb=4096) == 4
    need = lib.wq_gemm_w4a16_lora_workspace_bytes(0, 4, 128, 64, 16)
    assert need > lib.wq_gemm_workspace_bytes(0, 4, 128, 64)
    assert lib.wq_gemm_w4a16_lora_workspace_bytes(7, 4, 128, 64, 16) == 0


def test_rope_index_arrays_are_refused_only_off_4_bytes(lib):
    """The accepted addresses get as far as the check for overlaps, which refuses these calls (nothing is launched)."""
    for odd in (4, 8, 12):
        assert _rope(lib, pos=_p(3, odd), Qo=_p(0, 1024)) == 7 and _rope_cache(lib, slots=_p(4, odd), vc=_p(2)) == 7
    assert _rope(lib, pos=_p(3, 2), Qo=_p(0, 1024)) == 3 and _rope_cache(lib, slots=_p(4, 1), vc=_p(2)) == 3

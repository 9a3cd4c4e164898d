"""The attention-block operators on the GPU against the float64 oracle: head norm with rotation (and
the cache write), attention over a shared prefix, adapters beside a projection, and the three run
together as one block.

Tolerances (u is half a unit in the last place of the output type, relative: 2^-8 for
bf16's 8 significant bits, 2^-11 for fp16's 11; one rounding of a value is off by at most u of it):
- rotation: u |ref| plus float32 arithmetic of the norm and two products, 2^-18 (|a| + |b|) of a
  pair, bounded through the head's largest value;
- attention: the weights p enter the second product rounded to the type (each off by at most u of
  it; float32 elsewhere), so u |ref| + u sum p |v|, with 1e-5 for float32 sums; lse float32: 2e-5
  (1 + |lse|);
- adapters: the inner products enter the second product rounded to the type, so u |ref| + u sum
  |v| |b| + 1e-5 of that sum; the quantized layer adds one more rounding of its own output and its
  own 1e-2 (1 + |y|)."""
import numpy as np
import pytest

from bit_weight_quantized_wq_gb300 import inputs
from oracle import attention_block as ab
from oracle import int4_g128, linear, mxfp4
from tests._util import TOL, kernels_of

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(scope="module")
def B():
    import torch
    from bit_weight_quantized_wq_gb300 import binding
    binding.check_device()
    torch.cuda.init()
    return binding


@pytest.fixture(autouse=True)
def no_error_flags(B):
    B.read_error_flags()
    yield
    assert B.read_error_flags() == 0


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16}[name]


def _rand(seed, shape, dtype, scale=1.0):
    """The same values as a CUDA tensor of the type and as float64."""
    import torch
    t = (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * scale).to(_dt(dtype))
    return t.cuda(), t.double().numpy()


def _host(t):
    return t.detach().double().cpu().numpy()


def _within(got, ref, limit, what):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= limit)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - ref) / np.maximum(limit, 1e-300), 0)), bad.shape)
        raise AssertionError("%s: %d of %d off; worst at %s: got %r, want %r" % (what, bad.sum(), bad.size, i, got[i], ref[i]))


# ------------------------------------------------------------------------------- rotation
def _table(n, rot):
    import torch
    ang = np.arange(n)[:, None] * (1e4 ** (-np.arange(0, rot, 2) / rot))
    return torch.from_numpy(np.concatenate((np.cos(ang), np.sin(ang)), 1).astype(np.float32)).cuda()


def _rope_limit(ref, x, w, dtype):
    """u |ref| + 2^-18 of the head's largest value after the norm (|a| + |b| of any pair is below twice it)."""
    top = np.abs(ref).max(-1, keepdims=True)
    return U[dtype] * np.abs(ref) + 2.0 ** -17 * top


ROPE = [  # T, Hq, Hkv, d, rot, interleaved, norm
    (1, 32, 8, 128, 128, False, True),
    (1, 1, 1, 64, 16, True, False),
    (7, 28, 4, 128, 64, True, True),
    (13, 5, 5, 64, 64, False, True),
    (33, 3, 1, 256, 256, False, False),
    (5, 9, 3, 256, 64, True, True),
    (64, 16, 16, 64, 32, False, True),
    (600, 8, 1, 128, 32, False, True),
    (515, 7, 7, 64, 48, True, True),
    (1100, 64, 8, 64, 64, True, True),          # enough units for the kernel that walks over them
    (1301, 33, 3, 128, 96, False, True),
    (1000, 17, 4, 256, 128, False, False),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,Hq,Hkv,d,rot,interleaved,norm", ROPE)
def test_rope(B, dtype, T, Hq, Hkv, d, rot, interleaved, norm):
    import torch
    q, qf = _rand(T + 1, (T, Hq, d), dtype, 3.0)
    k, kf = _rand(T + 2, (T, Hkv, d), dtype, 0.1)
    (wq, wqf), (wk, wkf) = _rand(3, (d,), dtype), _rand(4, (d,), dtype)
    if not norm:
        wq = wqf = wk = wkf = None
    tab = _table(97, rot)
    pos = np.random.default_rng(T).integers(0, 97, T)
    p = torch.from_numpy(pos.astype(np.int32)).cuda()
    qo, ko = B.qk_norm_rope(q, k, p, tab, wq, wk, eps=1e-5, interleaved=interleaved)
    tabf = _host(tab)
    for got, x, w, what in ((qo, qf, wqf, "Q"), (ko, kf, wkf, "K")):
        ref = ab.norm_rotate(x, w, 1e-5, tabf, pos, interleaved)
        _within(_host(got), ref, _rope_limit(ref, x, w, dtype), what)
    # the same in place
    B.qk_norm_rope(q, k, p, tab, wq, wk, eps=1e-5, interleaved=interleaved, out=(q, k))
    assert torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("T,Hq,Hkv,d", [(1, 8, 2, 128), (50, 4, 4, 64), (9, 16, 2, 256), (700, 6, 2, 128), (1500, 24, 4, 128)])
def test_rope_cache(B, dtype, page, T, Hq, Hkv, d):
    """From the parts of a fused projection output into a cache; padding rows are not written, and
    neither is any other slot."""
    import torch
    x, xf = _rand(T, (T, (Hq + 2 * Hkv) * d), dtype)
    parts = [x[:, :Hq * d].view(T, Hq, d), x[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d), x[:, (Hq + Hkv) * d:].view(T, Hkv, d)]
    wk, wkf = _rand(5, (d,), dtype)
    tab = _table(64, 32)
    rng = np.random.default_rng(T + page)
    pos = rng.integers(0, 64, T)
    pages = (T + page - 1) // page + 2
    slots = rng.choice(pages * page, T, replace=False)
    if T > 1:
        slots[T // 2] = -1
    kc, kcf = _rand(6, (pages, Hkv, page, d), dtype)
    vc, vcf = _rand(7, (pages, Hkv, page, d), dtype)
    qo = B.qk_norm_rope_cache(parts[0], parts[1], parts[2], torch.from_numpy(pos.astype(np.int32)).cuda(), tab, kc, vc,
                              torch.from_numpy(slots.astype(np.int32)).cuda(), None, wk)
    tabf = _host(tab)
    f = [xf[:, :Hq * d].reshape(T, Hq, d), xf[:, Hq * d:(Hq + Hkv) * d].reshape(T, Hkv, d), xf[:, (Hq + Hkv) * d:].reshape(T, Hkv, d)]
    ref = ab.norm_rotate(f[0], None, 1e-6, tabf, pos, False)
    _within(_host(qo), ref, _rope_limit(ref, f[0], None, dtype), "Q")
    ref = ab.norm_rotate(f[1], wkf, 1e-6, tabf, pos, False)
    limit = np.zeros_like(kcf)
    for t in range(T):
        if slots[t] >= 0:
            kcf[slots[t] // page, :, slots[t] % page] = ref[t]
            limit[slots[t] // page, :, slots[t] % page] = _rope_limit(ref[t], f[1][t], wkf, dtype)
            vcf[slots[t] // page, :, slots[t] % page] = f[2][t]
    _within(_host(kc), kcf, limit, "k_cache")
    assert np.array_equal(_host(vc), vcf)


def test_rope_reports_indices_out_of_range(B):
    import torch
    q, _ = _rand(1, (3, 2, 64), "bf16")
    k, _ = _rand(2, (3, 1, 64), "bf16")
    kc, kcf = _rand(3, (2, 1, 16, 64), "bf16")
    vc, vcf = _rand(4, (2, 1, 16, 64), "bf16")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    B.qk_norm_rope_cache(q, k, k, i32(0, 1, 2), _table(8, 64), kc, vc, i32(-1, 32, 2 ** 31 - 1))
    assert B.read_error_flags() == 1 << 7
    assert np.array_equal(_host(kc), kcf) and np.array_equal(_host(vc), vcf)
    B.qk_norm_rope(q, k, i32(0, 8, -1), _table(8, 64))
    assert B.read_error_flags() == 1 << 7


def test_rope_rejects_bad_arguments(B):
    import torch
    q, _ = _rand(1, (3, 2, 64), "bf16")
    k, _ = _rand(2, (3, 1, 64), "bf16")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    tab = _table(8, 64)
    with pytest.raises(ValueError):
        B.qk_norm_rope(q.float(), k.float(), pos, tab)
    with pytest.raises(ValueError):
        B.qk_norm_rope(q, k.half(), pos, tab)
    with pytest.raises(ValueError):
        B.qk_norm_rope(q, k, pos.long(), tab)
    with pytest.raises(ValueError):
        B.qk_norm_rope(q, k[:2], pos, tab)
    with pytest.raises(ValueError):
        B.qk_norm_rope(q.transpose(0, 1), k, pos, tab)
    with pytest.raises(ValueError):
        B.qk_norm_rope(q.cpu(), k, pos, tab)
    with pytest.raises(ValueError):
        B.qk_norm_rope(q, k, pos, tab[:, :24].contiguous())
    with pytest.raises(ValueError):
        B.qk_norm_rope(q[:0], k[:0], pos[:0], tab)


# ------------------------------------------------------------------------------- attention
class Batch:
    """A batch on a shuffled cache whose unused rows hold NaN and infinities."""

    def __init__(self, seed, news, prefix, lens, Hq, Hkv, d, page, dtype, sharp=1.0):
        import torch
        rng = np.random.default_rng(seed)
        R = len(lens)
        self.blocks = [(n + page - 1) // page for n in lens]
        npre = (prefix + page - 1) // page
        pages = npre + sum(self.blocks) + 2
        perm = rng.permutation(pages)
        kc = rng.standard_normal((pages, Hkv, page, d))
        vc = rng.standard_normal((pages, Hkv, page, d))
        used = np.zeros((pages, page), bool)
        self.prefix_pages = perm[:npre]
        width = max(self.blocks) if R else 0
        self.table = np.full((R, width), -7, np.int32)
        at = npre
        for r in range(R):
            self.table[r, :self.blocks[r]] = perm[at:at + self.blocks[r]]
            at += self.blocks[r]
        for pl, n in [(self.prefix_pages, prefix)] + [(self.table[r], lens[r]) for r in range(R)]:
            for j in range(n):
                used[pl[j // page], j % page] = True
        for c, junk in ((kc, (np.nan, np.inf)), (vc, (np.inf, np.nan))):
            c[~used.any(1)] = junk[0]
            for p in range(pages):
                c[p, :, ~used[p]] = junk[1]
        q0 = np.concatenate(([0], np.cumsum(news)))
        T = int(q0[-1])
        to = lambda a: torch.from_numpy(a).to(_dt(dtype)).cuda()
        self.q, self.kc, self.vc = to(sharp * rng.standard_normal((T, Hq, d))), to(kc), to(vc)
        i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()
        self.args = [i32(self.prefix_pages), prefix, i32(self.table), i32(lens)]
        self.kw = dict(q_start=i32(q0), max_new=max(news))
        self.scale = d ** -0.5
        self.oracle = lambda: ab.attend(_host(self.q), _host(self.kc), _host(self.vc), self.prefix_pages, prefix, self.table,
                                        lens, q0, self.scale)
        self.dtype = dtype

    def run(self, B, **kw):
        return B.attn_shared_prefix(self.q, self.kc, self.vc, *self.args, **{**self.kw, **kw})

    def check(self, got):
        o, lse, oabs = self.oracle()
        u = U[self.dtype]
        _within(_host(got[0]), o, u * np.abs(o) + u * oabs + 1e-5, "O")
        l = _host(got[1])
        assert np.array_equal(np.isneginf(l), np.isneginf(lse))
        fine = np.isfinite(lse)
        _within(l[fine], lse[fine], 2e-5 * (1 + np.abs(lse[fine])), "lse")


ATTN = [  # new tokens, prefix, own lengths, Hq, Hkv
    ([1], 1, [1], 1, 1),
    ([1], 0, [1], 8, 2),
    ([1], 129, [0], 8, 2),
    ([1, 1, 1], 0, [0, 5, 0], 4, 4),                      # rows that see nothing
    ([1, 1], 500, [40, 3], 32, 8),
    ([1] * 5, 127, [1, 16, 17, 128, 129], 28, 4),
    ([1, 4, 2, 3], 300, [9, 4, 2, 200], 5, 5),
    ([4, 1, 4], 40, [2, 1, 0], 8, 1),                     # more new tokens than own keys
    ([3, 0, 2], 64, [30, 12, 70], 6, 2),                  # a request without new tokens
    ([40, 1], 200, [40, 90], 16, 2),                      # 320 rows of one request
    ([150], 10, [333], 4, 4),
    ([1] * 70, 333, [1 + 3 * i for i in range(70)], 8, 2),
    ([1] * 3, 4200, [700, 2, 1500], 8, 1),
    ([2] * 20, 1025, [5 + 7 * i for i in range(20)], 16, 1),
    ([1] * 1100, 70, [i % 5 for i in range(1100)], 2, 1),  # more requests than one round of the set-up
    ([1, 0, 3], 200, [1, 0, 64], 128, 1),                 # 128 query heads on one
    ([1, 2], 150, [64, 65], 9, 3),                        # tiles that end exactly, and one key later
]


@pytest.mark.parametrize("dtype,d,page", [("bf16", 128, 16), ("bf16", 64, 128), ("f16", 128, 64), ("f16", 64, 32)])
@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attn(B, case, dtype, d, page):
    news, prefix, lens, Hq, Hkv = ATTN[case]
    b = Batch(case, news, prefix, lens, Hq, Hkv, d, page, dtype, sharp=1.0 + case % 3)
    got = b.run(B)
    b.check(got)
    again = b.run(B)
    for x, y in zip(again, got):
        assert (x == y).all(), "two calls differ"


def test_attn_one_token_each_without_q_start_strided_q_no_own_keys(B):
    import torch
    b = Batch(5, [1] * 6, 700, [0] * 6, 8, 2, 128, 16, "bf16")
    o, lse = b.run(B)
    wide = torch.full((6, 3 * 8 * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 1024:2048] = b.q.view(6, -1)
    q = wide[:, 1024:2048].view(6, 8, 128)
    for got in (B.attn_shared_prefix(q, b.kc, b.vc, b.args[0], 700, None, None),
                B.attn_shared_prefix(q, b.kc, b.vc, b.args[0], 700, None, None, scale=128 ** -0.5)):
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)
    b.check((o, lse))


def test_attn_workspace_header_stays_zero_and_serves_other_calls(B):
    """One zeroed workspace for an attention call, a quantized layer and adapters in turn."""
    import torch
    b = Batch(81, [1, 2], 700, [100, 30], 8, 2, 64, 16, "bf16")
    K, N, M = 512, 256, 3
    pk = int4_g128.quantize(inputs.weights(5, N, K, 0.05))
    d = [torch.from_numpy(np.ascontiguousarray(p)).cuda() for p in pk]
    xb, xf = inputs.activations(6, M, K)
    X = torch.from_numpy(xb.view(np.int16)).cuda().view(torch.bfloat16)
    (a, w, s), _ = _adapter_set(3, 2, 16, K, N, "bf16")
    ad = torch.tensor([1, -1, 0], dtype=torch.int32, device="cuda")
    lib = B.load_library()
    need = max(lib.wq_attn_workspace_bytes(3, 2, 8, 2, 64, 2), lib.wq_gemm_w4a16_lora_workspace_bytes(0, M, K, N, 16),
               lib.wq_lora_workspace_bytes(M, K, N, 16))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(3):
        b.check(b.run(B, workspace=ws))
        y = B.gemm_w4a16("int4_g128", X, *d, workspace=ws)
        got = y, B.lora_add(y, X, a, w, ad, s, workspace=ws), B.gemm_w4a16_lora("int4_g128", X, *d, a, w, ad, s, workspace=ws)
        assert torch.equal(got[1], got[2])
        first = got if first is None else first
        assert all(torch.equal(p, q) for p, q in zip(got, first))
        assert int(ws[:64 * 1024 + 10 * 1024 * 1024].count_nonzero()) == 0


def test_attn_large_scores_and_shifted_scores(B):
    """Scores of several hundred: the running maximum moves often, and the softmax is one-hot."""
    for dtype in ("bf16", "f16"):
        b = Batch(11, [1, 2, 1], 900, [70, 300, 5], 8, 2, 128, 16, dtype, sharp=30.0)
        b.check(b.run(B))
    # scores that grow along the keys, so every tile raises the maximum
    b = Batch(12, [1, 1], 1500, [200, 10], 4, 1, 64, 16, "bf16")
    import torch
    ramp = torch.linspace(0, 3, 1500, device="cuda")
    for j in range(1500):
        b.kc[int(b.prefix_pages[j // 16]), :, j % 16] = ramp[j].to(torch.bfloat16)
    b.q.copy_(b.q.abs())
    b.check(b.run(B))


def test_attn_beyond_32_bit_offsets(B):
    """Pages whose element offsets pass 2^31 (and 2^32 bytes)."""
    import torch
    Hkv, page, d = 8, 64, 128
    pages = (2 ** 31) // (Hkv * page * d) + 40
    kc = torch.empty((pages, Hkv, page, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    ids = [pages - 1, 3, pages - 7, pages - 20]
    small = Batch(21, [1, 1], 100, [60, 64], 16, Hkv, d, page, "bf16")
    order = list(small.prefix_pages) + [small.table[0][0], small.table[1][0]]
    for new, old in zip(ids, order):
        kc[new], vc[new] = small.kc[int(old)], small.vc[int(old)]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    got = B.attn_shared_prefix(small.q, kc, vc, i32(ids[:2]), 100, i32([[ids[2]], [ids[3]]]), i32([60, 64]))
    small.check(got)
    # and the cache write at the far end
    k, kf = _rand(1, (2, Hkv, d), "bf16")
    far = (pages - 1) * page + 63
    B.qk_norm_rope_cache(small.q, k, k, i32([0, 0]), _table(4, 64), kc, vc, i32([far, 5]))
    assert torch.equal(vc[pages - 1, :, 63], k[0]) and torch.equal(vc[0, :, 5], k[1])
    del kc, vc
    torch.cuda.empty_cache()


def test_attn_propagates_nan_of_visible_keys_only(B):
    b = Batch(31, [1, 1], 40, [20, 20], 4, 2, 64, 16, "bf16")
    b.vc[int(b.table[0][0]), 0, 3, 5] = float("nan")
    o, lse = b.run(B)
    bad = np.isnan(_host(o))
    assert bad[0, :2, 5].all() and bad.sum() == 2 and not np.isnan(_host(lse)).any()


def test_attn_reports_indices_out_of_range(B):
    import torch
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    b = Batch(41, [1, 1], 40, [20, 20], 4, 2, 64, 16, "bf16")
    B.attn_shared_prefix(b.q, b.kc, b.vc, i32([0, 1, 10 ** 6]), 40, b.args[2], b.args[3])
    assert B.read_error_flags() == 1 << 7
    B.attn_shared_prefix(b.q, b.kc, b.vc, b.args[0], 40, b.args[2], i32([20, 33]))
    assert B.read_error_flags() == 1 << 7
    for q0 in ([0, 2, 2], [0, 1, 3], [-1, 1, 2], [1, 0, 2]):
        B.attn_shared_prefix(b.q, b.kc, b.vc, b.args[0], 40, b.args[2], b.args[3], q_start=i32(q0))
        assert B.read_error_flags() == 1 << 7, q0
    b.check(b.run(B))


def test_attn_rejects_bad_arguments(B):
    b = Batch(51, [1, 1], 40, [20, 20], 4, 2, 64, 16, "bf16")
    pp, P, bt, sl = b.args
    for bad in (lambda: B.attn_shared_prefix(b.q, b.kc.half(), b.vc, pp, P, bt, sl),
                lambda: B.attn_shared_prefix(b.q, b.kc[:, :, :8].contiguous(), b.vc[:, :, :8].contiguous(), pp, P, bt, sl),
                lambda: B.attn_shared_prefix(b.q, b.kc, b.vc, pp, 49, bt, sl),
                lambda: B.attn_shared_prefix(b.q, b.kc, b.vc, None, P, bt, sl),
                lambda: B.attn_shared_prefix(b.q, b.kc, b.vc, pp, P, bt, None),
                lambda: B.attn_shared_prefix(b.q, b.kc, b.vc, pp, P, bt.long(), sl),
                lambda: B.attn_shared_prefix(b.q, b.kc, b.vc, pp, P, bt[:1], sl),
                lambda: B.attn_shared_prefix(b.q, b.kc, b.vc, pp, P, bt, sl, max_new=2),
                lambda: B.attn_shared_prefix(b.q, b.kc, b.vc, pp, P, bt, sl, scale=0.0),
                lambda: B.attn_shared_prefix(b.q[:, :3], b.kc, b.vc, pp, P, bt, sl),
                lambda: B.attn_shared_prefix(b.q.cpu(), b.kc, b.vc, pp, P, bt, sl)):
        with pytest.raises(ValueError):
            bad()


# -------------------------------------------------------------------------------- adapters
def _adapter_set(seed, L, r, K, N, dtype, ranks=None):
    import torch
    a = torch.randn((L, r, K), generator=torch.Generator().manual_seed(seed)) * K ** -0.5
    b = torch.randn((L, N, r), generator=torch.Generator().manual_seed(seed + 1)) * 0.2
    if ranks is not None:
        for i, n in enumerate(ranks):
            a[i, n:] = 0
            b[i, :, n:] = 0
    a, b = a.to(_dt(dtype)), b.to(_dt(dtype))
    s = 0.25 + torch.rand(L, generator=torch.Generator().manual_seed(seed + 2))
    return (a.cuda(), b.cuda(), s.cuda()), (a.double().numpy(), b.double().numpy(), s.double().numpy())


LORA = [  # M, K, N, r, L, adapters of the rows
    (1, 128, 64, 8, 1, "one"),
    (1, 4096, 4096, 16, 3, "one"),
    (3, 8, 1, 8, 2, "mixed"),
    (5, 136, 33, 24, 4, "mixed"),
    (16, 1024, 512, 16, 16, "each"),
    (17, 512, 257, 64, 5, "mixed"),
    (64, 2048, 1000, 32, 48, "each"),
    (130, 264, 640, 128, 3, "runs"),
    (300, 1024, 384, 64, 7, "runs"),
    (300, 512, 129, 40, 300, "each"),
    (1000, 256, 320, 16, 6, "runs"),
    (513, 640, 250, 8, 4, "mixed"),
    (40, 128, 64, 16, 2, "none"),
    (1500, 256, 200, 64, 5, "runs"),
    (2100, 136, 72, 96, 9, "mixed"),
    (1025, 2048, 64, 8, 1, "one"),
    (1100, 512, 41, 128, 40, "each"),
    (1300, 512, 104, 128, 40, "each"),
    (700, 256, 200, 24, 64, "runs"),
    (16500, 64, 72, 8, 600, "each"),
    (600, 1024, 328, 40, 2, "runs"),
]


def _who(kind, M, L, seed):
    rng = np.random.default_rng(seed)
    if kind == "one":
        return np.full(M, L - 1, np.int32)
    if kind == "none":
        return np.full(M, -1, np.int32)
    if kind == "each":
        return (rng.permutation(M) % L).astype(np.int32)
    if kind == "mixed":
        return rng.integers(-1, L, M).astype(np.int32)
    cuts = np.sort(rng.choice(M, min(M - 1, 2 * L), replace=False))
    return np.repeat(rng.integers(-1, L, len(cuts) + 1), np.diff(np.concatenate(([0], cuts, [M])))).astype(np.int32)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", range(len(LORA)))
def test_lora_add(B, case, dtype):
    import torch
    M, K, N, r, L, kind = LORA[case]
    ranks = [max(1, r - 5 * (i % 3)) for i in range(L)]
    (a, b, s), (af, bf, sf) = _adapter_set(case, L, r, K, N, dtype, ranks)
    x, xf = _rand(case + 50, (M, K), dtype)
    base, basef = _rand(case + 60, (M, N), dtype)
    who = _who(kind, M, L, case)
    ad = torch.from_numpy(who).cuda()
    rk = torch.tensor(ranks, dtype=torch.int32, device="cuda")
    y = B.lora_add(base, x, a, b, ad, s, ranks=rk)
    delta, dabs = ab.adapters(xf, af, bf, who, sf)
    ref, u = basef + delta, U[dtype]
    _within(_host(y), ref, u * np.abs(ref) + (u + 1e-5) * dabs, "Y")
    assert np.array_equal(_host(y)[who < 0], basef[who < 0])
    assert torch.equal(y, B.lora_add(base, x, a, b, ad, s))                 # zeros past the ranks
    assert torch.equal(y, B.lora_add(base, x, a, b, ad, s, ranks=rk))       # two calls agree
    assert torch.equal(y, B.lora_add(base, x, a, b, ad, s, ranks=rk, out=base))   # in place


def test_lora_reports_indices_out_of_range(B):
    import torch
    (a, b, s), _ = _adapter_set(1, 2, 16, 256, 96, "bf16")
    x, _ = _rand(1, (4, 256), "bf16")
    base, _ = _rand(2, (4, 96), "bf16")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    good = B.lora_add(base, x, a, b, i32(0, 1, 0, 1), s)
    y = B.lora_add(base, x, a, b, i32(0, 2, -2, 1), s)
    assert B.read_error_flags() == 1 << 7
    assert torch.equal(y[0], good[0]) and torch.equal(y[3], good[3])
    B.lora_add(base, x, a, b, i32(0, 1, 0, 1), s, ranks=i32(17, -1))
    assert B.read_error_flags() == 1 << 7


def test_lora_rejects_bad_arguments(B):
    import torch
    (a, b, s), _ = _adapter_set(1, 2, 16, 256, 96, "bf16")
    x, _ = _rand(1, (4, 256), "bf16")
    base, _ = _rand(2, (4, 96), "bf16")
    ad = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: B.lora_add(base.half(), x, a, b, ad, s), lambda: B.lora_add(base, x, a, b, ad.long(), s),
                lambda: B.lora_add(base[:, :95], x, a, b, ad, s), lambda: B.lora_add(base, x, a[:, :12].contiguous(), b[:, :, :12].contiguous(), ad, s),
                lambda: B.lora_add(base, x[:, ::2], a, b, ad, s), lambda: B.lora_add(base, x, a, b, ad[:3], s),
                lambda: B.lora_add(base, x, a, b, ad, s[:1]), lambda: B.lora_add(base, x, a, b, ad, s, ranks=ad),
                lambda: B.lora_add(base.cpu(), x, a, b, ad, s),
                lambda: B.lora_add(base, x, a, b, ad, s, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("fmt", ["int4_g128", "mxfp4"])
@pytest.mark.parametrize("M", [1, 5, 16, 40, 100, 300])
def test_quantized_layer_with_adapters(B, fmt, M):
    import torch
    K, N, r, L = 512, 384, 16, 4
    W = inputs.weights(9, N, K, 0.05)
    pk = int4_g128.quantize(W) if fmt == "int4_g128" else mxfp4.quantize(W)
    d = [torch.from_numpy(np.ascontiguousarray(p)).cuda() for p in pk]
    xb, xf = inputs.activations(M, M, K)
    X = torch.from_numpy(xb.view(np.int16)).cuda().view(torch.bfloat16)
    (a, b, s), (af, bf, sf) = _adapter_set(M, L, r, K, N, "bf16")
    who = _who("mixed", M, L, M)
    y = B.gemm_w4a16_lora(fmt, X, d[0], d[1], d[2] if fmt == "int4_g128" else None, a, b, torch.from_numpy(who).cuda(), s)
    base = linear.linear_w4a16(fmt, xf, *pk)
    delta, dabs = ab.adapters(xf, af, bf, who, sf)
    u = U["bf16"]
    ref = base + delta
    _within(_host(y), ref, TOL * (1 + np.abs(base)) + u * (np.abs(ref) + np.abs(base)) + (u + 1e-5) * dabs, fmt)
    plain = B.gemm_w4a16(fmt, X, *d)
    assert torch.equal(y[torch.from_numpy(who < 0).cuda()], plain[torch.from_numpy(who < 0).cuda()])
    assert torch.equal(plain, B.gemm_w4a16(fmt, X, *d))     # the shared workspace's header is left at zero


@pytest.mark.parametrize("M,r,L", [(1, 8, 1), (19, 16, 5), (64, 64, 9), (130, 104, 3), (700, 40, 6), (1300, 104, 40), (640, 64, 2)])
def test_adapters_beside_a_quantized_layer_add_no_rounding_of_their_own(B, M, r, L):
    """Given the layer's output, which is rounded to bf16, the sum is rounded once: V's own rounding is
    carried along (it is left with u^2 of V, and float32 sums)."""
    import torch
    K, N = 512, 264
    W = inputs.weights(11, N, K, 0.05)
    d = [torch.from_numpy(np.ascontiguousarray(p)).cuda() for p in int4_g128.quantize(W)]
    xb, xf = inputs.activations(M, M, K)
    X = torch.from_numpy(xb.view(np.int16)).cuda().view(torch.bfloat16)
    (a, b, s), (af, bf, sf) = _adapter_set(M, L, r, K, N, "bf16")
    who = _who("mixed", M, L, M + 1)
    y = B.gemm_w4a16_lora("int4_g128", X, *d, a, b, torch.from_numpy(who).cuda(), s)
    base = _host(B.gemm_w4a16("int4_g128", X, *d))
    delta, dabs = ab.adapters(xf, af, bf, who, sf)
    ref, u = base + delta, U["bf16"]
    _within(_host(y), ref, u * np.abs(ref) + (u * u + 1e-5) * dabs, "Y")


# ------------------------------------------------------------------------- streams together
def test_on_a_side_stream(B):
    """Every call on a stream that is not the current one, inputs made there just before."""
    import torch
    b = Batch(61, [1, 2, 1], 600, [30, 40, 1], 8, 2, 64, 32, "bf16")
    here = b.run(B)
    (a, w, s), _ = _adapter_set(3, 2, 16, 256, 96, "bf16")
    x, _ = _rand(1, (4, 256), "bf16")
    base, _ = _rand(2, (4, 96), "bf16")
    ad = torch.zeros(4, dtype=torch.int32, device="cuda")
    y = B.lora_add(base, x, a, w, ad, s)
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    qk = B.qk_norm_rope(b.q, b.q, pos, _table(4, 64))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2000000)
        x2, q2 = x.clone(), b.q.clone()
    y2 = B.lora_add(base, x2, a, w, ad, s, stream=side)
    qk2 = B.qk_norm_rope(q2, q2, pos, _table(4, 64), stream=side)
    b.q = q2
    there = b.run(B, stream=side)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(here[0], there[0]) and torch.equal(here[1], there[1])
    assert torch.equal(qk[0], qk2[0]) and torch.equal(qk[1], qk2[1])


def test_calls_are_captured_in_a_graph(B):
    import torch
    b = Batch(71, [1] * 4, 300, [10, 20, 30, 40], 8, 2, 128, 16, "bf16")
    (a, w, s), _ = _adapter_set(3, 2, 16, 1024, 96, "bf16")
    base, _ = _rand(2, (4, 96), "bf16")
    ad = torch.tensor([0, 1, -1, 0], dtype=torch.int32, device="cuda")
    want = b.run(B)[0].clone()
    y = B.lora_add(base, want.view(4, -1), a, w, ad, s).clone()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        o, _ = b.run(B)
        B.lora_add(base, o.view(4, -1), a, w, ad, s)
    stream.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        o, _ = b.run(B)
        y2 = B.lora_add(base, o.view(4, -1), a, w, ad, s)
    o.zero_()
    y2.zero_()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(y2, y)


def test_the_three_together_as_one_block(B):
    """The example: a shared prompt prefilled, then requests with adapters decoding behind it."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "shared_prefix_block.py")
    spec = importlib.util.spec_from_file_location("shared_prefix_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.main() < 0.02


# --------------------------------------------------- what a call must not reach, drop or keep
def test_attn_requests_that_overlap_compute_nothing(B):
    """q_start that goes back and forth: each request by itself is in range, but together they have more
    tokens, and more partials, than the workspace is counted for (550 slots of own keys where it has 312).
    Nothing is computed: outputs and the bytes past the workspace's size keep what they held."""
    import torch
    T, R, Hq, Hkv, d = 640, 10, 32, 8, 64
    b = Batch(101, [T // R] * R, 70, [T] * R, Hq, Hkv, d, 16, "bf16")
    need = B.load_library().wq_attn_workspace_bytes(T, R, Hq, Hkv, d, T)
    ws = torch.zeros(3 * need, dtype=torch.uint8, device="cuda")
    ws[need:] = 0xA5
    o, lse = torch.full((T, Hq, d), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((T, Hq), 3.0, device="cuda")
    kw = dict(max_new=T, out=(o, lse), workspace=ws)
    for q0 in ([0, T] * (R // 2) + [T], [0] + [T, 0] * ((R - 1) // 2) + [0, T], [0, T, T - 1] + [T] * (R - 2)):
        b.run(B, q_start=torch.tensor(q0, dtype=torch.int32, device="cuda"), **kw)
        assert B.read_error_flags() == 1 << 7, q0
        assert (ws[need:] == 0xA5).all() and (o == 3).all() and (lse == 3).all(), q0
    want = b.run(B)
    got = b.run(B, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and (ws[need:] == 0xA5).all()


def test_a_captured_graph_keeps_the_workspace_it_was_captured_with(B):
    """Capture a small batch, then run a larger one on the same stream, which needs more workspace, and fill
    what the allocator hands out next: the graph's replay gives the same outputs and touches none of it."""
    import torch
    small, large = (Batch(111 + n, [1] * n, 300, [10 + i for i in range(n)], 8, 2, 128, 16, "bf16") for n in (2, 64))
    (a, w, s), _ = _adapter_set(3, 2, 16, 1024, 96, "bf16")
    stream = torch.cuda.Stream()

    def step(b):
        n = b.q.shape[0]
        o, lse = b.run(B)
        ad = torch.arange(n, dtype=torch.int32, device="cuda") % 3 - 1
        return o, lse, B.lora_add(torch.ones(n, 96, dtype=torch.bfloat16, device="cuda"), o.view(n, -1), a, w, ad, s)

    lib = B.load_library()
    sizes = [lib.wq_attn_workspace_bytes(2, 2, 8, 2, 128, 1), lib.wq_lora_workspace_bytes(2, 1024, 96, 16)]
    with torch.cuda.stream(stream):
        want = [x.clone() for x in step(small)]
    stream.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        got = step(small)
    with torch.cuda.stream(stream):
        step(large)
        others = [torch.full(((n + 255) // 256 * 256,), 0xA5, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    stream.synchronize()
    for x in got:
        x.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    assert all((t == 0xA5).all() for t in others)
    with torch.cuda.stream(stream):                       # and the larger workspace serves the smaller call
        again = step(small)
    stream.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(again, want))


@pytest.mark.parametrize("dtype,d,requests", [("bf16", 128, 3), ("f16", 64, 3), ("bf16", 64, 340), ("f16", 128, 340)])
@pytest.mark.parametrize("where", ["query", "only own key", "only own key, no prefix", "a run of keys", "beside a far lower score"])
def test_attn_nan_scores_reach_every_row_that_sees_them(B, where, dtype, d, requests):
    """A NaN score makes its rows NaN, lse too, however the line of keys is cut; all other rows keep their bits."""
    import torch
    lens = {"query": [40, 700, 3], "a run of keys": [9000, 64, 5], "beside a far lower score": [20, 2, 30]}.get(where, [20, 1, 30])
    prefix = 0 if where.endswith("no prefix") else 500
    Hq, Hkv = (8, 2) if requests == 3 else (32, 8)       # many rows are joined by other kernels than few
    b = Batch(91, [1] * requests, prefix, lens + [1] * (requests - 3), Hq, Hkv, d, 16, dtype)
    if where == "beside a far lower score":
        b.q[1, :4] = 8.0
        b.kc[int(b.table[1][0]), 0, 1] = -64.0
    clean = [x.clone() for x in b.run(B)]
    if requests == 3:
        b.check(clean)
    if where == "query":
        b.q[1, 2, 5] = float("nan")
        rows = [(1, 2)]
    elif where == "a run of keys":
        for j in range(640, 1280):
            b.kc[int(b.table[0][j // 16]), 1, j % 16] = float("nan")
        rows = [(0, h) for h in range(4, 8)]
    else:
        b.kc[int(b.table[1][0]), 0, 0] = float("nan")
        rows = [(1, h) for h in range(4)]
    o, lse = b.run(B)
    hit = torch.zeros(requests, Hq, dtype=torch.bool, device="cuda")
    for t, h in rows:
        hit[t, h] = True
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(o[~hit], clean[0][~hit]) and torch.equal(lse[~hit], clean[1][~hit])


@pytest.mark.parametrize("dtype,d,requests", [("bf16", 128, 3), ("f16", 64, 340)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_attn_nan_and_infinite_values_of_far_lower_scores(B, value, dtype, d, requests):
    """A value that is NaN or infinite reaches its rows also where its weight is too small for float32 (0 times
    it is NaN), in a segment of its own as in one with other keys."""
    import torch
    Hq, Hkv = (8, 2) if requests == 3 else (32, 8)
    b = Batch(95, [1] * requests, 500, [20, 1, 30] + [1] * (requests - 3), Hq, Hkv, d, 16, dtype)
    page = int(b.table[1][0])
    b.q[1, :4] = 8.0
    b.kc[page, 0, 0] = -64.0                   # score -4096 and below
    clean = [x.clone() for x in b.run(B)]
    b.vc[page, 0, 0, 7] = value
    o, lse = b.run(B)
    hit = torch.zeros(requests, Hq, d, dtype=torch.bool, device="cuda")
    hit[1, :4, 7] = True
    assert not torch.isfinite(o[hit]).any()
    assert torch.equal(o[~hit], clean[0][~hit]) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,N,r,L,kind", [(5, 128, 64, 8, 3, "mixed"), (16, 512, 256, 16, 16, "each"), (64, 256, 96, 40, 48, "each"),
                                            (40, 128, 33, 72, 20, "each"), (200, 128, 9001, 16, 5, "mixed"),
                                            (300, 128, 8200, 40, 4, "runs"), (1100, 1024, 72, 64, 6, "mixed")])
def test_lora_one_adapters_infinities_stay_its_own(B, M, K, N, r, L, kind, dtype):
    import torch
    (a, b, s), _ = _adapter_set(M, L, r, K, N, dtype)
    x, _ = _rand(M + 50, (M, K), dtype)
    base, _ = _rand(M + 60, (M, N), dtype)
    who = _who(kind, M, L, M)
    who[M // 2] = 1
    ad = torch.from_numpy(who).cuda()
    good = B.lora_add(base, x, a, b, ad, s)
    b[1, 3, 2], b[1, 5, 1], b[1, N - 1, r - 1] = float("inf"), float("nan"), float("-inf")
    y = B.lora_add(base, x, a, b, ad, s)
    mine = ad == 1
    assert torch.equal(y[~mine], good[~mine])
    broken = [3, 5, N - 1]
    assert not torch.isfinite(y[mine][:, broken]).any()
    rest = [n for n in range(N) if n not in broken]
    assert torch.equal(y[mine][:, rest], good[mine][:, rest])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,rank", [(4, 64, 8), (4, 64, 5), (700, 2048, 13)])
def test_lora_infinite_inner_products(B, M, K, rank, dtype):
    """An infinity in X gives an infinite sum where the definition does, not NaN: neither from what an infinite
    value's rounding leaves, nor from the zeros past an adapter's rank."""
    import torch
    r = (rank + 7) // 8 * 8
    (a, b, s), _ = _adapter_set(7, 2, r, K, 48, dtype)
    a[:, :, 0], b = 0.5, b.abs() + 0.01
    a[:, rank:], b[:, :, rank:] = 0, 0
    x, _ = _rand(8, (M, K), dtype)
    x[2, 0] = float("inf")
    base, _ = _rand(9, (M, 48), dtype)
    ad = torch.ones(M, dtype=torch.int32, device="cuda")
    ad[0], ad[1] = 0, -1
    y = B.lora_add(base, x, a, b, ad, s, ranks=torch.tensor([rank, rank], dtype=torch.int32, device="cuda"))
    assert (y[2] == float("inf")).all() and torch.isfinite(y[torch.arange(M) != 2]).all()


@pytest.mark.parametrize("M,K,N,r,L,kind", [(3, 256, 64, 8, 2, "mixed"), (16, 512, 256, 16, 16, "each"), (40, 512, 33, 72, 3, "mixed"),
                                            (130, 264, 640, 128, 3, "runs"), (700, 256, 200, 24, 6, "runs"),
                                            (1100, 1024, 328, 64, 7, "runs"), (1100, 1024, 41, 96, 7, "runs"),
                                            (1300, 1032, 104, 128, 9, "runs")])
def test_lora_f16_inner_products_beyond_the_type(B, M, K, N, r, L, kind):
    """s X A^T from some 10^2 to 10^7, by row and by half of the ranks, with B small: the result is ordinary."""
    import torch
    a = torch.randn((L, r, K), generator=torch.Generator().manual_seed(M)) * K ** -0.5
    a[:, :r // 2] *= torch.tensor([1.0, 200.0, 0.01])[torch.arange(L) % 3][:, None, None]
    b = torch.randn((L, N, r), generator=torch.Generator().manual_seed(M + 1)) * 2e-4
    a, b = a.half(), b.half()
    s = 0.25 + torch.rand(L, generator=torch.Generator().manual_seed(M + 2))
    x = (torch.randn((M, K), generator=torch.Generator().manual_seed(M + 3))
         * torch.tensor([1.0, 3e3, 1.2e4, 30.0])[torch.arange(M) % 4][:, None]).half()
    base, basef = _rand(M + 60, (M, N), "f16")
    who = _who(kind, M, L, M)
    y = B.lora_add(base, x.cuda(), a.cuda(), b.cuda(), torch.from_numpy(who).cuda(), s.cuda())
    delta, dabs = ab.adapters(x.double().numpy(), a.double().numpy(), b.double().numpy(), who, s.double().numpy())
    ref, u = basef + delta, U["f16"]
    assert np.abs(ref).max() < 60000
    _within(_host(y), ref, u * np.abs(ref) + (u + 1e-5) * dabs, "Y")


def test_rope_positions_and_slots_need_their_own_alignment_only(B):
    import torch
    q, _ = _rand(1, (5, 2, 64), "bf16")
    k, _ = _rand(2, (5, 1, 64), "bf16")
    kc, vc = torch.zeros(2, 2, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    kc2, vc2 = torch.zeros(2, 2, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    tab = _table(16, 64)
    pos = torch.tensor([9, 3, 5, 1, 0, 7], dtype=torch.int32, device="cuda")
    slots = torch.tensor([0, 0, 0, 17, 4, 31, -1, 2], dtype=torch.int32, device="cuda")
    want = B.qk_norm_rope(q, k, pos[1:].clone(), tab)
    got = B.qk_norm_rope(q, k, pos[1:], tab)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    want = B.qk_norm_rope_cache(q, k, k, pos[1:].clone(), tab, kc, vc, slots[3:].clone())
    got = B.qk_norm_rope_cache(q, k, k, pos[1:], tab, kc2, vc2, slots[3:])
    assert torch.equal(got, want) and torch.equal(kc2, kc) and torch.equal(vc2, vc)


def test_rope_refuses_a_pairing_that_is_no_truth_value(B):
    import torch
    q, _ = _rand(1, (3, 2, 64), "bf16")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        B.qk_norm_rope(q, q, pos, _table(8, 64), interleaved=np.array([True, False]))


# ------------------------------------------------- the many-row adapter kernels, by their names
def _kernels(f):
    """The adapter kernels that a call launches (the call, once more, captured in a graph)."""
    import torch
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        f()
    g = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(g, stream=stream):
        f()
    torch.cuda.synchronize()
    return [n for n in ("k_lora_shrink_tile", "k_lora_shrink_rows", "k_lora_expand_tile", "k_lora_expand")
            if any(n + "I" in k for k in kernels_of(g))]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,N,r,L,kind", [(1100, 1096, 328, 64, 7, "runs"), (2100, 1032, 72, 96, 9, "mixed"),
                                            (1300, 2048, 104, 128, 40, "each"), (1025, 1032, 48, 24, 3, "runs"),
                                            (4100, 520, 264, 40, 5, "runs"), (1100, 1024, 41, 104, 6, "mixed")])
def test_lora_many_rows_on_the_tensor_cores(B, M, K, N, r, L, kind, dtype):
    """Ranks beyond 64 (two parts of the grid), K that ends inside a step, several adapters a tile, several CTAs a
    cluster, ranks of their own: each on the kernels for many rows, whatever their rules become."""
    import torch
    ranks = [max(1, r - 5 * (i % 3)) for i in range(L)]
    (a, b, s), (af, bf, sf) = _adapter_set(M, L, r, K, N, dtype, ranks)
    x, xf = _rand(M + 50, (M, K), dtype)
    base, basef = _rand(M + 60, (M, N), dtype)
    who = _who(kind, M, L, M)
    ad, rk = torch.from_numpy(who).cuda(), torch.tensor(ranks, dtype=torch.int32, device="cuda")
    call = lambda: B.lora_add(base, x, a, b, ad, s, ranks=rk)
    assert _kernels(call) == ["k_lora_shrink_tile", "k_lora_expand_tile" if N % 8 == 0 else "k_lora_expand"]
    y = call()
    delta, dabs = ab.adapters(xf, af, bf, who, sf)
    ref, u = basef + delta, U[dtype]
    _within(_host(y), ref, u * np.abs(ref) + (u + 1e-5) * dabs, "Y")
    assert np.array_equal(_host(y)[who < 0], basef[who < 0])
    assert torch.equal(y, B.lora_add(base, x, a, b, ad, s)) and torch.equal(y, call())
    assert torch.equal(y, B.lora_add(base, x, a, b, ad, s, ranks=rk, out=base))


@pytest.mark.parametrize("fmt", ["int4_g128", "mxfp4"])
@pytest.mark.parametrize("M,K,N,r,L", [(1300, 1024, 264, 104, 5), (2100, 512, 136, 24, 3)])
def test_adapters_beside_a_quantized_layer_on_the_tensor_cores(B, fmt, M, K, N, r, L):
    """V in two parts through the kernels for many rows: the sum of the layer's output and the adapters' product
    is rounded once."""
    import torch
    W = inputs.weights(13, N, K, 0.05)
    pk = int4_g128.quantize(W) if fmt == "int4_g128" else mxfp4.quantize(W)
    d = [torch.from_numpy(np.ascontiguousarray(p)).cuda() for p in pk] + [None] * (3 - len(pk))
    xb, xf = inputs.activations(M, M, K)
    X = torch.from_numpy(xb.view(np.int16)).cuda().view(torch.bfloat16)
    (a, b, s), (af, bf, sf) = _adapter_set(M, L, r, K, N, "bf16")
    who = _who("runs", M, L, M + 1)
    ad = torch.from_numpy(who).cuda()
    call = lambda: B.gemm_w4a16_lora(fmt, X, *d, a, b, ad, s)
    assert _kernels(call) == ["k_lora_shrink_tile", "k_lora_expand_tile"]
    y = call()
    base = _host(B.gemm_w4a16(fmt, X, *d))
    delta, dabs = ab.adapters(xf, af, bf, who, sf)
    ref, u = base + delta, U["bf16"]
    _within(_host(y), ref, u * np.abs(ref) + (u * u + 1e-5) * dabs, "Y")
    assert torch.equal(y, call())


# --------------------------------------------------------------------- prompts through attention
@pytest.mark.parametrize("dtype,d,page", [("bf16", 128, 16), ("f16", 64, 128)])
@pytest.mark.parametrize("news,prefix,lens,Hq,Hkv", [([700], 0, [700], 8, 2), ([300, 1, 129], 200, [420, 5, 129], 4, 1),
                                                     ([513], 65, [513], 6, 2)])
def test_attn_prompts_of_several_row_tiles(B, dtype, d, page, news, prefix, lens, Hq, Hkv):
    """Requests whose new tokens fill several row tiles (of 64 tokens here and more), causal across them."""
    b = Batch(121, news, prefix, lens, Hq, Hkv, d, page, dtype)
    got = b.run(B)
    b.check(got)
    again = b.run(B)
    assert (again[0] == got[0]).all() and (again[1] == got[1]).all()

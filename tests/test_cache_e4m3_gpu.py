"""The 8-bit cache on the GPU against the float64 oracle: tokens quantized into pages, read back, and
attention over the pages.

Tolerances.  Codes, scales and what is read back in bf16 are exact; fp16 reads are rounded once.
Attention (u is half a unit in the last place of the output type, 2^-8 bf16, 2^-11 fp16): the output's
one rounding, u |ref|; the weights, rounded to fp16 for the second product (2^-11 each) and with the
error eps of their scores; the tensor core's float32 sums, n / 16 additions of at most 2^-22 each of sum
p |v|.  A score is off by d / 16 + 1 additions of 2^-22 of scale sum |q| |k| (`reach`), the float32 product
with the scale (2^-23 of it, and of the exponent that is added), and 2^-22 for the exponential, so eps =
2^-22 (10 reach + 64) log2(e); it enters numerator and sum.  Weights below 2^-31 of the largest lose
up to 2^-32 of it each: n 2^-32 of the largest |v|."""
import numpy as np
import pytest

from oracle import cache_e4m3 as c8

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


def i32(v):
    import torch
    return torch.tensor(np.asarray(v), dtype=torch.int32).cuda()


def _host(t):
    return t.detach().double().cpu().numpy()


class Cache:
    """A cache and its requests: the same arrays on the GPU and for the oracle."""

    def __init__(self, seed, lens, Hkv, d, page, spare=3, spread=0.0):
        import torch
        self.rng = np.random.default_rng(seed)
        self.Hkv, self.d, self.page = Hkv, d, page
        blocks = [-(-n // page) for n in lens]
        pages = sum(blocks) + spare
        perm = self.rng.permutation(pages)
        self.table = np.full((len(lens), max(blocks + [1])), -1, np.int32)
        at = 0
        for r, b in enumerate(blocks):
            self.table[r, :b] = perm[at:at + b]
            at += b
        self.host = [self.rng.integers(0, 256, (pages, Hkv, page, d)).astype(np.uint8) for _ in range(2)]   # NaN codes too
        self.host += [self.rng.integers(63, 192, (pages, Hkv)).astype(np.uint8) for _ in range(2)]
        self.dev = [torch.from_numpy(a.copy()).cuda() for a in self.host]
        self.spread = spread

    def new(self, seed, T, dtype, scale=1.0):
        """K, V [T, Hkv, d] as parts of one projection output: device tensors and float64."""
        import torch
        g = torch.Generator().manual_seed(seed)
        x = torch.randn(T, 2 * self.Hkv + 1, self.d, generator=g) * scale
        x = x * torch.exp(self.spread * torch.randn(T, 2 * self.Hkv + 1, 1, generator=g))
        x = x.to(_dt(dtype))
        dev = x.cuda()
        k, v = slice(0, self.Hkv), slice(self.Hkv, 2 * self.Hkv)
        return (dev[:, k], dev[:, v]), (x[:, k].double().numpy(), x[:, v].double().numpy())

    def append(self, B, kv, lens, news, q_start=True, pad=0, **kw):
        starts = np.concatenate(([0], np.cumsum(news)))
        B.kv_append_e4m3(*kv[0], *self.dev, i32(self.table), i32(lens), i32(starts) if q_start else None,
                         max(1, max(news)) if q_start else 1, **kw)
        c8.append(*kv[1], *self.host, self.table, lens, starts)

    def fill(self, B, lens, dtype="bf16", scale=1.0, seed=7):
        """Whole prompts at once."""
        self.append(B, self.new(seed, max(1, sum(lens)), dtype, scale), lens, list(lens))
        return self

    def check(self):
        import torch
        torch.cuda.synchronize()
        for got, want in zip(self.dev[2:], self.host[2:]):
            assert np.array_equal(got.cpu().numpy(), want)
        for got, want in zip(self.dev[:2], self.host[:2]):
            got = got.cpu().numpy()
            same = (got == want) | (((got & 127) == 127) & ((want & 127) == 127))
            assert same.all(), "%d codes differ, first at %s" % ((~same).sum(), np.argwhere(~same)[0])


# ------------------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hkv,d,page", [(1, 64, 16), (3, 128, 16), (2, 128, 64), (5, 64, 128), (8, 128, 128), (2, 64, 32)])
@pytest.mark.parametrize("spread", [0.0, 1.5])
def test_append_in_calls_of_all_sizes(B, dtype, Hkv, d, page, spread):
    """Prompts, then single tokens, then drafted ones, requests of unequal progress among them."""
    longest = [300, 1, 17, 129, 64, 2]
    c = Cache(1, longest, Hkv, d, page, spread=spread)
    lens = [0] * 6
    plan = [[200, 1, 5, 0, 63, 0], [1, 0, 1, 100, 1, 1], [1, 0, 1, 1, 0, 1], [7, 0, 3, 2, 0, 0], [90, 0, 7, 26, 0, 0], [1, 0, 0, 0, 0, 0]]
    for step, news in enumerate(plan):
        lens = [a + b for a, b in zip(lens, news)]
        c.append(B, c.new(step, sum(news), dtype, 3.0 ** step), lens, news)
        c.check()
    assert lens == longest


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_append_many_requests_one_token_each(B, dtype):
    lens = [int(n) for n in np.random.default_rng(3).integers(1, 200, 700)]
    c = Cache(4, lens, 2, 128, 16, spread=1.0)
    c.append(B, c.new(1, 700, dtype), lens, [1] * 700, q_start=False)
    c.check()
    c.append(B, c.new(2, 700, dtype, 50.0), lens, [1] * 700, q_start=False)         # the same places again: scales grow
    c.check()


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64), (64, 128)])
@pytest.mark.parametrize("most", [2, 16, 17, 18, 65, 130, 131])
def test_append_up_to_a_number_of_tokens(B, d, page, most):
    """One, two and more pages a request; requests with fewer than the most, none, or all of their tokens new."""
    lens = [most, 5 * page, 3 * page + 1, most + page - 1, 1, 2 * page, most + 1]
    c = Cache(12, lens, 3, d, page, spread=1.0).fill(B, [max(0, n - most) for n in lens])
    news = [most, most, most, most, 1, 0, max(1, most - 1)]
    news = [min(a, b) for a, b in zip(news, lens)]
    c.append(B, c.new(2, sum(news), "bf16", 4.0), lens, news)
    c.check()


@pytest.mark.parametrize("page,d", [(16, 128), (64, 64), (128, 128)])
def test_append_extreme_values(B, page, d):
    c = Cache(5, [page + 9], 2, d, page)
    (k, v), _ = c.new(1, page + 9, "bf16")
    k, v = k.contiguous(), v.contiguous()
    k[3, 0, 5], k[4, 1, 0], k[5, 0, 1] = float("nan"), float("inf"), -float("inf")
    k[page + 1] = float("nan")                                                       # one token of the second page ...
    v[:, 0] = 0
    v[:, 1] *= 1e30                                                                  # beyond the largest scale: saturates
    v[page:, 1] = 1e-30
    v[page + 2, 0] = 2.0 ** -126
    kv = (k, v), (_host(k), _host(v))
    c.append(B, kv, [page + 9], [page + 9])
    c.check()
    k2, v2 = k[:1] * 0 + 1, v[:1] * 0 - 1e38                                          # ... then another that lets scales grow far
    c.append(B, ((k2, v2), (_host(k2), _host(v2))), [page + 9], [1])
    c.check()


def test_append_scale_limits_and_ties(B):
    """Values on both sides of a step of the scale and of the codes, all bf16 patterns of a few binades."""
    import torch
    bits = torch.arange(0, 1 << 15, dtype=torch.int32)
    x = bits.to(torch.int16).view(torch.bfloat16)
    x = x[torch.isfinite(x.float())]
    x = torch.cat((x, -x))[: (2 * x.numel()) // 128 * 128].view(-1, 1, 128)
    T = x.shape[0]
    c = Cache(6, [16] * T, 1, 128, 16, spare=1)
    kv = (x.cuda(), x.flip(2).contiguous().cuda()), (x.double().numpy(), x.flip(2).double().numpy())
    c.append(B, kv, [1] * T, [1] * T, q_start=False)
    c.check()
    c.append(B, kv, [2] * T, [1] * T, q_start=False)
    c.check()


def test_append_leaves_padding_rows_and_requests_alone(B):
    c = Cache(7, [40, 33, 16], 2, 64, 16)
    kv = c.new(1, 64, "bf16")
    # 40 + 2 rows of two requests, an empty one, and rows behind them that belong to nobody
    starts = [0, 40, 42, 42]
    B.kv_append_e4m3(*kv[0], *c.dev, i32(c.table), i32([40, 33, 5]), i32(starts), 64)
    c8.append(*kv[1], *c.host, c.table, [40, 33, 5], starts)
    c.check()
    # one token a request; length 0: a row that pads the batch
    kv = c.new(2, 3, "bf16")
    B.kv_append_e4m3(*kv[0], *c.dev, i32(c.table), i32([39, 0, 16]), None, 1)
    c8.append(kv[1][0][[0, 2]], kv[1][1][[0, 2]], *c.host, c.table[[0, 2]], [39, 16], [0, 1, 2])
    c.check()


def test_append_reports_indices_out_of_range(B):
    c = Cache(8, [40, 33], 2, 64, 16)
    kv = c.new(1, 10, "bf16")
    bad_table = c.table.copy()
    bad_table[0, 2] = 99
    for table, lens, starts, most in ((c.table, [40, 33], [0, 5, 11], 8), (c.table, [40, 33], [-1, 5, 10], 8), (c.table, [40, 33], [0, 9, 5], 9),
                                      (c.table, [40, 49], [0, 0, 5], 8), (c.table, [40, -2], [0, 0, 5], 8), (c.table, [40, 3], [0, 0, 5], 8),
                                      (c.table, [40, 33], [0, 0, 5], 4), (bad_table, [40, 33], [0, 3, 3], 8), (bad_table, [40, 0], [0, 3, 3], 8)):
        B.kv_append_e4m3(*kv[0], *c.dev, i32(table), i32(lens), i32(starts), most)
        assert B.read_error_flags() == 1 << 7, (lens, starts)
    # rows 0 .. 4 of the first two belonged to a request in order; what is not a request's is as it was
    free = [p for p in range(c.host[0].shape[0]) if p not in c.table[:, :3]]
    for a, b in zip(c.dev, c.host):
        assert np.array_equal(a.cpu().numpy()[free], b[free])


# ------------------------------------------------------------------------------- reading back
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hkv,d,page", [(1, 64, 16), (3, 128, 32), (8, 128, 64), (5, 64, 128)])
def test_read(B, dtype, Hkv, d, page):
    import torch
    lens = [1, 130, 0, 64, 17]
    c = Cache(9, lens, Hkv, d, page, spread=2.0).fill(B, lens, "bf16", 5.0)
    take = [1, 77, 0, 64, 16]
    starts = np.concatenate(([0], np.cumsum(take)))
    T = int(starts[-1]) + 5
    out = [torch.full((T, Hkv, d), 7.0, dtype=_dt(dtype), device="cuda") for _ in range(2)]
    got = B.kv_read_e4m3(*c.dev, i32(c.table), i32(starts), T, dtype=_dt(dtype), out=out)
    for i in (0, 1):
        assert got[i] is out[i]
        want = np.concatenate([c8.tokens(c.host[i], c.host[i + 2], c.table[r], n) for r, n in enumerate(take)] + [np.full((5, Hkv, d), 7.0)])
        want = torch.from_numpy(want).clamp(-65504.0, 65504.0) if dtype == "f16" else torch.from_numpy(want)
        assert torch.equal(got[i].cpu(), want.to(_dt(dtype)))


@pytest.mark.parametrize("Hkv,d,page,lens", [(1, 128, 16, [700, 2, 0, 301]), (3, 64, 32, [999, 46]), (8, 128, 64, [9001, 1, 2047]),
                                             (40, 128, 16, [1500, 0, 723])])
def test_read_calls_of_all_sizes(B, Hkv, d, page, lens):
    import torch
    c = Cache(11, lens, Hkv, d, page)
    for i in (2, 3):                               # scales of a prompt's pages, some beyond fp16's exact powers
        c.host[i][:] = 127 + c.rng.integers(-17, 10, c.host[i].shape)
        c.dev[i].copy_(torch.from_numpy(c.host[i]))
    starts = np.concatenate(([0], np.cumsum(lens)))
    T = int(starts[-1])
    for dt in (torch.bfloat16, torch.float16):
        got = B.kv_read_e4m3(*c.dev, i32(c.table), i32(starts), T, dtype=dt)
        for i in (0, 1):
            want = np.concatenate([c8.tokens(c.host[i], c.host[i + 2], c.table[r], n) for r, n in enumerate(lens)])
            want = torch.from_numpy(want)
            want = (want.clamp(-65504.0, 65504.0) if dt == torch.float16 else want).to(dt)
            x = got[i].cpu()
            assert torch.equal(x.isnan(), want.isnan()) and torch.equal(x.nan_to_num(), want.nan_to_num())


def test_read_every_code_and_scale(B):
    """bf16 exactly (the largest binades of 2^64 * 448 are inside its range), fp16 rounded once and saturated."""
    import torch
    codes = torch.arange(256, dtype=torch.uint8).repeat(8).view(1, 1, 16, 128)
    pages = 129
    cache = codes.repeat(pages, 1, 1, 1).cuda()
    scales = torch.arange(63, 192, dtype=torch.uint8).view(pages, 1).cuda()
    table = i32(np.arange(pages)[:, None])
    starts = i32(np.arange(pages + 1) * 16)
    want = torch.from_numpy(c8.VALUES)[codes.long()].reshape(1, 16, 128) * torch.exp2(torch.arange(-64, 65).double())[:, None, None]
    for dt in (torch.bfloat16, torch.float16):
        k, v = B.kv_read_e4m3(cache, cache.clone(), scales, scales, table, starts, pages * 16, dtype=dt)
        w = want if dt == torch.bfloat16 else want.clamp(-65504.0, 65504.0)
        w = w.view(-1, 1, 128).to(dt)
        for x in (k.cpu(), v.cpu()):
            assert torch.equal(x.isnan(), w.isnan()) and torch.equal(x.nan_to_num(), w.nan_to_num())


def test_read_reports_indices_out_of_range(B):
    import torch
    c = Cache(10, [40, 33], 2, 64, 16)
    bad = c.table.copy()
    bad[1, 1] = -1
    for table, starts in ((bad, [0, 5, 38]), (c.table, [0, 49, 60]), (c.table, [0, 70, 71]), (c.table, [3, 1, 5])):
        out = [torch.full((64, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        B.kv_read_e4m3(*c.dev, i32(table), i32(starts), 64, out=out)
        assert B.read_error_flags() == 1 << 7, starts
        assert torch.all(out[0][60:] == 7)


# ------------------------------------------------------------------------------- attention
def _limit(ref, oabs, reach, n, vmax, dtype):
    eps = 2.0 ** -22 * (10 * reach[..., None] + 64) * 1.4427
    return U[dtype] * np.abs(ref) + (2.0 ** -11 + 2 * eps + (n / 16 + 8) * 2.0 ** -22) * oabs + n * 2.0 ** -32 * vmax


def _lse_limit(lse, reach, n):
    return 2.0 ** -22 * (10 * reach + 64) * 1.4427 + (n / 16 + 8) * 2.0 ** -23 + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0))


def _within(got, ref, limit, what):
    assert got.shape == ref.shape
    assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(np.isinf(got), np.isinf(ref)), what
    assert np.array_equal(got[np.isinf(ref)], ref[np.isinf(ref)]), what
    err = np.zeros_like(ref)
    np.subtract(got, ref, out=err, where=np.isfinite(ref))
    err = np.abs(err)
    bad = ~(err <= limit)
    assert not bad.any(), "%s: %d of %d outside, worst %g of its limit" % (what, bad.sum(), bad.size, np.nanmax(err / np.maximum(limit, 1e-300)))


def _attend(B, c, lens, news, Hq, dtype, seed=0, scale=None, q=None, rows=None, **kw):
    """Checks one call against the oracle; rows: of Q, where it is longer than the requests' tokens."""
    import torch
    starts = np.concatenate(([0], np.cumsum(news)))
    T = rows or int(starts[-1])
    if q is None:
        q = torch.randn(T, Hq, c.d, generator=torch.Generator().manual_seed(seed)).to(_dt(dtype)).cuda()
    o, lse = B.attn_e4m3(q, *c.dev, i32(c.table), i32(lens), i32(starts), max(1, max(news)), scale=scale, **kw)
    assert o.dtype == _dt(dtype) and lse.dtype == torch.float32
    check(c, q, o, lse, lens, starts, scale, dtype)
    return q, o, lse


def check(c, q, o, lse, lens, starts, scale, dtype):
    ref, ref_lse, oabs, reach = c8.attend(_host(q), *c.host, c.table, lens, starts, c.d ** -0.5 if scale is None else scale)
    n = max(max(lens), 1)
    vmax = max([np.abs(c8.tokens(c.host[1], c.host[3], c.table[r], k)).max() for r, k in enumerate(lens) if k] + [0.0])
    _within(_host(o)[:starts[-1]], ref[:starts[-1]], _limit(ref, oabs, reach, n, vmax, dtype)[:starts[-1]], "O")
    _within(_host(lse)[:starts[-1]], ref_lse[:starts[-1]], _lse_limit(ref_lse, reach, n)[:starts[-1]], "lse")


ATTN = [  # lens, new tokens, Hq, Hkv
    ([1], [1], 1, 1),
    ([500], [1], 8, 2),
    ([15, 16, 17, 1, 64, 65, 0], [1] * 7, 8, 2),
    ([100, 300, 37, 5], [4, 1, 3, 5], 4, 4),
    ([2100], [1], 16, 1),
    ([130, 260], [130, 7], 8, 2),
    ([700, 40], [3, 2], 14, 2),
    ([90, 3, 257], [2, 3, 9], 20, 1),
    ([128], [1], 128, 1),
    ([77, 200], [40, 1], 71, 1),
    ([300, 0, 20], [0, 0, 20], 6, 3),
]


@pytest.mark.parametrize("dtype,d,page", [("bf16", 128, 16), ("bf16", 64, 128), ("f16", 128, 64), ("f16", 64, 32)])
@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attend(B, case, dtype, d, page):
    lens, news, Hq, Hkv = ATTN[case]
    c = Cache(20 + case, lens, Hkv, d, page, spread=0.5).fill(B, lens)
    _attend(B, c, lens, news, Hq, dtype, case)


ROWS = [  # lens, new tokens, Hq, Hkv: rows of a head (new tokens x Hq / Hkv) on both sides of the kernels' limits
    ([200, 90, 64], [6, 8, 5], 8, 2),                              # 24, 32, 20: two row tiles
    ([300, 5, 70], [4, 4, 1], 16, 2),                              # 32 and 8 of the same call
    ([64, 60, 700], [10, 33, 12], 8, 2),                           # 40, 132, 48: key tiles in turn, and not
    ([5, 64, 63, 65, 129], [5, 9, 16, 10, 7], 16, 2),              # 40 .. 128 over one key tile, or two or three
    ([140, 300, 40], [32, 65, 33], 8, 2),                          # 128, 260, 132: on both sides of a lane and of an item
    ([200, 90, 300], [16, 13, 9], 8, 2),                           # 64, 52, 36
    ([70, 1100], [5, 6], 30, 3),                                   # 50, 60 of ten heads
    ([400, 60, 300, 90, 17], [100, 1, 1, 2, 1], 14, 2),            # decoding requests beside a prompt
    ([300, 40, 5, 260], [30, 1, 0, 2], 20, 1),                     # 600, 20, none, 40
    ([33, 2, 1, 500], [33, 2, 1, 0], 8, 1),                        # as long as the request
]


@pytest.mark.parametrize("dtype,d,page", [("bf16", 128, 16), ("bf16", 64, 32), ("f16", 128, 128), ("f16", 64, 64)])
@pytest.mark.parametrize("case", range(len(ROWS)))
def test_attend_rows_of_all_kinds(B, case, dtype, d, page):
    lens, news, Hq, Hkv = ROWS[case]
    c = Cache(60 + case, lens, Hkv, d, page, spread=0.5).fill(B, lens)
    _attend(B, c, lens, news, Hq, dtype, case)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("lens,news,Hq", [([9000], [1], 4), ([20001, 30], [7, 2], 4), ([9000, 77], [20, 1], 4), ([6000], [130], 2)])
def test_attend_few_requests_cut_in_many_pieces(B, dtype, d, lens, news, Hq):
    """Their pieces are joined by groups, then the groups."""
    c = Cache(70, lens, 1, d, 64, spread=0.5).fill(B, lens)
    _attend(B, c, lens, news, Hq, dtype, 1)


def test_attend_many_requests_of_both_kinds(B):
    rng = np.random.default_rng(6)
    news = [int(n) for n in rng.integers(0, 40, 90)]
    lens = [int(n + m) for n, m in zip(news, rng.integers(0, 90, 90))]
    c = Cache(71, lens, 2, 64, 16).fill(B, lens)
    _attend(B, c, lens, news, 8, "bf16")


def test_attend_many_requests(B):
    lens = [int(n) for n in np.random.default_rng(5).integers(0, 150, 600)]
    c = Cache(40, lens, 2, 64, 16).fill(B, lens)
    _attend(B, c, lens, [1] * 600, 8, "bf16")


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("news", [1, 5])
def test_attend_scales_that_differ_widely_between_pages(B, dtype, d, news):
    """A page's values may be 2^40 times another's, its keys 2^12 times: the weights follow what counts."""
    import torch
    lens = [220, 64]
    c = Cache(41, lens, 2, d, 16).fill(B, lens)
    rng = np.random.default_rng(0)
    c.host[2][:] = 127 - 8 + rng.integers(-9, 3, c.host[2].shape)
    c.host[3][:] = 127 + rng.integers(-40, 1, c.host[3].shape)
    for i in (2, 3):
        c.dev[i].copy_(torch.from_numpy(c.host[i]))
    _attend(B, c, lens, [news, news], 8, dtype)
    _attend(B, c, lens, [news, news], 8, dtype, scale=4.0)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("news", [1, 5, 70])
def test_attend_value_scales_a_hundred_powers_of_two_apart(B, dtype, d, news):
    """What a sum loses of a key is below 2^-33 of it here: in the limit's n 2^-32 of the largest value."""
    import torch
    lens = [news + 220, news + 64]
    c = Cache(77, lens, 2, d, 16).fill(B, lens)
    rng = np.random.default_rng(1)
    c.host[2][:] = 127 - 8 + rng.integers(-3, 2, c.host[2].shape)
    c.host[3][:] = 127 + rng.choice([-50, -49, 0, 49, 50], c.host[3].shape)
    for i in (2, 3):
        c.dev[i].copy_(torch.from_numpy(c.host[i]))
    # the output's type ends before the largest values do: those of fp16 are taken out by a page's exponent
    if dtype == "f16":
        c.host[3][:] -= 50
        c.host[3][:] = np.maximum(c.host[3], 63)
        c.dev[3].copy_(torch.from_numpy(c.host[3]))
    _attend(B, c, lens, [news, news], 8, dtype)


@pytest.mark.parametrize("where", [63, 191])
def test_attend_scales_at_their_limits(B, where):
    import torch
    lens = [150, 3]
    c = Cache(42, lens, 2, 64, 32).fill(B, lens)
    c.host[3][:] = where
    c.dev[3].copy_(torch.from_numpy(c.host[3]))
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    _attend(B, c, lens, [1, 1], 4, "bf16", q=q)


def test_attend_queries_of_all_magnitudes(B):
    """A query's power of two is taken out and put back: bf16 far beyond fp16's range, and far below."""
    import torch
    lens = [100] * 4
    c = Cache(43, lens, 1, 128, 16).fill(B, lens)
    q = torch.randn(4, 2, 128, generator=torch.Generator().manual_seed(1))
    q = (q * torch.tensor([1e30, 1e-30, 1.0, 1e-38])[:, None, None]).bfloat16().cuda()
    for scale in (1e-30, 0.1, 1e28):
        use = {1e-30: 0, 0.1: 2, 1e28: 1}[scale]
        o, lse = B.attn_e4m3(q, *c.dev, i32(c.table), i32(lens), scale=scale)
        one = Cache.__new__(Cache)
        one.host, one.table, one.d = c.host, c.table[use:use + 1], 128
        check(one, q[use:use + 1], o[use:use + 1], lse[use:use + 1], [100], [0, 1], float(np.float32(scale)), "bf16")


def test_attend_large_scores(B):
    lens = [400, 33]
    for dtype in ("bf16", "f16"):
        c = Cache(44, lens, 2, 128, 64).fill(B, lens, scale=8.0)
        _attend(B, c, lens, [2, 2], 4, dtype, scale=1.5)


def test_attend_one_token_each_without_q_start_strided_q_given_outputs(B):
    import torch
    lens = [90, 14, 260]
    c = Cache(45, lens, 2, 128, 32).fill(B, lens)
    wide = torch.randn(3, 12, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    q = wide[:, 2:10]
    out = torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 8, device="cuda")
    o, lse = B.attn_e4m3(q, *c.dev, i32(c.table), i32(lens), out=out)
    assert o is out[0] and lse is out[1]
    check(c, q, o, lse, lens, [0, 1, 2, 3], None, "bf16")


@pytest.mark.parametrize("news", [1, 70])
def test_attend_inputs_and_outputs_aligned_to_16_bytes_only(B, news):
    import torch
    lens = [news + 90, news + 7]
    c = Cache(74, lens, 2, 128, 32).fill(B, lens)
    T = 2 * news

    def at16(like):
        flat = torch.empty(like.numel() + 8, dtype=like.dtype, device="cuda")
        assert flat.data_ptr() % 32 == 0
        t = flat[16 // like.element_size():][:like.numel()].view(like.shape)
        t.copy_(like)
        return t
    q = at16(torch.randn(T, 8, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda())
    c.dev[0], c.dev[1] = (torch.cat((torch.zeros(16, dtype=torch.uint8, device="cuda"), x.flatten()))[16:].view(x.shape) for x in c.dev[:2])
    out = at16(torch.zeros(T, 8, 128, dtype=torch.bfloat16, device="cuda")), torch.empty(T * 8 + 1, device="cuda")[1:].view(T, 8)
    _, o, _ = _attend(B, c, lens, [news] * 2, 8, "bf16", q=q, out=out)
    assert o is out[0] and o.data_ptr() % 32 == 16


def test_attend_leaves_rows_behind_the_requests_alone(B):
    import torch
    lens = [90, 200]
    for news in ([1, 1], [30, 41]):
        c = Cache(46, lens, 2, 64, 32).fill(B, lens)
        T = sum(news) + 9
        out = torch.full((T, 8, 64), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((T, 8), 4.0, device="cuda")
        _attend(B, c, lens, news, 8, "bf16", rows=T, out=out)
        assert torch.all(out[0][sum(news):] == 3) and torch.all(out[1][sum(news):] == 4)


def test_attend_rows_without_keys(B):
    import torch
    lens = [0, 2, 40]
    c = Cache(47, lens, 2, 64, 16).fill(B, lens)
    _, o, lse = _attend(B, c, lens, [2, 5, 1], 4, "f16")
    assert torch.all(o[:5] == 0) and torch.all(lse[:5] == -float("inf")) and torch.all(torch.isfinite(lse[5:]))


@pytest.mark.parametrize("news", [1, 3, 70])
def test_attend_nan_of_visible_keys_and_values_only(B, news):
    """NaN codes behind a request's tokens reach nothing (caches start with some); visible ones do."""
    import torch
    lens = [150, 150]
    c = Cache(48, lens, 2, 64, 64).fill(B, lens)
    _attend(B, c, lens, [news, news], 4, "bf16")
    page, at = c.table[1, 0], 20
    for i in (0, 1):
        keep = c.host[i][page, 1, at, 3]
        c.host[i][page, 1, at, 3] = 0x7F
        c.dev[i].copy_(torch.from_numpy(c.host[i]))
        q = torch.randn(2 * news, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
        o, lse = B.attn_e4m3(q, *c.dev, i32(c.table), i32(lens), i32([0, news, 2 * news]), news)
        bad = torch.isnan(o)
        assert not bad[:news].any() and not bad[:, :2].any()
        assert bad[news:, 2:].all() if i == 0 else bad[news:, 2:, 3].all() and bad.sum() == 2 * news
        assert torch.isnan(lse[news:, 2:]).all() == (i == 0) and not torch.isnan(lse[:news]).any()
        c.host[i][page, 1, at, 3] = keep
        c.dev[i].copy_(torch.from_numpy(c.host[i]))


@pytest.mark.parametrize("byte", [0, 255])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (64, 32), (128, 128)])
@pytest.mark.parametrize("news", [1, 9, 70])
def test_attend_pages_of_no_request_reach_nothing(B, d, page, byte, news):
    """Pages that nothing was written to hold anything, scale bytes 0 and 255 too, the first page among them."""
    import torch
    lens = [news, news + 8, news + 67]
    c = Cache(72, lens, 2, d, page, spare=4)
    free = [p for p in range(c.host[0].shape[0]) if p not in c.table]
    c.table[c.table == 0] = free[0] if free[0] else 0
    c.fill(B, lens)
    free = [p for p in range(c.host[0].shape[0]) if p not in c.table]
    assert 0 in free
    for i, b in enumerate((0x7F, 0x7F, byte, byte)):
        c.host[i][free] = b
        c.dev[i].copy_(torch.from_numpy(c.host[i]))
    for dtype in ("bf16", "f16"):
        _attend(B, c, lens, [news] * 3, 8, dtype)


@pytest.mark.parametrize("news", [1, 9, 70])
def test_attend_scores_that_underflow(B, news):
    """scale times a query below float32's range: all visible keys weigh alike, the others still nothing."""
    import torch
    lens = [news + 30]
    c = Cache(73, lens, 1, 128, 16).fill(B, lens)
    q = (torch.randn(news, 4, 128, generator=torch.Generator().manual_seed(1)) * 2.0 ** -100).bfloat16().cuda()
    _attend(B, c, lens, [news], 4, "bf16", q=q, scale=float(np.float32(1e-30)))


def test_attend_and_append_beyond_32_bit_offsets(B):
    import torch
    pages, Hkv, page, d = 36000, 8, 128, 128                              # 4.7e9 codes
    k = torch.zeros(pages, Hkv, page, d, dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    ks, vs = (torch.full((pages, Hkv), 127, dtype=torch.uint8, device="cuda") for _ in range(2))
    c = Cache(49, [200], Hkv, d, page, spare=0)
    kv = c.new(1, 200, "bf16")
    c.append(B, kv, [200], [200])
    far = i32([[pages - 1, pages - 7]])
    B.kv_append_e4m3(*kv[0], k, v, ks, vs, far, i32([200]), i32([0, 200]), 200)
    q = torch.randn(1, 16, d, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    o, lse = B.attn_e4m3(q, k, v, ks, vs, far, i32([200]))
    check(c, q, o, lse, [200], [0, 1], None, "bf16")
    got = B.kv_read_e4m3(k, v, ks, vs, far, i32([0, 200]), 200)
    for i in (0, 1):
        assert np.array_equal(_host(got[i]), c8.tokens(c.host[i], c.host[i + 2], c.table[0], 200))


def test_attend_reports_indices_out_of_range(B):
    import torch
    lens = [90, 200]
    c = Cache(50, lens, 2, 64, 32).fill(B, lens)
    q = torch.randn(10, 4, 64).bfloat16().cuda()
    bad = c.table.copy()
    bad[1, 2] = 1 << 20
    for table, ln, starts, most in ((bad, lens, [0, 5, 10], 5), (c.table, [90, -1], [0, 5, 10], 5), (c.table, [90, 400], [0, 5, 10], 5),
                                    (c.table, lens, [0, 5, 11], 6), (c.table, lens, [0, 8, 3], 8), (c.table, lens, [-2, 5, 10], 8),
                                    (c.table, lens, [0, 5, 10], 4)):
        o, lse = B.attn_e4m3(q, *c.dev, i32(table), i32(ln), i32(starts), most)
        assert B.read_error_flags() == 1 << 7, (ln, starts)


def test_workspace_header_stays_zero_and_serves_other_calls(B):
    import torch
    from bit_weight_quantized_wq_gb300 import inputs
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    W = torch.from_numpy(inputs.weights(1, 256, 512, 0.02)).cuda()
    packed = B.quantize_int4_g128(W)
    X = torch.randn(3, 512, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    want = B.gemm_w4a16("int4_g128", X, *packed, workspace=ws).clone()
    for lens, news in (([5000], [1]), ([900, 20, 301], [2, 20, 100]), ([3000], [300])):
        c = Cache(51, lens, 2, 128, 64).fill(B, lens)
        _attend(B, c, lens, news, 8, "bf16", workspace=ws)
        assert not ws[:64 * 1024].any()
        assert torch.equal(B.gemm_w4a16("int4_g128", X, *packed, workspace=ws), want)


def test_same_bits_every_time(B):
    import torch
    for lens, news in (([6000, 11, 3000], [1, 1, 1]), ([700, 2000], [300, 90])):
        c = Cache(52, lens, 2, 128, 64).fill(B, lens)
        first = None
        for _ in range(5):
            q = torch.randn(sum(news), 8, 128, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
            got = B.attn_e4m3(q, *c.dev, i32(c.table), i32(lens), i32(np.concatenate(([0], np.cumsum(news)))), max(news))
            first = first or got
            assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_on_a_side_stream(B):
    import torch
    lens = [300, 70]
    side = torch.cuda.Stream()
    a, b = (Cache(53, lens, 2, 128, 16) for _ in range(2))
    kv = a.new(1, 370, "bf16")
    q = torch.randn(2, 8, 128, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    a.append(B, kv, lens, lens)
    want = B.attn_e4m3(q, *a.dev, i32(a.table), i32(lens))
    torch.cuda.synchronize()
    table, n, starts = i32(b.table), i32(lens), i32([0, 300, 370])
    B.kv_append_e4m3(*kv[0], *b.dev, table, n, starts, 300, stream=side)
    got = B.attn_e4m3(q, *b.dev, table, n, stream=side)
    back = B.kv_read_e4m3(*b.dev, table, starts, 370, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    b.host = a.host
    b.check()
    assert np.array_equal(_host(back[0])[300:], c8.tokens(a.host[0], a.host[2], a.table[1], 70))


def test_captured_and_replayed_over_growing_requests(B):
    """One captured decode step, replayed with new tokens and lengths in the same tensors."""
    import torch
    lens = [60, 15, 0]
    c = Cache(54, [90, 45, 16], 2, 64, 16)
    c.fill(B, lens)
    kv = c.new(1, 3, "bf16")
    k, v = kv[0][0].contiguous(), kv[0][1].contiguous()
    q = torch.randn(3, 8, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    table, n = i32(c.table), i32([61, 16, 0])
    ws = torch.zeros(B.load_library().wq_attn_e4m3_workspace_bytes(3, 3, 8, 2, 64, 1), dtype=torch.uint8, device="cuda")
    before = [t.clone() for t in c.dev]
    B.kv_append_e4m3(k, v, *c.dev, table, n)
    B.attn_e4m3(q, *c.dev, table, n, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.kv_append_e4m3(k, v, *c.dev, table, n)
        o, lse = B.attn_e4m3(q, *c.dev, table, n, workspace=ws)
    for t, saved in zip(c.dev, before):
        t.copy_(saved)
    live = [0, 1]
    for step in range(20):
        kv = c.new(100 + step, 3, "bf16", 1.0 + step)
        k.copy_(kv[0][0]), v.copy_(kv[0][1])
        now = [61 + step, 16 + step, 0]
        n.copy_(i32(now))
        graph.replay()
        c8.append(kv[1][0][live], kv[1][1][live], *c.host, c.table[live], now[:2], [0, 1, 2])
        c.check()
        check(c, q, o, lse, now, [0, 1, 2, 3], None, "bf16")


@pytest.mark.parametrize("dtype,Hq,d", [("bf16", 8, 128), ("f16", 24, 64)])
def test_decoding_requests_beside_prompts_call_after_call(B, dtype, Hq, d):
    """Appends and attention of both kinds of requests with nothing between the calls, eager and replayed: the same bits as
    with a synchronisation after each (the tokens that a call reads change with every step)."""
    import torch
    rng = np.random.default_rng(8)
    news = [1, 150, 1, 1, 2, 70, 1, 1]
    lens = [int(n) for n in 150 + rng.integers(0, 3000, 8)]
    T, starts = sum(news), i32(np.concatenate(([0], np.cumsum(news))))
    c = Cache(75, lens, 2, d, 64)
    c.append(B, c.new(1, sum(lens), dtype), lens, lens)
    table, n = i32(c.table), i32(lens)
    steps = [c.new(100 + i, T, dtype, 1.0 + i)[0] for i in range(12)]
    q = torch.randn(T, Hq, d, generator=torch.Generator().manual_seed(1)).to(_dt(dtype)).cuda()
    ws = torch.zeros(B.load_library().wq_attn_e4m3_workspace_bytes(T, 8, Hq, 2, d, 150), dtype=torch.uint8, device="cuda")
    fresh = [x.clone() for x in c.dev]

    def go(each, wait=False):
        for x, saved in zip(c.dev, fresh):
            x.copy_(saved)
        torch.cuda.synchronize()
        got = []
        for k, v in steps:
            got.append(each(k, v))
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return got

    def call(k, v):
        B.kv_append_e4m3(k, v, *c.dev, table, n, starts, 150)
        return B.attn_e4m3(q, *c.dev, table, n, starts, 150, workspace=ws)

    want = go(call, wait=True)
    assert not torch.equal(want[0][0], want[1][0])
    kv = [x.clone() for x in steps[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = call(*kv)

    def replayed(k, v):
        kv[0].copy_(k), kv[1].copy_(v)
        graph.replay()
        return o.clone(), lse.clone()
    for _ in range(5):
        for got in (go(call), go(replayed)):
            assert all(torch.equal(a, b) for x, y in zip(want, got) for a, b in zip(x, y))
    assert not ws[:64 * 1024].any()
    c.host = [x.cpu().numpy() for x in c.dev]
    check(c, q, *want[-1], lens, starts.cpu().numpy(), None, dtype)


@pytest.mark.parametrize("news", [1, 3, 70])
def test_attend_non_finite_queries_stay_in_their_rows(B, news):
    import torch
    lens = [news + 90, news + 300]
    c = Cache(76, lens, 2, 64, 32).fill(B, lens)
    for dtype in ("bf16", "f16"):
        q = torch.randn(2 * news, 8, 64, generator=torch.Generator().manual_seed(1)).to(_dt(dtype)).cuda()
        starts = [0, news, 2 * news]
        want = B.attn_e4m3(q, *c.dev, i32(c.table), i32(lens), i32(starts), news)
        bad = q.clone()
        bad[0, 1, 3], bad[-1, 6, 0], bad[-1, 7, 63] = float("nan"), float("inf"), -float("inf")
        got = B.attn_e4m3(bad, *c.dev, i32(c.table), i32(lens), i32(starts), news)
        hit = torch.zeros(2 * news, 8, dtype=torch.bool, device="cuda")
        hit[0, 1] = hit[-1, 6] = hit[-1, 7] = True
        for a, b in zip(got, want):
            assert torch.equal(a[~hit], b[~hit])
        assert not torch.isfinite(got[0][hit]).any()


def test_rejects_bad_arguments(B):
    import torch
    c = Cache(55, [40, 33], 2, 64, 16)
    (k, v), _ = c.new(1, 2, "bf16")
    q = torch.randn(2, 4, 64).bfloat16().cuda()
    table, lens, starts = i32(c.table), i32([40, 33]), i32([0, 1, 2])
    good = dict(K=k, V=v, k_cache=c.dev[0], v_cache=c.dev[1], k_scales=c.dev[2], v_scales=c.dev[3], block_table=table, lens=lens)
    for name, bad in (("K", k.float()), ("K", k.cpu()), ("K", k[:1]), ("V", v.half()), ("V", v[:, :1]), ("k_cache", c.dev[0].float()),
                      ("k_cache", c.dev[0][:, :, :, :32]), ("v_cache", c.dev[1][1:]), ("k_scales", c.dev[2].int()), ("v_scales", c.dev[3][:, :1]),
                      ("block_table", table.long()), ("block_table", table[0]), ("lens", lens[:1]), ("lens", lens.float()), ("lens", None),
                      ("q_start", lens), ("max_new", 0), ("K", k.transpose(1, 2)), ("k_cache", c.dev[0].transpose(0, 1))):
        with pytest.raises(ValueError):
            B.kv_append_e4m3(**dict(good, **{name: bad}))
    good = dict(Q=q, k_cache=c.dev[0], v_cache=c.dev[1], k_scales=c.dev[2], v_scales=c.dev[3], block_table=table, lens=lens)
    for name, bad in (("Q", q.float()), ("Q", q[:, :3]), ("Q", q[:, :, :32]), ("lens", lens.cpu()), ("scale", -1.0), ("scale", "x"),
                      ("out", (q, None, None)), ("out", (torch.empty_like(q).half(), None)), ("q_start", table), ("Q", q[:1]),
                      ("workspace", torch.zeros(1 << 10, dtype=torch.uint8, device="cuda")), ("max_new", 2)):
        with pytest.raises(ValueError):
            B.attn_e4m3(**dict(good, **{name: bad}))
    good = dict(k_cache=c.dev[0], v_cache=c.dev[1], k_scales=c.dev[2], v_scales=c.dev[3], block_table=table, starts=starts, tokens=2)
    for name, bad in (("dtype", torch.float32), ("tokens", 0), ("tokens", None), ("starts", lens), ("out", (k, None)), ("k_cache", c.dev[0].cpu())):
        with pytest.raises(ValueError):
            B.kv_read_e4m3(**dict(good, **{name: bad}))


def test_run_together_as_a_decoder_uses_them(B):
    """Norm and rotation, append, attention: a prompt, then single tokens; the cache read back at the end gives the
    16-bit cache that the 16-bit attention answers alike from."""
    import torch
    Hq, Hkv, d, page, n = 8, 2, 64, 16, 61
    c = Cache(56, [n], Hkv, d, page)
    g = torch.Generator().manual_seed(4)
    x = torch.randn(n, Hq + 2 * Hkv, d, generator=g).bfloat16().cuda()
    w = (1 + 0.1 * torch.randn(2, d, generator=g)).bfloat16().cuda()
    angle = torch.arange(64.0)[:, None] * 1e4 ** (-torch.arange(0, d, 2) / d)
    tab = torch.cat((angle.cos(), angle.sin()), 1).float().cuda()
    table = i32(c.table)
    outs = []
    for lo, hi in [(0, 50)] + [(t, t + 1) for t in range(50, n)]:
        q, k = B.qk_norm_rope(x[lo:hi, :Hq], x[lo:hi, Hq:Hq + Hkv], i32(range(lo, hi)), tab, w[0], w[1])
        v = x[lo:hi, Hq + Hkv:]
        starts = i32([0, hi - lo])
        B.kv_append_e4m3(k, v, *c.dev, table, i32([hi]), starts, hi - lo)
        c8.append(_host(k), _host(v), *c.host, c.table, [hi], [0, hi - lo])
        o, lse = B.attn_e4m3(q, *c.dev, table, i32([hi]), starts, hi - lo)
        check(c, q, o, lse, [hi], [0, hi - lo], None, "bf16")
        outs.append((q, o))
    c.check()
    k16, v16 = B.kv_read_e4m3(*c.dev, table, i32([0, n]), n)
    wide = torch.zeros(2, 4, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    for i, t in enumerate((k16, v16)):
        for j in range(4):
            rows = t[16 * j:16 * j + 16].transpose(0, 1)
            wide[i, j, :, :rows.shape[1]] = rows
    q, o = outs[-1]
    o16, _ = B.attn_shared_prefix(q, wide[0], wide[1], None, 0, i32([[0, 1, 2, 3]]), i32([n]))
    # both round the weights (2^-11, 2^-8) and the output (2^-8): sums of |v| p, at most max |v|
    assert (o16.float() - o.float()).abs().max() <= (2 * 2.0 ** -8 + 2.0 ** -8 + 2.0 ** -11) * float(v16.float().abs().max()) * 1.5


def test_example_of_a_served_block(B):
    """Prompts in pieces beside decoding requests, then a captured step with places whose request is done."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "quantized_cache_block.py")
    spec = importlib.util.spec_from_file_location("quantized_cache_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.main() < 2.0 ** -4


# ------------------------------------------------------------- items cut over many CTAs, neighbours in one of them
class LongCache:
    """Random codes and scales made on the GPU, for caches too long for the host's oracle."""

    def __init__(self, seed, lens, Hkv, d, page):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        blocks = [-(-n // page) for n in lens]
        pages = sum(blocks) + 3
        perm = torch.randperm(pages, generator=g, device="cuda").int().cpu().numpy()
        self.table, at = np.full((len(lens), max(blocks)), -1, np.int32), 0
        for r, b in enumerate(blocks):
            self.table[r, :b] = perm[at:at + b]
            at += b
        self.dev = []
        for _ in range(2):
            codes = torch.empty(pages, Hkv, page, d, dtype=torch.uint8, device="cuda")
            for i in range(0, pages, 512):
                x = torch.randn(codes[i:i + 512].shape, generator=g, device="cuda") * 64
                codes[i:i + 512] = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            self.dev.append(codes)
        self.dev += [torch.randint(119, 122, (pages, Hkv), generator=g, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.d, self.Hkv = d, Hkv

    def tokens(self, i, r, h, n):
        """Keys (i = 0) or values of the first n tokens of a request's head, float64."""
        import torch
        page = self.dev[i].shape[2]
        p = torch.from_numpy(self.table[r, :-(-n // page)]).long().cuda()
        x = torch.from_numpy(c8.VALUES).cuda()[self.dev[i][p, h].long()] * torch.exp2(self.dev[i + 2][p, h].double() - c8.BIAS)[:, None, None]
        return x.reshape(-1, self.d)[:n]

    def check(self, q, o, lse, lens, news, dtype):
        """All rows against float64, computed on the GPU."""
        import torch
        group, scale, t = q.shape[1] // self.Hkv, self.d ** -0.5, 0
        for r, (n, new) in enumerate(zip(lens, news)):
            for h in range(self.Hkv):
                k, v = self.tokens(0, r, h, n), self.tokens(1, r, h, n)
                heads = slice(h * group, (h + 1) * group)
                x = q[t:t + new, heads].double().reshape(-1, self.d)
                score = scale * (x @ k.T)
                hidden = torch.arange(n, device="cuda") > (n - new + torch.arange(new, device="cuda").repeat_interleave(group))[:, None]
                reach = scale * (x.abs() @ k.abs().T).amax(1)
                score.masked_fill_(hidden, -float("inf"))
                ref_lse, p = torch.logsumexp(score, 1), torch.softmax(score, 1)
                ref, oabs = (_host((p @ w).view(new, group, -1)) for w in (v, v.abs()))
                ref_lse, reach = _host(ref_lse.view(new, group)), _host(reach.view(new, group))
                what = "request %d, head %d: " % (r, h)
                _within(_host(o[t:t + new, heads]), ref, _limit(ref, oabs, reach, n, float(v.abs().max()), dtype), what + "O")
                _within(_host(lse[t:t + new, heads]), ref_lse, _lse_limit(ref_lse, reach, n), what + "lse")
            t += new


CUT = [  # lens, new tokens, Hq, Hkv, d, dtype: items of more than eight segments, the next one beginning where one ends
    ([74000], [1], 40, 5, 128, "bf16"),
    ([131071 - 997 * i for i in range(9)], [1] * 9, 64, 8, 128, "bf16"),
    ([int(32768 * 4 ** (i / 11)) for i in range(12)], [1] * 12, 64, 8, 128, "f16"),
    ([8000 + 8000 * i for i in range(8)], [4] * 8, 64, 8, 128, "bf16"),
    ([65000, 30011, 50000, 41000], [3, 2, 4, 1], 16, 16, 64, "f16"),
    ([25500], [128], 40, 5, 128, "bf16"),
    ([32663, 52569], [16, 64], 64, 8, 128, "bf16"),
    ([120000, 90000, 131071, 3000, 65536], [1, 1, 1, 200, 1], 64, 8, 128, "bf16"),
    ([11489, 18484, 42577, 49181], [1, 64, 24, 40], 24, 3, 64, "f16"),
]


@pytest.mark.parametrize("case", range(len(CUT)))
def test_attend_neighbouring_items_cut_in_groups(B, case):
    """Every row of every call is written, the same each time, and the workspace's header is left at zero."""
    import torch
    lens, news, Hq, Hkv, d, dtype = CUT[case]
    c = LongCache(80 + case, lens, Hkv, d, 64)
    T = sum(news)
    q = torch.randn(T, Hq, d, generator=torch.Generator().manual_seed(case)).to(_dt(dtype)).cuda()
    table, n, starts = i32(c.table), i32(lens), i32(np.concatenate(([0], np.cumsum(news))))
    ws = torch.zeros(B.load_library().wq_attn_e4m3_workspace_bytes(T, len(lens), Hq, Hkv, d, max(news)), dtype=torch.uint8, device="cuda")
    outs = [(torch.full((T, Hq, d), float("nan"), dtype=_dt(dtype), device="cuda"), torch.full((T, Hq), float("nan"), device="cuda"))
            for _ in range(30)]
    for i, out in enumerate(outs):                    # some with nothing between them, some each by itself
        B.attn_e4m3(q, *c.dev, table, n, starts, max(news), out=out, workspace=ws)
        if i >= 20:
            assert not ws[:64 * 1024].any()
    torch.cuda.synchronize()
    assert not ws[:64 * 1024].any()
    for o, lse in outs:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])
    c.check(q, *outs[0], lens, news, dtype)


# ---------------------------------------------------------------------------------- calls of many requests
def _read_directly(c, starts, T, dtype):
    """What a read gives, by indexing on the GPU; rows of no request are -1."""
    import torch
    rows, out = torch.arange(T, device="cuda"), []
    s = torch.tensor(starts, device="cuda")
    r = (torch.searchsorted(s, rows, right=True) - 1).clamp(0, len(starts) - 2)
    place, mine = rows - s[r], (rows >= s[0]) & (rows < s[-1])
    page = c.table[r, (place // 16).clamp(0, c.table.shape[1] - 1)].long().clamp(min=0)
    for i in (0, 1):
        x = torch.from_numpy(c8.VALUES).cuda()[c.dev[i][page, :, place % 16].long()] * torch.exp2(c.dev[i + 2][page].double() - c8.BIAS)[..., None]
        out.append(torch.where(mine[:, None, None], x, -1.0).to(dtype))
    return out


class ManyRequests:
    """Requests of random tokens in pages of 16, on the GPU alone."""

    def __init__(self, seed, lens, Hkv, d):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        blocks = -(-torch.tensor(lens) // 16)
        pages = int(blocks.sum()) + 1
        perm = torch.randperm(pages, generator=g, device="cuda").int()
        most = max(1, int(blocks.max()))
        at = torch.arange(most)[None] < blocks[:, None]
        self.table = torch.full((len(lens), most), -1, dtype=torch.int32)
        self.table[at] = perm[:int(blocks.sum())].cpu()
        self.table = self.table.cuda()
        codes = torch.randint(0, 254, (2, pages, Hkv, 16, d), generator=g, device="cuda", dtype=torch.uint8)
        codes[(codes & 127) == 127] = 5
        scales = torch.randint(110, 130, (2, pages, Hkv), generator=g, device="cuda", dtype=torch.uint8)
        self.dev = [codes[0], codes[1], scales[0], scales[1]]


@pytest.mark.parametrize("Hkv,d", [(2, 64), (1, 64), (8, 128)])
@pytest.mark.parametrize("R", [256, 257, 1000, 70000])
def test_read_of_many_requests(B, R, Hkv, d):
    """Empty ones among them, rows before the first and behind the last left as they were."""
    import torch
    rng = np.random.default_rng(R)
    lens = rng.choice([0, 0, 1, 1, 2, 3, 17, 40], R) if R < 10000 else rng.choice([0, 1, 2], R)
    lens[rng.integers(0, R, 3)] = 300
    lens[R // 3:R // 3 + 400] = 0                     # more empty ones in a row than threads
    c = ManyRequests(R, lens.tolist(), Hkv, d)
    for lead in (0, 5):
        starts = np.concatenate(([lead], lead + np.cumsum(lens)))
        T = int(starts[-1]) + 7
        want = _read_directly(c, starts.tolist(), T, torch.bfloat16)
        out = [torch.full((T, Hkv, d), -1.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        B.kv_read_e4m3(*c.dev, c.table, i32(starts), T, out=out)
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_read_of_many_requests_reports_starts_out_of_range(B):
    import torch
    lens = [3] * 900
    c = ManyRequests(1, lens, 2, 64)
    good = np.concatenate(([0], np.cumsum(lens)))
    for at, value in ((0, -1), (1, -5), (450, 0), (450, 1 << 30), (899, 2), (900, 2701), (900, 5)):
        starts = good.copy()
        starts[at] = value
        B.kv_read_e4m3(*c.dev, c.table, i32(starts), 2700)
        assert B.read_error_flags() == 1 << 7, (at, value)
    B.kv_read_e4m3(*c.dev, c.table, i32(good), 2700)
    assert B.read_error_flags() == 0


@pytest.mark.parametrize("R", [128, 129, 700, 3000])
@pytest.mark.parametrize("kind", ["single tokens and prompts", "pieces", "nearly all empty"])
def test_append_to_many_requests(B, R, kind):
    """More requests than a CTA's threads: empty ones, single tokens and pieces of several pages among them, a padded batch."""
    rng = np.random.default_rng(R)
    if kind == "single tokens and prompts":
        news = np.ones(R, int)
        news[rng.integers(0, R, 4)] = [200, 77, 16, 129]
    elif kind == "pieces":
        news = rng.integers(0, 60, R) if R < 1000 else rng.integers(0, 20, R)
        news[R // 2] = 64
    else:
        news = np.zeros(R, int)
        news[rng.integers(0, R, 5)] = [300, 1, 40, 17, 2]
        news[0], news[-1] = 0, 33
    news = [int(n) for n in news]
    lens = [int(n + m) for n, m in zip(news, rng.integers(0, 40, R))]
    c = Cache(90, lens, 1, 64, 16, spread=1.0).fill(B, [n - m for n, m in zip(lens, news)])
    c.append(B, c.new(2, sum(news) + 3, "bf16", 4.0), lens, news)
    c.check()
    c.append(B, c.new(3, sum(news), "bf16", 4.0), [0] * R, news)          # all of them padding: nothing is written
    c.check()


def test_append_to_many_requests_reports_indices_out_of_range(B):
    import torch
    R = 600
    news, lens = [1] * R, [30] * R
    news[7] = 25
    c = Cache(91, lens, 1, 64, 16).fill(B, lens)
    kv, _ = c.new(1, sum(news), "bf16")
    starts = np.concatenate(([0], np.cumsum(news)))
    for which, at, value in (("starts", 300, 0), ("starts", 300, 1 << 30), ("starts", 0, -1), ("starts", R, sum(news) + 1), ("starts", 301, 360),
                             ("lens", 599, -1), ("lens", 0, 1 << 20), ("lens", 7, 24), ("table", 599, -1), ("table", 0, 1 << 20)):
        a = dict(starts=starts.copy(), lens=np.array(lens), table=c.table.copy())
        a[which][(at, 1) if which == "table" else at] = value
        B.kv_append_e4m3(*kv, *c.dev, i32(a["table"]), i32(a["lens"]), i32(a["starts"]), 25)
        assert B.read_error_flags() == 1 << 7, (which, at, value)
    B.kv_append_e4m3(*kv, *c.dev, i32(c.table), i32(lens), i32(starts), 25)
    assert B.read_error_flags() == 0


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("prompts", [{0: 60, 399: 90}, {0: 33}, {399: 100}, {31: 40, 32: 41, 33: 42, 300: 70}, {200: 50}])
def test_attend_prompts_far_apart_among_many_requests(B, dtype, d, prompts):
    """Hundreds of single tokens and of empty requests lie between, before and behind them."""
    news = [1] * 400
    for r in list(range(40, 120)) + list(range(330, 399)):
        news[r] = 0
    for r, n in prompts.items():
        news[r] = n
    lens = [n + m for n, m in zip(news, np.random.default_rng(9).integers(0, 40, 400).tolist())]
    c = Cache(92, lens, 2, d, 16).fill(B, lens)
    _attend(B, c, lens, news, 8, dtype)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("news", [1, 5, 70])
@pytest.mark.parametrize("apart", [10, 20, 30, 60])
def test_attend_elements_where_a_page_of_large_scale_holds_zeros(B, dtype, d, news, apart):
    """One value of the first page raises its scale by 2^apart, its others are zeros: the outputs' other elements come from
    the other pages alone, to what wq.h says: 2^-11 of sum p |v| and n 2^-32 * 448 max p 2^e."""
    import torch
    lens = [news + 150, news + 60]
    c = Cache(93, lens, 2, d, 16).fill(B, lens)
    c.host[2][:] = 127 - 8
    c.host[3][:] = 127 - 8 - (apart if dtype == "f16" else 0)
    first = c.table[:, 0]
    c.host[1][first] = 0
    c.host[1][first, :, 3, 7] = 0x7E                                     # 448
    c.host[3][first] += apart
    for i in (1, 2, 3):
        c.dev[i].copy_(torch.from_numpy(c.host[i]))
    starts = [0, news, 2 * news]
    q = torch.randn(2 * news, 8, d, generator=torch.Generator().manual_seed(1)).to(_dt(dtype)).cuda()
    o, lse = B.attn_e4m3(q, *c.dev, i32(c.table), i32(lens), i32(starts), news)
    ref, ref_lse, oabs, reach = c8.attend(_host(q), *c.host, c.table, lens, starts, d ** -0.5)
    # 2^e of the largest scale for max p 2^e: p is at most 1
    largest = 2.0 ** (int(c.host[3].max()) - 127)
    eps = 2.0 ** -22 * (10 * reach[..., None] + 64) * 1.4427
    n = max(lens)
    limit = U[dtype] * np.abs(ref) + (2.0 ** -11 + 2 * eps + (n / 16 + 8) * 2.0 ** -22) * oabs + n * 2.0 ** -32 * 448 * largest
    if dtype == "f16":
        limit += 2.0 ** -25                                              # half the lowest step of the output's type
    others = np.arange(d) != 7
    _within(_host(o)[..., others], ref[..., others], limit[..., others], "O")
    _within(_host(lse), ref_lse, _lse_limit(ref_lse, reach, n), "lse")


@pytest.mark.parametrize("dtype,d,page", [("bf16", 128, 16), ("f16", 64, 64), ("bf16", 64, 32), ("f16", 128, 128)])
@pytest.mark.parametrize("lens,news", [([40, 90], [3, 6]), ([33, 700], [8, 16]), ([100, 64], [30, 7]), ([150, 400], [70, 130]), ([20000, 70], [70, 70])])
def test_attend_nan_among_new_values_reaches_no_row_before_them(B, dtype, d, page, lens, news):
    """A NaN in the value of a new token makes that element NaN in the rows that see the token, and changes no other bit."""
    import torch
    c = Cache(94, lens, 2, d, page).fill(B, lens)
    T, table, n, starts = sum(news), i32(c.table), i32(lens), i32([0, news[0], sum(news)])
    q = torch.randn(T, 8, d, generator=torch.Generator().manual_seed(1)).to(_dt(dtype)).cuda()
    clean = c.dev[1].clone()
    want = B.attn_e4m3(q, *c.dev, table, n, starts, max(news))
    first = [0, news[0]]
    for marks in ([(1, -1, 0, 5)], [(0, -1, 1, d - 1)], [(1, 0, 1, 0)], [(0, news[0] // 2, 0, 17), (0, news[0] - 1, 0, 18), (1, news[1] // 3, 1, 33)],
                  [(1, -2, 0, 62), (0, 1, 1, 40)]):
        c.dev[1].copy_(clean)
        nan = torch.zeros(T, 8, d, dtype=torch.bool, device="cuda")
        for r, i, h, col in marks:                    # request, new token, key/value head, element
            i %= news[r]
            at = lens[r] - news[r] + i
            c.dev[1][int(c.table[r, at // page]), h, at % page, col] = 0x7F if (i & 1) else 0xFF
            nan[first[r] + i:first[r] + news[r], 4 * h:4 * h + 4, col] = True
        o, lse = B.attn_e4m3(q, *c.dev, table, n, starts, max(news))
        assert torch.equal(torch.isnan(o), nan), marks
        assert torch.equal(o[~nan], want[0][~nan]) and torch.equal(lse, want[1])


def test_attend_nan_values_of_new_tokens_in_items_that_are_joined(B):
    """The same where the rows' keys are cut over many CTAs, for few rows and for many."""
    import torch
    for lens, news, Hq in (([30000], [4], 8), ([26000], [40], 16), ([26000], [200], 4)):
        c = LongCache(95, lens, 1, 128, 64)
        q = torch.randn(news[0], Hq, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
        args = i32(c.table), i32(lens), i32([0, news[0]]), news[0]
        want = B.attn_e4m3(q, *c.dev, *args)
        i = 2 * news[0] // 3
        at = lens[0] - news[0] + i
        c.dev[1][int(c.table[0, at // 64]), 0, at % 64, 70] = 0x7F
        o, lse = B.attn_e4m3(q, *c.dev, *args)
        nan = torch.zeros_like(o, dtype=torch.bool)
        nan[i:, :, 70] = True
        assert torch.equal(torch.isnan(o), nan) and torch.equal(o[~nan], want[0][~nan]) and torch.equal(lse, want[1])


# ------------------------------------------------------------------------------ calls of unusual shape
@pytest.mark.parametrize("dtype,d,page", [("bf16", 128, 16), ("f16", 64, 128)])
@pytest.mark.parametrize("lens,news,Hq,Hkv", [([20, 0, 300], [70, 40, 50], 8, 2), ([1, 64, 65], [300, 65, 64], 4, 4), ([0], [90], 8, 1),
                                              ([250, 40], [3, 1], 128, 1), ([130], [130], 7, 7)])
def test_attend_more_new_tokens_than_keys_and_wide_groups(B, dtype, d, page, lens, news, Hq, Hkv):
    c = Cache(96, lens, Hkv, d, page).fill(B, lens) if sum(lens) else Cache(96, lens, Hkv, d, page)
    _attend(B, c, lens, news, Hq, dtype)


@pytest.mark.parametrize("news", [1, 6, 90])
def test_attend_queries_inside_a_fused_projection(B, news):
    import torch
    lens = [news + 70, news + 3]
    c = Cache(97, lens, 2, 128, 32).fill(B, lens)
    x = torch.randn(2 * news, 8 + 4 + 1, 128, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    x[:, 8:] = float("nan")
    _attend(B, c, lens, [news, news], 8, "bf16", q=x[:, :8])


@pytest.mark.parametrize("most", [1, 100])
def test_calls_of_requests_without_new_tokens(B, most):
    """A batch that is all padding: nothing is written, nothing reported."""
    import torch
    lens = [40, 0, 7]
    c = Cache(98, lens, 2, 64, 16).fill(B, lens)
    before = [x.clone() for x in c.dev]
    starts, table, n = i32([0, 0, 0, 0]), i32(c.table), i32(lens)
    out = torch.full((5, 8, 64), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((5, 8), 4.0, device="cuda")
    q = torch.randn(5, 8, 64).bfloat16().cuda()
    B.attn_e4m3(q, *c.dev, table, n, starts, most, out=out)
    B.kv_append_e4m3(q[:, :2], q[:, 2:4], *c.dev, table, n, starts, most)
    read = [torch.full((5, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    B.kv_read_e4m3(*c.dev, table, starts, 5, out=read)
    torch.cuda.synchronize()
    assert torch.all(out[0] == 3) and torch.all(out[1] == 4) and all(torch.all(x == 5) for x in read)
    assert all(torch.equal(a, b) for a, b in zip(before, c.dev))


@pytest.mark.parametrize("lens,news", [([90, 200], [1, 1]), ([90, 9000], [40, 3])])
def test_attend_without_lse(B, lens, news):
    """The C call may leave lse out; O is the same."""
    import ctypes

    import torch
    c = Cache(99, lens, 2, 64, 32).fill(B, lens)
    T, most = sum(news), max(news)
    q = torch.randn(T, 8, 64, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    table, n, starts = i32(c.table), i32(lens), i32(np.concatenate(([0], np.cumsum(news))))
    want, _ = B.attn_e4m3(q, *c.dev, table, n, starts, most)
    lib, o = B.load_library(), torch.empty_like(q)
    ws = torch.zeros(lib.wq_attn_e4m3_workspace_bytes(T, 2, 8, 2, 64, most), dtype=torch.uint8, device="cuda")
    p = lambda t: ctypes.c_void_p(t.data_ptr())   # noqa: E731
    st = lib.wq_attn_e4m3(0, p(q), 512, T, 2, 8, 2, 64, *[p(x) for x in c.dev], c.dev[0].shape[0], 32, p(table), c.table.shape[1], p(n), p(starts),
                          most, 0.125, p(o), None, p(ws), ws.numel(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    torch.cuda.synchronize()
    assert st == 0 and torch.equal(o, want)


@pytest.mark.parametrize("prompts", [{0: 40, 700: 50, 1299: 60}, {600: 300}])
def test_attend_more_requests_than_a_cta_has_threads(B, prompts):
    news = [1] * 1300
    for r, n in prompts.items():
        news[r] = n
    lens = [n + m for n, m in zip(news, np.random.default_rng(10).integers(0, 30, 1300).tolist())]
    c = Cache(100, lens, 1, 64, 16).fill(B, lens)
    _attend(B, c, lens, news, 4, "bf16")

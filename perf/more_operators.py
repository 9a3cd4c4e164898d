"""Cases and plain forms of the operators around a cache of keys and values held in 8 bits.

Three operators of a served decoder whose cache is quantized, in the order a token meets them:

- ``append``: new keys and values quantized as they are written to a cache in pages (E4M3 codes, one
  power-of-two scale, an E8M0 byte, for each page and head, that grows with what the page holds);
- ``attend``: attention of a batch of requests over that cache, new tokens causal, with the
  log-sum-exp beside the output;
- ``read``: the cached tokens of requests read back in 16 bits, one request after the other.

``run`` computes them in elementary torch operations in float32, rounded once at the end, or, with
``own`` set, through ``bit_weight_quantized_wq_gb300.binding``.  ``exact`` computes the same outputs
in float64, written separately from the plain forms.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
LOWEST, HIGHEST = -64, 64        # exponents that a scale can have
STORED = 127                     # a scale's byte is its exponent + 127


# ------------------------------------------------------------------------------- the cases
def _case(name, op, requests, longest, new, hq, hkv, d, page, dtype="bf16", mixed=False):
    """`requests` of up to `longest` tokens, their last 1 .. `new` tokens new in this call (with
    `mixed`: every eighth request's; the others have one)."""
    return {"name": name, "op": op, "requests": requests, "longest": longest, "new": new, "hq": hq, "hkv": hkv, "d": d,
            "page": page, "dtype": dtype, "mixed": mixed}


def listed():
    return [
        # one request decoding: a token of LLaMA-3-8B's key and value heads (latency only)
        _case("append_decode_1", "append", 1, 700, 1, 32, 8, 128, 16),
        # drafted tokens of a decode batch, heads of 64, fp16
        _case("append_verify_96_f16", "append", 96, 3001, 4, 16, 16, 64, 32, dtype="f16"),
        # a prefill batch: pieces of seven prompts
        _case("append_prompts_7", "append", 7, 4099, 2047, 64, 8, 128, 64),
        # one request handed over to a 16-bit cache (latency only)
        _case("read_request_1", "read", 1, 700, 1, 32, 8, 128, 16),
        # a batch of long requests read back, fp16
        _case("read_batch_24_f16", "read", 24, 8191, 1, 64, 8, 128, 64, dtype="f16"),
        # one short request decoding, LLaMA-3-8B's heads (latency only)
        _case("attend_decode_1", "attend", 1, 500, 1, 32, 8, 128, 16),
        # one request behind a very long document, Qwen2.5-72B's heads
        _case("attend_decode_1_long", "attend", 1, 131071, 1, 64, 8, 128, 64),
        # a wide decode batch of long requests, Qwen2.5-72B's heads
        _case("attend_decode_64", "attend", 64, 16384, 1, 64, 8, 128, 64),
        # drafted tokens being verified: up to four new tokens a request, as many key as query heads of 64, fp16
        _case("attend_verify_48_f16", "attend", 48, 5003, 4, 16, 16, 64, 32, dtype="f16"),
        # pieces of three prompts over what the cache holds of them already
        _case("attend_prompts_3", "attend", 3, 10007, 2047, 32, 8, 128, 16),
        # decoding requests with a piece of a prompt among them, seven query heads a key head
        _case("attend_mixed_16", "attend", 16, 4096, 500, 28, 4, 128, 128, mixed=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = ((32, 8), (64, 8), (28, 4), (16, 16), (8, 1), (40, 8), (5, 5))


def draw(rng):
    most = {c["op"]: max(_cost(x) for x in listed() if x["op"] == c["op"]) for c in listed()}
    while True:
        op = rng.choice(("append", "attend", "attend", "read"))
        hq, hkv = rng.choice(HEADS)
        if op == "read":
            new = 1
        elif rng.random() < 0.6:
            new = rng.choice((1, 1, 1, 2, 4, 7))
        else:
            new = _log_int(rng, 8, 2047)
        c = _case("", op, _log_int(rng, 1, 128), _log_int(rng, max(new, 8), 65536), new, hq, hkv, rng.choice((64, 128)),
                  rng.choice((16, 32, 64, 128)), rng.choice(("bf16", "bf16", "f16")), new > 1 and rng.random() < 0.3)
        # the plain attention pads all requests to the longest and to the most new tokens
        padded = c["requests"] * c["longest"] * max(2 * new * hq, hkv * c["d"])
        if _cost(c) <= most[op] and padded <= 4e9:
            del c["name"]
            return c


def _cost(case):
    w = work(case)
    return w["flops"] / 1.0e15 + w["bytes"] / 6.0e12


# --------------------------------------------------------- what a case fixes without its seed
def _new_tokens(case):
    """New tokens of each request, from the most down to about half of that."""
    n = case["new"]
    each = [n - n * ((3 * r) % 5) // 8 for r in range(case["requests"])]
    return [n if r % 8 == 0 else 1 for r in range(case["requests"])] if case["mixed"] else each


def _lengths(case):
    """Tokens of each request after the call, spread evenly from the new ones alone to the longest
    (one request: the longest; shuffled by the seed)."""
    r, lo, hi = case["requests"], case["new"], case["longest"]
    return [hi - (hi - lo) * i // max(1, r - 1) for i in range(r)]


def work(case):
    """Bytes and operations of one pass: each input read once, each output written once."""
    d, hq, hkv, page = case["d"], case["hq"], case["hkv"], case["page"]
    new, lens = _new_tokens(case), _lengths(case)
    t, keys, pages = sum(new), sum(lens), sum((n + page - 1) // page for n in lens)
    if case["op"] == "append":
        return {"bytes": 2 * t * hkv * d * 3 + 4 * len(lens), "flops": 2 * t * hkv * d * 3}
    if case["op"] == "read":
        return {"bytes": 2 * keys * hkv * d * 3 + 2 * pages * hkv + 4 * pages, "flops": 2 * keys * hkv * d}
    # new tokens see the keys up to their own; lengths are shuffled against the numbers of new tokens
    pairs = sum(new) * sum(lens) / len(lens) - sum(n * (n - 1) / 2 for n in new)
    return {"bytes": 2 * keys * hkv * d + 2 * pages * hkv + 4 * pages + 2 * 2 * t * hq * d + 4 * t * hq,
            "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------------------------ inputs
def _scale_bytes(amax):
    """The lowest exponents e with amax <= 448 * 2^e, as scale bytes (448 = 0.875 * 2^9)."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return (torch.where(amax > 0, e, LOWEST).clamp(LOWEST, HIGHEST) + STORED).to(torch.uint8)


def _encode(x, scale):
    """E4M3 codes of float32 x at the scale bytes `scale` (the same number of dimensions)."""
    y = (x * torch.exp2(STORED - scale.float())).clamp(-448.0, 448.0)
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    r, hq, hkv, d, page = case["requests"], case["hq"], case["hkv"], case["d"], case["page"]
    order = torch.randperm(r, generator=torch.Generator().manual_seed(seed))
    lens, new = torch.tensor(_lengths(case))[order], torch.tensor(_new_tokens(case))
    blocks = (lens + page - 1) // page
    pages = int(blocks.sum()) + 3
    perm = torch.randperm(pages, generator=g, device="cuda")[:pages - 3].to(torch.int32)
    table = torch.full((r, int(blocks.max())), -1, dtype=torch.int32)
    table[torch.arange(table.shape[1])[None] < blocks[:, None]] = perm.cpu()
    s = {"case": case, "block_table": table.cuda(), "lens": lens.to(torch.int32).cuda()}
    # keys after norm and rotation have a few strong channels, values are even; tokens differ in size
    strong = 1 + 5.0 * (torch.rand(hkv, 1, d, generator=g, device="cuda") < 0.04)
    for name, channel in (("k", strong), ("v", torch.ones_like(strong))):
        cache = torch.empty(pages, hkv, page, d, dtype=torch.uint8, device="cuda")
        scales = torch.empty(pages, hkv, dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 28) // (hkv * page * d))
        for a in range(0, pages, step):
            b = min(pages, a + step)
            x = torch.randn(b - a, hkv, page, d, generator=g, device="cuda") * channel
            x = (x * torch.exp(0.3 * torch.randn(b - a, 1, page, 1, generator=g, device="cuda"))).to(dt).float()
            scales[a:b] = _scale_bytes(x.abs().amax((2, 3)))
            cache[a:b] = _encode(x, scales[a:b, :, None, None])
        s[name + "_cache"], s[name + "_scales"] = cache, scales
    t = int(new.sum())
    starts = lens if case["op"] == "read" else new
    s["starts"] = torch.cat((torch.zeros(1, dtype=torch.long), starts.cumsum(0))).to(torch.int32).cuda()
    s["tokens"] = int(starts.sum())
    if case["op"] == "append":
        # the key and value parts of a fused projection's output
        x = torch.randn(t, 2 * hkv, d, generator=g, device="cuda") * torch.cat((strong, torch.ones_like(strong)))[:, 0]
        x = (x * torch.exp(0.3 * torch.randn(t, 1, 1, generator=g, device="cuda"))).to(dt)
        s["k"], s["v"] = x[:, :hkv], x[:, hkv:]
    elif case["op"] == "attend":
        # one query head in four attends sharply
        sharp = 1 + 2.0 * (torch.arange(hq, device="cuda") % 4 == 0)
        s["q"] = (torch.randn(t, hq, d, generator=g, device="cuda") * sharp[:, None] / 2).to(dt)
        s["scale"] = 1.0 / math.sqrt(d)
    return s


# ------------------------------------------------------------------------- the plain forms
def _request_of(starts, tokens):
    """The request of each row, and the row's place among that request's rows."""
    at = torch.arange(tokens, device="cuda")
    r = torch.searchsorted(starts[1:], at, right=True)
    return r, at - starts[r]


def _plain_append(s):
    case = s["case"]
    page = case["page"]
    starts, lens, table = s["starts"].long(), s["lens"].long(), s["block_table"].long()
    new = starts[1:] - starts[:-1]
    r, i = _request_of(starts, s["tokens"])
    position = lens[r] - new[r] + i
    to, at = table[r, position // page], position % page
    # the page that a request's new tokens continue, and the tokens that it held
    held = (lens - new) % page
    goes_on = table[torch.arange(len(lens), device="cuda"), (lens - new) // page][held > 0]
    held = held[held > 0]
    for name in ("k", "v"):
        x, cache, scales = s[name].float(), s[name + "_cache"], s[name + "_scales"]
        top = x.abs().amax(-1)
        need = torch.zeros(scales.shape, device="cuda").index_reduce_(0, to, top, "amax")
        grown = _scale_bytes(need)
        before = scales[goes_on]
        grown[goes_on] = torch.maximum(grown[goes_on], before)
        scales[to] = grown[to]
        # tokens held already, at the page's new scale
        old = cache[goes_on]
        kept = old.view(torch.float8_e4m3fn).float() * torch.exp2(before.float() - STORED)[:, :, None, None]
        kept = _encode(kept, grown[goes_on][:, :, None, None])
        before_new = (torch.arange(page, device="cuda") < held[:, None])[:, None, :, None]
        cache[goes_on] = torch.where(before_new, kept, old)
        cache[to, :, at] = _encode(x, grown[to][:, :, None])
    return _cache_of(s)


def _cache_of(s):
    """The updated cache: codes as the E4M3 values they are, scale bytes."""
    return {"k_cache": s["k_cache"].view(torch.float8_e4m3fn), "v_cache": s["v_cache"].view(torch.float8_e4m3fn),
            "k_scales": s["k_scales"], "v_scales": s["v_scales"]}


def _plain_read(s):
    case = s["case"]
    r, position = _request_of(s["starts"].long(), s["tokens"])
    page, at = s["block_table"].long()[r, position // case["page"]], position % case["page"]
    most = torch.finfo(DTYPES[case["dtype"]]).max
    out = {}
    for name in ("k", "v"):
        x = s[name + "_cache"][page, :, at].view(torch.float8_e4m3fn).float()
        x = x * torch.exp2(s[name + "_scales"][page].float() - STORED)[..., None]
        out[name] = x.clamp(-most, most).to(DTYPES[case["dtype"]])
    return out


def _plain_attend(s):
    case = s["case"]
    r, hkv, d, most = case["requests"], case["hkv"], case["d"], case["new"]
    group, t = case["hq"] // hkv, s["tokens"]
    table, starts, lens = s["block_table"].long().clamp(min=0), s["starts"].long(), s["lens"].long()

    def pages_of(name):
        x = s[name + "_cache"][table].view(torch.float8_e4m3fn).float()
        x = x * torch.exp2(s[name + "_scales"][table].float() - STORED)[..., None, None]
        return x.transpose(1, 2).reshape(r, hkv, -1, d)

    q = s["q"].float().view(t, hkv, group, d) * s["scale"]
    new = starts[1:] - starts[:-1]
    request, place = _request_of(starts, t)
    padded = (starts[:-1, None] + torch.arange(most, device="cuda")).clamp(max=t - 1)
    qs = q[padded].permute(0, 2, 1, 3, 4).reshape(r, hkv, most * group, d)
    x = (qs @ pages_of("k").transpose(2, 3)).view(r, hkv, most, group, -1)
    seen = (lens - new)[:, None] + torch.arange(most, device="cuda") + 1
    seen = torch.minimum(seen, lens[:, None])
    hidden = torch.arange(x.shape[-1], device="cuda") >= seen[:, :, None]
    x = x.masked_fill_(hidden[:, None, :, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.view(r, hkv, most * group, -1) @ pages_of("v")).view(r, hkv, most, group, d)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + torch.log(total))[..., 0]
    return {"o": o.permute(0, 2, 1, 3, 4)[request, place].reshape(t, -1, d).to(DTYPES[case["dtype"]]),
            "lse": lse.permute(0, 2, 1, 3)[request, place].reshape(t, -1)}


# -------------------------------------------------------------------------------- one pass
def _own(s):
    from bit_weight_quantized_wq_gb300 import binding as wq

    case = s["case"]
    if case["op"] == "append":
        wq.kv_append_e4m3(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["block_table"],
                          s["lens"], q_start=s["starts"], max_new=case["new"])
        return _cache_of(s)
    if case["op"] == "read":
        k, v = wq.kv_read_e4m3(s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["block_table"], s["starts"],
                               s["tokens"], dtype=DTYPES[case["dtype"]])
        return {"k": k, "v": v}
    o, lse = wq.attn_e4m3(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["block_table"], s["lens"],
                          q_start=s["starts"], max_new=case["new"], scale=s["scale"])
    return {"o": o, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "read": _plain_read, "attend": _plain_attend}[state["case"]["op"]](state)


# ------------------------------------------------------------------------- in 64 bits
def _value_table():
    """The 256 values of E4M3: 1.mmm * 2^(e - 7), 0.mmm * 2^-6 where e is 0; 0x7f and 0xff are NaN."""
    def value(c):
        e, m = (c >> 3) & 15, c & 7
        x = math.ldexp(8 + m, e - 10) if e else math.ldexp(m, -9)
        return math.nan if c & 127 == 127 else -x if c & 128 else x
    return torch.tensor([value(c) for c in range(256)], dtype=torch.float64, device="cuda")


def _to_grid(y):
    """float64 y rounded to E4M3, ties to even: steps of 2^-3 of a value's binade, of 2^-9 below 2^-6."""
    y = y.clamp(-448.0, 448.0)
    step = torch.exp2((torch.frexp(y)[1] - 1).clamp(min=-6).double() - 3)
    return torch.round(y / step) * step


def _exact_append(s):
    """One request and one page of it at a time."""
    page, value = s["case"]["page"], _value_table()
    starts, lens, table = s["starts"].tolist(), s["lens"].tolist(), s["block_table"].tolist()
    out = {}
    for name in ("k", "v"):
        codes, scales = s[name + "_cache"].long(), s[name + "_scales"].clone()
        cache = value[codes]
        for r, n in enumerate(lens):
            first = n - (starts[r + 1] - starts[r])
            for block in range(first // page, (n + page - 1) // page):
                lo, hi, p = max(first, block * page), min(n, (block + 1) * page), table[r][block]
                x = s[name][starts[r] + lo - first:starts[r] + hi - first].double().transpose(0, 1)      # [hkv, tokens, d]
                top = x.abs().amax((1, 2))
                e = torch.ceil(torch.log2(top / 448.0))
                e = torch.where(top > 448.0 * torch.exp2(e), e + 1, torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e))
                e = torch.where(top > 0, e, LOWEST).clamp(LOWEST, HIGHEST)
                held = lo - block * page
                if held:
                    was = scales[p].double() - STORED
                    e = torch.maximum(e, was)
                    cache[p, :, :held] = _to_grid(cache[p, :, :held] * torch.exp2(was - e)[:, None, None])
                cache[p, :, held:held + hi - lo] = _to_grid(x * torch.exp2(-e)[:, None, None])
                scales[p] = (e + STORED).to(torch.uint8)
        out[name + "_cache"], out[name + "_scales"] = cache, scales
    return {k: out[k] for k in ("k_cache", "v_cache", "k_scales", "v_scales")}


def _request_pages(s, name, r, h, value):
    """Keys or values of one head of a request, in order: [tokens in its pages, d]."""
    blocks = -(-int(s["lens"][r]) // s["case"]["page"])
    p = s["block_table"][r, :blocks].long()
    x = value[s[name + "_cache"][p, h].long()] * torch.exp2(s[name + "_scales"][p, h].double() - STORED)[:, None, None]
    return x.reshape(-1, s["case"]["d"])


def _exact_read(s):
    case, value = s["case"], _value_table()
    starts = s["starts"].tolist()
    out = {n: torch.empty(s["tokens"], case["hkv"], case["d"], dtype=torch.float64, device="cuda") for n in ("k", "v")}
    for name, x in out.items():
        for r in range(case["requests"]):
            for h in range(case["hkv"]):
                x[starts[r]:starts[r + 1], h] = _request_pages(s, name, r, h, value)[:starts[r + 1] - starts[r]]
    return out


def _exact_attend(s):
    case, value = s["case"], _value_table()
    group = case["hq"] // case["hkv"]
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    o = torch.empty(s["tokens"], case["hq"], case["d"], dtype=torch.float64, device="cuda")
    lse = torch.empty(s["tokens"], case["hq"], dtype=torch.float64, device="cuda")
    for r in range(case["requests"]):
        a, b, n = starts[r], starts[r + 1], lens[r]
        last = torch.arange(n - (b - a), n, device="cuda")
        for h in range(case["hkv"]):
            mine = slice(h * group, (h + 1) * group)
            ks, vs = (_request_pages(s, name, r, h, value)[:n] for name in ("k", "v"))
            score = torch.einsum("tgd,jd->tgj", s["q"][a:b, mine].double(), ks) * s["scale"]
            score = torch.where(torch.arange(n, device="cuda") <= last[:, None, None], score, float("-inf"))
            lse[a:b, mine] = torch.logsumexp(score, -1)
            o[a:b, mine] = torch.einsum("tgj,jd->tgd", torch.softmax(score, -1), vs)
    return {"o": o, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "attend": _exact_attend}[case["op"]](s)

"""Cases and plain forms of the attention-block operators beside the quantized layers.

Three operators of a served decoder's attention block, in the order a token meets them:

- ``adapt``: low-rank adapters of many requests at once beside a shared projection (the
  projection's output given, or the projection itself in INT4 g128 / MXFP4 in the same call);
- ``rotate``: the norm of every query and key head and the rotation by position in one pass,
  keys and values written to their places in a cache kept in pages;
- ``attend``: attention of a batch whose requests share a long prefix, over that cache.

``run`` computes them in elementary torch operations in float32, rounded once at the end, or,
with ``own`` set, through ``bit_weight_quantized_wq_gb300.binding``.  ``exact`` computes the same
outputs in float64, written separately from the plain forms.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------- the cases
def _rotate(name, tokens, hq, hkv, d, rot, page, interleaved=False, norm=True, cache=True, dtype="bf16"):
    return {"name": name, "op": "rotate", "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "rot": rot, "page": page,
            "interleaved": interleaved, "norm": norm, "cache": cache, "dtype": dtype}


def _attend(name, requests, prefix, suffix, new, hq, hkv, d, page, dtype="bf16"):
    return {"name": name, "op": "attend", "requests": requests, "prefix": prefix, "suffix": suffix, "new": new, "hq": hq,
            "hkv": hkv, "d": d, "page": page, "dtype": dtype}


def _adapt(name, rows, k, n, rank, adapters, requests, base="given", dtype="bf16"):
    return {"name": name, "op": "adapt", "rows": rows, "k": k, "n": n, "rank": rank, "adapters": adapters,
            "requests": requests, "base": base, "dtype": dtype}


def listed():
    return [
        # one request decoding: a single token of LLaMA-3-8B's heads (latency only)
        _rotate("rotate_decode_1", 1, 32, 8, 128, 128, 16),
        # a decode batch of a model with as many key as query heads, half of each head rotated in
        # adjacent pairs, no norms, fp16
        _rotate("rotate_decode_61_f16", 61, 16, 16, 64, 32, 32, interleaved=True, norm=False, dtype="f16"),
        # a prefill chunk without a cache (keys returned as a tensor), odd length
        _rotate("rotate_chunk_2047", 2047, 32, 8, 128, 128, 16, cache=False),
        # a long prefill of Qwen2.5-72B's heads into the cache
        _rotate("rotate_prefill_8192", 8192, 64, 8, 128, 128, 64),
        # two requests behind a short system prompt (latency only)
        _attend("attend_decode_2", 2, 500, 40, 1, 32, 8, 128, 16),
        # the ordinary decode batch: 32 requests of LLaMA-3-8B's heads on an 8k shared document
        _attend("attend_decode_32", 32, 8192, 700, 1, 32, 8, 128, 16),
        # drafted tokens being verified: up to four new tokens a request, heads of 64, fp16, odd lengths
        _attend("attend_verify_48_f16", 48, 5003, 333, 4, 16, 16, 64, 32, dtype="f16"),
        # a wide batch of Qwen2.5-72B's heads on a 32k shared prefix
        _attend("attend_decode_256", 256, 32768, 1024, 1, 64, 8, 128, 64),
        # three requests, each with an adapter of its own, on a square projection (latency only)
        _adapt("adapt_decode_3", 3, 4096, 4096, 16, 8, 3),
        # a full decode batch on the fused gate+up projection, 48 adapters resident
        _adapt("adapt_decode_64", 64, 4096, 28672, 32, 48, 64),
        # the INT4 fused QKV projection with adapters in one call
        _adapt("adapt_int4_decode_16", 16, 4096, 6144, 16, 16, 16, base="int4_g128"),
        # prompts of eleven requests in one prefill batch, Qwen2.5-72B's O projection
        _adapt("adapt_prefill_4001", 4001, 8192, 8192, 64, 8, 11),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


HEADS = ((32, 8), (64, 8), (28, 4), (16, 16), (8, 1), (40, 8), (5, 5))


def draw(rng):
    most = {c["op"]: max(_cost(x) for x in listed() if x["op"] == c["op"]) for c in listed()}
    while True:
        op = rng.choice(("rotate", "attend", "adapt"))
        hq, hkv = rng.choice(HEADS)
        dtype = rng.choice(("bf16", "bf16", "f16"))
        page = rng.choice((16, 32, 64, 128))
        if op == "rotate":
            d = rng.choice((64, 128, 128, 256))
            c = _rotate("", _log_int(rng, 1, 8192), hq, hkv, d, rng.choice((d, d, d // 2, d // 4)), page,
                        rng.random() < 0.4, rng.random() < 0.7, rng.random() < 0.7, dtype)
        elif op == "attend":
            new = rng.choice((1, 1, 1, 2, 4, 7))
            prefix = 0 if rng.random() < 0.05 else _log_int(rng, 16, 32768)
            c = _attend("", _log_int(rng, 1, 256), prefix, _log_int(rng, max(new, 8), 2048), new, hq, hkv,
                        rng.choice((64, 128)), page, dtype)
        else:
            base = rng.choice(("given", "given", "int4_g128", "mxfp4"))
            rows = _log_int(rng, 1, 4096)
            c = _adapt("", rows, 128 * _log_int(rng, 4, 64), _log_int(rng, 256, 28672), 8 * rng.randint(1, 8),
                       _log_int(rng, 1, 64), min(rows, _log_int(rng, 1, 256)), base,
                       "bf16" if base != "given" else dtype)
        if _cost(c) <= most[op]:
            del c["name"]
            return c


def _cost(case):
    w = work(case)
    return w["flops"] / 1.5e15 + w["bytes"] / 6.0e12


# --------------------------------------------------------- what a case fixes without its seed
def _new_tokens(case):
    """New tokens of each request: 1 .. new."""
    return [1 + (5 * r) % case["new"] for r in range(case["requests"])]


def _suffix_lengths(case):
    """Own lengths, spread evenly from the new tokens to the longest (shuffled by the seed)."""
    r, lo, hi = case["requests"], case["new"], case["suffix"]
    return [hi - (hi - lo) * i // max(1, r - 1) for i in range(r)]


def _ranks(case):
    """The adapters' own ranks: the largest, every third adapter half of it (a multiple of 8)."""
    r = case["rank"]
    return [max(8, r // 16 * 8) if a % 3 == 2 else r for a in range(case["adapters"])]


def _request_adapters(case):
    """The adapter of each request; every ninth request has none."""
    return [-1 if i % 9 == 8 else i % case["adapters"] for i in range(case["requests"])]


def _request_rows(case):
    """Rows of each request: one each, the rest spread unevenly (a batch of prompts)."""
    rows, n = case["rows"], case["requests"]
    weight = [1 + (7 * i) % 5 for i in range(n)]
    left = rows - n
    got = [1 + left * w // sum(weight) for w in weight]
    got[0] += rows - sum(got)
    return got


def work(case):
    """Bytes and operations of one pass: each input read once, each output written once."""
    if case["op"] == "rotate":
        t, d = case["tokens"], case["d"]
        heads = case["hq"] + (2 if case["cache"] else 1) * case["hkv"]
        return {"bytes": 2 * 2 * t * heads * d + 4 * t * case["rot"] + 8 * t,
                "flops": t * (case["hq"] + case["hkv"]) * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    if case["op"] == "attend":
        d, hq, hkv = case["d"], case["hq"], case["hkv"]
        new, lens = _new_tokens(case), _suffix_lengths(case)
        t = sum(new)
        keys = case["prefix"] + sum(lens)
        pairs = t * case["prefix"] + sum(new) * sum(lens) / len(lens)
        return {"bytes": 2 * 2 * keys * hkv * d + 2 * 2 * t * hq * d + 4 * t * hq, "flops": 4 * d * hq * pairs}
    m, k, n = case["rows"], case["k"], case["n"]
    ranks, rows, who = _ranks(case), _request_rows(case), _request_adapters(case)
    used = sorted(set(a for a in who if a >= 0))
    flops = sum(2 * r * ranks[a] * (k + n) for r, a in zip(rows, who) if a >= 0)
    bytes_ = 2 * m * (k + n) + 2 * sum(ranks[a] for a in used) * (k + n)
    if case["base"] == "given":
        bytes_ += 2 * m * n
    else:
        bytes_ += n * k * 17 // 32
        flops += 2 * m * n * k
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------------------------------ inputs
def _pages(g, tokens, page):
    """A permutation of just enough pages (and three more) for `tokens` tokens."""
    n = (tokens + page - 1) // page
    return n + 3, torch.randperm(n + 3, generator=g, device="cuda")[:n].to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    s = {"case": case}
    if case["op"] == "rotate":
        t, hq, hkv, d, page = case["tokens"], case["hq"], case["hkv"], case["d"], case["page"]
        # Q, K and V as a fused projection leaves them, with outlying channels before the norms
        x = normal(t, (hq + 2 * hkv) * d) * (1 + 9 * (torch.rand((hq + 2 * hkv) * d, generator=g, device="cuda") < 0.01)).to(dt)
        s["q"] = x[:, :hq * d].view(t, hq, d)
        s["k"] = x[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
        s["v"] = x[:, (hq + hkv) * d:].view(t, hkv, d)
        s["wq"], s["wk"] = (1 + normal(2, d, scale=0.1, dtype=torch.float32)).to(dt) if case["norm"] else (None, None)
        most = 32768
        freq = 1e6 ** (-torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
        angle = torch.arange(most, device="cuda", dtype=torch.float64)[:, None] * freq
        s["table"] = torch.cat((angle.cos(), angle.sin()), 1).float()
        if t < 256:      # decode: one token of each request, at its own place
            s["positions"] = torch.randint(0, most, (t,), generator=g, device="cuda").to(torch.int32)
        else:            # prompts: consecutive places
            s["positions"] = ((torch.arange(t, device="cuda") + torch.randint(0, most, (1,), generator=g, device="cuda")) % most).to(torch.int32)
        if case["cache"]:
            pages, order = _pages(g, t, page)
            i = torch.arange(t, device="cuda")
            s["slots"] = (order[i // page] * page + i % page).to(torch.int32)
            s["k_cache"], s["v_cache"] = normal(pages, hkv, page, d), normal(pages, hkv, page, d)
    elif case["op"] == "attend":
        r, hq, hkv, d, page = case["requests"], case["hq"], case["hkv"], case["d"], case["page"]
        new = torch.tensor(_new_tokens(case))
        order = torch.randperm(r, generator=torch.Generator().manual_seed(seed))
        lens = torch.tensor(_suffix_lengths(case))[order]
        blocks = (lens + page - 1) // page
        prefix_blocks = (case["prefix"] + page - 1) // page
        total = int(blocks.sum()) + prefix_blocks
        pages, perm = _pages(g, total * page, page)
        s["prefix_pages"] = perm[:prefix_blocks].contiguous()
        width = (case["suffix"] + page - 1) // page
        table = torch.full((r, width), -1, dtype=torch.int32)
        table[torch.arange(width)[None] < blocks[:, None]] = perm[prefix_blocks:].cpu()
        s["block_table"] = table.cuda()
        s["suffix_lens"] = lens.to(torch.int32).cuda()
        s["q_start"] = torch.cat((torch.zeros(1, dtype=torch.long), new.cumsum(0))).to(torch.int32).cuda()
        # normed and rotated queries and keys; one query head in four attends sharply
        s["q"] = normal(int(new.sum()), hq, d) * (1 + 2.0 * (torch.arange(hq, device="cuda") % 4 == 0))[:, None].to(dt)
        s["k_cache"], s["v_cache"] = normal(pages, hkv, page, d), normal(pages, hkv, page, d)
        s["scale"] = 1.0 / math.sqrt(d)
    else:
        m, k, n, rank, adapters = case["rows"], case["k"], case["n"], case["rank"], case["adapters"]
        s["x"] = normal(m, k)
        ranks = torch.tensor(_ranks(case), dtype=torch.int32)
        live = (torch.arange(rank)[None] < ranks[:, None]).cuda()
        s["a"] = normal(adapters, rank, k, scale=k ** -0.5) * live[:, :, None].to(dt)
        s["b"] = normal(adapters, n, rank, scale=0.1) * live[:, None, :].to(dt)
        s["ranks"] = ranks.cuda()
        s["scales"] = 0.5 + 1.5 * torch.rand(adapters, generator=g, device="cuda")
        shuffled = torch.randperm(adapters, generator=torch.Generator().manual_seed(seed)).tolist() + [-1]
        who = torch.tensor([shuffled[a] for a in _request_adapters(case)], dtype=torch.int32)
        s["adapter"] = who.repeat_interleave(torch.tensor(_request_rows(case))).cuda()
        if case["base"] == "given":
            s["base"] = normal(m, n)
        else:
            s["wq"] = torch.randint(-2 ** 31, 2 ** 31, (n, k // 8), generator=g, device="cuda").to(torch.int32)
            if case["base"] == "int4_g128":
                s["ws"] = (0.004 + 0.004 * torch.rand(n, k // 128, generator=g, device="cuda")).half()
                s["wz"] = torch.randint(6, 10, (n, k // 128), generator=g, device="cuda").half()
            else:
                s["ws"] = torch.randint(117, 121, (n, k // 32), generator=g, device="cuda").to(torch.uint8)
                s["wz"] = None
    return s


# ------------------------------------------------------------------------- the plain forms
def _head_norm(x, w):
    x = x.float()
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _turn(x, cos, sin, rot, interleaved):
    a = x[..., 0:rot:2] if interleaved else x[..., :rot // 2]
    b = x[..., 1:rot:2] if interleaved else x[..., rot // 2:rot]
    y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1 if interleaved else -2)
    return torch.cat((y.flatten(-2), x[..., rot:]), -1)


def _plain_rotate(s):
    case = s["case"]
    rot, dt = case["rot"], DTYPES[case["dtype"]]
    row = s["table"][s["positions"].long()][:, None]
    cos, sin = row[..., :rot // 2], row[..., rot // 2:]
    q = _turn(_head_norm(s["q"], s["wq"]), cos, sin, rot, case["interleaved"]).to(dt)
    k = _turn(_head_norm(s["k"], s["wk"]), cos, sin, rot, case["interleaved"]).to(dt)
    if not case["cache"]:
        return {"q": q, "k": k}
    page, at = s["slots"].long() // case["page"], s["slots"].long() % case["page"]
    s["k_cache"][page, :, at] = k
    s["v_cache"][page, :, at] = s["v"]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s):
    case = s["case"]
    r, p, hkv, d, most = case["requests"], case["prefix"], case["hkv"], case["d"], case["new"]
    group = case["hq"] // hkv
    t = s["q"].shape[0]
    q = s["q"].float().view(t, hkv, group, d) * s["scale"]
    # scores against the prefix, all tokens at once: [hkv, t, group, p]
    kp = s["k_cache"][s["prefix_pages"].long()].transpose(0, 1).reshape(hkv, -1, d)[:, :p].float()
    vp = s["v_cache"][s["prefix_pages"].long()].transpose(0, 1).reshape(hkv, -1, d)[:, :p].float()
    sp = (q.permute(1, 0, 2, 3).reshape(hkv, t * group, d) @ kp.transpose(1, 2)).view(hkv, t, group, p)
    # scores against each request's own keys, tokens padded to the most a request has
    start = s["q_start"].long()
    new = start[1:] - start[:-1]
    request = torch.searchsorted(start[1:], torch.arange(t, device="cuda"), right=True)
    place = torch.arange(t, device="cuda") - start[request]
    padded = (start[:-1, None] + torch.arange(most, device="cuda")).clamp(max=t - 1)
    table = s["block_table"].long()
    ks = s["k_cache"][table].transpose(1, 2).reshape(r, hkv, -1, d).float()
    vs = s["v_cache"][table].transpose(1, 2).reshape(r, hkv, -1, d).float()
    qs = q[padded].permute(0, 2, 1, 3, 4).reshape(r, hkv, most * group, d)
    ss = (qs @ ks.transpose(2, 3)).view(r, hkv, most, group, -1)
    seen = s["suffix_lens"].long()[:, None] - new[:, None] + torch.arange(most, device="cuda") + 1
    hidden = torch.arange(ss.shape[-1], device="cuda") >= seen[:, :, None]
    ss = ss.masked_fill(hidden[:, None, :, None], float("-inf"))
    of_token = ss.permute(0, 2, 1, 3, 4)[request, place]                        # [t, hkv, group, s]
    top = of_token.amax(-1)
    if p:
        top = torch.maximum(top, sp.amax(-1).transpose(0, 1))
    safe = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    es = torch.exp(of_token - safe[..., None])
    ep = torch.exp(sp - safe.transpose(0, 1)[..., None])
    total = es.sum(-1) + ep.sum(-1).transpose(0, 1)
    spread = torch.zeros(r, most, hkv, group, es.shape[-1], device="cuda")
    spread[request, place] = es
    os_ = (spread.permute(0, 2, 1, 3, 4).reshape(r, hkv, most * group, -1) @ vs).view(r, hkv, most, group, d)
    o = os_.permute(0, 2, 1, 3, 4)[request, place]
    o = o + (ep.reshape(hkv, t * group, p) @ vp).view(hkv, t, group, d).transpose(0, 1)
    o = o / torch.where(total > 0, total, torch.ones_like(total))[..., None]
    return {"o": o.reshape(t, hkv * group, d).to(DTYPES[case["dtype"]]),
            "lse": (safe + torch.log(total)).reshape(t, hkv * group)}


def _codes(wq):
    shift = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    return ((wq[:, :, None] >> shift) & 15).flatten(1)


def _dequantized(s):
    q = _codes(s["wq"])
    if s["case"]["base"] == "int4_g128":
        w = (q.float().view(q.shape[0], -1, 128) - s["wz"].float()[..., None]) * s["ws"].float()[..., None]
    else:
        value = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")[q.long()]
        w = value.view(q.shape[0], -1, 32) * torch.exp2(s["ws"].float() - 127)[..., None]
    return w.flatten(1)


def _plain_adapt(s):
    case = s["case"]
    x, adapter = s["x"].float(), s["adapter"].long()
    base = s["base"].float() if case["base"] == "given" else x @ _dequantized(s).t()
    # every adapter's product for every row, those that are not the row's own set to zero
    mine = adapter[:, None] == torch.arange(case["adapters"], device="cuda")
    v = (x @ s["a"].float().flatten(0, 1).t()).view(case["rows"], case["adapters"], case["rank"])
    v = (v * (mine * s["scales"])[..., None]).flatten(1)
    y = base + v @ s["b"].float().permute(0, 2, 1).flatten(0, 1)
    return {"y": y.to(DTYPES[case["dtype"]])}


# -------------------------------------------------------------------------------- one pass
def _own(s):
    from bit_weight_quantized_wq_gb300 import binding as wq

    case = s["case"]
    if case["op"] == "rotate":
        if case["cache"]:
            q = wq.qk_norm_rope_cache(s["q"], s["k"], s["v"], s["positions"], s["table"], s["k_cache"], s["v_cache"],
                                      s["slots"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS,
                                      interleaved=case["interleaved"])
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        q, k = wq.qk_norm_rope(s["q"], s["k"], s["positions"], s["table"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS,
                               interleaved=case["interleaved"])
        return {"q": q, "k": k}
    if case["op"] == "attend":
        o, lse = wq.attn_shared_prefix(s["q"], s["k_cache"], s["v_cache"], s["prefix_pages"], case["prefix"],
                                       s["block_table"], s["suffix_lens"], q_start=s["q_start"], max_new=case["new"],
                                       scale=s["scale"])
        return {"o": o, "lse": lse}
    if case["base"] == "given":
        return {"y": wq.lora_add(s["base"], s["x"], s["a"], s["b"], s["adapter"], s["scales"], ranks=s["ranks"])}
    return {"y": wq.gemm_w4a16_lora(case["base"], s["x"], s["wq"], s["ws"], s["wz"], s["a"], s["b"], s["adapter"],
                                    s["scales"], ranks=s["ranks"])}


def run(state):
    if own:
        return _own(state)
    return {"rotate": _plain_rotate, "attend": _plain_attend, "adapt": _plain_adapt}[state["case"]["op"]](state)


# ------------------------------------------------------------------------- in 64 bits
def _exact_rotate(s):
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    row = s["table"].double()[s["positions"].long()]
    turn = torch.complex(row[:, :half], row[:, half:])[:, None]

    def heads(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + EPS) * w.double()
        y = x.clone()
        first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, half), slice(half, rot))
        z = torch.complex(x[..., first], x[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    q, k = heads(s["q"], s["wq"]), heads(s["k"], s["wk"])
    if not case["cache"]:
        return {"q": q, "k": k}
    out = {"q": q}
    for name, new in (("k_cache", k), ("v_cache", s["v"].double())):
        pool = s[name].double().transpose(1, 2).flatten(0, 1)                  # [slots, hkv, d]
        pool[s["slots"].long()] = new
        out[name] = pool.view(-1, case["page"], case["hkv"], case["d"]).transpose(1, 2).contiguous()
    return out


def _exact_attend(s):
    case = s["case"]
    p, hkv, d = case["prefix"], case["hkv"], case["d"]
    group = case["hq"] // hkv
    t = s["q"].shape[0]
    start, lens, table = s["q_start"].tolist(), s["suffix_lens"].tolist(), s["block_table"].long()
    o = torch.empty(t, case["hq"], d, dtype=torch.float64, device="cuda")
    lse = torch.empty(t, case["hq"], dtype=torch.float64, device="cuda")
    for h in range(hkv):
        mine = slice(h * group, (h + 1) * group)
        q = s["q"][:, mine].double()
        kp = s["k_cache"][s["prefix_pages"].long(), h].reshape(-1, d)[:p].double()
        vp = s["v_cache"][s["prefix_pages"].long(), h].reshape(-1, d)[:p].double()
        score = torch.einsum("tgd,pd->tgp", q, kp) * s["scale"]
        lse_p = torch.logsumexp(score, -1)
        o_p = torch.einsum("tgp,pd->tgd", torch.softmax(score, -1), vp)
        del score
        for r in range(case["requests"]):
            a, b, n = start[r], start[r + 1], lens[r]
            ks = s["k_cache"][table[r], h].reshape(-1, d)[:n].double()
            vs = s["v_cache"][table[r], h].reshape(-1, d)[:n].double()
            score = torch.einsum("tgd,jd->tgj", q[a:b], ks) * s["scale"]
            last = torch.arange(n - (b - a), n, device="cuda")
            score = torch.where(torch.arange(n, device="cuda") <= last[:, None, None], score, float("-inf"))
            lse_s = torch.logsumexp(score, -1)
            both = torch.logaddexp(lse_p[a:b], lse_s)
            lse[a:b, mine] = both
            o[a:b, mine] = (torch.exp(lse_p[a:b] - both)[..., None] * o_p[a:b]
                            + torch.exp(lse_s - both)[..., None] * torch.einsum("tgj,jd->tgd", torch.softmax(score, -1), vs))
    return {"o": o, "lse": lse}


def _exact_adapt(s):
    case = s["case"]
    x = s["x"].double()
    if case["base"] == "given":
        y = s["base"].double()
    else:
        n, k = case["n"], case["k"]
        words = s["wq"].long() & 0xffffffff
        w = torch.empty(n, k, dtype=torch.float64, device="cuda")
        for i in range(8):
            code = (words >> (4 * i)) & 15
            if case["base"] == "int4_g128":
                w[:, i::8] = code.double()
            else:
                low, e = (code & 1).double(), ((code >> 1) & 3).double()
                size = torch.where(e > 0, torch.exp2(e - 1) * (1 + low / 2), low / 2)
                w[:, i::8] = torch.where(code >= 8, -size, size)
        if case["base"] == "int4_g128":
            w = (w - s["wz"].double().repeat_interleave(128, 1)) * s["ws"].double().repeat_interleave(128, 1)
        else:
            w = w * torch.exp2(s["ws"].double() - 127).repeat_interleave(32, 1)
        y = x @ w.t()
    for a, rank in enumerate(s["ranks"].tolist()):
        rows = torch.nonzero(s["adapter"] == a)[:, 0]
        if rows.numel():
            v = x[rows] @ s["a"][a, :rank].double().t()
            y[rows] += s["scales"][a].double() * (v @ s["b"][a, :, :rank].double().t())
    return {"y": y}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rotate": _exact_rotate, "attend": _exact_attend, "adapt": _exact_adapt}[case["op"]](s)

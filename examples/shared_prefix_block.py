"""One attention block of a served decoder, end to end: a system prompt is prefilled once, then
several requests, each with its own low-rank adapter, decode behind it.

    python examples/shared_prefix_block.py

A token's way through the block: quantized QKV projection with the request's adapter
(``gemm_w4a16_lora``), head norms, rotation and the write to the cache's pages
(``qk_norm_rope_cache``), attention over the shared prefix and the request's own pages
(``attn_shared_prefix``), quantized output projection with adapter.  ``reference`` computes the same
in float64 from the dequantized weights, and ``main`` compares the two.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_weight_quantized_wq_gb300 import binding as wq  # noqa: E402

EPS, PAGE = 1e-6, 16


class Block:
    """Weights, adapters, cache and page bookkeeping of the block."""

    def __init__(self, hidden=512, hq=8, hkv=2, d=64, adapters=3, rank=16, pages=64, max_pos=4096, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.hq, self.hkv, self.d = hidden, hq, hkv, d

        def normal(*shape, scale):
            return torch.randn(*shape, generator=g, device="cuda") * scale

        self.w = {"qkv": normal((hq + 2 * hkv) * d, hidden, scale=hidden ** -0.5), "o": normal(hidden, hq * d, scale=(hq * d) ** -0.5)}
        self.packed = {name: wq.quantize_int4_g128(w) for name, w in self.w.items()}
        self.a = {n: normal(adapters, rank, w.shape[1], scale=w.shape[1] ** -0.5).bfloat16() for n, w in self.w.items()}
        self.b = {n: normal(adapters, w.shape[0], rank, scale=0.1).bfloat16() for n, w in self.w.items()}
        self.scales = 0.5 + torch.rand(adapters, generator=g, device="cuda")
        self.q_norm, self.k_norm = (1 + normal(2, d, scale=0.1)).bfloat16()
        freq = 1e4 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
        angle = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * freq
        self.table = torch.cat((angle.cos(), angle.sin()), 1).float()
        self.k_cache = torch.zeros(pages, hkv, PAGE, d, dtype=torch.bfloat16, device="cuda")
        self.v_cache = torch.zeros_like(self.k_cache)
        self.free = list(range(pages))[::-1]

    def pages_for(self, tokens):
        return [self.free.pop() for _ in range((tokens + PAGE - 1) // PAGE)]

    def step(self, x, adapter, positions, slots, attend):
        """x [T, hidden] bf16 -> [T, hidden]; ``attend``: the page arguments of attn_shared_prefix."""
        hq, hkv, d = self.hq, self.hkv, self.d
        y = wq.gemm_w4a16_lora("int4_g128", x, *self.packed["qkv"], self.a["qkv"], self.b["qkv"], adapter, self.scales)
        q, k, v = y[:, :hq * d], y[:, hq * d:(hq + hkv) * d], y[:, (hq + hkv) * d:]
        q = wq.qk_norm_rope_cache(q.view(-1, hq, d), k.view(-1, hkv, d), v.view(-1, hkv, d), positions, self.table, self.k_cache,
                                  self.v_cache, slots, q_weight=self.q_norm, k_weight=self.k_norm, eps=EPS)
        o, _ = wq.attn_shared_prefix(q, self.k_cache, self.v_cache, **attend)
        return wq.gemm_w4a16_lora("int4_g128", o.view(-1, hq * d), *self.packed["o"], self.a["o"], self.b["o"], adapter, self.scales)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def serve(block, prompt, requests):
    """``prompt`` [P, hidden]: the shared prefix; ``requests``: list of (adapter, [S, hidden]) whose
    tokens come one a step.  Returns the outputs of every request's tokens, in their order."""
    P, R = prompt.shape[0], len(requests)
    longest = max(x.shape[0] for _, x in requests)
    prefix = block.pages_for(P)
    # the prompt as one request without a prefix: its tokens attend among themselves
    block.step(prompt, i32([-1] * P), i32(list(range(P))), i32([prefix[j // PAGE] * PAGE + j % PAGE for j in range(P)]),
               dict(prefix_pages=None, prefix_len=0, block_table=i32([prefix]), suffix_lens=i32([P]), q_start=i32([0, P]), max_new=P))
    own = [block.pages_for(x.shape[0]) for _, x in requests]
    width = max(len(p) for p in own)
    table = i32([p + [-1] * (width - len(p)) for p in own])
    out = [[] for _ in requests]
    for step in range(longest):
        live = [r for r in range(R) if step < requests[r][1].shape[0]]
        x = torch.stack([requests[r][1][step] for r in live])
        attend = dict(prefix_pages=i32(prefix), prefix_len=P, block_table=table[live].contiguous(), suffix_lens=i32([step + 1] * len(live)))
        y = block.step(x, i32([requests[r][0] for r in live]), i32([P + step] * len(live)),
                       i32([own[r][step // PAGE] * PAGE + step % PAGE for r in live]), attend)
        for i, r in enumerate(live):
            out[r].append(y[i])
    return [torch.stack(o) for o in out]


def reference(block, prompt, adapter, tokens):
    """A request's outputs in float64: the prompt without an adapter, then its tokens with its own."""
    hq, hkv, d = block.hq, block.hkv, block.d

    def dequantized(name):
        codes, scales, zeros = block.packed[name]
        q = torch.stack([(codes >> (4 * i)) & 15 for i in range(8)], -1).flatten(1).double()
        return (q - zeros.double().repeat_interleave(128, 1)) * scales.double().repeat_interleave(128, 1)

    def project(name, x, who):
        y = x @ dequantized(name).t()
        return y if who < 0 else y + block.scales[who].double() * (x @ block.a[name][who].double().t()) @ block.b[name][who].double().t()

    x = torch.cat((prompt, tokens)).double()
    P, n = prompt.shape[0], x.shape[0]
    y = torch.cat((project("qkv", x[:P], -1), project("qkv", x[P:], adapter)))

    def turned(h, w):
        h = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * w.double()
        c, s = block.table[:n, None, :d // 2].double(), block.table[:n, None, d // 2:].double()
        return torch.cat((h[..., :d // 2] * c - h[..., d // 2:] * s, h[..., d // 2:] * c + h[..., :d // 2] * s), -1)

    q = turned(y[:, :hq * d].view(n, hq, d), block.q_norm)
    k = turned(y[:, hq * d:(hq + hkv) * d].view(n, hkv, d), block.k_norm).repeat_interleave(hq // hkv, 1)
    v = y[:, (hq + hkv) * d:].view(n, hkv, d).repeat_interleave(hq // hkv, 1)
    score = torch.einsum("qhd,khd->hqk", q, k) * d ** -0.5
    score = score.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), float("-inf"))
    o = torch.einsum("hqk,khd->qhd", torch.softmax(score, -1), v).reshape(n, -1)
    return project("o", o[P:], adapter)


def main():
    block = Block()
    g = torch.Generator(device="cuda").manual_seed(1)
    prompt = torch.randn(75, block.hidden, generator=g, device="cuda").bfloat16()
    requests = [(r % 4 - 1, torch.randn(5 + 7 * r, block.hidden, generator=g, device="cuda").bfloat16()) for r in range(5)]
    worst = 0.0
    for (who, tokens), got in zip(requests, serve(block, prompt, requests)):
        want = reference(block, prompt, who, tokens)
        worst = max(worst, float((got.double() - want).norm() / want.norm()))
    print("largest relative error of a request: %.4f" % worst)
    # every tensor between the operators is bf16: about ten roundings of 2^-9 on the way
    assert worst < 0.02 and wq.read_error_flags() == 0
    return worst


if __name__ == "__main__":
    main()

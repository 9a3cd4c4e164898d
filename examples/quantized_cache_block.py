"""One attention block of a served decoder over an 8-bit cache: prompts come in pieces, beside requests
that decode already, and then all decode in one captured step.

    python examples/quantized_cache_block.py

A token's way through the block: quantized QKV projection (``gemm_w4a16``), head norms and rotation
(``qk_norm_rope``), keys and values to the cache's pages as E4M3 codes (``kv_append_e4m3``), attention over
the pages (``attn_e4m3``), quantized output projection.  The captured step has a fixed number of places;
a request that is done keeps its place with length 0, which writes nothing and reads nothing.
``reference`` computes the same in float64 from the dequantized weights with keys and values that are not
rounded, and ``main`` compares the two; ``handed_over`` reads a request's pages back in 16 bits.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_weight_quantized_wq_gb300 import binding as wq  # noqa: E402

EPS, PAGE = 1e-6, 32


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Block:
    """Weights and cache of the block; places 0 .. R - 1, each with the pages of its request."""

    def __init__(self, requests, longest, hidden=512, hq=8, hkv=2, d=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.hidden, self.hq, self.hkv, self.d = hidden, hq, hkv, d

        def normal(*shape, scale):
            return torch.randn(*shape, generator=g, device="cuda") * scale

        shapes = {"qkv": ((hq + 2 * hkv) * d, hidden), "o": (hidden, hq * d)}
        self.packed = {n: wq.quantize_int4_g128(normal(*s, scale=s[1] ** -0.5)) for n, s in shapes.items()}
        self.q_norm, self.k_norm = (1 + normal(2, d, scale=0.1)).bfloat16()
        freq = 1e4 ** (-torch.arange(0, d, 2, device="cuda", dtype=torch.float64) / d)
        angle = torch.arange(longest, device="cuda", dtype=torch.float64)[:, None] * freq
        self.table = torch.cat((angle.cos(), angle.sin()), 1).float()
        blocks = (longest + PAGE - 1) // PAGE
        codes = (requests * blocks, hkv, PAGE, d)
        # codes of K and V, then the scales; never initialised: what no token was written to is not used
        self.cache = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in (codes, codes, codes[:2], codes[:2])]
        self.block_table = torch.randperm(codes[0], generator=g, device="cuda").int().view(requests, blocks)

    def step(self, x, positions, lens, q_start=None, max_new=1):
        """x [T, hidden] bf16 -> [T, hidden]; ``lens``: tokens of each place with this call's."""
        hq, hkv, d = self.hq, self.hkv, self.d
        y = wq.gemm_w4a16("int4_g128", x, *self.packed["qkv"]).view(-1, hq + 2 * hkv, d)
        q, k = wq.qk_norm_rope(y[:, :hq], y[:, hq:hq + hkv], positions, self.table, self.q_norm, self.k_norm, EPS)
        wq.kv_append_e4m3(k, y[:, hq + hkv:], *self.cache, self.block_table, lens, q_start, max_new)
        o, _ = wq.attn_e4m3(q, *self.cache, self.block_table, lens, q_start, max_new)
        return wq.gemm_w4a16("int4_g128", o.view(-1, hq * d), *self.packed["o"])

    def handed_over(self, place, tokens):
        """Keys and values [tokens, hkv, d] of a place in bf16, for a 16-bit cache."""
        return wq.kv_read_e4m3(*self.cache, self.block_table[place:place + 1], i32([0, tokens]), tokens)


def prefill(block, xs, prompts, piece):
    """The prompts' tokens, up to ``piece`` of each a call; places that have none left have none of the call's rows."""
    done, out = [0] * len(xs), [[] for _ in xs]
    while done != prompts:
        news = [min(piece, p - n) for p, n in zip(prompts, done)]
        starts = [sum(news[:r]) for r in range(len(news) + 1)]
        x = torch.cat([x[n:n + m] for x, n, m in zip(xs, done, news)])
        positions = [n + i for n, m in zip(done, news) for i in range(m)]
        done = [n + m for n, m in zip(done, news)]
        y = block.step(x, i32(positions), i32(done), i32(starts), max(news))
        for r in range(len(xs)):
            out[r].append(y[starts[r]:starts[r + 1]])
    return out


def decode(block, xs, prompts):
    """A token of every place a step, in one captured graph."""
    R = len(xs)
    x = torch.zeros(R, block.hidden, dtype=torch.bfloat16, device="cuda")
    positions, lens = i32([0] * R), i32([0] * R)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.step(x, positions, lens)                   # workspaces; all places of length 0: nothing is written
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        y = block.step(x, positions, lens)
    out = [[] for _ in xs]
    for step in range(max(t.shape[0] - p for t, p in zip(xs, prompts))):
        at = [p + step if p + step < t.shape[0] else -1 for t, p in zip(xs, prompts)]
        for r in range(R):
            if at[r] >= 0:
                x[r].copy_(xs[r][at[r]])
        positions.copy_(i32([max(n, 0) for n in at])), lens.copy_(i32([n + 1 for n in at]))
        graph.replay()
        for r in range(R):
            if at[r] >= 0:
                out[r].append(y[r:r + 1].clone())
    return out


def reference(block, x):
    """Outputs, keys and values of a request's tokens in float64."""
    hq, hkv, d, n = block.hq, block.hkv, block.d, x.shape[0]

    def project(name, x):
        codes, scales, zeros = block.packed[name]
        q = torch.stack([(codes >> (4 * i)) & 15 for i in range(8)], -1).flatten(1).double()
        return x @ ((q - zeros.double().repeat_interleave(128, 1)) * scales.double().repeat_interleave(128, 1)).t()

    def turned(h, w):
        h = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * w.double()
        c, s = block.table[:n, None, :d // 2].double(), block.table[:n, None, d // 2:].double()
        return torch.cat((h[..., :d // 2] * c - h[..., d // 2:] * s, h[..., d // 2:] * c + h[..., :d // 2] * s), -1)

    y = project("qkv", x.double()).view(n, -1, d)
    q, k, v = turned(y[:, :hq], block.q_norm), turned(y[:, hq:hq + hkv], block.k_norm), y[:, hq + hkv:]
    wide = lambda t: t.repeat_interleave(hq // hkv, 1)   # noqa: E731
    score = torch.einsum("qhd,khd->hqk", q, wide(k)) * d ** -0.5
    score = score.masked_fill(torch.ones(n, n, device="cuda").triu(1).bool(), float("-inf"))
    o = torch.einsum("hqk,khd->qhd", torch.softmax(score, -1), wide(v)).reshape(n, -1)
    return project("o", o), k, v


def main():
    prompts, answers = [75, 1, 130, 40], [9, 30, 17, 1]
    longest = max(p + n for p, n in zip(prompts, answers))
    block = Block(len(prompts), longest)
    g = torch.Generator(device="cuda").manual_seed(1)
    xs = [torch.randn(p + n, block.hidden, generator=g, device="cuda").bfloat16() for p, n in zip(prompts, answers)]
    out = [a + b for a, b in zip(prefill(block, xs, prompts, 50), decode(block, xs, prompts))]
    off = lambda got, want: float((got.double() - want).norm() / want.norm())   # noqa: E731
    worst = worst_kv = 0.0
    for r, x in enumerate(xs):
        y, k, v = reference(block, x)
        got_k, got_v = block.handed_over(r, x.shape[0])
        worst = max(worst, off(torch.cat(out[r]), y))
        worst_kv = max(worst_kv, off(got_k, k), off(got_v, v))
    print("largest relative error of a request: %.4f; of its keys or values: %.4f" % (worst, worst_kv))
    # a code is off by 2^-4 of its value at most, 0.026 on average over a binade; in the output the keys' and
    # the values' add up as independent errors, some 0.037, with about ten roundings of 2^-9 on the way
    assert worst_kv < 2 ** -4 and worst < 2 ** -4 and wq.read_error_flags() == 0
    return worst


if __name__ == "__main__":
    main()

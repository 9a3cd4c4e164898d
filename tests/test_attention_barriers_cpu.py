"""A model of the attention kernel's barriers, run in random order on the CPU.

The kernel's warps hand tiles to one another through barriers whose waits are by parity: such a wait
is only sound while the waiting warp is at most one phase behind or ahead, and a slip shows as a product
on a tile that is still loading, rarely and only on some timings.  The model runs the warps' loops as
coroutines in random order, with copies and products that land late and out of order, over random
items; it checks at each use that the tile is the one the warp means, that no barrier gets an arrival
too many, and that all warps come to their end.  Ring sizes and the products' lead are read from the
kernel's source.  Two protocols that are wrong have to be caught."""
import os
import random
import re

import pytest

from bit_weight_quantized_wq_gb300 import build as wqbuild

SOURCE = open(os.path.join(wqbuild.CSRC, "attn.cu")).read()


def _constants():
    stages = re.search(r"kStages = D == 128 \? (\d+) : (\d+);", SOURCE)
    items = re.search(r"constexpr int kItems = (\d+);", SOURCE)
    lead = re.search(r"k_ahead\(bool rows\) \{ return rows \? (\d+) : (\d+); \}", SOURCE)
    return [int(v) for v in stages.groups()], int(items.group(1)), [int(v) for v in lead.groups()]


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase, self.bytes = count, count, 0, 0

    def arrive(self):
        assert self.left > 0, "an arrival too many"
        self.left -= 1
        self.check()

    def land(self):                                   # copied bytes
        self.bytes -= 1
        self.check()

    def check(self):
        if self.left == 0 and self.bytes == 0:
            self.phase, self.left = self.phase + 1, self.count

    def passed(self, parity):
        return (self.phase & 1) != (parity & 1)


def simulate(seed, stages, ring_items, lead, lanes_skip_slots=False, wait_for_products=True, steps=400000):
    rnd = random.Random(seed)
    items = [(rnd.randint(1, rnd.choice((1, 2, 5, 12))), rnd.random() < 0.4) for _ in range(rnd.randint(1, 12))]   # tiles, rows mode
    bars = lambda count, n: [Barrier(count) for _ in range(n)]   # noqa: E731
    full, empty = [bars(1, stages) for _ in "KV"], [bars(2, stages) for _ in "KV"]
    q_full, q_empty = bars(1, 2), bars(2, 2)
    s_full, p_full = [bars(1, 2) for _ in range(2)], [bars(1, 2) for _ in range(2)]
    pv_done, o_full, o_empty = bars(1, 2), bars(1, 2), bars(1, 2)
    item_full, item_empty = bars(1, ring_items), bars(6, ring_items)
    ring, kv, q = [None] * ring_items, [[None] * stages for _ in "KV"], [None] * 2
    scores, weights = [[None] * 2 for _ in range(2)], [[None] * 2 for _ in range(2)]
    out, products, late, actors, ended = [[], []], [0, 0], [], [], []

    def later(f):
        late.append([rnd.randint(1, 60) if rnd.random() < 0.9 else rnd.randint(60, 700), f])

    def next_item(i):
        while not item_full[i % ring_items].passed(i // ring_items):
            yield
        assert ring[i % ring_items] == i, "an item that is not this one"

    def scheduler():
        for i in range(len(items) + 1):
            while not item_empty[i % ring_items].passed((i // ring_items) ^ 1):
                yield
            ring[i % ring_items] = i if i < len(items) else None
            item_full[i % ring_items].arrive()
        ended.append("scheduler")

    def copies(rg):                                   # rg 0: K (and Q), 1: V
        n_copied = n_q = 0
        for i, (n, rows) in enumerate(items):
            yield from next_item(i)
            for half in range((2 if rows else 1) if rg == 0 else 0):
                s = n_q & 1
                while not q_empty[s].passed((n_q >> 1) ^ 1):
                    yield
                q_full[s].bytes += 1
                q_full[s].arrive()

                def land(s=s, what=(i, half)):
                    q[s] = what
                    q_full[s].land()
                later(land)
                n_q += 1
            for j in range(n):
                s = n_copied % stages
                while not empty[rg][s].passed((n_copied // stages) ^ 1):
                    yield
                full[rg][s].bytes += 1
                full[rg][s].arrive()
                kv[rg][s] = "loading"

                def land(s=s, what=(i, j)):
                    kv[rg][s] = what
                    full[rg][s].land()
                later(land)
                n_copied += 1
            item_empty[i % ring_items].arrive()
        ended.append("copies")

    def tensor_core(queue):                           # one lane's products, in order
        while True:
            if queue:
                for _ in range(rnd.randint(1, 12)):
                    yield
                queue.pop(0)()
            yield

    def given_back(rg, slot, rows):                   # by each lane, or twice by the tile's own
        for _ in range(2 if lanes_skip_slots and not rows else 1):
            empty[rg][slot].arrive()

    def product_warp(l):
        seen, n_q, n_out, n_s, n_p, queue = [0, 0], 0, 0, 0, 0, []
        actors.append(tensor_core(queue))
        for i, (n, rows) in enumerate(items):
            yield from next_item(i)
            halves, ahead = (2, lead[0]) if rows else (1, lead[1])
            for a in range(halves):
                while not q_full[(n_q + a) & 1].passed((n_q + a) >> 1):
                    yield
            my_q = (n_q + (l if rows else 0)) & 1
            order = []
            for j in range(n + ahead):
                order += [(1, j - ahead)] if j >= ahead else []
                order += [(0, j)] if j < n else []
            for rg, j in order:
                slot, phase = seen[rg] % stages, seen[rg] // stages
                seen[rg] += 1
                mine = rows or ((j ^ i) & 1) == l
                if not mine and lanes_skip_slots:
                    continue
                while not full[rg][slot].passed(phase):
                    yield
                if not mine:                          # the other lane's tile: waited for and given back all the same
                    assert kv[rg][slot] == (i, j)
                    empty[rg][slot].arrive()
                    continue
                if rg == 0:
                    def run(i=i, j=j, slot=slot, rows=rows, b=n_s & 1, my_q=my_q):
                        assert q[my_q] == (i, l if rows else 0) and kv[0][slot] == (i, j), "a product on the wrong tile"
                        scores[l][b] = (i, j)
                        s_full[l][b].arrive()
                        given_back(0, slot, rows)
                    n_s += 1
                else:
                    first, last = (j == 0 if rows else j < 2), j + (1 if rows else 2) >= n
                    if first:
                        while not o_empty[l].passed(n_out ^ 1):
                            yield
                        n_out += 1
                    while not p_full[l][n_p & 1].passed(n_p >> 1):
                        yield

                    def run(i=i, j=j, slot=slot, rows=rows, b=n_p & 1, first=first, last=last):
                        assert kv[1][slot] == (i, j) and weights[l][b] == scores[l][b] == (i, j), "a product on the wrong tile"
                        if first:
                            out[l] = []
                        out[l].append((i, j))
                        products[l] += 1
                        pv_done[l].arrive()
                        if last:
                            o_full[l].arrive()
                        given_back(1, slot, rows)
                    n_p += 1
                queue.append(run)

            def give_back(slots=tuple((n_q + a) & 1 for a in range(halves))):
                for s in slots:
                    q_empty[s].arrive()
            queue.append(give_back)
            n_q += halves
            item_empty[i % ring_items].arrive()
        while queue:
            yield
        ended.append("products")

    def softmax(l):
        n, n_out, v_end = 0, 0, 0
        for i, (tiles, rows) in enumerate(items):
            yield from next_item(i)
            mine = list(range(tiles)) if rows else list(range(l ^ (i & 1), tiles, 2))
            v_end += tiles
            for j in mine:
                b = n & 1
                while not s_full[l][b].passed(n >> 1):
                    yield
                assert scores[l][b] == (i, j), "scores of another tile"
                if j != mine[0] and rnd.random() < 0.4:       # the output is rescaled
                    while wait_for_products and not pv_done[l].passed(n - 1):
                        yield
                    assert products[l] == n, "rescaled beside a product"
                for _ in range(rnd.randint(1, 40)):
                    yield
                if j == tiles - 1:                            # rows past the end are zeroed
                    slot = (v_end - 1) % stages
                    while not full[1][slot].passed((v_end - 1) // stages):
                        yield
                    assert kv[1][slot] == (i, j), "zeros into another tile"
                weights[l][b] = (i, j)
                p_full[l][b].arrive()
                n += 1
            if mine:
                while not o_full[l].passed(n_out):
                    yield
                n_out += 1
                assert out[l] == [(i, j) for j in mine], "an output of other tiles"
                for _ in range(rnd.randint(1, 20)):
                    yield
                o_empty[l].arrive()
            item_empty[i % ring_items].arrive()
        ended.append("softmax")

    actors += [scheduler(), copies(0), copies(1), softmax(0), softmax(1), product_warp(0), product_warp(1)]
    for _ in range(steps):
        if len(ended) == 7:
            return
        for entry in list(late):
            entry[0] -= 1
            if entry[0] <= 0:
                late.remove(entry)
                entry[1]()
        actor = rnd.choice(actors)
        for _ in range(rnd.randint(1, 3)):
            if next(actor, "end") == "end":
                break
    raise AssertionError("the warps wait for one another")


def _caught(**wrong):
    stages, ring_items, lead = _constants()
    for seed in range(400):
        try:
            simulate(seed, stages[seed & 1], ring_items, lead, steps=60000, **wrong)
        except AssertionError:
            return True
    return False


@pytest.mark.parametrize("d", [128, 64])
def test_every_wait_sees_the_tile_it_means(d):
    stages, ring_items, lead = _constants()
    for seed in range(120):
        simulate(seed, stages[0] if d == 128 else stages[1], ring_items, lead)


def test_lanes_that_skip_each_others_slots_are_caught():
    """Each lane waits for its own tiles only: a wait by parity then passes one phase early."""
    assert _caught(lanes_skip_slots=True)


def test_rescaling_without_a_wait_is_caught():
    assert _caught(wait_for_products=False)

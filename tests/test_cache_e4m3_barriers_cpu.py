"""A model of the barriers of the 8-bit cache's attention kernel for many rows, run in random order on the CPU.

The kernel's warps hand segments, codes, widened tiles, scores, weights and outputs to one another through
barriers whose waits are by parity: such a wait is only sound while the waiting warp is at most one phase
behind or ahead, and a slip would show as a product on a tile that is still being written, rarely and only
on some timings.  The model runs the warps' loops as coroutines in random order, with copies and products
that end late, over random segments; it checks at each use that what is there is what the warp means, that
no barrier gets an arrival too many, and that all warps come to their end.  Each lane has two softmax warps
here (four in the kernel).  Ring sizes and how far the scores run ahead are read from the kernel's source.
Protocols that are wrong have to be caught."""
import os
import random
import re

import pytest

from bit_weight_quantized_wq_gb300 import build as wqbuild

SOURCE = open(os.path.join(wqbuild.CSRC, "attn_e4m3.cu")).read()
WARPS = 2                                             # softmax warps of a lane


def _constant(name):
    return int(re.search(r"constexpr int %s = (\d+);" % name, SOURCE).group(1))


def _constants():
    ahead = re.search(r"const int ahead = turns.step == 1 \? (\d+) : (\d+);", SOURCE)
    return dict(raw_stages=_constant("kRawStages"), wide_stages=_constant("kWideStages"), scale_ring=_constant("kScaleRing"),
                ring=_constant("kSegments"), ahead=[int(v) for v in ahead.groups()])


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.phase, self.pending = count, count, 0, 0

    def arrive(self, copies=0):
        assert self.left > 0, "an arrival too many"
        self.left, self.pending = self.left - 1, self.pending + copies
        self.turn()

    def land(self):
        self.pending -= 1
        self.turn()

    def turn(self):
        if self.left == 0 and self.pending == 0:
            self.phase, self.left = self.phase + 1, self.count

    def passed(self, parity):
        return (self.phase & 1) != (parity & 1)


def simulate(seed, raw_stages, wide_stages, scale_ring, ring, ahead, skip_slots=False, no_meeting=False, steps=400000):
    rnd = random.Random(seed)
    # tiles, and whether both lanes have the same rows and take the tiles in turn
    segments = [(rnd.choice((0, 1, 1, 2, 3, 5, 12)), rnd.random() < 0.5) for _ in range(rnd.randint(1, 12))]
    bars = lambda count, n: [Barrier(count) for _ in range(n)]   # noqa: E731
    raw_full, raw_empty = bars(1, raw_stages), bars(4, raw_stages)
    full, empty = [bars(2, wide_stages) for _ in "KV"], [bars(2, wide_stages) for _ in "KV"]
    q_full, q_empty = bars(WARPS, 2), bars(1, 2)
    s_full, p_full = [bars(1, 2) for _ in range(2)], [bars(WARPS, 2) for _ in range(2)]
    pv_done, o_full, o_empty = bars(1, 2), bars(1, 2), bars(WARPS, 2)
    n_actors = 1 + 4 + 2 + 2 * WARPS
    seg_full, seg_empty, meeting = bars(1, ring), bars(n_actors, ring), Barrier(2 * WARPS)
    seg, raw, scales = [None] * ring, [None] * raw_stages, [None] * scale_ring
    wide = [[[None, None] for _ in range(wide_stages)] for _ in "KV"]
    q, statistics = [[None] * WARPS for _ in range(2)], [[None] * WARPS for _ in range(2)]
    scores, weights = [[None] * 2 for _ in range(2)], [[[None] * WARPS for _ in range(2)] for _ in range(2)]
    out, products, late, actors, ended = [[], []], [0, 0], [], [], []

    def until(bar, parity):
        while not bar.passed(parity):
            yield

    def pause(most):
        for _ in range(rnd.randint(0, most)):
            yield

    def taken(i, l):                                  # the tiles of segment i that lane l takes
        n, turns = segments[i]
        return list(range(l, n, 2)) if turns else list(range(n))

    def segment(i):
        yield from until(seg_full[i % ring], i // ring)
        assert seg[i % ring] == i, "a segment that is not this one"

    def walk():
        for i in range(len(segments)):
            yield from until(seg_empty[i % ring], (i // ring) ^ 1)
            seg[i % ring] = i
            seg_full[i % ring].arrive()
        ended.append("walk")

    def copies():
        t = 0
        for i, (n, _) in enumerate(segments):
            yield from segment(i)
            for j in range(n):
                s = t % raw_stages
                yield from until(raw_empty[s], (t // raw_stages) ^ 1)
                scales[t % scale_ring], raw[s] = (i, j), "loading"
                raw_full[s].arrive(1)

                def land(s=s, what=(i, j)):
                    raw[s] = what
                    raw_full[s].land()
                late.append([rnd.randint(1, 60) if rnd.random() < 0.9 else rnd.randint(60, 700), land])
                t += 1
            seg_empty[i % ring].arrive()
        ended.append("copies")

    def widen(v, half):
        t = 0
        for i, (n, _) in enumerate(segments):
            yield from segment(i)
            for j in range(n):
                rs, ws = t % raw_stages, t % wide_stages
                yield from until(raw_full[rs], t // raw_stages)
                yield from until(empty[v][ws], (t // wide_stages) ^ 1)
                wide[v][ws][half] = "being written"
                yield from pause(8)
                assert raw[rs] == (i, j), "codes of another tile"
                wide[v][ws][half] = (i, j)
                full[v][ws].arrive(), raw_empty[rs].arrive()
                t += 1
            seg_empty[i % ring].arrive()
        ended.append("widen")

    def tensor_core(queue):
        while True:
            if queue:
                yield from pause(12)
                queue.pop(0)()
            yield

    def product_warp(l):
        tiles, s_cnt, p_cnt, items, queue = [0, 0], 0, 0, 0, []
        actors.append(tensor_core(queue))

        def place(v, j, mine):
            t = tiles[v]
            tiles[v] += 1
            slot = t % wide_stages
            if mine or not skip_slots:
                yield from until(full[v][slot], t // wide_stages)
            if not mine:
                empty[v][slot].arrive()
            return slot

        for i, (n, turns) in enumerate(segments):
            yield from segment(i)
            mine = taken(i, l)
            if mine:
                yield from until(q_full[l], items)
            lead = ahead[1] if turns else ahead[0]
            for step in range(n + lead):
                j = step - lead
                if j >= 0:                            # O += W V
                    slot = yield from place(1, j, j in mine)
                    if j in mine:
                        if j == mine[0]:
                            yield from until(o_empty[l], items ^ 1)
                        yield from until(p_full[l][p_cnt & 1], p_cnt >> 1)

                        def run(i=i, j=j, slot=slot, b=p_cnt & 1, first=j == mine[0], last=j == mine[-1]):
                            assert wide[1][slot] == [(i, j)] * 2 and weights[l][b] == [(i, j)] * WARPS, "a product on the wrong tile"
                            out[l][:] = [] if first else out[l]
                            out[l].append((i, j))
                            products[l] += 1
                            pv_done[l].arrive()
                            if last:
                                o_full[l].arrive()
                            empty[1][slot].arrive()
                        queue.append(run)
                        p_cnt += 1
                if step < n:                          # S = Q K^T
                    j = step
                    slot = yield from place(0, j, j in mine)
                    if j in mine:
                        def run(i=i, j=j, slot=slot, b=s_cnt & 1, last=j == mine[-1]):
                            assert wide[0][slot] == [(i, j)] * 2 and q[l] == [i] * WARPS, "a product on the wrong tile"
                            scores[l][b] = (i, j)
                            s_full[l][b].arrive()
                            empty[0][slot].arrive()
                            if last:
                                q_empty[l].arrive()
                        queue.append(run)
                        s_cnt += 1
            items += bool(mine)
            seg_empty[i % ring].arrive()
        while queue:
            yield
        ended.append("products")

    def softmax(l, w):
        cnt, items, q_items, tile, meets = 0, 0, 0, 0, 0

        def put_q(i):
            nonlocal q_items
            if taken(i, l):
                yield from until(q_empty[l], q_items ^ 1)
                yield from pause(10)
                q[l][w] = i
                q_full[l].arrive()
                q_items += 1

        def meet():
            nonlocal meets
            if not no_meeting:
                meeting.arrive()
                yield from until(meeting, meets)
                meets += 1

        yield from segment(0)
        yield from put_q(0)
        for i, (n, turns) in enumerate(segments):
            mine = taken(i, l)
            for j in mine:
                b, at = cnt & 1, tile + j
                yield from until(s_full[l][b], cnt >> 1)
                yield from until(full[1][at % wide_stages], at // wide_stages)
                assert scores[l][b] == (i, j), "scores of another tile"
                assert scales[at % scale_ring] == (i, j), "scales of another tile"
                if j != mine[0] and rnd.random() < 0.4:       # the output is rescaled
                    yield from until(pv_done[l], cnt - 1)
                    assert products[l] == cnt, "rescaled beside a product"
                yield from pause(30)
                assert scores[l][b] == (i, j) and scales[at % scale_ring] == (i, j), "overwritten while in use"
                weights[l][b][w] = (i, j)
                p_full[l][b].arrive()
                cnt += 1
            tile += n
            if i + 1 < len(segments):                 # the next queries, before this output is taken
                yield from segment(i + 1)
                yield from put_q(i + 1)
            if mine:
                yield from until(o_full[l], items)
                items += 1
                assert out[l] == [(i, j) for j in mine], "an output of other tiles"
            if turns:                                 # the first lane reads the second one's output and statistics
                statistics[l][w] = i
                yield from meet()
                if l == 0:
                    yield from pause(20)
                    assert statistics[1][w] == i and (n < 2 or out[1] == [(i, j) for j in range(1, n, 2)]), "another segment's"
                yield from meet()
            else:
                yield from pause(20)
            if mine:
                assert out[l] == [(i, j) for j in mine], "an output overwritten"
                o_empty[l].arrive()
            seg_empty[i % ring].arrive()
        ended.append("softmax")

    actors += [walk(), copies()] + [widen(v, h) for v in (0, 1) for h in (0, 1)]
    actors += [product_warp(0), product_warp(1)] + [softmax(l, w) for l in (0, 1) for w in range(WARPS)]
    for _ in range(steps):
        if len(ended) == n_actors + 1:
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


def _caught(wrong, **more):
    for seed in range(400):
        try:
            simulate(seed, **dict(_constants(), **wrong), steps=60000, **more)
        except AssertionError:
            return True
    return False


@pytest.mark.parametrize("part", range(4))
def test_every_wait_sees_what_it_means(part):
    for seed in range(60 * part, 60 * part + 60):
        simulate(seed, **_constants())


@pytest.mark.parametrize("wrong,more", [
    ({}, dict(skip_slots=True)),                      # lanes that give back a place that they have not waited for
    ({}, dict(no_meeting=True)),                      # the first lane reads the second one's statistics at any time
    (dict(ahead=[3, 3]), {}),                         # scores over weights that their product has not read yet
    (dict(ahead=[2, 5]), {}),
    (dict(scale_ring=4), {}),                         # scales overwritten while the softmax is behind
])
def test_wrong_protocols_are_caught(wrong, more):
    assert _caught(wrong, **more)

"""A model of how the 8-bit cache's attention cuts its work and joins it again, run in random order on the CPU.

The rules are the kernels' own (``csrc/line.cuh``, compiled here for the host): the share of the line that a
CTA takes, the tiles of an item that fall into it, and which counter a CTA adds to after it has left its
part of an item.  The model runs the CTAs of a call in random order, at random speeds, each from one
visible step to the next, and checks that every item's output is written once, from all of its parts and from no
other item's, that no place of a part is in use twice, and that all counters are 0 at the end.  A rule that counts a group
of a single segment has to be caught: the next item's first group may have the same counter."""
import ctypes
import heapq
import os
import random
import shutil
import subprocess

import pytest

from bit_weight_quantized_wq_gb300 import build as wqbuild

RULES = r"""
#include "line.cuh"
extern "C" {
long long share_of(long long total, long long ctas, int heaviest, int exactly) { return wq::line_share(total, ctas, heaviest, exactly); }
int tile_of(long long b, long long s, int n, int w) { return wq::tile_at(b, s, n, w); }
int cta_of(long long at, long long share) { return wq::quotient(at, share); }
static int put(const wq::Join& j, int* out) {
  out[0] = j.counter, out[1] = j.first, out[2] = j.step, out[3] = j.n;
  return j.final;
}
int first_of(int c0, int c1, int cta, int ctas, int* out) { return put(wq::first_join(c0, c1, cta, ctas), out); }
int final_of(int c0, int c1, int* out) { return put(wq::final_join(c0, c1), out); }
int group() { return wq::kGroup; }
}
"""


class Rules:
    def __init__(self, folder):
        source, lib = os.path.join(folder, "rules.cpp"), os.path.join(folder, "rules.so")
        with open(source, "w") as f:
            f.write(RULES)
        subprocess.run([shutil.which("g++") or "g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", wqbuild.CSRC, source, "-o", lib],
                       check=True)
        self.lib = ctypes.CDLL(lib)
        i, big = ctypes.c_int, ctypes.c_longlong
        self.lib.share_of.argtypes, self.lib.share_of.restype = [big, big, i, i], big
        self.lib.tile_of.argtypes, self.lib.cta_of.argtypes = [big, big, i, i], [big, big]
        self.group = self.lib.group()

    def _join(self, f, *args):
        out = (ctypes.c_int * 4)()
        final = bool(f(*args, out))
        return tuple(out) + (final,)                  # counter, first, step, n, final

    def first(self, c0, c1, cta, ctas):
        return self._join(self.lib.first_of, c0, c1, cta, ctas)

    def final(self, c0, c1):
        return self._join(self.lib.final_of, c0, c1)


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    return Rules(str(tmp_path_factory.mktemp("rules")))


class Counted(Rules):
    """The rule that counts every group, one of a single segment too."""

    def __init__(self, rules):
        self.__dict__.update(rules.__dict__)

    def first(self, c0, c1, cta, ctas):
        if c1 - c0 + 1 <= self.group:
            return self.final(c0, c1)
        first = c0 + (cta - c0) // self.group * self.group
        return ctas + first, first, 1, min(self.group, c1 - first + 1), False


def cut(rules, items, ctas, heaviest, constant, exactly):
    """Items (tiles, weight) on the line -> for each CTA its segments (item, whole, first CTA, last CTA, line units)."""
    total = sum(n * w + constant for n, w in items)
    share = rules.lib.share_of(total, ctas, heaviest, exactly)
    assert share * ctas >= total and (not exactly or share == max(heaviest, -(-total // ctas)))
    segments, at = [[] for _ in range(ctas)], 0
    for item, (n, w) in enumerate(items):
        c0, c1 = at // share, (at + (n - 1) * w) // share
        assert (rules.lib.cta_of(at, share), rules.lib.cta_of(at + (n - 1) * w, share)) == (c0, c1)
        done = 0
        for cta in range(c0, c1 + 1):
            lo, hi = (rules.lib.tile_of(b, at, n, w) for b in (cta * share, (cta + 1) * share))
            assert lo == done and hi > lo             # each tile once, some in every CTA between the first and the last
            segments[cta].append((item, lo == 0 and hi == n, c0, c1, (hi - lo) * w + constant))
            done = hi
        assert done == n
        at += n * w + constant
    return segments


def simulate(rules, seed, items, ctas, heaviest, constant, exactly, timed):
    rnd = random.Random(seed)
    segments = cut(rules, items, ctas, heaviest, constant, exactly)
    counters, parts, written = [0] * (2 * ctas), {}, [0] * len(items)

    def cta_runs(cta):
        speed = rnd.uniform(0.9, 1.1)
        for item, whole, c0, c1, cost in segments[cta]:
            yield cost * speed
            if whole:
                written[item] += 1
                continue
            place = (cta, cta == c0)
            assert place not in parts, "two parts in one place"
            parts[place] = (item, frozenset([cta]))
            turn = rules.first(c0, c1, cta, ctas)
            while True:
                yield 2
                counter, first, step, n, final = turn
                counters[counter] += 1
                if counters[counter] < n:
                    break
                yield 1
                counters[counter] = 0
                have = frozenset()
                for c in range(first, first + n * step, step):
                    assert parts.get((c, c == c0), (None,))[0] == item, "joined before it was there"
                    assert not have & parts[c, c == c0][1], "joined twice"
                    have |= parts[c, c == c0][1]
                yield 8
                if final:
                    assert have == frozenset(range(c0, c1 + 1)), "joined from some of its parts"
                    written[item] += 1
                    break
                parts[first, first == c0] = (item, have)
                turn = rules.final(c0, c1)

    def wait(cost):
        return cost if timed else rnd.expovariate(1.0)

    queue = []
    for cta in range(ctas):
        run = cta_runs(cta)
        cost = next(run, None)
        if cost is not None:
            queue.append((wait(cost), cta, run))
    heapq.heapify(queue)
    while queue:
        now, cta, run = queue[0]
        cost = next(run, None)
        if cost is None:
            heapq.heappop(queue)
        else:
            heapq.heapreplace(queue, (now + wait(cost), cta, run))
    assert written == [1] * len(items), "an item that is not written, or written twice"
    assert not any(counters), "a counter that is not 0"


FEW, MANY = dict(constant=60, exactly=False), dict(constant=80, exactly=True)


def few(rnd, requests, keys, heads):
    """Items of up to 8 rows, or of up to 32 in two weights."""
    wide = rnd.random() < 0.5
    items = []
    for n in keys(rnd, requests):
        items += [(-(-n // 64), rnd.choice((8, 12)) if wide else 8)] * heads
    return dict(FEW, items=items, heaviest=12 if wide else 8, ctas=152 * (3 if wide else 4))


def many(rnd, requests, keys, heads):
    items = []
    for n in keys(rnd, requests):
        for _ in range(heads):
            items += [(-(-max(1, n - 100 * i) // 64), 10) for i in range(rnd.choice((0, 0, 1, 2)))] + [(-(-n // 64), rnd.choice((5, 10)))]
    return dict(MANY, items=items, heaviest=10, ctas=152)


def lengths(low, high):
    return lambda rnd, r: [int(low * (high / low) ** rnd.random()) for _ in range(r)]


LINES = [                                             # kernel, requests, their keys, key/value heads
    (few, (8, 16), lengths(1000, 65536), 8),          # decoding requests over long caches
    (few, (9, 9), lengths(131000, 131071), 8),
    (few, (1, 3), lengths(5000, 131071), 5),
    (few, (1, 1), lengths(20000, 131071), 38),
    (few, (1, 600), lengths(1, 3000), 2),
    (many, (1, 6), lengths(1000, 65536), 8),          # pieces of prompts over long caches
    (many, (1, 3), lengths(64, 30000), 5),
    (many, (20, 90), lengths(1, 4096), 2),
]
KNOWN = [                                             # two neighbours with one counter, were every group counted
    dict(FEW, items=[(2048, 8)] * 72, heaviest=8, ctas=608),           # 9 requests of 131071 keys, 8 heads
    dict(FEW, items=[(1157, 8)] * 5, heaviest=8, ctas=608),            # one of 74000 keys, 5 heads
    dict(MANY, items=[(n, 10) for n in (397, 398, 398, 399)] * 5, heaviest=10, ctas=152),         # one of 25500 keys, 128 new tokens, 40 heads on 5
]


@pytest.mark.parametrize("timed", [True, False])
@pytest.mark.parametrize("line", range(len(LINES)))
def test_every_cut_item_is_joined_once_from_all_its_parts(rules, line, timed):
    kernel, (least, most), keys, heads = LINES[line]
    for seed in range(40):
        rnd = random.Random(1000 * line + seed)
        call = kernel(rnd, rnd.randint(least, most), keys, heads)
        if seed % 4 == 3:
            call["ctas"] = rnd.choice((1, 2, 17, 100, 148, 592))       # other devices' sizes
        simulate(rules, seed, timed=timed, **call)


@pytest.mark.parametrize("timed", [True, False])
@pytest.mark.parametrize("call", KNOWN)
def test_neighbours_that_are_cut_in_groups(rules, call, timed):
    for seed in range(30):
        simulate(rules, seed, timed=timed, **call)


def _caught(rules, timed, calls):
    for seed, call in enumerate(calls):
        try:
            simulate(rules, seed, timed=timed, **call)
        except AssertionError:
            return True
    return False


@pytest.mark.parametrize("call", KNOWN)
def test_groups_of_one_that_are_counted_are_caught(rules, call):
    assert _caught(Counted(rules), False, [call] * 60)


def test_groups_of_one_that_are_counted_are_caught_at_a_device_s_speeds(rules):
    assert _caught(Counted(rules), True, [KNOWN[0]] * 30)


def test_groups_of_one_that_are_counted_are_caught_in_random_calls(rules):
    rnd = random.Random(7)
    assert _caught(Counted(rules), False, [few(rnd, rnd.randint(8, 16), lengths(1000, 65536), 8) for _ in range(200)])

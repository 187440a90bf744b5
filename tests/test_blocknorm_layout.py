"""Threads, shared memory and division of rows of the norms around a block: what
the host plans holds what a CTA lays out, for every vector width that a call's
addresses can ask for, and the units cover every row once.  Both sides are
restated here from k_blocknorm.cu, k_blocknorm_bwd.cu and blocknorm.cuh, with
their constants, and compared over many shapes."""
import os
import random
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "convolution_nhwc_implicit_gb300", "csrc")
TEXT = open(os.path.join(CSRC, "blocknorm.cuh")).read()
SMS, SMEM, STATIC = 152, 227 * 1024, 2048


def constant(name):
    return int(re.search(rf"\b{name} = (\d+)[;,]", TEXT)[1])


MAX_C, THREADS, MOST, CLUSTER, SETS, MEET = (constant(k) for k in ("kMaxC", "kThreads", "kMostThreads", "kCluster", "kClusterSets", "kMeet"))
SUMS = 4


def up(a, b):
    return -(-a // b)


def element(es, vec):
    return 4 if es * vec < 4 else es


BWD_STAGES = 3


def fwd_stages(es, k):
    return 2 if k == 2 and es == 4 else 3


class Part:
    def __init__(self, c, rb, k, threads, pair=False):
        self.rb, self.k, self.ctas = rb, k, 2 if pair else 1                    # (CTAs of a row)
        want = up(c, 8 * k * self.ctas)
        if want > 32:
            self.tpr = up(want, 32) * 32
        else:
            self.tpr = 1
            while self.tpr < want:
                self.tpr *= 2
        self.slots = threads // self.tpr if self.tpr <= threads else 1
        self.threads = self.tpr * self.slots
        self.whole = self.joined = False

    def smem(self, es):
        maps = self.threads * 8 * self.k * es
        if self.rb:
            return 2 * fwd_stages(es, self.k) * self.rb * maps + (self.threads * 2 * 8 * self.k * 4 if self.k > 1 else 0)
        return BWD_STAGES * (4 * maps + self.threads // min(self.tpr, 32) * 16)

    def wave(self, es):
        n = min(228 * 1024 // (self.smem(es) + 1024 + 256), MOST // self.threads)
        return SMS * max(n, 1) // self.ctas

    def divide_rows(self, rows, sets, wave):
        self.run = max(up(up(rows, wave), sets) * sets, sets)
        self.S = self.units = self.grid = up(rows, self.run)

    def divide_images(self, n, hw, sets, wave):
        best = None
        for s in range(1, 1025):
            each = up(up(hw, s), sets)
            if s > 1 and up(hw, each * sets) != s:
                continue
            cost = up(n * s, wave) * (each + 4)
            if best is None or cost < best:
                best, self.S, self.run = cost, s, hw if s == 1 else each * sets
        self.units = self.grid = n * self.S


def plan(n, hw, c, es, layers=True):
    rows = n * hw
    warp = 256 < c <= 512 and rows > 1024 and (c * es % 16 != 0 or (es == 2 and layers))
    k = 2 if c > 2048 or warp else 1
    fwd = Part(c, 1, k, THREADS)
    if k == 1 and rows > fwd.wave(es) * fwd.slots:
        fwd.rb = 2
    gated = Part(c, fwd.rb, k, THREADS)
    fwd.divide_rows(rows, fwd.slots * fwd.rb, fwd.wave(es))
    if fwd.rb == 2 and hw >= 4 * fwd.slots:
        gated.divide_images(n, hw, 2 * gated.slots, gated.wave(es))
    else:
        gated.rb = 1
        gated.divide_rows(rows, gated.slots, gated.wave(es))
    pair = c > 8 * MOST
    bwd = Part(c, 0, 1, 1 if pair else MOST, pair)
    bgate = Part(c, 0, 1, 1 if pair else MOST, pair)
    if hw < bwd.slots:
        bgate = Part(c, 0, 1, up(bwd.tpr * hw, 32) * 32)
    w = bgate.wave(es)
    bwd.divide_rows(rows, bwd.slots, bwd.wave(es))
    bgate.divide_images(n, hw, bgate.slots, w)

    def cluster(d, images, each):
        most = CLUSTER // images if images <= CLUSTER else 0
        if pair or not most or up(each, most * d.slots) > SETS:
            return
        d.run = up(each, most * d.slots) * d.slots
        d.S = up(each, d.run)
        d.units = d.grid = images * d.S
        d.joined = True

    cluster(bwd, 1, rows)
    cluster(bgate, n, hw)
    if not bgate.joined:
        bgate.whole = bgate.S == 1
        if bgate.whole and n > w:
            bgate.grid = w
    return fwd, gated, bwd, bgate


def shapes(count, seed):
    rng = random.Random(seed)
    for _ in range(count):
        c = min(MAX_C, int(2 ** rng.uniform(0, 13.2)))
        n, hw = int(2 ** rng.uniform(0, 9)), int(2 ** rng.uniform(0, 14))
        yield n, hw, c, rng.choice([2, 4])
    for c in (1, 2, 8, 9, 255, 256, 257, 264, 512, 513, 1024, 2047, 2048, 2049, 2056, 4095, 4096, 4097, 8191, 8192):
        for es in (2, 4):
            for n, hw in ((1, 1), (16, 1), (17, 3), (5000, 1), (3, 50), (8, 6400)):
                yield n, hw, c, es


def widths(c, es):
    return [v for v in ((8, 2, 1) if es == 2 else (4, 1)) if c % v == 0]


def test_threads_and_shared_memory():
    for n, hw, c, es in shapes(4000, 1):
        cp = up(c, 4) * 4
        for d in plan(n, hw, c, es) + plan(n, hw, c, es, False):
            assert d.threads % 32 == 0 and 32 <= d.threads <= MOST and (d.tpr < 32 or d.tpr % 32 == 0)
            assert d.tpr * 8 * d.k * d.ctas >= c > d.tpr * 8 * d.k * (d.ctas - 1) and (d.slots <= 15 or d.tpr <= 32)     # (named barriers 1 .. slots)
            if d.tpr > 32:
                assert d.slots * up(d.tpr // 32, 2) <= MEET
            if d.rb == 0 and d.slots == 1:
                assert d.tpr >= 32                                             # (a part of a warp never holds a CTA's sums alone)
            if d.ctas == 2:
                assert d.rb == 0 and d.slots == 1 and d.tpr > 32 and not d.joined
            for vec in widths(c, es):
                el = element(es, vec)
                assert 8 * d.k % vec == 0
                total = d.smem(el)
                assert total + STATIC <= SMEM, (n, hw, c, es, vec, d.__dict__)
                if d.rb:
                    ring = 2 * fwd_stages(el, d.k) * d.rb * d.threads * 8 * d.k * el
                    assert ring % 16 == 0 and ring + (d.threads * 16 * 8 if d.k > 1 else 0) <= total
                    continue
                ring = BWD_STAGES * 4 * d.threads * 8 * d.k * el
                stats = BWD_STAGES * (d.threads // min(d.tpr, 32)) * 16
                assert ring + stats <= total
                if d.ctas == 1:
                    sums = SUMS * 4 * 8 * d.threads                            # the threads' sums, four pairs of each
                    if d.slots > 1:
                        assert sums <= ring
                    if d.joined:
                        assert (sums if d.slots > 1 else 0) + SUMS * cp * 4 <= ring
                    if d.whole:
                        assert 2 * 4 * 8 * d.threads + 2 * c * 4 <= ring


def test_units_cover_every_row_once():
    for n, hw, c, es in shapes(1500, 2):
        rows = n * hw
        fwd, gated, bwd, bgate = plan(n, hw, c, es)
        for d, is_gated in ((fwd, False), (gated, True), (bwd, False), (bgate, True)):
            per_image = is_gated and (d.rb != 1)                               # (one row at a time: runs of all rows)
            span, images = (hw, n) if per_image else (rows, 1)
            assert d.units == images * d.S and d.S >= 1
            runs = [(min(span, s * d.run), min(span, (s + 1) * d.run)) for s in range(d.S)]
            assert runs[0][0] == 0 and runs[-1][1] == span and all(a[1] == b[0] and a[0] < a[1] for a, b in zip(runs, runs[1:] + [(span, 0)]))
            assert d.run * d.S + 2 * d.slots * 4 < 2 ** 31
            if d.rb:
                assert d.grid == d.units
            elif d.joined:
                assert d.grid == d.units <= CLUSTER
            elif d.whole:
                assert d.grid <= d.units and d.S == 1
            else:
                assert d.grid == d.units

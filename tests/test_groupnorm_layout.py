"""Shared memory of group norm's one-launch form: what the host asks for holds
what a CTA lays out, for every block of groups (the last of an image may have
fewer channels, and then more thread rows) and every vector width that a call's
addresses can ask for.  Both sides are restated here from k_groupnorm.cu, with
its constants, and compared over many shapes."""
import os
import random
import re

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "convolution_nhwc_implicit_gb300", "csrc", "k_groupnorm.cu")
TEXT = open(SRC).read()


def constant(name):
    m = re.search(rf"\b{name} = ([\d *]+)[;,]", TEXT)
    n = 1
    for f in m[1].split("*"):
        n *= int(f)
    return n


THREADS, RESIDENT, MOST, MAX_C = (constant(k) for k in ("kThreads", "kResident", "kResidentMost", "kMaxC"))
SMEM = 227 * 1024


def folds(vectors):
    return vectors <= 32 and vectors & (vectors - 1) == 0


def thread_rows(vectors):
    return 1 if vectors >= THREADS else THREADS // vectors


def entries(channels, vec):
    return (THREADS // 32 if folds(channels // vec) else thread_rows(channels // vec)) * channels


def ceil_div(a, b):
    return -(-a // b)


def plan(es, groups, cg, pixels, maps, most_k, sms_left):
    """(groups, channels, CTAs, pixels) of the form, or None where it is not taken."""
    c = groups * cg
    wide = 16 // es
    widest = wide if c % wide == 0 else (2 if c % 2 == 0 and es == 2 else 1)
    gb = 1
    while gb < groups and (gb * cg % widest or gb * cg * es < 64):
        gb += 1
    cb = gb * cg
    if cb > THREADS and cb // widest > THREADS:
        return None
    size = lambda k: ceil_div(pixels, k) * cb * es * maps  # noqa: E731
    k = 1
    while k < most_k and size(k) > RESIDENT:
        k += 1
    if size(k) > MOST:
        return None
    while k < most_k and k < sms_left and size(k) > 8 * 1024:
        k += 1
    run = ceil_div(pixels, k)
    return gb, cb, ceil_div(pixels, run), run


def host(es, groups, cg, gb, cb, run, maps, vec):
    last = (groups - (groups - 1) // gb * gb) * cg
    return 2 * gb * 8 + cb * 8 + max(entries(cb, vec), entries(last, vec)) * 8 + cb * 4 + 16 + run * cb * es * maps, last


def test_constants_are_the_sources():
    assert (THREADS, RESIDENT, MOST, MAX_C) == (256, 50 * 1024, 88 * 1024, 8192)


def test_what_a_cta_lays_out_fits():
    rng = random.Random(1)
    checked = short = 0
    while checked < 60000:
        es, maps, groups, cg = rng.choice([2, 4]), rng.choice([1, 2]), rng.randint(1, 40), rng.randint(1, 300)
        c, pixels = groups * cg, rng.randint(1, 30000 if rng.random() < 0.5 else 300)
        if c > MAX_C:
            continue
        p = plan(es, groups, cg, pixels, maps, rng.randint(1, 8) if maps == 2 else 8, rng.randint(1, 8))
        if p is None:
            continue
        gb, cb, k, run = p
        assert 1 <= k <= 8 and (k - 1) * run < pixels <= k * run        # every CTA has pixels
        for vec in {16 // es, 2 if es == 2 else 1, 1}:
            if c % vec or cb % vec or cb // vec > THREADS:
                continue
            need, last = host(es, groups, cg, gb, cb, run, maps, vec)
            assert need <= SMEM
            most = max(entries(cb, vec), entries(last, vec))
            for channels in {cb, last}:
                assert channels % vec == 0 and channels // vec <= THREADS
                assert entries(channels, vec) <= most
                # the runs start on 16 bytes after the sums and (forward) the pivots
                start = ceil_div(2 * gb * 8 + cb * 8 + most * 8 + (cb * 4 if maps == 1 else 0), 16) * 16
                vectors = channels // vec
                per = thread_rows(vectors) * vectors
                taken = ceil_div(run, thread_rows(vectors)) * per       # one past the last thread's last vector, at most
                assert taken - per < run * vectors
                assert start + maps * run * channels * es <= need
                short += channels < cb
            checked += 1
    assert short > 1000

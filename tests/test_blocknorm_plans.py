"""The plans of the norms around a block as the library makes them, against what
test_blocknorm_layout.py restates of them: the threads, grids, clusters, shared
memory and scratch of every launch, on a fake runtime that leaves a line for each.
(Its device runs every cluster that is asked about, as a GB300 does.)

Which forward rows take sixteen channels a thread is restated here: beyond 2048
channels, and from 257 to 512 for more rows than four sets of eight channels a
thread, where sixteen gain; below, they lost up to a quarter (512 channels, 2432
rows of bf16, layer norm and rms norm: 3.7 us and 4.4)."""
import ctypes

import pytest
from fake_cuda import load
from test_blocknorm_layout import SUMS, THREADS, Part, plan, shapes, up, widths


class Params(ctypes.Structure):
    _fields_ = [(k, ctypes.c_void_p) for k in ("scale", "gate", "post_gamma", "post_beta", "pre_gamma", "pre_beta")]


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    out = load(tmp_path_factory.mktemp("fake"))
    p, i64 = ctypes.c_void_p, ctypes.c_int64
    out.conv_plan_create_blocknorm.argtypes = [ctypes.c_int] * 6 + [ctypes.c_float, ctypes.c_int, ctypes.POINTER(p)]
    out.conv_run_blocknorm.argtypes = [p, p, i64, p, i64, p, p, i64, p, i64, p, p]
    out.conv_run_blocknorm_bwd.argtypes = [p, p, i64, p, i64, p, p] + [p, i64] * 4 + [p, p, p]
    out.conv_plan_destroy.argtypes = [p]
    for k in ("conv_plan_workspace", "conv_plan_workspace_bwd"):
        getattr(out, k).argtypes = [p, ctypes.POINTER(ctypes.c_size_t)]
    return out


# Addresses that no launch follows: a part of the address space for each tensor.
def place(i, shift=0):
    return (i + 1 << 42) + shift


def launches(lib):
    lines = lib.fake_log().decode().split("\n")[:-1]
    lib.fake_clear()
    out = []
    for line in lines:
        name, grid, threads, smem, cluster = line.split()
        out.append((name, tuple(map(int, grid.split(","))), int(threads), int(smem), int(cluster)))
    return out


def forward(n, hw, c, es, layers):
    """The forward launches without a gate and with one."""
    rows, eight, ragged = n * hw, Part(c, 1, 1, THREADS), c * es % 16 != 0
    many = 256 < c <= 512 and rows > 4 * eight.wave(es) * eight.slots
    out = []
    for is_gated, sixteen in ((False, many and (ragged or (es == 2 and layers))), (True, many and ragged)):
        d = Part(c, 1, 2 if sixteen or c > 2048 else 1, THREADS)
        if d.k == 1 and rows > d.wave(es) * d.slots:
            d.rb = 2
        if is_gated and d.rb == 2 and hw >= 4 * d.slots:
            d.divide_images(n, hw, 2 * d.slots, d.wave(es))
        else:
            d.rb = 1 if is_gated else d.rb
            d.divide_rows(rows, d.slots * d.rb, d.wave(es))
        out.append(d)
    return out


def many_rows():
    for c in (257, 264, 384, 510, 512):
        for es in (2, 4):
            for n, hw in ((1, 1024), (1, 1025), (4, 608), (1, 4864), (1, 4865), (8, 1600)):
                yield from ((n, hw, c, es), (n, hw, c, es))            # (with layer norms, and without)


def test_launches_are_the_restated_ones(lib):
    kinds = {"layers": (1, 1), "rms": (2, 2)}
    for number, (n, hw, c, es) in enumerate([*many_rows(), *shapes(1200, 11)]):
        post, pre = kinds["layers" if number % 2 else "rms"]
        h = ctypes.c_void_p()
        assert lib.conv_plan_create_blocknorm(n, hw, 1, c, post, pre, 1e-5, 0 if es == 4 else 1, ctypes.byref(h)) == 0
        fwd, gated = forward(n, hw, c, es, post == 1)
        _, _, bwd, bgate = plan(n, hw, c, es)
        parts = max(0 if d.joined else d.grid for d in (bwd, bgate))
        sizes = ctypes.c_size_t(9), ctypes.c_size_t(9)
        assert lib.conv_plan_workspace(h, ctypes.byref(sizes[0])) == 0 and lib.conv_plan_workspace_bwd(h, ctypes.byref(sizes[1])) == 0
        assert (sizes[0].value, sizes[1].value) == (0, parts * SUMS * up(c, 4) * 4 * 4)
        lib.fake_clear()
        for vec in widths(c, es):
            shift = {8: 0, 4: 0, 2: 4, 1: es}[vec]            # (what makes the accesses that narrow)
            for gate in (None, place(20)):
                w, d = Params(gate=gate), Params(place(21), place(22) if gate else None, place(23), None, place(25), None)
                x, f, y, z, dy, dz, dx, df = (place(i, shift) for i in range(8))
                where = (n, hw, c, es, vec, gate)
                assert lib.conv_run_blocknorm(h, x, 0, f, 0, ctypes.byref(w), y, 0, z, 0, place(10), None) == 0
                (name, grid, threads, smem, cluster), = launches(lib)
                one = gated if gate else fwd
                el = 4 if es * vec < 4 else es
                assert "bn_fwd_kernel" in name and (grid, threads, cluster) == ((one.grid, 1, 1), one.threads, 1), where
                assert smem == one.smem(el), where
                assert lib.conv_run_blocknorm_bwd(h, x, 0, f, 0, ctypes.byref(w), place(10), dy, 0, dz, 0, dx, 0, df, 0, ctypes.byref(d),
                                                  place(11) if parts else None, None) == 0
                (name, grid, threads, smem, cluster), *join = launches(lib)
                one = bgate if gate else bwd
                assert "bn_bwd_kernel" in name and (grid, threads) == ((one.grid * one.ctas, 1, 1), one.threads), where
                assert smem == one.smem(el) and cluster == (one.grid if one.joined else one.ctas), where
                assert [j[0].count("bn_join_kernel") for j in join] == ([] if one.joined else [1]), where
                if join:
                    images = 0 if not gate or one.whole else up(n, 16)
                    assert join[0][1] == (up(c, 16), 1 + images, 1), where
        lib.conv_plan_destroy(h)


def test_every_instance_that_is_built_is_reached(lib):
    built, i = set(), 0
    while name := lib.fake_kernel(i):
        if b"bn_fwd_kernel" in name or b"bn_bwd_kernel" in name:
            built.add(name.decode())
        i += 1
    reached = set()
    channels = (3, 8, 12, 250, 251, 256, 301, 302, 320, 511, 512, 1000, 1001, 1002, 2500, 2501, 2502, 5000, 5001, 5002)
    for c in channels:
        for es in (2, 4):
            for rows in (1, 2, 200000, 200001):
                for kind in (1, 2):
                    h = ctypes.c_void_p()
                    assert lib.conv_plan_create_blocknorm(1, rows, 1, c, kind, kind, 1e-5, 0 if es == 4 else 1, ctypes.byref(h)) == 0
                    x, f, y, z, dy, dz, dx, df = (place(i) for i in range(8))
                    lib.fake_clear()
                    for whole in (True, False):
                        assert lib.conv_run_blocknorm(h, x, 0, f, 0, None, y if whole else None, 0, z, 0, None, None) == 0
                        assert lib.conv_run_blocknorm_bwd(h, x, 0, f, 0, None, place(10), dy if whole else None, 0, dz, 0, dx, 0, df, 0, None,
                                                          place(11), None) == 0
                    reached |= {line[0] for line in launches(lib)}
                    lib.conv_plan_destroy(h)
    assert len(built) > 60 and built - reached == set()

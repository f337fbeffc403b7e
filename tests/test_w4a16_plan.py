"""What csrc/w4a16_plan.hpp decides, from that very header compiled for the host: every item of a ragged grouped call is
taken by exactly one workgroup of its launches, whatever the offsets hold nothing leaves the operands, a tile's copies
have landed when they are read and no slot is refilled before."""

import ctypes
import itertools
import os
import subprocess

import numpy as np
import pytest

from mxfp4_block_scaled_amd import ops

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "mxfp4_block_scaled_amd", "csrc")
i32, i64 = ctypes.c_int32, ctypes.c_int64


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("plan") / "plan.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wno-unknown-pragmas", "-I", CSRC,
                    os.path.join(HERE, "w4a16_plan_host.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    lib.items.restype = lib.matrix_items.restype = lib.weight_row.restype = i64
    lib.items.argtypes = [i32, ctypes.c_void_p, i32, i64, i32, i32, i64, i64, ctypes.c_void_p]
    lib.matrix_items.argtypes = [i64, i64, i64, ctypes.c_void_p]
    lib.grouped_plan.argtypes = [i64, i32, i64, i64, i32, i32, ctypes.c_void_p]
    lib.segment.argtypes = [ctypes.c_void_p, i32, i64]
    lib.weight_row.argtypes = [i32, i32, i64, i32, i32]
    lib.share.restype = ctypes.c_uint32
    return lib


def plan(host, R, E, N, K, swiglu, nv=0):
    out = np.zeros(18, np.int64)
    n = host.grouped_plan(R, E, N, K, int(nv), int(swiglu), out.ctypes.data)
    return [tuple(int(v) for v in row) for row in out.reshape(3, 6)[:n]]


def taken(host, launch, offs, R):
    bm, _, lo, hi, groups, ntiles = launch
    out = np.zeros((groups + 1, 4), np.int64)
    n = host.items(bm, offs.ctypes.data, len(offs) - 1, R, lo, hi, ntiles, groups, out.ctypes.data)
    return out[:n]


def counts_of(kind, E, rng):
    if kind == "empty":
        return np.zeros(E, int)
    if kind == "one":
        c = np.zeros(E, int)
        c[rng.integers(E)] = 700
        return c
    if kind == "edges":
        return rng.choice([0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 256, 257], E)
    if kind == "few":
        return rng.integers(0, 4, E)
    return (rng.zipf(1.3, E) % 2000).astype(int)


@pytest.mark.parametrize("kind", ["empty", "one", "edges", "few", "zipf"])
@pytest.mark.parametrize("E", [1, 2, 63, 64, 65, 255, 256, 257, 1024])
def test_every_item_is_taken_once(host, E, kind):
    rng = np.random.default_rng(E)
    for N, K, swiglu, before, behind in [(16, 128, 0, 0, 0), (528, 1152, 0, 3, 70), (4096, 7168, 1, 0, 5),
                                         (7168, 2048, 0, 1, 0), (1040, 256, 0, 0, 0)]:
        counts = counts_of(kind, E, rng)
        R = int(counts.sum()) + before + behind
        if R == 0 or R * (N // 64 + 1) > 2_000_000:
            continue
        offs = (before + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)
        launches = plan(host, R, E, N, K, swiglu, E % 2)
        for c in range(1, max(2, int(counts.max()) + 1)):  # an expert of c rows belongs to one launch
            assert sum(lo < c <= hi for _, _, lo, hi, _, _ in launches) == 1
        for launch in launches:
            bm, bn, lo, hi, groups, ntiles = launch
            assert ntiles == -(-N // bn)
            want = {(e, n, int(offs[e]) + u * bm, min(bm, int(c) - u * bm))
                    for e, c in enumerate(counts) if lo < c <= hi for u in range(-(-int(c) // bm)) for n in range(ntiles)}
            got = [tuple(map(int, v)) for v in taken(host, launch, offs, R)]
            assert len(got) == len(set(got)) and set(got) == want, launch


@pytest.mark.parametrize("E", [3, 64, 200, 300])
def test_wild_offsets_stay_inside(host, E):
    """Offsets that descend, are negative or lie past R: no item leaves rows, experts or n-tiles."""
    rng = np.random.default_rng(E)
    for trial in range(40):
        R = int(rng.integers(1, 3000))
        offs = rng.integers(-R, 3 * R, E + 1).astype(np.int32)
        if trial % 4 == 0:
            offs = np.sort(offs)
        if trial % 5 == 0:
            offs[rng.integers(E + 1)] = rng.choice([-2 ** 31, 2 ** 31 - 1])
        for launch in plan(host, R, E, 1040, 512, 0) + [(64, 128, 0, 2 ** 31 - 1, 256, 9), (128, 256, 16, 2 ** 31 - 1, 200, 5)]:
            got = taken(host, launch, offs, R)
            if len(got):
                e, n, row0, m = got.T
                assert (0 <= e).all() and (e < E).all() and (0 <= n).all() and (n < launch[5]).all()
                assert (row0 >= 0).all() and (m > 0).all() and (m <= launch[0]).all() and (row0 + m <= R).all()


@pytest.mark.parametrize("units,ntiles", itertools.product([1, 2, 7, 8, 9, 33, 129], [1, 5, 8, 16, 29, 61]))
def test_every_tile_of_a_matrix_is_taken_once(host, units, ntiles):
    groups = 8 * -(-units * ntiles // 8)
    out = np.zeros((groups, 2), np.int64)
    n = host.matrix_items(units, ntiles, groups, out.ctypes.data)
    assert n == units * ntiles
    assert {tuple(v) for v in out[:n].tolist()} == set(itertools.product(range(units), range(ntiles)))


@pytest.mark.parametrize("n,s", itertools.product([0, 1, 4, 7, 56, 57, 112], range(1, 9)))
def test_slices_cover_k(host, n, s):
    bounds = [host.share(n, i, s) for i in range(s + 1)]
    assert bounds[0] == 0 and bounds[-1] == n and bounds == sorted(bounds)
    if n >= s:  # as the plan has it: none is empty
        assert len(set(bounds)) == s + 1


@pytest.mark.parametrize("S", [0, 1, 2, 63, 64, 65, 130, 4097, 9000])
def test_segment_search(host, S):
    rng = np.random.default_rng(S)
    lens = rng.choice([0, 0, 1, 2, 70], S)
    offs = (3 + np.concatenate([[0], np.cumsum(lens)])).astype(np.int32)
    top = int(offs[-1])
    for t in {0, 1, 2, 3, 4, top - 1, top, top + 1, *map(int, rng.integers(0, top + 1, 200))}:
        want = int(np.searchsorted(offs[1:], t, side="right"))
        assert host.segment(offs.ctypes.data, S, t) == want, t
    wild = rng.integers(-5, 50, S + 1).astype(np.int32)  # not ascending: it ends, inside [0, S]
    assert all(0 <= host.segment(wild.ctypes.data, S, t) <= S for t in range(-1, 52))


# rows, weight rows, waves, slots of activations of the tiles that are built
TILES = [(128, 256, 4, 2), (64, 256, 4, 3), (64, 128, 4, 3)]


@pytest.mark.parametrize("BM,BN,NW,NA", TILES)
@pytest.mark.parametrize("P", [4, 8])
def test_copies_have_landed_and_slots_are_free(host, BM, BN, NW, NA, P):
    IA, IB = BM * 8 // 64 // NW, BN * 4 // 64 // NW
    slices = [0] if (BM, BN) != (64, 128) else [0, 2, 4, 6, 14]  # a K slice's first stage
    for st0, stages, has_sc in itertools.product(slices, [2, 4, 6, 8, 10, 14, 24, 26, 112], [True, False]):
        nst = st0 + stages
        outstanding, slot = [], {}

        def issue(op, at, what, copies):
            slot[op, at] = what
            outstanding.extend([(op, what)] * copies)

        issue("S", (st0 // P) & 1, st0 // P, has_sc)
        issue("B", host.code_slot(0), st0 // 2, IB)
        for i in range(min(NA - 1, stages)):
            issue("A", i, st0 + i, IA)
        for st in range(st0, nst):
            i = (st - st0) % host.turn(NA)
            scales = i % 2 == 1 and has_sc and host.begins_scales(st - 1, st0, P, nst)
            allowed = host.in_flight(i, NA, IA, IB, int(st + 1 >= nst), int(bool(scales)))
            del outstanding[:max(0, len(outstanding) - allowed)]
            assert not {("A", st), ("B", st // 2), ("S", st // P)} & set(outstanding)
            # behind the barrier every wave is done with stage st - 1
            if host.issues_codes(i, st, nst):
                at = host.code_slot(i + 2)
                assert slot.get(("B", at), -1) < st // 2
                issue("B", at, st // 2 + 1, IB)
            if i % 2 == 0 and host.begins_scales(st, st0, P, nst):
                at = (st // P + 1) & 1
                assert slot.get(("S", at), -1) < st // P
                issue("S", at, st // P + 1, has_sc)
            if host.issues_a(st, NA, nst):
                at = host.a_slot(i + NA - 1, NA)
                assert slot.get(("A", at), -1) < st
                issue("A", at, st + NA - 1, IA)
            assert slot["A", host.a_slot(i, NA)] == st and slot["B", host.code_slot(i)] == st // 2
            assert slot["S", (st // P) & 1] == st // P and i % 2 == st % 2
        assert not outstanding


def test_swizzles(host):
    """A row's chunks stay its own, and the 16 lanes of an LDS cycle (16 rows, one chunk) hit 8 or 4 of the chunks evenly."""
    for f, chunks in ((host.swizzle_a, 8), (host.swizzle_b, 4)):
        for r in range(256):
            assert sorted(c ^ f(r) for c in range(chunks)) == list(range(chunks))
    for base in range(0, 256, 16):
        assert sorted(host.swizzle_a(base + r) for r in range(16)) == sorted(list(range(8)) * 2)
        # 64-byte rows: four rows are a turn of the banks
        assert sorted((4 * (r & 1) + host.swizzle_b(base + r)) for r in range(16)) == sorted(list(range(8)) * 2)


@pytest.mark.parametrize("swiglu", [0, 1])
@pytest.mark.parametrize("BN", [128, 256])
@pytest.mark.parametrize("N", [32, 96, 256, 288, 4096, 7200])
def test_weight_rows(host, N, BN, swiglu):
    """Every weight row below N is some tile's, once; none lies more than 256 rows past N (what the byte bounds allow)."""
    if swiglu and BN == 128:
        pytest.skip("no such tile")
    half = N // 2
    rows = [host.weight_row(swiglu, BN, half, n, r) for n in range(-(-N // BN)) for r in range(BN)]
    assert min(rows) >= 0 and max(rows) < N + 257
    if swiglu:  # the first BN / 2 are gate rows (past half: not stored), the others their up rows
        gate = [r for i, r in enumerate(rows) if i % BN < BN // 2]
        up = [r for i, r in enumerate(rows) if i % BN >= BN // 2]
        assert gate == list(range(len(gate))) and up == [half + r for r in gate]
    else:
        assert rows == list(range(len(rows)))


def test_the_library_has_this_plan(host):
    if not os.path.exists(ops.lib_path()):
        pytest.skip("library not built (run __graft_entry__.build())")
    fn = ops.load().mxf_w16_grouped_plan
    fn.argtypes = [i64, i32, i64, i64, i32, i32, ctypes.c_void_p]
    for R, E, N, K, sw in [(1, 1, 16, 128, 0), (48, 256, 4096, 7168, 1), (512, 4, 4096, 7168, 0), (12288, 256, 7168, 2048, 0),
                           (12288, 32, 4096, 7168, 1), (6000, 8, 2048, 2048, 0)]:
        for nv in (0, 1):
            out = np.zeros((3, 5), np.int64)
            n = fn(R, E, N, K, nv, sw, out.ctypes.data)
            assert [tuple(v[:5]) for v in plan(host, R, E, N, K, sw, nv)] == [tuple(v) for v in out[:n].tolist()]


def test_runs_of_a_streaming_workgroup(host):
    """Four runs of weight rows where K is short, workgroups are many and the weights MXFP4, else one."""
    runs = lambda R, E, N, K, nv: plan(host, R, E, N, K, 0, nv)[0][1] // 64  # noqa: E731
    assert runs(384, 256, 7168, 2048, 0) == runs(192, 128, 4096, 512, 0) == 4
    assert runs(384, 256, 7168, 2048, 1) == runs(384, 256, 7168, 2176, 0) == runs(96, 64, 4096, 512, 0) == 1

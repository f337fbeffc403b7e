"""The product of two quantised matrices replayed on the CPU with the functions that its kernels run
(csrc/fp4_pair_plan.hpp, compiled for the host): a stage's codes and scales are where its lanes read them, nothing that is
read is being refilled, every element of K is multiplied once, whatever stage a K slice begins at, and each result leaves
once. The order of a stage (wait for all copies and the other waves, send the next stage's copies and perhaps the next
scale group's, read) is written down here as the kernels have it."""

import ctypes
import os
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "mxfp4_block_scaled_amd", "csrc")
FLYING, NOTHING = -2, -1


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("pair") / "pair.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wno-unknown-pragmas", "-I", CSRC,
                    os.path.join(HERE, "fp4_pair_host.cpp"), "-o", so], check=True)
    lib = ctypes.CDLL(so)
    i64, p = ctypes.c_int64, ctypes.c_void_p
    lib.plan.argtypes = [i64, i64, i64, ctypes.c_int, p]
    lib.past.argtypes = [ctypes.c_int, ctypes.c_int, i64]
    lib.copies.argtypes = lib.scales.argtypes = [ctypes.c_int, i64, p]
    lib.blocks.argtypes = [ctypes.c_int, p]
    lib.scales_at.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, p]
    lib.few_scales.argtypes = [ctypes.c_int, i64, ctypes.c_int, p]
    lib.share.restype = ctypes.c_uint32
    return lib


def table(fn, shape, *args, dtype=np.int64):
    out = np.zeros(shape, dtype)
    fn(*args, out.ctypes.data)
    return out


def spread(src, n):
    """n consecutive byte offsets from each of src."""
    return (src[..., None] + np.arange(n)).reshape(-1)


class Operand:
    """One operand of `rows` rows (a tile's, all of them in the matrix) with its two slots and two scale groups."""

    def __init__(self, host, rows, K, nv):
        self.host, self.rows, self.K, self.nv = host, rows, K, nv
        self.wrow, self.srow = K // 2, K // (16 if nv else 32)
        self.W = 2 if nv else 1
        self.slot = np.full((2, rows * 128), NOTHING)
        self.group = np.full((2, rows * 32), NOTHING)
        self.copy = table(host.copies, rows * 8, rows, self.wrow)
        self.scale = table(host.scales, rows * 2, rows, self.srow)
        self.at = table(host.blocks, (rows, 2, 4), rows, dtype=np.int32)
        assert self.at.min() >= 0 and self.at.max() + 16 <= rows * 128
        self.flying = []

    def issue(self, slot, st):
        assert 0 <= st * 128 < self.wrow  # the scalar offset, below any resource's size
        self.slot[slot] = FLYING
        self.flying.append((self.slot[slot], spread(self.copy + st * 128, 16)))

    def issue_scales(self, grp):
        assert 0 <= grp * 32 < self.srow
        self.group[grp & 1] = FLYING
        self.flying.append((self.group[grp & 1], spread(self.scale + grp * 32, 16)))

    def land(self):
        for where, what in self.flying:
            where[:] = what
        self.flying = []

    def read(self, slot, st):
        """All lanes' reads of a stage: the blocks of K that they take."""
        G = self.host.group_stages(int(self.nv))
        held = self.group[(st // G) & 1]
        sat = table(self.host.scales_at, (self.rows, 2), self.rows, st, int(self.nv), dtype=np.int32)
        assert sat.min() >= 0 and sat.max() + 4 * self.W <= self.rows * 32 and not (sat % 4).any()
        rows, taken = np.arange(self.rows)[:, None], []
        for g in range(2):
            past = self.host.past(g, st, self.K)
            for s in range(4):
                block = st * 8 + 4 * g + s
                assert bool(past) == (block * 32 >= self.K)
                codes = self.slot[slot][self.at[:, g, s, None] + np.arange(16)]
                assert np.array_equal(codes, rows * self.wrow + block * 16 + np.arange(16))  # (past K: the next row's)
                if past:
                    continue
                # byte s of the lane's dword, or half s % 2 of its dword s / 2
                scales = held[sat[:, g, None] + self.W * s + np.arange(self.W)]
                assert np.array_equal(scales, rows * self.srow + block * self.W + np.arange(self.W))
                taken.append(block)
        return taken


@pytest.mark.parametrize("nv", [False, True])
@pytest.mark.parametrize("rows", [64, 128, 256])
@pytest.mark.parametrize("K,slices", [(128, 1), (256, 1), (384, 1), (640, 2), (1152, 4), (1408, 2), (2048, 8), (2944, 8), (7040, 4),
                                      (7168, 8)])
def test_every_block_is_taken_once(host, rows, nv, K, slices):
    stages = -(-K // 256)
    G, taken = host.group_stages(int(nv)), []
    for k in range(slices):
        st0, nst = host.share(stages, k, slices), host.share(stages, k + 1, slices)
        assert st0 < nst
        op = Operand(host, rows, K, nv)
        op.issue_scales(st0 // G)
        op.issue(0, st0)
        for st in range(st0, nst):
            i = (st - st0) & 1
            op.land()  # waits for all copies; the barrier: every wave is done with the stage before
            if st + 1 < nst:
                op.issue(i ^ 1, st + 1)
            if host.begins_scales(st, st0, int(nv), nst):
                op.issue_scales(st // G + 1)
            taken += op.read(i, st)
        assert not op.flying
    assert sorted(taken) == list(range(K // 32))


@pytest.mark.parametrize("nv", [False, True])
def test_slices_that_begin_anywhere_in_a_scale_group(host, nv):
    K = 256 * 23
    for st0 in range(9):
        for nst in range(st0 + 1, min(st0 + 11, 24)):
            G, op = host.group_stages(int(nv)), Operand(host, 64, K, nv)
            op.issue_scales(st0 // G)
            op.issue(0, st0)
            for st in range(st0, nst):
                op.land()
                if st + 1 < nst:
                    op.issue((st - st0 + 1) & 1, st + 1)
                if host.begins_scales(st, st0, int(nv), nst):
                    op.issue_scales(st // G + 1)
                assert op.read((st - st0) & 1, st) == list(range(8 * st, 8 * st + 8))


@pytest.mark.parametrize("nv", [False, True])
@pytest.mark.parametrize("K", [128, 256, 384, 1152, 2048, 2944, 7168])
def test_few_tiles(host, nv, K):
    """Eight waves share K, each with two slots and the scales of two stages in registers; copies, then loads, return in
    the order they were sent, and a stage begins once at most the next one's are in flight."""
    stages, taken = -(-K // 256), []
    copies, loads = host.few_copies(), host.few_loads()
    assert copies == 2 * 32 * 8 // 64 and loads == 2  # both operands'
    for wave in range(8):
        st0, nst = host.share(stages, wave, 8), host.share(stages, wave + 1, 8)
        op = Operand(host, 32, K, nv)
        queue, scales = [], {}

        def issue(slot, st):
            assert 0 <= st * 128 < op.wrow and 0 <= st * 8 * op.W < op.srow
            op.slot[slot] = FLYING
            queue.extend([("codes", slot, st)] * copies + [("scales", slot, st)] * loads)

        def wait(most):
            while len(queue) > most:
                kind, slot, st = queue.pop(0)
                if kind == "codes" and ("codes", slot, st) not in queue:
                    op.slot[slot] = spread(op.copy + st * 128, 16)
                if kind == "scales" and ("scales", slot, st) not in queue:
                    scales[slot] = st

        if st0 < nst:
            issue(0, st0)
        for st in range(st0, nst):
            i = (st - st0) & 1
            if st + 1 < nst:
                issue(i ^ 1, st + 1)
                wait(copies + loads)
            else:
                wait(0)
            assert scales[i] == st
            at = table(host.few_scales, (32, 2), st, op.srow, int(nv))
            assert np.array_equal(at, np.arange(32)[:, None] * op.srow + (st * 8 + 4 * np.arange(2)) * op.W)
            for g in range(2):
                past = host.past(g, st, K)
                for s in range(4):
                    block = st * 8 + 4 * g + s
                    codes = op.slot[i][op.at[:, g, s, None] + np.arange(16)]
                    assert np.array_equal(codes, np.arange(32)[:, None] * op.wrow + block * 16 + np.arange(16))
                    assert bool(past) == (block * 32 >= K)
                    if not past:
                        taken.append(block)
        assert not queue
    assert sorted(taken) == list(range(K // 32))


@pytest.mark.parametrize("fn", [1, 2, 4])
@pytest.mark.parametrize("es", [2, 4])
def test_each_result_leaves_once(host, fn, es):
    PF = 256 // (32 * es) if fn * 32 * es > 256 else fn  # fragments of a pass: a wave's 8 KB
    chunks = PF * 32 * es // 16
    for p in range(fn // PF):
        area = np.full(8192, NOTHING)
        for lane in range(64):
            g, r = lane >> 5, lane & 31
            for f in range(PF):
                for j in range(4):
                    at = host.out_to(f, j, g, r, es, chunks)
                    assert 0 <= at <= 8192 - 4 * es and at % (4 * es) == 0 and (area[at:at + 4 * es] == NOTHING).all()
                    cols = 32 * (p * PF + f) + 8 * j + 4 * g + np.arange(4)  # accumulators 4 j .. 4 j + 3
                    area[at:at + 4 * es] = np.repeat(1000 * r + cols, es)
        seen = set()
        for r in range(32):
            for c in range(chunks):
                at = host.out_from(r, c, chunks)
                assert 0 <= at <= 8192 - 16 and at % 16 == 0
                first = 32 * p * PF + c * (16 // es)
                assert np.array_equal(area[at:at + 16], np.repeat(1000 * r + first + np.arange(16 // es), es))
                seen |= {(r, first + k) for k in range(16 // es)}
        assert len(seen) == 32 * 32 * PF


def test_few_tiles_sums(host):
    """Lane l's accumulator v is element (l % 32, 8 (v / 4) + 4 (l / 32) + v % 4) of the tile (B is the first operand)."""
    at = {}
    for lane in range(64):
        for v in range(16):
            at[(lane % 32, 8 * (v // 4) + 4 * (lane // 32) + v % 4)] = 65 * v + lane
    for r in range(32):
        for c in range(32):
            assert host.few_sum(r, c) == at[(r, c)] < 16 * 65


@pytest.mark.parametrize("nv", [0, 1])
def test_slices_have_stages_and_tiles_their_waves(host, nv):
    """Whatever the sizes: no slice without a stage, and the plan is one of the launchers' shapes."""
    rng = np.random.default_rng(nv)
    out = np.zeros(3, np.int32)
    for _ in range(3000):
        M, N, K = int(2 ** rng.uniform(0, 18)), 16 * int(2 ** rng.uniform(0, 13)), 128 * int(2 ** rng.uniform(0, 12))
        host.plan(M, N, K, nv, out.ctypes.data)
        bm, bn, slices = out.tolist()
        assert (bm, bn) in ((32, 32), (64, 64), (64, 128), (128, 128), (256, 256)) and slices in (1, 2, 4, 8)
        assert bm > 32 or slices == 1
        stages = -(-K // 256)
        assert all(host.share(stages, k, slices) < host.share(stages, k + 1, slices) for k in range(slices))

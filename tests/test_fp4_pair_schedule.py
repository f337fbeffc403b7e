"""The schedule of the product of two quantised matrices (csrc/fp4_pair.hpp, csrc/fp4_pair.hip), replayed on the CPU
from a copy of its formulas: where each copy lands, which bytes each lane reads for each matrix step, that every element
of K is multiplied once with its own scale, that no offset leaves its slot or its rows, and what the waits guarantee."""

import numpy as np
import pytest

SHAPES = [(64, 64, 2, 2), (64, 128, 2, 2), (128, 128, 2, 2), (256, 256, 4, 2)]


def swz(r):
    return (r & 7) ^ ((r >> 3) & 1)


def copies(rows, waves, wrow, st):
    """(LDS byte, source byte offset) of each 16-byte copy of a stage, all waves and lanes."""
    per = rows * 8 // 64 // waves
    for w in range(waves):
        for q in range(per):
            for lane in range(64):
                chunk = (w * per + q) * 64 + lane
                r = chunk >> 3
                yield (w * per + q) * 1024 + 16 * lane, r * wrow + 16 * ((chunk & 7) ^ swz(r)) + st * 128


@pytest.mark.parametrize("rows,waves", [(64, 4), (128, 4), (256, 8)])
def test_copies_fill_a_slot_once_and_stay_in_their_rows(rows, waves):
    wrow = 7 * 128
    for st in (0, 6):
        where = {}
        for lds, src in copies(rows, waves, wrow, st):
            assert lds not in where and 0 <= lds <= rows * 128 - 16
            where[lds] = src
        assert len(where) == rows * 8
        for r in range(rows):  # row r holds the 128 bytes of the stage, its chunks swapped among themselves
            got = sorted(where[r * 128 + 16 * p] for p in range(8))
            assert got == [r * wrow + st * 128 + 16 * c for c in range(8)]


@pytest.mark.parametrize("rows,waves", [(64, 4), (128, 4), (256, 8), (32, 1)])
def test_each_lane_reads_its_rows_blocks(rows, waves):
    """Step s, lane group g: the 32-block 4 g + s of row r, for both operands alike."""
    content = np.zeros(rows * 128, np.int64)
    if rows == 32:  # the few-tile kernel: a wave's own slot, four copies of a stage
        for q in range(4):
            for lane in range(64):
                r = 8 * q + (lane >> 3)
                content[1024 * q + 16 * lane:1024 * q + 16 * lane + 16] = (
                    r * 128 + 16 * ((lane & 7) ^ swz(r)) + np.arange(16))
    else:
        for lds, src in copies(rows, waves, 128, 0):
            content[lds:lds + 16] = src + np.arange(16)
    seen = np.zeros((rows, 128), int)
    for r in range(rows):
        for g in range(2):
            base = r * 128 + 16 * ((4 * g) ^ swz(r))
            for s in range(4):
                at = base ^ (16 * s)
                assert r * 128 <= at <= r * 128 + 112
                got = content[at:at + 16]
                assert np.array_equal(got, r * 128 + 16 * (4 * g + s) + np.arange(16))
                seen[r, 16 * (4 * g + s):16 * (4 * g + s) + 16] += 1
    assert (seen == 1).all()


@pytest.mark.parametrize("nv", [False, True])
@pytest.mark.parametrize("bm,bn,wm,wn", SHAPES)
def test_scales_of_a_group(bm, bn, wm, wn, nv):
    """A group is 32 scale bytes a row, the first 16 of 32 rows, then their second; the lane of row r and group g finds those of its blocks 4 g .. 4 g + 3."""
    NW, G, W = wm * wn, 2 if nv else 4, 2 if nv else 1
    SB = 32 // G
    ISA, ISB = bm * 2 // 64, bn * 2 // 64
    IS = -(-(ISA + ISB) // NW)
    srow = 96
    for grp in (0, 2):
        sa, sb = np.full(bm * 32, -1), np.full(bn * 32, -1)
        for wave in range(NW):
            for q in range(IS):
                p = wave + NW * q
                if p >= ISA + ISB:
                    continue
                into, part = (sa, p) if p < ISA else (sb, p - ISA)
                for lane in range(64):
                    lds = part * 1024 + 16 * lane
                    assert (into[lds:lds + 16] == -1).all() and lds + 16 <= into.size
                    into[lds:lds + 16] = (32 * part + lane % 32) * srow + 16 * (lane // 32) + grp * 32 + np.arange(16)
        for rows, held in ((bm, sa), (bn, sb)):
            for r in range(rows):
                for st in range(grp * G, grp * G + G):
                    for g in range(2):
                        off = SB * (st % G) + 4 * W * g
                        at = 1024 * (r // 32) + 512 * (off >> 4) + 16 * (r % 32) + (off & 15)
                        for s in range(4):  # block 4 g + s of the stage: one byte, or two of 16 elements each
                            block = (st * 8 + 4 * g + s) * W
                            got = held[at + s * W:at + s * W + W]
                            assert np.array_equal(got, r * srow + block + np.arange(W))


@pytest.mark.parametrize("bm,bn,wm,wn", SHAPES)
@pytest.mark.parametrize("nst", [1, 2, 3, 5, 8])
def test_slots_hold_what_is_read(bm, bn, wm, wn, nst):
    """Stage st waits for all copies, meets the other waves, sends those of st + 1 to the other slot and reads its own."""
    slot, flying = {}, [(0, 0)]
    for st in range(nst):
        for i, s in flying:  # vmcnt 0
            slot[i] = s
        flying = []
        if st + 1 < nst:
            flying.append(((st + 1) & 1, st + 1))
            assert ((st + 1) & 1) != (st & 1)
        assert slot[st & 1] == st
    assert not flying


@pytest.mark.parametrize("nst", [1, 2, 3, 7])
def test_few_tiles_wait_for_their_copies(nst):
    """A stage is 8 copies, then 2 loads, in order; with at most 10 outstanding the stage before has its copies."""
    outstanding, landed = [], set()

    def issue(st):
        outstanding.extend([("copy", st)] * 8 + [("load", st)] * 2)

    def wait(most):
        while len(outstanding) > most:
            landed.add(outstanding.pop(0))

    issue(0)
    for st in range(nst):
        if st + 1 < nst:
            issue(st + 1)
            wait(10)
        else:
            wait(0)
        assert ("copy", st) in landed and not any(o == ("copy", st) for o in outstanding)


@pytest.mark.parametrize("K", [128, 256, 384, 640, 7168])
def test_the_half_past_k_is_dropped(K):
    """Lane group 1 of a stage whose second 128 elements lie past K takes zero scales; nothing else past K is read."""
    for st in range(-(-K // 256)):
        for g in range(2):
            past = g == 1 and st * 256 + 128 >= K
            for s in range(4):
                inside = (st * 8 + 4 * g + s) * 32 < K
                assert inside != past


@pytest.mark.parametrize("fn", [1, 2, 4])
@pytest.mark.parametrize("es", [2, 4])
def test_the_epilogue_writes_each_column_once(fn, es):
    """32 rows x PF fragments through a wave's 8 KB: runs of four columns in, 16-byte pieces out."""
    PF = 256 // (32 * es) if fn * 32 * es > 256 else fn
    RB = PF * 32 * es
    nch = RB // 16
    assert fn % PF == 0 and 32 * RB <= 8192
    for p in range(fn // PF):
        area = np.full(8192, -1)
        for lane in range(64):
            g, r = lane >> 5, lane & 31
            for f in range(PF):
                for j in range(4):
                    cols = 32 * (p * PF + f) + 8 * j + 4 * g + np.arange(4)  # the accumulators 4 j .. 4 j + 3
                    if es == 2:
                        at = RB * r + 16 * ((4 * f + j) ^ (r & (nch - 1))) + 8 * g
                    else:
                        at = RB * r + 16 * ((8 * f + 2 * j + g) ^ (r & (nch - 1)))
                    assert (area[at:at + 4 * es] == -1).all()
                    area[at:at + 4 * es] = np.repeat(r * 1000 + cols, es)
        out = {}
        for k in range(nch // 2):
            for lane in range(64):
                idx = lane + 64 * k
                rr, c = idx // nch, idx % nch
                got = area[RB * rr + 16 * (c ^ (rr & (nch - 1))):][:16:es]
                for i, v in enumerate(got):
                    out[(rr, 32 * p * PF + c * (16 // es) + i)] = v
        assert len(out) == 32 * 32 * PF
        assert all(v == r * 1000 + c for (r, c), v in out.items())

"""Host replay of the tiled FP4 x bf16 kernel's copy schedule and lane layout (csrc/w4a16_tile_body.hpp), for each tile
shape it is built in: every copy's source and LDS bytes, coverage of a slot, what each fragment read returns (every
row's k of the stage exactly once, the same k for both operands), the scale byte it is multiplied with, and the
hand-over of the three slots."""

import pytest

SHAPES = [(128, 256, 4, False), (128, 256, 4, True), (64, 256, 4, False), (64, 256, 4, True),
          (64, 128, 4, False)]
# rows per wave: 128 in the 128 x 256 tiles of experts, else 64
WAVES = [(*shape, 64) for shape in SHAPES] + [(*shape, 128) for shape in SHAPES[:2]]


def swz_a(r):
    return (r & 7) ^ ((r >> 3) & 1)


def swz_b(r):
    return (r >> 2) & 3


def copies(BM, BN, NW):
    """(operand, wave, lane) -> LDS byte offset and (row, 16-byte chunk of the row's stage bytes)."""
    IA, IB = BM * 8 // 64 // NW, BN * 4 // 64 // NW
    for wave in range(NW):
        for q in range(IB):
            for lane in range(64):
                chunk = (wave * IB + q) * 64 + lane
                r = chunk >> 2
                yield "B", (wave * IB + q) * 1024 + 16 * lane, (r, (chunk & 3) ^ swz_b(r))
        for q in range(IA):
            for lane in range(64):
                chunk = (wave * IA + q) * 64 + lane
                r = chunk >> 3
                yield "A", (wave * IA + q) * 1024 + 16 * lane, (r, (chunk & 7) ^ swz_a(r))
        if wave < BN // 64:
            for lane in range(64):
                yield "S", wave * 1024 + 16 * lane, (64 * wave + lane, 0)


@pytest.mark.parametrize("BM,BN,NW,swiglu,WM", WAVES)
def test_slot_is_filled_and_read_in_one_layout(BM, BN, NW, swiglu, WM):
    WMN = BM // WM
    WNN = NW // WMN
    FN = BN // WNN // 32
    slot = {"A": {}, "B": {}, "S": {}}
    for op, at, what in copies(BM, BN, NW):
        assert at not in slot[op]
        slot[op][at] = what
    assert sorted(slot["A"]) == list(range(0, BM * 128, 16))
    assert sorted(slot["B"]) == list(range(0, BN * 64, 16))
    assert sorted(slot["S"]) == list(range(0, BN * 16, 16))
    for name, per in (("A", 8), ("B", 4)):
        assert sorted(slot[name].values()) == [(r, c) for r in range(len(slot[name]) // per) for c in range(per)]
    rows_seen, cols_seen = [], []
    for wave in range(NW):
        wm, wn = wave // WNN, wave % WNN
        for f in range(FN):
            for r32 in range(32):
                if swiglu:
                    row = (0 if f < FN // 2 else BN // 2) + FN * 16 * wn + 32 * (f % (FN // 2)) + r32
                else:
                    row = 32 * (FN * wn + f) + r32
                assert slot["S"][16 * row] == (row, 0)
                for g in range(2):
                    for odd in range(2):  # the 32 codes k = 32 (2 odd + g) + ... of the 128-k slot
                        at = (row * 64 + 16 * (g ^ swz_b(row))) ^ (32 * odd)
                        assert slot["B"][at] == (row, 2 * odd + g)
                if wm == 0:
                    cols_seen.append(row)
        for f in range(WM // 32):
            for r32 in range(32):
                r = WM * wm + 32 * f + r32
                if wn == 0:
                    rows_seen.append(r)
                for g in range(2):
                    base = r * 128 + 16 * ((4 * g) ^ swz_a(r))
                    for j in range(4):
                        # MFMA j, group g: k = 32 g + 8 j + [0, 8), 16 bytes of bf16
                        assert slot["A"][base ^ (16 * j)] == (r, 4 * g + j)
    assert sorted(rows_seen) == list(range(BM)) and sorted(cols_seen) == list(range(BN))


@pytest.mark.parametrize("BM,BN,NW,swiglu,WM", WAVES)
def test_output_columns_are_those_of_the_weight_rows(BM, BN, NW, swiglu, WM):
    WNN = NW // (BM // WM)
    FN = BN // WNN // 32
    OF = FN // 2 if swiglu else FN
    half = 4096
    seen = []
    for n_tile in (0, 3):
        for wn in range(WNN):
            col0 = (n_tile * BN >> (1 if swiglu else 0)) + OF * 32 * wn
            for f in range(OF):
                for c in range(32):
                    def src(frag):
                        if swiglu:
                            r = (0 if frag < FN // 2 else BN // 2) + FN * 16 * wn + 32 * (frag % (FN // 2)) + c
                            return (0 if r < BN // 2 else half - BN // 2) + n_tile * (BN // 2) + r
                        return n_tile * BN + 32 * (FN * wn + frag) + c
                    assert src(f) == col0 + 32 * f + c
                    if swiglu:
                        assert src(f + FN // 2) == half + col0 + 32 * f + c
                    seen.append(col0 + 32 * f + c)
    assert len(seen) == len(set(seen))


@pytest.mark.parametrize("es", [2, 4])
@pytest.mark.parametrize("OF", [1, 2, 4])
def test_epilogue_staging_round_trip(OF, es):
    """32 rows x PF fragments through 8 KB: the 8- or 16-byte runs written are what the 16-byte pieces read back."""
    PF = 256 // (32 * es) if OF * 32 * es > 256 else OF
    assert OF % PF == 0
    RB, NCH = PF * 32 * es, PF * 32 * es // 16
    assert 32 * RB <= 8192
    lds = {}
    for r in range(32):
        for f in range(PF):
            for j in range(4):
                for g in range(2):
                    cols = [32 * f + 8 * j + 4 * g + i for i in range(4)]
                    if es == 2:
                        at = RB * r + 16 * ((4 * f + j) ^ (r & (NCH - 1))) + 8 * g
                    else:
                        at = RB * r + 16 * ((8 * f + 2 * j + g) ^ (r & (NCH - 1)))
                    for i, c in enumerate(cols):
                        assert at + i * es not in lds
                        lds[at + i * es] = (r, c)
    for k in range(NCH // 2):
        for lane in range(64):
            idx = lane + 64 * k
            rr, c = idx // NCH, idx % NCH
            got = [lds[RB * rr + 16 * (c ^ (rr & (NCH - 1))) + i * es] for i in range(16 // es)]
            assert got == [(rr, c * (16 // es) + i) for i in range(16 // es)]
    assert 64 * (NCH // 2) == 32 * NCH


@pytest.mark.parametrize("nst", [2, 4, 6, 8, 10, 32, 112])
@pytest.mark.parametrize("NA", [2, 3])
@pytest.mark.parametrize("P", [4, 8])
@pytest.mark.parametrize("st0", [0, 2, 4, 6, 14])  # a K slice's first stage
@pytest.mark.parametrize("IA,IB,has_sc", [(4, 2, True), (4, 2, False), (4, 4, True), (2, 4, True), (2, 2, False)])
def test_slots_are_handed_over(nst, NA, P, st0, IA, IB, has_sc):
    """A stage is computed only after its copies landed, and a slot refilled only after every wave is done with it."""
    outstanding, A, B, S = [], {}, {}, {}

    def issue_a(slot, st):
        A[slot] = st
        outstanding.extend([("A", st)] * IA)

    def issue_b(slot, h):
        B[slot] = h
        outstanding.extend([("B", h)] * IB)

    def issue_s(grp):
        S[grp & 1] = grp
        if has_sc:
            outstanding.append(("S", grp))

    end = st0 + nst

    def next_s(st):
        return (st % P == 0 or st == st0) and (st // P + 1) * P < end

    issue_s(st0 // P)
    issue_b(0, st0 // 2)
    for i in range(min(NA - 1, nst)):
        issue_a(i, st0 + i)
    U = 12 if NA == 3 else 4
    for st in range(st0, end):
        i = (st - st0) % U
        if NA == 2 or st + 1 >= end:
            allowed = 0
        elif i % 2 == 0:
            allowed = IA
        elif has_sc and next_s(st - 1):
            allowed = IA + IB + 1
        else:
            allowed = IA + IB
        del outstanding[:max(0, len(outstanding) - allowed)]
        needed = {("A", st), ("B", st // 2), ("S", st // P)}
        assert not needed & set(outstanding)
        # after the barrier every wave is done with stage st - 1: what it and older stages read may be refilled
        if i % 2 == 0 and st + 2 < end:
            slot = (i // 2 + 1) % 2
            assert B.get(slot, -1) < (st // 2)
            issue_b(slot, st // 2 + 1)
        if i % 2 == 0 and next_s(st):
            assert S.get((st // P + 1) & 1, -1) < st // P
            issue_s(st // P + 1)
        if st + NA - 1 < end:
            slot = (i + NA - 1) % NA
            assert A.get(slot, -1) < st
            issue_a(slot, st + NA - 1)
        assert A[i % NA] == st and B[(i // 2) % 2] == st // 2 and S[(st // P) & 1] == st // P and i % 2 == st % 2
    assert not outstanding


@pytest.mark.parametrize("nv", [False, True])
def test_scale_bytes(nv):
    """A scale group is 16 bytes of a row: stage st finds the scales of its two 32-k groups in one dword of it."""
    P, per = (4, 16) if nv else (8, 32)
    for st in range(40):
        dword = st & 3 if nv else (st & 7) >> 1
        for g in range(2):
            for k in range(0, 32, 8):
                byte = 2 * g + k // 16 if nv else 2 * (st & 1) + g
                assert 16 * (st // P) + 4 * dword + byte == (64 * st + 32 * g + k) // per


def first_segment(ends, S, t):
    """The kernel's 64-way search over seg_off[1:]."""
    lo, hi = 0, S
    while lo < hi:
        step = (hi - lo + 63) // 64
        p = [lo + lane * step < hi and ends[lo + lane * step] > t for lane in range(64)]
        probes = (hi - lo + step - 1) // step
        f = p.index(True) if any(p) else probes
        lo, hi = (lo if f == 0 else lo + (f - 1) * step + 1), (hi if f == probes else lo + f * step)
        if step == 1:
            break
    return lo


@pytest.mark.parametrize("S", [0, 1, 2, 63, 64, 65, 130, 4097])
def test_segment_search(S):
    ends = [(i * 5) // 3 for i in range(S)]  # some empty
    for t in range(-1, (ends[-1] if S else 0) + 2):
        assert first_segment(ends, S, t) == next((s for s in range(S) if ends[s] > t), S)


def place(w, units, ntiles, group=8):
    grp, rem = divmod(w, ntiles * group)
    width = min(group, units - grp * group)
    return rem // width, grp * group + rem % width


@pytest.mark.parametrize("units", [1, 2, 3, 7, 8, 9, 32, 129])
@pytest.mark.parametrize("ntiles", [1, 5, 8, 9, 16, 28, 61])
def test_every_tile_is_placed_once(units, ntiles):
    seen = [place(w, units, ntiles) for w in range(units * ntiles)]
    assert sorted(seen) == [(n, u) for n in range(ntiles) for u in range(units)]
    if units <= 8:  # n-tile by n-tile
        assert seen == sorted(seen)

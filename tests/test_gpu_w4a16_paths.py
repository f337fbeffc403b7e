"""moe_grouped_gemm_w4a16 in each of its kernels, by name: every case asserts from the library's rule that the kernel it
is meant for runs it. Long K (slots, scale groups and super-steps turn over), NaN beside rows, offsets and pairs outside
their range, extreme scales, stray writes. Against 64 bits; an fp32 result is off by at most (K / 16 + 32) 2^-23
sum |a w| (weights and products exact, K / 16 dependent instructions of at most 32 additions)."""

import pytest
import torch

from mxfp4_block_scaled_amd import ops
from tests.test_gpu_canary import Guarded
from tests.w4a16_exact import close, grouped_paths, product, silu_mul, weights

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
ANY = 2 ** 31 - 1
STREAM, S64, T128 = (16, 64), (64, 128), (128, 256)
T64 = (64, 256)

# tile, (rows of the experts), N: the launch that takes the experts of more than 16 rows
SHAPES = {
    "64x128": (S64, [(16, ANY)], [130, 17, 0, 200, 9, 64, 65], 8208),
    "64x256": (T64, [(16, ANY)], [130, 17, 0, 250, 64, 65, 80, 90], 10256),
    "64x256 swiglu": (T64, [(16, ANY)], [130, 17, 0, 200, 9, 64, 65], 8224),
    "128x256": (T128, [(16, ANY)], [1000, 530, 20], 7200),
    "large": (T128, [(16, 64), (64, ANY)], [500, 300, 193, 129, 128, 100, 65, 64, 40, 33, 17, 16, 10, 1, 0, 1200], 7200),
}


def launch_of(name, counts, N, K, fmt, swiglu, R):
    """The launches are those that `name` stands for, and each has an expert to work on."""
    tile, classes, _, _ = SHAPES[name]
    paths = grouped_paths(R, len(counts), N, K, fmt, swiglu)
    assert paths[0][2:] == (0, 16) and [p[2:] for p in paths[1:]] == classes
    assert paths[-1][:2] == tile and (len(classes) == 1 or paths[1][:2] == T64)
    for _, _, lo, hi in paths[1:]:
        assert any(lo < c <= hi for c in counts)


def offsets(counts, before=0):
    return torch.tensor([before] + counts, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()


def check(counts, N, K, fmt, swiglu, dtype, gather, before=0, behind=0, scales=None, shift=0):
    """One call against 64 bits; rows outside every expert stay as they were."""
    R = sum(counts) + before + behind
    gen = torch.Generator(device="cuda").manual_seed(R + N + K)
    topk = 2 if gather and R % 2 == 0 else 1
    a = (torch.randn(R // topk, K, device="cuda", generator=gen) * 2.0 ** shift).to(BF)
    pair = torch.randperm(R, device="cuda", generator=gen).to(torch.int32) if gather else None
    src = (pair // topk).long() if gather else torch.arange(R, device="cuda")
    w, s = weights((len(counts), N), K, fmt, gen, scales)
    out = torch.full((R, N // 2 if swiglu else N), 7.0, dtype=dtype, device="cuda")
    ops.moe_grouped_gemm_w4a16(a, offsets(counts, before), w, s, fmt, sorted_pair=pair, topk=topk, swiglu=swiglu, out=out)
    at = before
    assert (out[:before] == 7).all() and (out[R - behind:] == 7).all()
    for e, c in enumerate(counts):
        if c:
            acc, mag = product(a[src[at:at + c]], w[e], s[e], fmt)
            mag = mag * (K / 16 + 32) * 2.0 ** -23
            if swiglu:
                acc, mag = silu_mul(acc, mag)
            close(out[at:at + c], acc, mag, f"expert {e} of {c} rows")
        at += c


@pytest.mark.parametrize("counts", [[1, 4, 0, 3, 2], [5, 16, 9, 1, 13], [40, 0, 130]], ids=["few", "to16", "more"])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("K", [2688, 4096, 7168, 7296])
def test_streaming_kernel_over_a_long_k(K, fmt, swiglu, counts):
    """Several super-steps of 512 k a wave, unequal shares, a last one that is not full."""
    N, R = 96, sum(counts) + 5
    assert grouped_paths(R, len(counts), N, K, fmt, swiglu) == [(*STREAM, 0, ANY)]
    check(counts, N, K, fmt, swiglu, F32 if K % 512 else BF, K != 4096, 2, 3)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("K", [1152, 2176, 7296])
@pytest.mark.parametrize("name", SHAPES)
def test_tiles_over_a_long_k(name, K, fmt):
    """Slots, scale groups and the K loop turn over in every tile shape, both formats, and with SwiGLU where it is built;
    experts of at most 16 rows stream beside them."""
    _, _, counts, N = SHAPES[name]
    for swiglu in {"64x128": [False], "64x256": [False], "64x256 swiglu": [True]}.get(name, [False, True]):
        if K == 7296 and name == "large":
            counts = [200, 100, 64, 33, 17, 10, 1, 0] + [150] * 8  # fewer rows of wider matrices
            N = 14368
        launch_of(name, counts, N, K, fmt, swiglu, sum(counts) + 4)
        check(counts, N, K, fmt, swiglu, BF if swiglu else F32, not swiglu, 3, 1)


TILED = [n for n in SHAPES if n != "64x256 swiglu"]


@pytest.mark.parametrize("name", TILED)
def test_a_bad_row_stays_alone(name):
    """NaN and infinite rows change no other row of their tile."""
    _, _, counts, N = SHAPES[name]
    K, R = 640, sum(counts)
    launch_of(name, counts, N, K, "mxfp4", False, R)
    gen = torch.Generator(device="cuda").manual_seed(5)
    w, s = weights((len(counts), N), K, "mxfp4", gen)
    a = torch.randn(R, K, device="cuda", generator=gen).to(BF)
    want = ops.moe_grouped_gemm_w4a16(a, offsets(counts), w, s)
    bad = a.clone()
    rows = sorted({0, counts[0] // 2, counts[0], counts[0] + 3, R // 2, R - 1})
    for i, r in enumerate(rows):
        bad[r, i] = [float("nan"), float("inf"), float("-inf")][i % 3]
    got = ops.moe_grouped_gemm_w4a16(bad, offsets(counts), w, s)
    keep = torch.ones(R, dtype=torch.bool, device="cuda")
    keep[rows] = False
    assert torch.equal(got[keep], want[keep])
    assert not torch.isfinite(got[rows]).all(1).any()


@pytest.mark.parametrize("name", TILED)
def test_offsets_are_held_to_the_rows(name):
    """Offsets below 0 and past R are taken as 0 and R; nothing beside y is written."""
    _, _, counts, N = SHAPES[name]
    K, R, E = 256, sum(counts), len(counts)
    launch_of(name, counts, N, K, "mxfp4", False, R)
    gen = torch.Generator(device="cuda").manual_seed(6)
    w, s = weights((E, N), K, "mxfp4", gen)
    a = torch.randn(R, K, device="cuda", generator=gen).to(BF)
    offs = offsets(counts)
    y, z = Guarded((R, N), F32, 7), Guarded((R, N), F32, 8)
    ops.moe_grouped_gemm_w4a16(a, offs, w, s, out=y.t)
    wild = offs.clone()
    wild[0], wild[E] = -5, R + 1000
    ops.moe_grouped_gemm_w4a16(a, wild, w, s, out=z.t)
    torch.cuda.synchronize()
    y.check("y")
    z.check("y of wild offsets")
    assert torch.equal(y.t, z.t)


@pytest.mark.parametrize("name", TILED)
def test_pairs_outside_their_range_spoil_their_rows_only(name):
    _, _, counts, N = SHAPES[name]
    counts = counts[:-1] + [counts[-1] + sum(counts) % 2]
    K, R, topk = 384, sum(counts), 2
    launch_of(name, counts, N, K, "mxfp4", False, R)
    gen = torch.Generator(device="cuda").manual_seed(7)
    w, s = weights((len(counts), N), K, "mxfp4", gen)
    a = torch.randn(R // topk, K, device="cuda", generator=gen).to(BF)
    pair = torch.randperm(R, device="cuda", generator=gen).to(torch.int32)
    want = ops.moe_grouped_gemm_w4a16(a, offsets(counts), w, s, sorted_pair=pair, topk=topk)
    rows = [0, 40, R // 2, R - 1]
    pair[rows] = torch.tensor([-1, R, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    got = ops.moe_grouped_gemm_w4a16(a, offsets(counts), w, s, sorted_pair=pair, topk=topk)
    keep = torch.ones(R, dtype=torch.bool, device="cuda")
    keep[rows] = False
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("name", TILED)
def test_extreme_scales(name):
    """UE8M0 bytes at both ends of 2 .. 252, and every UE4M3 byte."""
    _, _, counts, N = SHAPES[name]
    for fmt, scales, shift in (("mxfp4", (2, 7), 60), ("mxfp4", (248, 253), -60), ("nvfp4", (0, 0x7F), 0)):
        launch_of(name, counts, N, 640, fmt, False, sum(counts))
        check(counts, N, 640, fmt, False, F32, False, scales=scales, shift=shift)


@pytest.mark.parametrize("name", list(SHAPES))
def test_writes_stay_inside(name):
    _, _, counts, N = SHAPES[name]
    swiglu, R = "swiglu" in name, sum(counts)
    gen = torch.Generator(device="cuda").manual_seed(9)
    for fmt, dt, K in (("mxfp4", BF, 640), ("nvfp4", F32, 384)):
        launch_of(name, counts, N, K, fmt, swiglu, R)
        w, s = weights((len(counts), N), K, fmt, gen)
        a = torch.randn(R, K, device="cuda", generator=gen).to(BF)
        y = Guarded((R, N // 2 if swiglu else N), dt, 10)
        want = ops.moe_grouped_gemm_w4a16(a, offsets(counts), w, s, fmt, swiglu=swiglu, out_dtype=dt)
        ops.moe_grouped_gemm_w4a16(a, offsets(counts), w, s, fmt, swiglu=swiglu, out=y.t)
        torch.cuda.synchronize()
        y.check(name)
        assert torch.equal(y.t, want)


@pytest.mark.parametrize("E", [65, 256, 257, 600])
def test_tiles_beside_many_experts(E):
    """The lookup's forms for more experts than lanes, and than a lane holds, in the tiled kernels."""
    counts = [(7 * i) % 5 for i in range(E)]
    counts[3], counts[E // 2], counts[E - 1], counts[E - 2] = 70, 17, 200, 33
    N, K = 4112, 256
    paths = grouped_paths(sum(counts), E, N, K, "mxfp4", False)
    assert len(paths) > 1
    check(counts, N, K, "mxfp4", False, F32, True)

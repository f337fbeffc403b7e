"""GPU parity of moe_grouped_gemm_w4a16 (ragged rows by expert, bf16 activations, FP4 weights)
against products in 64 bits.

Tolerance, from arithmetic: weights and products are exact, so an fp32 result is off by the
accumulation alone. An instruction adds at most 32 products to the accumulator; counting every
one of its additions as a rounding of 2^-23 (rounded or cut off) gives, for the K / 16 dependent
instructions of the longest chain and the 32 additions inside one,
|acc - exact| <= (K / 16 + 32) 2^-23 sum |a w| = d. SwiGLU passes errors on as
1.1 dg (|u| + du) + |silu(g)| du (sup |silu'| < 1.1), plus 2^-19 |h| for the hardware exponential
and reciprocal; the rounding to bf16 is half a step, 2^-8 of the value."""

import numpy as np
import pytest
import torch

import oracle
from mxfp4_block_scaled_amd import datagen as dg
from mxfp4_block_scaled_amd import ops

pytestmark = pytest.mark.gpu


def weights(E, N, K, fmt, seed):
    g = np.random.default_rng(seed)
    w = g.integers(0, 256, (E, N, K // 2), dtype=np.uint8)
    if fmt == "nvfp4":
        s = g.integers(0, 0x50, (E, N, K // 16), dtype=np.uint8)
        hat = np.stack([oracle.dequant_nvfp4_weights(w[e], s[e]) for e in range(E)])
    else:
        s = g.integers(118, 131, (E, N, K // 32), dtype=np.uint8)
        hat = np.stack([oracle.dequant_weights(w[e], s[e]) for e in range(E)])
    return torch.from_numpy(w).cuda(), torch.from_numpy(s).cuda(), torch.from_numpy(hat).double()


def reference(a, src, offs, hat, swiglu):
    """(y, bound without the output rounding) in 64 bits; rows outside every expert are NaN."""
    E, N, K = hat.shape
    R = src.numel()
    cols = N // 2 if swiglu else N
    y = torch.full((R, cols), float("nan"), dtype=torch.float64)
    d = torch.zeros((R, cols), dtype=torch.float64)
    c = (K / 16 + 32) * 2.0 ** -23
    for e in range(E):
        rows = slice(offs[e], offs[e + 1])
        x = a[src[rows]].double()
        acc, mag = x @ hat[e].T, c * (x.abs() @ hat[e].abs().T)
        if swiglu:
            g, u = acc[:, :cols], acc[:, cols:]
            dg_, du = mag[:, :cols], mag[:, cols:]
            silu = g * torch.sigmoid(g)
            y[rows] = silu * u
            d[rows] = 1.1 * dg_ * (u.abs() + du) + silu.abs() * du + 2.0 ** -19 * (silu * u).abs()
        else:
            y[rows], d[rows] = acc, mag
    return y, d


def assert_close(got, want, d, what):
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    got = got.cpu().double()
    inside = ~torch.isnan(want)
    err = (got - want).abs()[inside]
    lim = (d + half * (want.abs() + d) + 1e-38)[inside]
    assert (err <= lim).all(), f"{what}: error {float((err / lim).max()):.3g} of its bound"


CASES = [
    # counts per expert; rows before and behind them; N, K, fmt, swiglu, dtype
    ([1], 0, 0, 16, 128, "mxfp4", False, torch.float32),
    ([0, 3, 0, 16, 1, 0], 0, 0, 64, 512, "mxfp4", False, torch.bfloat16),
    ([5, 0, 16, 2], 3, 4, 96, 640, "nvfp4", True, torch.bfloat16),
    ([16, 17, 0, 64, 1], 0, 0, 272, 384, "mxfp4", False, torch.float32),
    ([17, 33, 64, 2], 1, 9, 528, 1152, "nvfp4", False, torch.float32),
    ([63, 64, 65], 0, 0, 160, 256, "mxfp4", True, torch.float32),
    ([65, 0, 256, 257], 7, 5, 256, 128, "mxfp4", False, torch.bfloat16),
    ([300, 1, 20], 0, 2, 544, 896, "mxfp4", True, torch.bfloat16),
    ([130, 70], 0, 0, 48, 2048, "nvfp4", False, torch.bfloat16),
    ([200, 90, 513], 0, 0, 576, 320 * 2, "nvfp4", True, torch.float32),
    ([8] * 70, 0, 0, 80, 256, "mxfp4", False, torch.float32),  # more experts than lanes
    # wide enough for the tiled kernels beside the streaming one (more than 2560 streamed workgroups)
    ([300, 1, 20, 64, 65, 0, 16, 17, 257], 3, 5, 4112, 128, "mxfp4", False, torch.float32),
    ([130, 63, 500, 40], 0, 0, 4128, 384, "nvfp4", True, torch.bfloat16),
    ([90, 33, 128, 5, 700], 1, 0, 3616, 640, "mxfp4", True, torch.float32),
    ([256, 129, 18, 2, 0, 260], 0, 7, 4368, 1152, "nvfp4", False, torch.bfloat16),
    # large enough for a tiled launch per class of experts (1024 and more 128 x 256 tiles)
    ([500, 300, 200, 130, 100, 90, 65, 64, 40, 33, 20, 17, 16, 10, 5, 3, 1, 0, 0, 2, 1, 1, 1, 1], 2, 1, 7440, 128,
     "mxfp4", False, torch.bfloat16),
    ([1, 300, 200, 0, 100, 90, 65, 64, 40, 33, 700, 17, 16, 10, 5], 0, 0, 11296, 128, "nvfp4", True, torch.float32),
    ([3] * 260 + [40, 70], 0, 0, 1040, 256, "mxfp4", False, torch.float32),  # more experts than a lane batch holds
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}e{sum(c[0])}r-{c[3]}x{c[4]}-{c[5]}-{'swiglu' if c[6] else 'y'}")
@pytest.mark.parametrize("gather", [False, True])
def test_against_64_bits(case, gather):
    counts, before, behind, N, K, fmt, swiglu, dtype = case
    E, R = len(counts), sum(counts) + before + behind
    offs = [before + int(c) for c in np.cumsum([0] + counts)]
    w, s, hat = weights(E, N, K, fmt, R + N)
    topk = 1 if not gather else 2 if R % 2 == 0 else 1
    g = torch.Generator().manual_seed(R)
    pair = torch.randperm(R, generator=g).to(torch.int32)
    src = (pair // topk).long() if gather else torch.arange(R)
    a = torch.from_numpy(dg.activations(R, R // topk if gather else R, K).view(np.int16)).view(torch.bfloat16)
    out = torch.full((R, N // 2 if swiglu else N), 7.0, dtype=dtype, device="cuda")
    y = ops.moe_grouped_gemm_w4a16(a.cuda(), torch.tensor(offs, dtype=torch.int32).cuda(), w, s, fmt,
                                   sorted_pair=pair.cuda() if gather else None, topk=topk, swiglu=swiglu, out=out)
    torch.cuda.synchronize()
    want, d = reference(a, src, offs, hat, swiglu)
    assert_close(y, want, d, "y")
    outside = torch.isnan(want[:, 0])
    assert int(outside.sum()) == before + behind
    assert (y.cpu()[outside] == 7.0).all(), "rows outside every expert were written"


@pytest.mark.parametrize("fmt,swiglu,N,dtype", [("mxfp4", False, 4240, torch.float32), ("nvfp4", True, 4256, torch.bfloat16)])
@pytest.mark.parametrize("rows", ["few", "mixed"])
def test_many_experts_of_a_short_k(fmt, swiglu, N, dtype, rows):
    """128 experts of wide matrices with a short K, where a workgroup streams several runs of weight rows."""
    E, K = 128, 256
    g = np.random.default_rng(N)
    counts = np.zeros(E, int)
    if rows == "few":
        counts[g.permutation(E)[:100]] = 1
        counts[3], counts[77] = 9, 18
    else:
        counts = g.integers(0, 6, E)
        counts[5], counts[90], counts[127] = 30, 80, 17
    R = int(counts.sum())
    offs = np.concatenate([[0], np.cumsum(counts)])
    w = torch.from_numpy(g.integers(0, 256, (E, N, K // 2), dtype=np.uint8))
    lo, hi = (0, 0x50) if fmt == "nvfp4" else (118, 131)
    s = torch.from_numpy(g.integers(lo, hi, (E, N, K // (16 if fmt == "nvfp4" else 32)), dtype=np.uint8))
    a = torch.randn(R, K).to(torch.bfloat16)
    y = ops.moe_grouped_gemm_w4a16(a.cuda(), torch.from_numpy(offs.astype(np.int32)).cuda(), w.cuda(), s.cuda(), fmt,
                                   swiglu=swiglu, out_dtype=dtype)
    decode = oracle.dequant_nvfp4_weights if fmt == "nvfp4" else oracle.dequant_weights
    for e in (0, 3, 5, 41, 77, 90, 127):
        rows_e = slice(offs[e], offs[e + 1])
        if counts[e]:
            hat = torch.from_numpy(decode(w[e].numpy(), s[e].numpy()))[None].double()
            x = a[rows_e]
            want, d = reference(x, torch.arange(len(x)), [0, len(x)], hat, swiglu)
            assert_close(y[rows_e], want, d, f"expert {e}")


def test_one_row_is_its_own():
    """A row does not depend on what else its expert or the others hold: NaN and infinite rows beside it change
    nothing, and each row alone gives the bits that it gives among others of the same class."""
    E, N, K = 3, 4096, 256
    w, s, _ = weights(E, N, K, "mxfp4", 5)
    for counts in ([4, 9, 2], [40, 20, 61], [100, 500, 80], [50, 60, 600]):
        R = sum(counts)
        offs = torch.tensor(np.cumsum([0] + counts), dtype=torch.int32).cuda()
        a = torch.randn(R, K, generator=torch.Generator().manual_seed(R)).to(torch.bfloat16).cuda()
        want = ops.moe_grouped_gemm_w4a16(a, offs, w, s)
        bad = a.clone()
        rows = [0, counts[0], R - 1]
        bad[rows[0]], bad[rows[1]], bad[rows[2], 3] = float("nan"), float("inf"), float("-inf")
        got = ops.moe_grouped_gemm_w4a16(bad, offs, w, s)
        keep = torch.ones(R, dtype=torch.bool, device="cuda")
        keep[rows] = False
        assert torch.equal(got[keep], want[keep])
        assert not torch.isfinite(got[rows]).all(dim=1).any()


def test_offsets_are_held_to_the_rows():
    """Offsets outside [0, R] are taken as 0 and R; every write stays inside y."""
    for R, N in ((40, 64), (700, 4096)):
        check_offsets(R, N)


def check_offsets(R, N):
    E, K = 3, 128
    w, s, hat = weights(E, N, K, "mxfp4", 9)
    a = torch.randn(R, K).to(torch.bfloat16)
    raw = torch.full((3 * R, N), 3.0, device="cuda")
    y = raw[R:2 * R]
    ops.moe_grouped_gemm_w4a16(a.cuda(), torch.tensor([-5, 4, 30, 1000], dtype=torch.int32).cuda(), w, s, out=y)
    want, d = reference(a, torch.arange(R), [0, 4, 30, R], hat, False)
    assert_close(y, want, d, "y")
    assert (raw[:R] == 3).all() and (raw[2 * R:] == 3).all()


@pytest.mark.parametrize("R,N", [(40, 64), (800, 4096)])
def test_pairs_outside_the_rows_stay_inside_a(R, N):
    """Entries of sorted_pair outside their range spoil their own rows only."""
    E, K, topk = 2, 256, 2
    w, s, _ = weights(E, N, K, "mxfp4", 10)
    a = torch.randn(R // topk, K).to(torch.bfloat16).cuda()
    offs = torch.tensor([0, 12, R], dtype=torch.int32).cuda()
    pair = torch.randperm(R).to(torch.int32).cuda()
    want = ops.moe_grouped_gemm_w4a16(a, offs, w, s, sorted_pair=pair, topk=topk)
    bad = pair.clone()
    bad[3], bad[20], bad[R - 1] = -1, R + 5, 2 ** 31 - 1
    got = ops.moe_grouped_gemm_w4a16(a, offs, w, s, sorted_pair=bad, topk=topk)
    keep = torch.ones(R, dtype=torch.bool, device="cuda")
    keep[[3, 20, R - 1]] = False
    assert torch.equal(got[keep], want[keep])


def test_extreme_scale_bytes():
    """UE8M0 bytes at both ends of 2..252 in the streamed and the tiled kernel."""
    g = np.random.default_rng(3)
    for counts, N, K in (([3], 64, 256), ([30], 64, 256), ([700], 4096, 128)):
        for lo, hi, shift in ((2, 6, 60), (248, 252, -60)):
            w = g.integers(0, 256, (1, N, K // 2), dtype=np.uint8)
            s = g.integers(lo, hi + 1, (1, N, K // 32), dtype=np.uint8)
            hat = torch.from_numpy(oracle.dequant_weights(w[0], s[0]))[None].double()
            a = (torch.randn(counts[0], K) * 2.0 ** shift).to(torch.bfloat16)
            offs = [0, counts[0]]
            y = ops.moe_grouped_gemm_w4a16(a.cuda(), torch.tensor(offs, dtype=torch.int32).cuda(),
                                           torch.from_numpy(w).cuda(), torch.from_numpy(s).cuda(), out_dtype=torch.float32)
            want, d = reference(a, torch.arange(counts[0]), offs, hat, False)
            assert_close(y, want, d, f"scales {lo}..{hi}")


def test_every_ue4m3_scale():
    for R, N, K in ((2, 128, 1024), (33, 128, 1024), (700, 4096, 256)):
        check_ue4m3(R, N, K)


def check_ue4m3(R, N, K):
    w = np.random.default_rng(4).integers(0, 256, (1, N, K // 2), dtype=np.uint8)
    s = (np.arange(N * K // 16) % 0x7F).astype(np.uint8).reshape(1, N, K // 16)
    hat = torch.from_numpy(oracle.dequant_nvfp4_weights(w[0], s[0]))[None].double()
    a = torch.randn(R, K).to(torch.bfloat16)
    y = ops.moe_grouped_gemm_w4a16(a.cuda(), torch.tensor([0, R], dtype=torch.int32).cuda(),
                                   torch.from_numpy(w).cuda(), torch.from_numpy(s).cuda(), "nvfp4",
                                   out_dtype=torch.float32)
    want, d = reference(a, torch.arange(R), [0, R], hat, False)
    assert_close(y, want, d, "y")


def test_no_rows():
    w, s, _ = weights(2, 32, 128, "mxfp4", 1)
    z = torch.zeros(3, dtype=torch.int32, device="cuda")
    y = ops.moe_grouped_gemm_w4a16(torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"), z, w, s)
    assert y.shape == (0, 32)


@pytest.mark.parametrize("T,lo,hi", [(9, 0, 3), (9, 2, 6), (700, 3, 6), (700, 5, 5)])
def test_the_pairs_of_some_experts(T, lo, hi):
    """Experts lo .. hi - 1 with their own pairs and offsets give those experts' rows of the whole call."""
    E, N, K, topk = 6, 4112, 512, 2
    w, s, _ = weights(E, N, K, "mxfp4", 12)
    a = torch.from_numpy(dg.activations(13, T, K).view(np.int16)).view(torch.bfloat16).cuda()
    ids, gates, offs, sp, pr = ops.moe_route_permute(torch.from_numpy(dg.logits(13, T, E)).cuda(), topk)
    whole = ops.moe_grouped_gemm_w4a16(a, offs, w, s, sorted_pair=sp, topk=topk, out_dtype=torch.float32)
    o = offs.tolist()
    mine = ops.moe_grouped_gemm_w4a16(a, (offs[lo:hi + 1] - offs[lo]).contiguous() if hi > lo else offs[:2] * 0,
                                      w[lo:max(hi, lo + 1)], s[lo:max(hi, lo + 1)], sorted_pair=sp[o[lo]:o[hi]].clone(),
                                      topk=topk, out_dtype=torch.float32)
    assert mine.shape == (o[hi] - o[lo], N)
    err = (mine - whole[o[lo]:o[hi]]).abs()
    # another kernel may run an expert in the smaller call: the same products in another order
    x = a.float().abs()[(sp[o[lo]:o[hi]] // topk).long()]
    hat = torch.from_numpy(np.stack([oracle.dequant_weights(w[e].cpu().numpy(), s[e].cpu().numpy()) for e in range(lo, hi)])
                           ).float().cuda() if hi > lo else None
    for e in range(lo, hi):
        rows = slice(o[e] - o[lo], o[e + 1] - o[lo])
        assert (err[rows] <= 2 * (K / 16 + 32) * 2.0 ** -23 * (x[rows] @ hat[e - lo].abs().t().contiguous()) * 1.01).all()
    with pytest.raises(RuntimeError, match="sorted_pair"):
        ops.moe_grouped_gemm_w4a16(a, offs, w, s, sorted_pair=sp)  # topk forgotten

"""GPU parity of fp4_gemm_w4a16_lora against the formula in 64 bits.

Tolerance, from arithmetic: the projection is off by (K / 16 + 32) 2^-23 sum |a w| (weights and
products exact, see test_gpu_w4a16_grouped.py) and by 2^-24 for each of its K slices' sums. The low-rank product
of the first factor is off by the same with sum |a A|, scaled, plus one rounding; through the
second factor that is sum_r dlow |B|, to which come 2^-16 of sum |low B| where low is split into two
bf16 terms (each rounds by 2^-8 of what it holds) and (rank + 32) 2^-23 of it for the sum."""

import numpy as np
import pytest
import torch

import oracle
from mxfp4_block_scaled_amd import datagen as dg
from mxfp4_block_scaled_amd import ops
from tests.test_gpu_w4a16_grouped import weights

pytestmark = pytest.mark.gpu


def adapters(L, rank, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(L, rank, K, generator=g).mul(K ** -0.5).to(torch.bfloat16),
            torch.randn(L, N, rank, generator=g).to(torch.bfloat16), torch.rand(L, generator=g) + 0.5)


def reference(a, hat, offs, adapter, la, lb, scaling):
    K, rank = a.shape[1], la.shape[1]
    x = a.double()
    c = (K / 16 + 32) * 2.0 ** -23
    y = x @ hat.T
    d = (c + 32 * 2.0 ** -24) * (x.abs() @ hat.abs().T)
    for s, l in enumerate(adapter):
        if not 0 <= l < la.shape[0]:
            continue
        rows = slice(max(offs[s], 0), max(offs[s + 1], 0))
        A, B, sc = la[l].double(), lb[l].double(), float(scaling[l])
        low = sc * (x[rows] @ A.T)
        dlow = abs(sc) * (c + 16 * 2.0 ** -24) * (x[rows].abs() @ A.abs().T) + 2.0 ** -23 * low.abs()
        y[rows] += low @ B.T
        d[rows] += dlow @ B.abs().T + (2.0 ** -16 + (rank + 32) * 2.0 ** -23) * (low.abs() @ B.abs().T)
    return y, d


def close(got, want, d):
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    err, lim = (got.cpu().double() - want).abs(), d + half * (want.abs() + d)
    assert (err <= lim).all(), f"error {float((err / lim).max()):.3g} of its bound"


def bf16(seed, M, K):
    return torch.from_numpy(dg.activations(seed, M, K).view(np.int16)).view(torch.bfloat16)


CASES = [
    # segment lengths; rows before and behind them; N, K, rank, L, fmt, dtype
    ([1], 0, 0, 16, 512, 8, 1, "mxfp4", torch.float32),
    ([1], 0, 0, 4096, 2048, 32, 3, "nvfp4", torch.bfloat16),
    ([1] * 64, 0, 0, 272, 3584, 16, 24, "mxfp4", torch.float32),
    ([3, 0, 20, 0, 1, 17], 2, 5, 80, 1024, 24, 4, "mxfp4", torch.float32),
    ([64], 0, 0, 336, 512, 128, 2, "nvfp4", torch.float32),
    ([65], 0, 0, 144, 512, 8, 2, "mxfp4", torch.float32),
    ([1] * 70, 1, 3, 256, 512, 40, 9, "mxfp4", torch.bfloat16),
    ([100, 0, 0, 31, 200, 1, 7], 0, 20, 528, 1536, 72, 5, "nvfp4", torch.float32),
    ([5, 700, 60], 0, 0, 1040, 512, 64, 2, "mxfp4", torch.bfloat16),
    ([1] * 300, 5, 0, 272, 1024, 16, 7, "nvfp4", torch.float32),  # single rows, sliced
    ([100, 0, 1900, 3, 97], 0, 0, 1040, 512, 24, 3, "mxfp4", torch.bfloat16),  # 64 x 128 tiles, low in K slices
    ([7] * 300, 1, 2, 1040, 1536, 8, 5, "mxfp4", torch.float32),  # the same with short segments
    ([100, 3, 0, 90, 1, 200, 2, 371], 4, 6, 1520, 1024, 24, 5, "nvfp4", torch.bfloat16),  # sliced, long segments
    ([3] * 10 + [0] * 80 + [6] * 100 + [1], 0, 1, 1520, 512, 40, 6, "mxfp4", torch.float32),  # empty ones between
    ([1, 2] * 200 + [400], 2, 0, 1296, 512, 8, 3, "mxfp4", torch.float32),
    ([150, 50], 0, 0, 4112, 2048, 128, 2, "nvfp4", torch.float32),  # a wide adapter: few tiles, not sliced
    ([900, 3200], 0, 4, 4352, 512, 16, 2, "mxfp4", torch.float32),  # 128 x 256 tiles
    ([2049, 1, 2046], 0, 0, 4096, 512, 120, 3, "nvfp4", torch.bfloat16),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}s{sum(c[0])}r-{c[3]}x{c[4]}-r{c[5]}-{c[7]}")
def test_against_64_bits(case):
    lens, before, behind, N, K, rank, L, fmt, dtype = case
    M, S = sum(lens) + before + behind, len(lens)
    offs = [before + int(v) for v in np.cumsum([0] + lens)]
    adapter = [(i * 7 + 1) % (L + 1) - 1 for i in range(S)]  # -1 among them
    if S == 1:
        adapter = [L - 1]
    w, s, hat = weights(1, N, K, fmt, M + N)
    la, lb, scaling = adapters(L, rank, N, K, M)
    a = bf16(M, M, K)
    c = ops.fp4_gemm_w4a16_lora(a.cuda(), w[0], s[0], torch.tensor(offs, dtype=torch.int32).cuda(),
                                torch.tensor(adapter, dtype=torch.int32).cuda(), la.cuda(), lb.cuda(), scaling.cuda(),
                                fmt, out_dtype=dtype)
    want, d = reference(a, hat[0], offs, adapter, la, lb, scaling)
    close(c, want, d)


@pytest.mark.parametrize("M", [9, 130])
def test_no_adapter_is_the_projection(M):
    """S = 0, L = 0, every adapter -1 or outside [0, L), or segments that hold no row: the projection alone."""
    N, K, rank = 96, 1024, 16
    w, s, hat = weights(1, N, K, "mxfp4", 2)
    la, lb, scaling = (t.cuda() for t in adapters(2, rank, N, K, 4))
    a = bf16(1, M, K)
    want, d = reference(a, hat[0], [], [], la, lb, scaling)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    first = None
    for offs, ad, L in (([0], [], 2), ([0, M], [-1], 2), ([0, 4, M], [2, -9], 2), ([0, M], [0], 0), ([M, M], [1], 2),
                        ([0, 0, 0], [0, 1], 2)):
        c = ops.fp4_gemm_w4a16_lora(a.cuda(), w[0], s[0], i32(offs), i32(ad), la[:L], lb[:L], scaling[:L])
        close(c, want, d)
        first = c if first is None else first
        assert torch.equal(c, first)


@pytest.mark.parametrize("M", [8, 200])
def test_rows_and_adapters_stay_apart(M):
    """NaN in one request's rows, in an adapter nobody names and in the old workspace changes no other row."""
    N, K, rank, L = 272, 512, 24, 3
    w, s, _ = weights(1, N, K, "mxfp4", 6)
    la, lb, scaling = (t.cuda() for t in adapters(L, rank, N, K, 7))
    a = bf16(2, M, K).cuda()
    cut = M // 2 + 1
    offs = torch.tensor([0, cut, M], dtype=torch.int32).cuda()
    ad = torch.tensor([1, 0], dtype=torch.int32).cuda()
    want = ops.fp4_gemm_w4a16_lora(a, w[0], s[0], offs, ad, la, lb, scaling)
    need = ops.load().fp4_w4a16_lora_workspace_bytes(M, N, K, rank)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    la[2], lb[2], scaling[2] = float("nan"), float("nan"), float("nan")
    a[cut + 1] = float("nan")
    got = ops.fp4_gemm_w4a16_lora(a, w[0], s[0], offs, ad, la, lb, scaling, workspace=ws)
    keep = [t for t in range(M) if t != cut + 1]
    assert torch.equal(got[keep], want[keep]) and torch.isnan(got[cut + 1]).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("M,N,K,rank", [(9, 272, 512, 24), (777, 1520, 512, 24), (200, 4112, 512, 128),
                                        (4100, 4352, 512, 16)])
def test_an_adapter_that_is_not_finite_reaches_its_own_rows_only(M, N, K, rank, bad):
    """One of the adapters in use holds a NaN or an infinity: the requests beside it keep their results bit for
    bit, and its own rows show it (sliced; 64 x 128 tiles, 128 x 256 tiles)."""
    L = 3
    w, s, _ = weights(1, N, K, "mxfp4", 6)
    la, lb, scaling = (t.cuda() for t in adapters(L, rank, N, K, 7))
    a = bf16(2, M, K).cuda()
    lo, hi = M // 2 - 3, M // 2 + 2  # inside one tile, with rows of others (and of none) before and behind
    offs = torch.tensor([0, lo - 1, lo, hi, M - 1, M], dtype=torch.int32).cuda()
    ad = torch.tensor([1, -1, 2, 0, 2], dtype=torch.int32).cuda()
    want = ops.fp4_gemm_w4a16_lora(a, w[0], s[0], offs, ad, la, lb, scaling)
    lb[2, 5, 3] = lb[2, N - 1, rank - 1] = bad
    got = ops.fp4_gemm_w4a16_lora(a, w[0], s[0], offs, ad, la, lb, scaling)
    own = torch.zeros(M, dtype=torch.bool, device="cuda")
    own[lo:hi] = own[M - 1] = True
    assert torch.equal(got[~own], want[~own])
    cols = torch.zeros(N, dtype=torch.bool, device="cuda")
    cols[5] = cols[N - 1] = True
    assert not torch.isfinite(got[own][:, cols]).any() and torch.equal(got[own][:, ~cols], want[own][:, ~cols])


@pytest.mark.parametrize("M,N,K,rank", [(9, 272, 512, 24), (200, 4112, 512, 128), (4100, 4352, 512, 16)])
def test_an_infinite_first_product_stays_infinite(M, N, K, rank):
    w, s, _ = weights(1, N, K, "mxfp4", 6)
    la, lb, scaling = adapters(1, rank, N, K, 7)
    la[0, rank - 1, 17] = float("inf")
    a = bf16(2, M, K)
    assert (a[:, 17] != 0).all() and (lb[0, :, rank - 1] != 0).all()
    got = ops.fp4_gemm_w4a16_lora(a.cuda(), w[0], s[0], torch.tensor([0, M], dtype=torch.int32).cuda(),
                                  torch.zeros(1, dtype=torch.int32).cuda(), la.cuda(), lb.cuda(), scaling.cuda(),
                                  out_dtype=torch.float32)
    want = float("inf") * a[:, 17, None].float().sign() * lb[0, None, :, rank - 1].float().sign()
    assert torch.equal(got.cpu(), want)


def test_no_rows():
    w, s, _ = weights(1, 32, 512, "mxfp4", 1)
    la, lb, scaling = (t.cuda() for t in adapters(1, 8, 32, 512, 1))
    z = torch.zeros(2, dtype=torch.int32, device="cuda")
    c = ops.fp4_gemm_w4a16_lora(torch.empty(0, 512, dtype=torch.bfloat16, device="cuda"), w[0], s[0], z, z[:1], la, lb,
                                scaling)
    assert c.shape == (0, 32)


def single_terms(M, N, K, rank, seed, scaling):
    """An adapter 0 whose first product is one term a row and nothing else, so that its fp32 value is known exactly:
    low[t][0] = fp32(scaling * a[t][17] * lora_a[0][17]). Adapter 1 is all zeros."""
    g = torch.Generator().manual_seed(seed)
    a = bf16(seed, M, K)
    la, lb = torch.zeros(2, rank, K, dtype=torch.bfloat16), torch.zeros(2, N, rank, dtype=torch.bfloat16)
    la[0, 0, 17] = 1.3828125  # all eight bits of a bf16 in use
    lb[0] = torch.randn(N, rank, generator=g).to(torch.bfloat16)
    sc = torch.tensor([scaling, 1.0])
    low = (a[:, 17].float() * la[0, 0, 17].float()) * sc[0]  # the product of two bf16 is exact in fp32
    return a, la, lb, sc, low


# sliced; 64 x 128 tiles; 128 x 256 tiles
PATHS = [(9, 272, 512, 24), (777, 1520, 512, 24), (200, 4112, 512, 128), (4100, 4352, 512, 16)]


@pytest.mark.parametrize("scaling", [1.1, -2.9e38])
@pytest.mark.parametrize("M,N,K,rank", PATHS)
def test_the_first_product_is_held_in_fp32(M, N, K, rank, scaling):
    """With one term a row and a weight of next to nothing the result is low * B: low has 24 bits, B 8, and a path
    that holds low in fp32 only rounds in the sums of the at most three products it may split that into (2^-23 each,
    rounded or cut off) and, the weights' part being below 2^-23 of it, once more. The larger scaling makes some low
    greater than the largest bf16 and others larger than the largest fp32."""
    w, s, hat = weights(1, N, K, "mxfp4", 6)
    s = (s - 118) // 6 + 2  # 2^-125 .. 2^-123
    a, la, lb, sc, low = single_terms(M, N, K, rank, 2, scaling)
    a[:, 17] = torch.linspace(0.06, 0.9, M).to(torch.bfloat16)
    low = (a[:, 17].float() * la[0, 0, 17].float()) * sc[0]
    edge = (low.abs() > torch.finfo(torch.bfloat16).max) & torch.isfinite(low)
    if abs(scaling) > 2:
        lb = (lb.float() * 2.0 ** -30).to(torch.bfloat16)
        assert torch.isinf(low).any() and torch.isfinite(low).any()
        if M > 4000:
            assert edge.any()
    got = ops.fp4_gemm_w4a16_lora(a.cuda(), w[0], s[0], torch.tensor([0, M], dtype=torch.int32).cuda(),
                                  torch.zeros(1, dtype=torch.int32).cuda(), la.cuda(), lb.cuda(), sc.cuda()).cpu()
    B = lb[0, :, 0].double()
    want = low.double()[:, None] * B
    fin = torch.isfinite(low)
    err, lim = (got.double() - want).abs()[fin], (4 * 2.0 ** -23 * want.abs() + K * 2.0 ** -110)[fin]
    assert (err <= lim).all(), f"{float((err / lim).max()):.3g} of its bound"
    assert torch.equal(got[~fin].double(), want[~fin])


@pytest.mark.parametrize("whole", [True, False])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf")])
@pytest.mark.parametrize("M,N,K,rank", PATHS)
def test_an_infinite_second_factor_gives_signed_infinities(M, N, K, rank, bad, whole):
    """low * B with B infinite is the infinity of their signs, whatever the bits of low, and NaN where low is 0; the
    same in every path, in segments that fill tiles and in ones that do not."""
    w, s, _ = weights(1, N, K, "mxfp4", 6)
    a, la, lb, sc, low = single_terms(M, N, K, rank, 2, 1.1)
    a[M // 2], low[M // 2] = 0, 0
    assert (low != 0).sum() == M - 1
    lo, hi = (0, M) if whole else (M // 3, M - 2)
    args = (torch.tensor([0, lo, hi, M], dtype=torch.int32).cuda(), torch.tensor([1, 0, 1], dtype=torch.int32).cuda(),
            la.cuda())
    plain = ops.fp4_gemm_w4a16_lora(a.cuda(), w[0], s[0], *args, lb.cuda(), sc.cuda())
    cols = [5, N - 1]
    lb[0, cols, 0] = bad
    got = ops.fp4_gemm_w4a16_lora(a.cuda(), w[0], s[0], *args, lb.cuda(), sc.cuda()).cpu()
    want = plain.cpu().clone()
    for c in cols:
        want[lo:hi, c] = low[lo:hi] * bad
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and int(torch.isnan(want).sum()) == len(cols)
    assert torch.equal(got.nan_to_num(7.0, posinf=float("inf"), neginf=float("-inf")),
                       want.nan_to_num(7.0, posinf=float("inf"), neginf=float("-inf")))

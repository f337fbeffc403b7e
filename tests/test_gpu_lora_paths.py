"""fp4_gemm_w4a16_lora in each of its forms, by name: every case asserts from the library's rule which tiles and how many
K slices its call takes. Against 64 bits, with the first product's fp32 sums in the bound:
dlow = |scaling| (K / 16 + 48) 2^-23 sum |a A| + 2^-23 |low|, and the result is off by
(K / 16 + 32 + rank) 2^-23 (sum |a W| + sum |low B|) + sum dlow |B| (an fp32 low splits into three bf16 terms exactly,
so each 16 ranks are three dependent instructions, or 16 fused multiply-adds)."""

import pytest
import torch

from mxfp4_block_scaled_amd import ops
from tests.test_gpu_canary import Guarded
from tests.w4a16_exact import close, lora_path, product, weights

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32

CASES = [
    # lengths of the segments; rows before and behind; N, K, rank, L, fmt, dtype; K slices of the projection and of the
    # first product, rows of its workgroups, tile
    ([1000, 0, 3, 997], 0, 0, 4096, 4096, 64, 3, "mxfp4", F32, (0, 4, 32, 128, 256)),
    ([700, 1290], 4, 6, 4096, 4096, 40, 2, "nvfp4", BF, (0, 4, 32, 128, 256)),
    ([2100, 1, 1899], 0, 0, 2064, 2048, 128, 4, "mxfp4", BF, (0, 2, 32, 128, 256)),
    ([1300, 2700], 0, 0, 2064, 7168, 8, 2, "nvfp4", F32, (0, 2, 32, 128, 256)),
    ([9] * 220, 10, 10, 4096, 3584, 24, 7, "mxfp4", F32, (0, 1, 16, 128, 256)),  # short segments
    ([600, 0, 890], 5, 5, 4112, 4096, 32, 3, "nvfp4", F32, (0, 4, 32, 64, 128)),
    ([1000], 0, 0, 7168, 2048, 120, 1, "mxfp4", BF, (0, 2, 32, 64, 128)),
    ([11] * 130, 0, 3, 4112, 4608, 72, 5, "mxfp4", F32, (0, 1, 16, 64, 128)),
    ([1] * 64, 0, 0, 4096, 7168, 16, 24, "mxfp4", F32, (8, 8, 16, 64, 128)),  # sliced: a decode batch
    ([1] * 33 + [30], 0, 1, 4096, 7168, 64, 9, "nvfp4", BF, (8, 14, 16, 64, 128)),
    ([7, 0, 300, 1, 400], 9, 60, 1520, 2048, 24, 5, "nvfp4", F32, (3, 8, 16, 64, 128)),
    ([1], 0, 0, 2048, 2048, 32, 4, "mxfp4", BF, (8, 8, 16, 64, 128)),
]


def make(case, seed):
    lens, before, behind, N, K, rank, L, fmt, dtype, want = case
    S, M = len(lens), sum(lens) + before + behind
    path = lora_path(M, N, K, rank, S)
    assert (*path[:3], *path[4:]) == want, path
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
    w, s = weights((N,), K, fmt, gen)
    offs = [before]
    for n in lens:
        offs.append(offs[-1] + n)
    adapter = [(7 * i + 1) % (L + 1) - 1 if S > 1 else L - 1 for i in range(S)]
    t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    return (rn(M, K).to(BF), w, s, t(offs), t(adapter), (rn(L, rank, K) * K ** -0.5).to(BF), rn(L, N, rank).to(BF),
            torch.rand(L, device="cuda", generator=gen) + 0.5, fmt), offs, adapter


def reference(args, offs, adapter):
    a, w, s, _, _, la, lb, scaling, fmt = args
    K, rank = a.shape[1], la.shape[1]
    y, mag = product(a, w, s, fmt)
    extra = torch.zeros_like(y)
    for i, l in enumerate(adapter):
        if 0 <= l < la.shape[0] and offs[i + 1] > offs[i]:
            rows, sc = slice(offs[i], offs[i + 1]), scaling[l].double()
            A, B, x = la[l].double().t().contiguous(), lb[l].double().t().contiguous(), a[rows].double()
            low = sc * (x @ A)
            dlow = sc * (K / 16 + 48) * 2.0 ** -23 * (x.abs() @ A.abs()) + 2.0 ** -23 * low.abs()
            y[rows] += low @ B
            mag[rows] += low.abs() @ B.abs()
            extra[rows] = dlow @ B.abs()
    return y, (K / 16 + 32 + rank) * 2.0 ** -23 * mag + extra


IDS = [f"{len(c[0])}s{sum(c[0])}r-{c[3]}x{c[4]}-r{c[5]}-{c[7]}-{c[9][3]}x{c[9][4]}" for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_against_64_bits(case):
    args, offs, adapter = make(case, 1)
    close(ops.fp4_gemm_w4a16_lora(*args, out_dtype=case[8]), *reference(args, offs, adapter))


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_writes_and_rows_stay_apart(case):
    """Result and workspace stay inside their buffers, whatever the workspace held; NaN in one row and in an adapter
    nobody names changes no other row; the call repeats itself bit for bit."""
    args, offs, adapter = make(case, 2)
    a, w, s, so, sa, la, lb, scaling, fmt = args
    M, (L, rank, K), N, dtype = a.shape[0], la.shape, w.shape[0], case[8]
    want = ops.fp4_gemm_w4a16_lora(*args, out_dtype=dtype)
    need = ops.load().fp4_w4a16_lora_workspace_bytes(M, N, K, rank)
    c, ws = Guarded((M, N), dtype, 3), Guarded((need,), torch.uint8, 4)
    ws.t.fill_(255)  # NaN
    la, lb, scaling = (torch.cat([t, torch.full_like(t[:1], float("nan"))]) for t in (la, lb, scaling))
    bad = a.clone()
    bad[M // 2, 3] = float("nan")
    ops.fp4_gemm_w4a16_lora(bad, w, s, so, sa, la, lb, scaling, fmt, out=c.t, workspace=ws.t)
    torch.cuda.synchronize()
    c.check("c")
    ws.check("workspace")
    keep = torch.arange(M, device="cuda") != M // 2
    assert torch.equal(c.t[keep], want[keep]) and torch.isnan(c.t[M // 2]).all()


@pytest.mark.parametrize("case", [CASES[i] for i in (0, 2, 4, 5, 8, 10)], ids=[IDS[i] for i in (0, 2, 4, 5, 8, 10)])
def test_replays_match_eager(case):
    """Captured twice, with inputs that change between the replays and eager calls beside them."""
    one, other = make(case, 5)[0], make(case, 6)[0]
    dtype = case[8]
    eager = [ops.fp4_gemm_w4a16_lora(*x, out_dtype=dtype).clone() for x in (one, other)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ops.fp4_gemm_w4a16_lora(*one, out_dtype=dtype)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ops.fp4_gemm_w4a16_lora(*one, out_dtype=dtype))
        graphs.append(g)
    kept = one[0].clone()
    for rep in range(4):
        one[0].copy_(other[0] if rep % 2 else kept)
        want = ops.fp4_gemm_w4a16_lora(*one, out_dtype=dtype).clone()
        assert rep % 2 or torch.equal(want, eager[0])
        for g in graphs:
            g.replay()
        ops.fp4_gemm_w4a16_lora(*other, out_dtype=dtype)
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)

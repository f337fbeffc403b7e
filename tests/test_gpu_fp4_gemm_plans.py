"""fp4_gemm in each of its kernels by name: every tile shape with 1, 2, 4 and 8 K slices in both formats (the plan is
asserted), against 64 bits and with a one in each row of either operand, which leaves the other's values exactly."""

import ctypes

import pytest
import torch

from mxfp4_block_scaled_amd import ops
from tests.test_gpu_fp4_gemm import _check, _operand, _values

pytestmark = pytest.mark.gpu

# format, tile, K slices: sizes
PLANS = [
    ("mxfp4", 32, 32, 1, (24, 528, 1152)), ("nvfp4", 32, 32, 1, (24, 528, 1152)),
    ("mxfp4", 64, 64, 1, (66, 5552, 128)), ("mxfp4", 64, 64, 2, (100, 4256, 6528)),
    ("mxfp4", 64, 64, 4, (35, 4288, 6784)), ("mxfp4", 64, 64, 8, (1, 16, 15232)),
    ("mxfp4", 64, 128, 1, (515, 6560, 128)), ("mxfp4", 64, 128, 2, (261, 5808, 29568)),
    ("mxfp4", 64, 128, 4, (135, 4160, 12672)), ("mxfp4", 64, 128, 8, (1, 4144, 30592)),
    ("mxfp4", 128, 128, 1, (450, 6208, 128)), ("mxfp4", 128, 128, 2, (280, 3408, 16896)),
    ("mxfp4", 128, 128, 4, (66, 5712, 7424)), ("mxfp4", 128, 128, 8, (71, 2928, 11392)),
    ("mxfp4", 256, 256, 1, (4397, 1808, 128)), ("mxfp4", 256, 256, 2, (520, 7728, 11136)),
    ("mxfp4", 256, 256, 4, (263, 6560, 13824)), ("mxfp4", 256, 256, 8, (130, 5760, 14208)),
    ("nvfp4", 64, 64, 1, (97, 6464, 128)), ("nvfp4", 64, 64, 2, (4915, 144, 6016)),
    ("nvfp4", 64, 64, 4, (4277, 48, 6912)), ("nvfp4", 64, 64, 8, (1, 16, 8064)),
    ("nvfp4", 64, 128, 1, (130, 6544, 128)), ("nvfp4", 64, 128, 2, (169, 4208, 6272)),
    ("nvfp4", 64, 128, 4, (35, 4288, 6784)), ("nvfp4", 64, 128, 8, (1, 2064, 12032)),
    ("nvfp4", 128, 128, 1, (323, 5472, 128)), ("nvfp4", 128, 128, 2, (237, 4160, 5120)),
    ("nvfp4", 128, 128, 4, (67, 5792, 4992)), ("nvfp4", 128, 128, 8, (97, 2176, 5760)),
    ("nvfp4", 256, 256, 1, (4397, 1808, 128)), ("nvfp4", 256, 256, 2, (518, 7424, 6528)),
    ("nvfp4", 256, 256, 4, (324, 5872, 7040)), ("nvfp4", 256, 256, 8, (133, 5664, 7808)),
]


def _ones(rows, K, fmt, seed):
    """(codes, scales, k): row r is zero but for a one at k[r]."""
    k = torch.randint(0, K, (rows,), generator=torch.Generator().manual_seed(seed))
    k[-1] = K - 1
    q = torch.zeros((rows, K // 2), dtype=torch.uint8)
    q[torch.arange(rows), k // 2] = torch.where(k % 2 == 0, 2, 32).to(torch.uint8)
    nv = fmt == "nvfp4"
    s = torch.full((rows, K // (16 if nv else 32)), 0x38 if nv else 127, dtype=torch.uint8)
    return q.cuda(), s.cuda(), k.cuda()


@pytest.mark.parametrize("fmt,bm,bn,slices,size", PLANS)
def test_each_kernel(fmt, bm, bn, slices, size):
    M, N, K = size
    out = (ctypes.c_int32 * 3)()
    fn = ops.load().mxf_fp4_pair_plan
    fn.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int, ctypes.c_void_p]
    fn(M, N, K, ops.WEIGHT_FMTS[fmt], out)
    assert list(out) == [bm, bn, slices]
    a, sa = _operand(M, K, fmt, M)
    b, sb = _operand(N, K, fmt, N + 1)
    for dt in (torch.float32, torch.bfloat16):
        got = ops.fp4_gemm(a, sa, b, sb, fmt, out_dtype=dt)
        _check(got, a, sa, b, sb, fmt)
        assert torch.equal(got, ops.fp4_gemm(a, sa, b, sb, fmt, out_dtype=dt))
    a, sa = _operand(M, K, fmt, M + 2, wide=True)
    q, s, k = _ones(N, K, fmt, 3)
    assert torch.equal(ops.fp4_gemm(a, sa, q, s, fmt, out_dtype=torch.float32).double(), _values(a, sa, fmt)[:, k])
    b, sb = _operand(N, K, fmt, N + 3, wide=True)
    q, s, k = _ones(M, K, fmt, 4)
    assert torch.equal(ops.fp4_gemm(q, s, b, sb, fmt, out_dtype=torch.float32).double(), _values(b, sb, fmt)[:, k].t())

"""fp4_gemm with tensor scales at both ends of fp32: their product is what counts, not the order they are applied in.

The sum v is off as in test_gpu_fp4_gemm.py. With g_a = m_a 2^i and g_b = m_b 2^j the result is v (m_a m_b) 2^(i + j): two
roundings of half a step (2^-24 of the value each; none for powers of two), and where it lies below 2^-126 one to a
multiple of 2^-149."""

import pytest
import torch

from mxfp4_block_scaled_amd import ops
from tests.test_gpu_fp4_gemm import _operand, _plan, _values

pytestmark = pytest.mark.gpu

# the few-tile kernel, unsliced tiles, K slices
SIZES = [(24, 528, 1152, "32 x 32"), (130, 6544, 128, "64 x 128"), (4400, 1808, 128, "256 x 256"),
         (100, 272, 16256, "64 x 64, sliced")]
SCALES = [(2.0 ** 117, 2.0 ** -100), (2.0 ** -126, 2.0 ** 100), (1.7 * 2.0 ** 116, 1.3 * 2.0 ** -110),
          (1.9 * 2.0 ** -126, 1.1 * 2.0 ** 90), (2.0 ** -126, 2.0 ** -20), (3.0 * 2.0 ** -140, 2.0 ** 110), (2.0 ** -80, 2.0 ** -80)]


@pytest.mark.parametrize("M,N,K,plan", SIZES)
def test_far_scales(M, N, K, plan):
    assert _plan(M, N, K, "nvfp4") == plan
    a, sa = _operand(M, K, "nvfp4", 1)
    b, sb = _operand(N, K, "nvfp4", 2)
    x, y = _values(a, sa, "nvfp4"), _values(b, sb, "nvfp4")
    v, size = torch.mm(x, y.t().contiguous()), torch.mm(x.abs(), y.abs().t().contiguous())
    for ga, gb in SCALES:
        for p, q in ((ga, gb), (gb, ga)):
            tp, tq = torch.tensor([p]).cuda(), torch.tensor([q]).cuda()
            g = float(tp) * float(tq)
            want = v * g
            for dt, step in ((torch.float32, 2.0 ** -23), (torch.bfloat16, 2.0 ** -23 + 2.0 ** -8)):
                got = ops.fp4_gemm(a, sa, b, sb, "nvfp4", tp, tq, out_dtype=dt)
                tol = (K / 8 + 16) * 2.0 ** -23 * size * g + step * want.abs() + (2.0 ** -149 if dt == torch.float32 else 2.0 ** -133)
                assert ((got.double() - want).abs() <= tol).all(), (p, q, dt)
            if p in (2.0 ** 117, 2.0 ** -126) and g >= 2.0 ** -40:  # powers of two, far from the ends: exact
                plain = ops.fp4_gemm(a, sa, b, sb, "nvfp4", out_dtype=torch.float32)
                got = ops.fp4_gemm(a, sa, b, sb, "nvfp4", tp, tq, out_dtype=torch.float32)
                assert torch.equal(got.double(), plain.double() * g)


def test_no_scale_beside_a_far_one():
    a, sa = _operand(40, 512, "nvfp4", 3)
    b, sb = _operand(64, 512, "nvfp4", 4)
    plain = ops.fp4_gemm(a, sa, b, sb, out_dtype=torch.float32)
    for g in (2.0 ** 100, 2.0 ** -100, 0.0):
        t = torch.tensor([g]).cuda()
        for args in ((t, None), (None, t)):
            got = ops.fp4_gemm(a, sa, b, sb, "nvfp4", *args, out_dtype=torch.float32)
            assert torch.equal(got, plain * g)

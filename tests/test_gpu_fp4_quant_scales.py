"""fp4_quantize with a tensor scale anywhere in fp32's range, subnormal ones included: scales and codes of the definition,
and the transposed form alike. With bf16 values and powers of two x / d is exact enough for equality (as in
test_gpu_fp4_quant.py), else codes beside a border may be one step off."""

import numpy as np
import pytest
import torch

from mxfp4_block_scaled_amd import ops
from tests import train_exact as ex
from tests.test_gpu_fp4_quant import _compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("g", [2.0 ** 127, 2.0 ** 126, 2.0 ** 124, 3.0e38, 2.0 ** 99, 2.0 ** -79, 2.0 ** -110, 2.0 ** -126, 2.0 ** -130,
                               3 * 2.0 ** -137, 2.0 ** -149])
@pytest.mark.parametrize("size", [0.4, 2.5, 600.0, 2500.0])
def test_a_scale_from_either_end(g, size):
    """Blocks around size x g: s from its subnormals to 448."""
    rows, cols = 40, 96
    gen = torch.Generator().manual_seed(int(size * 10))
    x = torch.rand((rows, cols), generator=gen, dtype=torch.float64) * 2 - 1
    x = x * torch.exp2(-torch.randint(0, 3, (rows, 1), generator=gen).double()) * size
    x = (x * g).clamp(-3.3e38, 3.3e38).float().bfloat16()
    gt = torch.tensor([g], dtype=torch.float32)
    assert float(gt) > 0
    exact = float(np.log2(float(gt))).is_integer()
    xd = x.double().numpy()
    d = ops.fp4_quantize(x.cuda(), "nvfp4", gt.cuda(), transposed=True)
    _compare(d["q"], d["q_scale"], xd, "nvfp4", float(gt), None, exact)
    _compare(d["qt"], d["qt_scale"], ex.transposed(xd), "nvfp4", float(gt), None, exact)


@pytest.mark.parametrize("shuffled", [False, True])
def test_mxfp4_rows_are_those_of_the_activations_for_every_value(shuffled):
    """Every finite bf16 value, in blocks of neighbours and in mixed ones."""
    bits = torch.arange(65536, dtype=torch.int32)
    bits = bits[(bits & 0x7F80) != 0x7F80]
    if shuffled:
        bits = bits[torch.randperm(bits.numel(), generator=torch.Generator().manual_seed(1))]
    x = bits.to(torch.int16).view(torch.bfloat16).view(-1, 64).cuda()
    q, s = ops.mxfp4_quantize_act(x, "e2m1")
    d = ops.fp4_quantize(x, "mxfp4")
    assert torch.equal(d["q"], q) and torch.equal(d["q_scale"], s)

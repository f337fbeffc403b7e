"""The operators of training with nothing to work on: a linear layer's step of no tokens, as an expert or a shard that
got none runs it. The C entry points refuse sizes without a meaning there (a maximum of no values, a sum over K = 0);
the binding answers them: scale 1, products of zeros."""

import pytest
import torch

from mxfp4_block_scaled_amd import ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_a_linear_layers_step_of_no_tokens(fmt):
    O, I = 256, 384
    nv = fmt == "nvfp4"
    w = torch.randn((O, I)).bfloat16().cuda()
    x, dy = (torch.empty((0, n), dtype=torch.bfloat16).cuda() for n in (I, O))
    gx, gw, gy = (ops.nvfp4_tensor_scale(t) if nv else None for t in (x, w, dy))
    if nv:
        assert gx.tolist() == [1.0] and gx.dtype == torch.float32 and gx.device == x.device
    qx, qw = (ops.fp4_quantize(t, fmt, g, transposed=True) for t, g in ((x, gx), (w, gw)))
    rnd = torch.empty((0, O), dtype=torch.uint8).cuda()
    qd = ops.fp4_quantize(dy, fmt, gy, rnd=rnd, transposed=True)
    y = ops.fp4_gemm(qx["q"], qx["q_scale"], qw["q"], qw["q_scale"], fmt, gx, gw)
    dx = ops.fp4_gemm(qd["q"], qd["q_scale"], qw["qt"], qw["qt_scale"], fmt, gy, gw)
    dw = ops.fp4_gemm(qd["qt"], qd["qt_scale"], qx["qt"], qx["qt_scale"], fmt, gy, gx, out_dtype=torch.float32)
    assert y.shape == (0, O) and dx.shape == (0, I)
    assert dw.shape == (O, I) and dw.dtype == torch.float32 and not dw.any()
    given = torch.full((O, I), 7.0).cuda()
    assert ops.fp4_gemm(qd["qt"], qd["qt_scale"], qx["qt"], qx["qt_scale"], fmt, gy, gx, out=given) is given
    assert not given.any()
    for a in ("q", "qt"):
        back = ops.fp4_dequantize(qx[a], qx[a + "_scale"], fmt, gx)
        assert back.shape == ((0, I) if a == "q" else (I, 0)) and back.dtype == torch.bfloat16


def test_refusals_stay():
    x = torch.empty((0, 64), dtype=torch.bfloat16).cuda()
    q, s = torch.empty((24, 0), dtype=torch.uint8).cuda(), torch.empty((24, 0), dtype=torch.uint8).cuda()
    with pytest.raises(RuntimeError):
        ops.fp4_gemm(q, s, q, s)  # N % 16
    with pytest.raises(RuntimeError):
        ops.fp4_gemm(q[:16], s[:16], q[:16], s[:16], out_dtype=torch.float16)
    with pytest.raises(RuntimeError):
        ops.fp4_gemm(q[:16], s[:16], q[:16], s[:16], out=torch.empty((16, 8)).cuda())
    with pytest.raises(RuntimeError):
        ops.fp4_dequantize(q, s, out_dtype=torch.float16)
    with pytest.raises(RuntimeError):
        ops.nvfp4_tensor_scale(x.half())
    with pytest.raises(RuntimeError):
        ops.nvfp4_tensor_scale(torch.empty((3, 16), dtype=torch.bfloat16).cuda())  # 48 values

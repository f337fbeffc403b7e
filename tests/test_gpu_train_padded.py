"""A 4-bit linear layer whose inputs are no multiple of 128, the products' step of K: the columns are filled up with
zeros before they are quantised, which adds nothing to any sum."""

import pytest
import torch

from mxfp4_block_scaled_amd import ops
from tests import train_exact as ex

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,I,O", [(5, 96, 64), (300, 2880, 320)])
def test_columns_filled_up(fmt, T, I, O):
    g = torch.Generator().manual_seed(I)
    x, w = (torch.randn(s, generator=g).bfloat16().cuda() for s in ((T, I), (O, I)))
    nv = fmt == "nvfp4"
    plain = [ops.fp4_quantize(t, fmt) for t in (x, w)]
    with pytest.raises(RuntimeError):
        ops.fp4_gemm(plain[0]["q"], plain[0]["q_scale"], plain[1]["q"], plain[1]["q_scale"], fmt)
    full = [ops.fp4_quantize(torch.nn.functional.pad(t, (0, -I % 128)), fmt, transposed=True) for t in (x, w)]
    for p, f in zip(plain, full):  # the same codes, then zeros
        assert torch.equal(f["q"][:, :I // 2], p["q"]) and not f["q"][:, I // 2:].any()
        assert torch.equal(f["q_scale"][:, :p["q_scale"].shape[1]], p["q_scale"])
    y = ops.fp4_gemm(full[0]["q"], full[0]["q_scale"], full[1]["q"], full[1]["q_scale"], fmt, out_dtype=torch.float32)
    u, v = (ex.values(p["q"].cpu().numpy(), p["q_scale"].cpu().numpy(), fmt) for p in plain)
    K = I + -I % 128
    assert (abs(y.double().cpu().numpy() - u @ v.T) <= (K / 8 + 16) * 2.0 ** -23 * (abs(u) @ abs(v).T) + 1e-40).all()
    # the transposed results have rows for the columns added: all zeros
    assert not full[1]["qt"][I:].any() and (not nv or not full[1]["qt_scale"][I:].any())

"""The router's losses and gradient for expert counts that end early in a wave's last steps of 64 (columns past the
experts cost whole steps), few rows of them, and memory around the result; tolerances of test_gpu_route_loss.py."""

import pytest
import torch

from mxfp4_block_scaled_amd import ops
from tests.test_gpu_route_loss import _case, _check

pytestmark = pytest.mark.gpu

WIDTHS = [129, 130, 160, 191, 192, 257, 300, 384, 447, 448, 513, 700, 959, 960]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("E", WIDTHS)
def test_widths(E, bf16):
    for T in (1, 9, 70):  # fewer rows than a wave takes, a workgroup's waves without any, two launches
        _check(*_case(T, E, 6, T + E, bf16), None, None)
    _check(*_case(67, E, 3, E, bf16), None, [0, 1, 1, 40, 66])


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("E", WIDTHS)
@pytest.mark.parametrize("T", [1, 6])
def test_nothing_around_the_gradient_is_written(T, E, bf16):
    logits, ids, gates, dgates = (t.cuda() for t in _case(T, E, 5, E, bf16))
    d = ops.moe_balance_loss(logits, ids)
    dl = torch.tensor([0.3, 0.1]).cuda()
    want = ops.moe_route_backward(logits, ids, gates, dgates, d, dl)
    room = torch.full((T * E + 2048,), 7.0, dtype=logits.dtype).cuda()
    at = room[1024:]
    ops._call("moe_route_backward", logits.get_device(), logits.data_ptr(), ops.DTYPES[logits.dtype], ids.data_ptr(),
              gates.data_ptr(), dgates.data_ptr(), dl.data_ptr(), d["lse"].data_ptr(), d["counts"].data_ptr(),
              d["tokens"].data_ptr(), None, 1, T, E, 5, at.data_ptr())
    assert torch.equal(at[:T * E].view(T, E), want)
    assert (room[:1024] == 7).all() and (at[T * E:] == 7).all()

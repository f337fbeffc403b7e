"""moe_combine_backward against its definition in 64 bits.

dy is one product in fp32 and one rounding, so equal to torch's. dgates adds at most ceil(H / 64) + 16 terms after each
other (16 columns a pass and thread, then lanes and waves): off by at most that many 2^-24 of the sum of magnitudes."""

import numpy as np
import pytest
import torch

from mxfp4_block_scaled_amd import ops

pytestmark = pytest.mark.gpu


def _case(T, H, k, dd, yd, drop, seed, extra=0):
    g = torch.Generator().manual_seed(seed)
    dout = torch.randn((T, H), generator=g).to(dd)
    rows = T * k + extra
    y = torch.randn((rows, H), generator=g).to(yd)
    pair_row = torch.randperm(rows, generator=g)[:T * k].to(torch.int32)
    if drop:
        gone = torch.rand(T * k, generator=g) < drop
        pair_row[gone] = torch.tensor([-1, rows, 2 ** 31 - 1, -2 ** 31], dtype=torch.int64)[torch.arange(int(gone.sum())) % 4].to(torch.int32)
    gates = torch.randn((T, k), generator=g)
    return dout, y, gates, pair_row


def _check(dout, y, gates, pair_row):
    T, H = dout.shape
    k = gates.shape[1]
    sentinel = torch.full_like(y, 3.0).cuda()
    dy, dgates = ops.moe_combine_backward(dout.cuda(), y.cuda(), gates.cuda(), pair_row.cuda(), dy=sentinel)
    want = torch.full_like(y, 3.0)
    row = pair_row.long()
    p = ((row >= 0) & (row < y.shape[0])).nonzero().flatten()
    want[row[p]] = (gates.flatten()[p, None] * dout.float()[p // k]).to(y.dtype)
    assert torch.equal(dy.cpu(), want)
    terms = np.zeros((T * k, H))
    terms[p] = dout.double().numpy()[p.numpy() // k] * y.double().numpy()[row[p].numpy()]
    got = dgates.double().cpu().numpy().reshape(-1)
    tol = (-(-H // 64) + 16) * 2.0 ** -24 * abs(terms).sum(1)
    assert (abs(got - terms.sum(1)) <= tol).all()


@pytest.mark.parametrize("k", range(1, 9))
@pytest.mark.parametrize("T,H", [(1, 8), (3, 7168), (300, 264), (257, 1544)])
def test_bf16(T, H, k):
    _check(*_case(T, H, k, torch.bfloat16, torch.bfloat16, 0.0, T + k))


@pytest.mark.parametrize("dd,yd", [(torch.float32, torch.float32), (torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("T,H,k,drop", [(5, 64, 3, 0.5), (400, 1032, 6, 0.2), (260, 20000, 2, 1.0)])
def test_types_and_dropped_pairs(dd, yd, T, H, k, drop):
    """Pairs outside y's rows add nothing, have no gradient and write no row; rows that none names keep what they held."""
    _check(*_case(T, H, k, dd, yd, drop, T, extra=5))


def test_each_result_alone_in_place_and_empty():
    dout, y, gates, pair_row = (t.cuda() for t in _case(40, 512, 4, torch.bfloat16, torch.bfloat16, 0.1, 9))
    dy, dgates = ops.moe_combine_backward(dout, y, gates, pair_row, dy=torch.zeros_like(y))
    assert ops.moe_combine_backward(dout, y, gates, pair_row, want_dgates=False, dy=torch.zeros_like(y))[1] is None
    none, alone = ops.moe_combine_backward(dout, y, gates, pair_row, want_dy=False)
    assert none is None and torch.equal(alone, dgates)
    held = y.clone()
    named = pair_row[(pair_row >= 0) & (pair_row < y.shape[0])].long()
    _, again = ops.moe_combine_backward(dout, held, gates, pair_row, dy=held)
    assert torch.equal(again, dgates) and torch.equal(held[named], dy[named])
    e = ops.moe_combine_backward(dout[:0], y, gates[:0], pair_row[:0])
    assert e[0].shape == y.shape and e[1].shape == (0, 4)


def test_no_rows_at_all():
    dout = torch.ones((3, 64)).cuda()
    dy, dgates = ops.moe_combine_backward(dout, torch.empty((0, 64)).cuda(), torch.ones((3, 2)).cuda(),
                                          torch.zeros(6, dtype=torch.int32).cuda())
    assert dy.shape == (0, 64) and not dgates.any()


def test_infinities_stay_with_their_pair():
    dout, y, gates, pair_row = _case(300, 128, 2, torch.bfloat16, torch.bfloat16, 0.0, 11)
    y[pair_row[9].long(), 5] = torch.inf
    y[pair_row[10].long(), 7] = torch.nan
    _, dgates = ops.moe_combine_backward(dout.cuda(), y.cuda(), gates.cuda(), pair_row.cuda())
    assert (~dgates.isfinite()).flatten().nonzero().flatten().tolist() == [9, 10]

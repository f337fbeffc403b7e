"""moe_balance_loss and moe_route_backward against their definition in 64 bits and against differences.

Tolerances: a probability is exp2 of fp32 (x - m) log2(e): the product is off by at most 1.5 |x - m| 2^-24, the
instruction and the division by the sum a few 2^-23, so p is within (2 |x - m| + 16) 2^-24 relative: 1e-5 covers
spreads up to 70. Sums of positive terms keep that. A gradient is held to 1e-5 of the sum of its terms' magnitudes,
and for bf16 results half a step (2^-8) of its value more."""

import numpy as np
import pytest
import torch

from mxfp4_block_scaled_amd import ops
from tests import train_exact as ex

pytestmark = pytest.mark.gpu
RTOL = 1e-5


def _case(T, E, k, seed, bf16=False, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn((T, E), generator=g) * spread
    if bf16:
        logits = logits.bfloat16()
    x = logits.float()
    top = torch.sort(x, dim=1, descending=True, stable=True)
    ids = top.indices[:, :k].to(torch.int32).contiguous()
    gates = torch.softmax(top.values[:, :k], 1)
    dgates = torch.randn((T, k), generator=g)
    return logits, ids, gates, dgates


def _check(logits, ids, gates, dgates, mask, offsets, dlosses=(0.7, -0.3)):
    T, E = logits.shape
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32)
    d = ops.moe_balance_loss(dev(logits), dev(ids), dev(mask), dev(off))
    dl = torch.tensor(dlosses, dtype=torch.float32)
    got = ops.moe_route_backward(dev(logits), dev(ids), dev(gates), dev(dgates), d, dev(dl), dev(off))
    x = logits.double().numpy()
    m = np.ones(T, bool) if mask is None else mask.numpy().astype(bool)
    want = ex.balance(x, ids.numpy(), m, [0, T] if offsets is None else offsets)
    assert np.array_equal(d["counts"].cpu().numpy(), want["counts"])
    assert np.array_equal(d["tokens"].cpu().numpy(), want["tokens"])
    np.testing.assert_allclose(d["prob_mean"].cpu().numpy(), want["prob_mean"], rtol=RTOL, atol=1e-37)
    np.testing.assert_allclose(d["lse"].cpu().numpy(), want["lse"], rtol=RTOL, atol=RTOL)
    np.testing.assert_allclose(d["losses"].cpu().numpy(), want["losses"], rtol=2 * RTOL, atol=1e-9)
    grad, size = ex.route_gradient(x, ids.numpy(), gates.double().numpy(), dgates.double().numpy(), want,
                                   dl.double().numpy())
    tol = RTOL * size + 1e-37 + (2.0 ** -8 * abs(grad) if logits.dtype == torch.bfloat16 else 0)
    assert (abs(got.double().cpu().numpy() - grad) <= tol).all()
    return d, got


@pytest.mark.parametrize("T,E,k,bf16", [(1, 1, 1, False), (1, 4, 2, True), (3, 60, 4, True), (64, 256, 6, False),
                                        (65, 256, 6, False), (129, 64, 8, True), (200, 65, 1, False), (257, 500, 8, True),
                                        (130, 1024, 8, False), (777, 128, 3, False)])
def test_one_sequence(T, E, k, bf16):
    _check(*_case(T, E, k, T + E, bf16), None, None)


@pytest.mark.parametrize("T,offsets", [
    (40, [0, 7, 7, 40]), (300, [0, 1, 2, 3, 130, 130, 300]), (300, [5, 64, 128, 200]), (300, [0, 0, 0]), (300, [300, 300]),
    (500, list(range(0, 501))), (64, list(range(0, 65))), (1000, [0, 999, 1000]), (128, [64, 64, 128]),
])
def test_sequences(T, offsets):
    """Sequences of one token, empty ones, tokens before, behind and outside all of them."""
    mask = (torch.rand(T, generator=torch.Generator().manual_seed(T)) < 0.7).to(torch.uint8)
    _check(*_case(T, 96, 4, T), mask, offsets)
    _check(*_case(T, 33, 2, T, True), mask.bool(), offsets)


@pytest.mark.parametrize("T,offsets", [(64, sorted([i // 2 for i in range(129)])), (20000, [0, 17, 16000, 19990]),
                                       (70000, [3, 100, 40000, 40001, 69990, 70000])])
def test_many_tokens_and_more_sequences_than_lanes(T, offsets):
    """Workgroups that take their tokens in several turns; 128 sequences in one workgroup, half of them empty."""
    _check(*_case(T, 24, 2, T), None, offsets)


@pytest.mark.parametrize("T,S", [(1, 65), (16, 100), (50, 3000), (700, 65), (700, 5000)])
def test_runs_of_empty_sequences(T, S):
    """Many sequences, nearly all of them empty: before the tokens, between them (inside a workgroup's tokens and at
    their ends) and behind them; tokens of no sequence at both ends."""
    g = torch.Generator().manual_seed(T + S)
    cuts = sorted(torch.randint(0, T + 1, (6,), generator=g).tolist()) + [T]
    runs = torch.multinomial(torch.ones(7), S + 1, replacement=True, generator=g).tolist()
    offsets = sorted(cuts[k] for k in runs)
    _check(*_case(T, 40, 3, S), None, offsets)
    _check(*_case(T, 70, 2, S, True), None, [0] * (S // 2) + [min(3, T)] * (S + 1 - S // 2))


@pytest.mark.parametrize("S", [1, 64, 65, 4000])
def test_no_tokens_in_many_sequences(S):
    d = ops.moe_balance_loss(torch.empty((0, 96)).cuda(), torch.empty((0, 2), dtype=torch.int32).cuda(),
                             seg_offsets=torch.zeros(S + 1, dtype=torch.int32).cuda())
    assert d["losses"].tolist() == [0.0, 0.0] and d["counts"].shape == (S, 96)
    assert not d["counts"].any() and not d["prob_mean"].any() and not d["tokens"].any()


def test_views_of_larger_tensors():
    logits, ids, gates, dgates = (t.cuda() for t in _case(130, 64, 4, 8))
    mask = torch.ones(200, dtype=torch.uint8).cuda()
    mask[40] = 0
    a = ops.moe_balance_loss(logits, ids, mask[1:131])
    b = ops.moe_balance_loss(logits, ids, mask[1:131].clone())
    assert torch.equal(a["losses"], b["losses"]) and int(a["tokens"][0]) == 129
    dl = torch.tensor([9.0, 0.3, 0.2]).cuda()
    x = ops.moe_route_backward(logits, ids, gates, dgates, a, dl[1:])
    assert torch.equal(x, ops.moe_route_backward(logits, ids, gates, dgates, a, dl[1:].clone()))
    with pytest.raises(RuntimeError, match="contiguous"):
        ops.moe_balance_loss(logits.t().contiguous().t(), ids)
    with pytest.raises(RuntimeError, match="seg_offsets"):
        ops.moe_balance_loss(logits, ids, seg_offsets=torch.zeros(1, dtype=torch.int32).cuda())


@pytest.mark.parametrize("T", [30, 400])
def test_nothing_counts(T):
    logits, ids, gates, dgates = _case(T, 48, 3, 1)
    d, _ = _check(logits, ids, gates, dgates, torch.zeros(T, dtype=torch.uint8), [0, 20, T])
    assert d["losses"].tolist() == [0.0, 0.0]
    assert torch.isneginf(d["lse"]).all()


@pytest.mark.parametrize("T", [50, 300])
def test_ruled_out_experts_and_dropped_pairs(T):
    """-inf logits, rows of nothing but -inf, the type's lowest value, ids outside the experts, the same id twice."""
    logits, ids, gates, dgates = _case(T, 70, 4, 2)
    logits[:, ::3] = -torch.inf
    logits[5] = -torch.inf
    logits[T - 1] = -torch.inf
    logits[7, :] = torch.finfo(torch.float32).min
    logits[8, 1:] = torch.finfo(torch.float32).min
    ids[3, 1] = -1
    ids[4, 0] = 70
    ids[9, 2] = ids[9, 0]
    x = logits.double().numpy()
    want = ex.balance(x, ids.numpy(), np.ones(T, bool), [0, T])
    d = ops.moe_balance_loss(logits.cuda(), ids.cuda())
    assert np.array_equal(d["counts"].cpu().numpy(), want["counts"])
    assert d["tokens"].tolist() == [T - 2, T - 2, 1]
    np.testing.assert_allclose(d["prob_mean"].cpu().numpy(), want["prob_mean"], rtol=RTOL, atol=1e-37)
    assert torch.isneginf(d["lse"]).nonzero().flatten().tolist() == [5, T - 1]
    dl = torch.tensor([0.5, 0.0])  # (lse near -3e38 squared is infinite: no z)
    got = ops.moe_route_backward(logits.cuda(), ids.cuda(), gates.cuda(), dgates.cuda(), d, dl.cuda())
    want["lse"] = np.where(abs(want["lse"]) > 1e30, 0.0, want["lse"])
    grad, size = ex.route_gradient(x, ids.numpy(), gates.double().numpy(), dgates.double().numpy(), want, dl.double().numpy())
    assert (abs(got.double().cpu().numpy() - grad) <= RTOL * size + 1e-37).all()


def test_a_nan_row_spoils_the_losses_and_its_own_gradient_only():
    logits, ids, gates, dgates = _case(200, 40, 2, 3)
    logits[17, 3] = torch.nan
    logits[18, 4] = torch.inf
    d = ops.moe_balance_loss(logits.cuda(), ids.cuda())
    assert d["losses"].isnan().all()
    assert int(d["counts"].sum()) == 400
    dl = torch.ones(2).cuda()
    got = ops.moe_route_backward(logits.cuda(), ids.cuda(), gates.cuda(), dgates.cuda(), d, dl)
    bad = got.isnan().any(1).nonzero().flatten().tolist()
    assert bad == [17, 18]


@pytest.mark.parametrize("T", [60, 200])
def test_a_row_of_nothing_but_nan_counts(T):
    """NaN is not -inf: such a row, alone or beside -inf, is no row ruled out; it spoils the losses."""
    logits, ids, gates, dgates = _case(T, 40, 2, 4)
    logits[17] = torch.nan
    logits[18] = -torch.inf
    logits[19, 1:], logits[19, 0] = -torch.inf, torch.nan
    d = ops.moe_balance_loss(logits.cuda(), ids.cuda())
    assert d["losses"].isnan().all()
    assert d["tokens"].tolist() == [T - 1, T - 1, 1] and int(d["counts"].sum()) == 2 * (T - 1)
    assert d["lse"].isnan().nonzero().flatten().tolist() == [17, 19]
    got = ops.moe_route_backward(logits.cuda(), ids.cuda(), gates.cuda(), dgates.cuda(), d, torch.ones(2).cuda())
    assert got.isnan().any(1).nonzero().flatten().tolist() == [17, 19]


def test_no_tokens():
    d = ops.moe_balance_loss(torch.empty((0, 32)).cuda(), torch.empty((0, 2), dtype=torch.int32).cuda(),
                             seg_offsets=torch.zeros(4, dtype=torch.int32).cuda())
    assert d["losses"].tolist() == [0.0, 0.0] and d["tokens"].tolist() == [0] * 5
    assert not d["counts"].any() and not d["prob_mean"].any()
    got = ops.moe_route_backward(torch.empty((0, 32)).cuda(), torch.empty((0, 2), dtype=torch.int32).cuda(),
                                 torch.empty((0, 2)).cuda(), torch.empty((0, 2)).cuda())
    assert got.shape == (0, 32)


def test_each_part_alone():
    logits, ids, gates, dgates = _case(90, 64, 4, 5)
    d = ops.moe_balance_loss(logits.cuda(), ids.cuda())
    dl = torch.tensor([0.4, 0.2]).cuda()
    both = ops.moe_route_backward(logits.cuda(), ids.cuda(), gates.cuda(), dgates.cuda(), d, dl)
    one = ops.moe_route_backward(logits.cuda(), ids.cuda(), gates.cuda(), dgates.cuda())
    other = ops.moe_route_backward(logits.cuda(), ids.cuda(), balance=d, dlosses=dl)
    assert torch.equal(both, one + other)
    for bad in (dict(gates=gates.cuda()), dict(balance=d), {}):
        with pytest.raises(RuntimeError):
            ops.moe_route_backward(logits.cuda(), ids.cuda(), **bad)


def test_sequences_spread_over_several_devices():
    """Counts and tokens of the parts added up (the sequences that hold any counted again): each part's gradient is its
    piece of the whole's. Every term of a token is formed from the same values in the same order, so bit for bit."""
    logits, ids, gates, dgates = (t.cuda() for t in _case(400, 96, 4, 9))
    dl = torch.tensor([0.6, 0.2]).cuda()
    offs = [torch.tensor(o, dtype=torch.int32).cuda() for o in ([0, 150, 150, 400], [0, 100, 100, 220], [0, 50, 50, 180])]
    # the first part: tokens 0..99 of sequence 0 and 150..269 of sequence 2
    own = [torch.cat((torch.arange(0, 100), torch.arange(150, 270))), torch.cat((torch.arange(100, 150), torch.arange(270, 400)))]
    whole = ops.moe_balance_loss(logits, ids, seg_offsets=offs[0])
    want = ops.moe_route_backward(logits, ids, gates, dgates, whole, dl, offs[0])
    part = [ops.moe_balance_loss(logits[o], ids[o], seg_offsets=f) for o, f in zip(own, offs[1:])]
    counts = part[0]["counts"] + part[1]["counts"]
    tokens = part[0]["tokens"] + part[1]["tokens"]
    tokens[-1] = (tokens[:-2] > 0).sum()
    assert torch.equal(counts, whole["counts"]) and torch.equal(tokens, whole["tokens"])
    for o, f, d in zip(own, offs[1:], part):
        d = dict(d, counts=counts, tokens=tokens)
        got = ops.moe_route_backward(logits[o], ids[o], gates[o], dgates[o], d, dl, f)
        assert torch.equal(got, want[o.cuda()])


def test_against_differences():
    """dlogits is the derivative of dlosses . losses + dgates . gates (counts held): differences of the 64-bit forms."""
    T, E, k = 9, 12, 3
    logits, ids, gates, dgates = _case(T, E, k, 6)
    offsets, dl = [0, 4, 9], np.array([1.3, 0.6])
    x, dg = logits.double().numpy(), dgates.double().numpy()

    def loss(v):
        d = ex.balance(v, ids.numpy(), np.ones(T, bool), offsets)
        sel = np.take_along_axis(v, ids.numpy().astype(np.int64), 1)
        sel = np.exp(sel - sel.max(1, keepdims=True))
        return (d["losses"] * dl).sum() + (sel / sel.sum(1, keepdims=True) * dg).sum()

    off = torch.tensor(offsets, dtype=torch.int32).cuda()
    d = ops.moe_balance_loss(logits.cuda(), ids.cuda(), seg_offsets=off)
    got = ops.moe_route_backward(logits.cuda(), ids.cuda(), gates.cuda(), dgates.cuda(), d,
                                 torch.tensor(dl, dtype=torch.float32).cuda(), off).double().cpu().numpy()
    h = 1e-5  # off by h^2 of the third derivative, and 1e-16 / h
    for t in range(T):
        for e in range(E):
            a, b = x.copy(), x.copy()
            a[t, e] += h
            b[t, e] -= h
            assert abs((loss(a) - loss(b)) / (2 * h) - got[t, e]) <= 1e-6 + 1e-5 * abs(got[t, e])


def test_same_result_every_time_and_captured():
    logits, ids, gates, dgates = (t.cuda() for t in _case(5000, 256, 6, 7))
    off = torch.tensor([0, 100, 3000, 5000], dtype=torch.int32).cuda()
    dl = torch.tensor([0.01, 0.001]).cuda()

    def step():
        d = ops.moe_balance_loss(logits, ids, seg_offsets=off)
        return [d["losses"], d["counts"], d["prob_mean"], ops.moe_route_backward(logits, ids, gates, dgates, d, dl, off)]

    want = step()
    graph = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    with torch.cuda.graph(graph):
        held = step()
    for i in range(3):
        for t in held:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), i
        assert all(torch.equal(a, b) for a, b in zip(step(), want)), i

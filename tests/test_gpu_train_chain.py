"""The operators of training as they are used together: the backward pass of an expert layer's combine and router with
its losses, and a 4-bit linear layer with its gradients, each against 64-bit forms; large tensors' far ends."""

import numpy as np
import pytest
import torch

from mxfp4_block_scaled_amd import ops
from tests import train_exact as ex

pytestmark = pytest.mark.gpu


def _experts(E, H, I, seed):
    g = torch.Generator().manual_seed(seed)
    w = [torch.randint(0, 256, s, dtype=torch.uint8, generator=g).cuda() for s in ((E, 2 * I, H // 2), (E, H, I // 2))]
    s = [torch.randint(117, 121, t, dtype=torch.uint8, generator=g).cuda() for t in ((E, 2 * I, H // 32), (E, H, I // 32))]
    return w, s


@pytest.mark.parametrize("T", [1, 24, 300])
def test_router_and_combine_of_an_expert_layer(T):
    """loss = <dout, out> + 0.02 balance + 0.003 z; dlogits by the operators and by differentiating the 64-bit form, in
    which the experts' rows are constants and the counts have no gradient."""
    E, k, H, I = 16, 3, 512, 256
    g = torch.Generator().manual_seed(T)
    x = torch.randn((T, H), generator=g).bfloat16().cuda()
    logits = torch.randn((T, E), generator=g)
    dout = torch.randn((T, H), generator=g).bfloat16()
    mask = (torch.rand(T, generator=g) < 0.8).to(torch.uint8)
    off = torch.tensor([0, T // 3, T // 3, T], dtype=torch.int32)
    (w1, w2), (s1, s2) = _experts(E, H, I, T)
    r = ops.moe_layer(x, logits.cuda(), w1, s1, w2, s2, k, act_fmt="bf16")
    bal = ops.moe_balance_loss(logits.cuda(), r["topk_ids"], mask.cuda(), off.cuda())
    assert bal["counts"].sum() == int(bal["tokens"][3]) * k == int(mask.sum()) * k
    dy, dgates = ops.moe_combine_backward(dout.cuda(), r["y"], r["gates"], r["pair_row"])
    dl = torch.tensor([0.02, 0.003])
    got = ops.moe_route_backward(logits.cuda(), r["topk_ids"], r["gates"], dgates, bal, dl.cuda(), off.cuda()).cpu().double()

    v = logits.double().requires_grad_()
    ids = r["topk_ids"].cpu().long()
    y = r["y"].double().cpu()[r["pair_row"].cpu().long()].view(T, k, H)
    gates = torch.softmax(torch.gather(v, 1, ids), 1)
    loss = (dout.double()[:, None] * gates[..., None] * y).sum()
    p, lse = torch.softmax(v, 1), torch.logsumexp(v, 1)
    parts = []
    for a, b in zip(off.tolist()[:-1], off.tolist()[1:]):
        use = [t for t in range(a, b) if mask[t]]
        if use:
            c = torch.bincount(ids[use].flatten(), minlength=E).double()
            parts.append(E / (k * len(use)) * (c * p[use].mean(0)).sum())
    if parts:
        loss = loss + 0.02 * sum(parts) / len(parts) + 0.003 * (lse[mask.bool()] ** 2).mean()
        assert abs(float(bal["losses"][0]) - float(sum(parts).detach() / len(parts))) < 1e-5 * E
    loss.backward()
    # dgates: 512 products added in fp32, |terms| in all at most `size`; dlogits adds k of them weighted by gates
    size = (dout.double()[:, None] * y).abs().sum(2).max(1, keepdim=True).values
    assert ((got - v.grad).abs() <= 2e-5 * (v.grad.abs() + size)).all()
    want = (gates.detach()[..., None] * dout.double()[:, None]).view(T * k, H)
    assert ((dy.cpu().double()[r["pair_row"].cpu().long()] - want).abs() <= (2.0 ** -8 + 1e-5) * want.abs()).all()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("T,I,O", [(1, 128, 128), (40, 256, 384), (300, 640, 256), (1000, 2048, 1152)])
def test_linear_layer_and_its_gradients(fmt, T, I, O):
    """y = x^ W^^T, dx = dy^ W^ and dW = dy^^T x^, each operand coded along the sum of its product: against 64-bit
    products of the values the codes stand for. T need not be a multiple of anything: rows are filled up with zeros."""
    g = torch.Generator().manual_seed(T)
    x, w, dy = (torch.randn(s, generator=g).bfloat16().cuda() for s in ((T, I), (O, I), (T, O)))
    rnd = torch.randint(0, 256, (T, O), dtype=torch.uint8, generator=g).cuda()
    nv = fmt == "nvfp4"
    gs = [ops.nvfp4_tensor_scale(t) if nv else None for t in (x, w, dy)]
    qx, qw = (ops.fp4_quantize(t, fmt, s, transposed=True) for t, s in ((x, gs[0]), (w, gs[1])))
    qd = ops.fp4_quantize(dy, fmt, gs[2], rnd=rnd, transposed=True)

    def value(q, name, s):
        return ex.values(q[name].cpu().numpy(), q[name + "_scale"].cpu().numpy(), fmt, float(s) if nv else 1.0)

    for a, an, ga, b, bn, gb, dt in ((qx, "q", 0, qw, "q", 1, torch.bfloat16), (qd, "q", 2, qw, "qt", 1, torch.bfloat16),
                                     (qd, "qt", 2, qx, "qt", 0, torch.float32)):
        got = ops.fp4_gemm(a[an], a[an + "_scale"], b[bn], b[bn + "_scale"], fmt, gs[ga], gs[gb], out_dtype=dt)
        u, v = value(a, an, gs[ga]), value(b, bn, gs[gb])
        want, size, K = u @ v.T, abs(u) @ abs(v).T, u.shape[1]
        tol = (K / 8 + 16) * 2.0 ** -23 * size + (2.0 ** -8 * abs(want) if dt == torch.bfloat16 else 0)
        assert got.shape == want.shape and (abs(got.double().cpu().numpy() - want) <= tol + 1e-40).all()
    # the layer's forward differs from the unquantised one by what two codes of a block can be off
    y = ops.fp4_gemm(qx["q"], qx["q_scale"], qw["q"], qw["q_scale"], fmt, gs[0], gs[1], out_dtype=torch.float32)
    full = x.double() @ w.double().t().contiguous()
    assert float((y.double() - full).norm() / full.norm()) < 0.35


def test_the_whole_step_captured():
    """Forward and backward in one graph, replayed on new inputs beside eager work."""
    T, E, k, H = 200, 32, 4, 256
    g = torch.Generator().manual_seed(1)

    def inputs():
        logits = torch.randn((T, E), generator=g).cuda()
        y = torch.randn((T * k, H), generator=g).bfloat16().cuda()
        return logits, y, torch.randn((T, H), generator=g).bfloat16().cuda()

    dl = torch.tensor([0.01, 0.001]).cuda()
    w = torch.randn((256, H), generator=g).bfloat16().cuda()

    def step(logits, y, dout):
        ids, gates, _, _, pr = ops.moe_route_permute(logits, k)
        out = ops.moe_unpermute_combine(y, gates, pr, T, k)
        bal = ops.moe_balance_loss(logits, ids)
        dy, dgates = ops.moe_combine_backward(dout, y, gates, pr)
        dlogits = ops.moe_route_backward(logits, ids, gates, dgates, bal, dl)
        s, sw = ops.nvfp4_tensor_scale(out), ops.nvfp4_tensor_scale(w)
        q, qw = ops.fp4_quantize(out, "nvfp4", s, transposed=True), ops.fp4_quantize(w, "nvfp4", sw)
        z = ops.fp4_gemm(q["q"], q["q_scale"], qw["q"], qw["q_scale"], "nvfp4", s, sw)
        return dlogits, dy, bal["losses"], bal["counts"], q["qt"], z

    sets = [inputs() for _ in range(3)]
    want = [step(*s) for s in sets]
    held = [t.clone() for t in sets[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*held)
    for i in (1, 2, 0, 1):
        for a, b in zip(held, sets[i]):
            a.copy_(b)
        graph.replay()
        eager = step(*sets[i])
        torch.cuda.synchronize()
        for a, b, c in zip(got, want[i], eager):
            assert torch.equal(a, b) and torch.equal(b, c), i


def test_offsets_past_32_bits():
    """More than 2^31 elements: the far end of each result equals the same rows computed alone."""
    rows, cols = 300_000, 7168
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    x.zero_()
    x[:256].normal_()
    x[-256:].normal_()
    d = ops.fp4_quantize(x, "nvfp4", transposed=True)
    tail = ops.fp4_quantize(x[-256:].contiguous(), "nvfp4", transposed=True)
    assert torch.equal(d["q"][-256:], tail["q"]) and torch.equal(d["q_scale"][-256:], tail["q_scale"])
    first = rows // 128 * 128  # the last tile of rows begins here
    last = ops.fp4_quantize(x[first:].contiguous(), "nvfp4", rows=False, transposed=True)
    assert torch.equal(d["qt"][:, first // 2:], last["qt"]) and torch.equal(d["qt_scale"][:, first // 16:], last["qt_scale"])
    alone = ops.fp4_quantize(x, "nvfp4")
    assert torch.equal(alone["q"][-256:], tail["q"])
    back = ops.fp4_dequantize(alone["q"], alone["q_scale"])
    assert torch.equal(back[-256:], ops.fp4_dequantize(tail["q"], tail["q_scale"]))
    x[-1, -1] = 300.0
    assert float(ops.nvfp4_tensor_scale(x)) == 0.125
    del back, alone, d
    # combine: 300000 rows of y, two a token
    gates = torch.rand((rows // 2, 2), device="cuda")
    pair_row = torch.arange(rows, dtype=torch.int32, device="cuda")
    dout = torch.zeros((rows // 2, cols), dtype=torch.bfloat16, device="cuda")
    dout[-64:].normal_()
    dy, dg = ops.moe_combine_backward(dout, x, gates, pair_row)
    ey, eg = ops.moe_combine_backward(dout[-64:].contiguous(), x[-128:].contiguous(), gates[-64:].contiguous(),
                                      pair_row[:128].contiguous())
    assert torch.equal(dy[-128:], ey)
    torch.testing.assert_close(dg[-64:], eg, rtol=1e-5, atol=1e-2)  # (another split of the sum: 7168 terms of up to 300)
    del dy, dout
    # product: 5 GB of results
    a, b = (torch.randint(0, 256, (n, 64), dtype=torch.uint8, device="cuda") for n in (40_000, 32_768))
    sa, sb = (torch.full((n, 8), 0x38, dtype=torch.uint8, device="cuda") for n in (40_000, 32_768))
    c = ops.fp4_gemm(a, sa, b, sb, out_dtype=torch.float32)
    assert torch.equal(c[-200:], ops.fp4_gemm(a[-200:].contiguous(), sa[-200:].contiguous(), b, sb, out_dtype=torch.float32))
    del c, x
    # router: 2^21 + 5 tokens of 1024 experts
    T, E = (1 << 21) + 5, 1024
    logits = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
    logits[-100:].normal_()
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    off = torch.tensor([0, T - 100, T], dtype=torch.int32, device="cuda")
    bal = ops.moe_balance_loss(logits, ids, seg_offsets=off)
    assert bal["counts"][:, 0].tolist() == [T - 100, 100] and bal["tokens"].tolist() == [T - 100, 100, T, 2]
    np.testing.assert_allclose(bal["prob_mean"][1].cpu().numpy(), torch.softmax(logits[-100:].double(), 1).mean(0).cpu().numpy(), rtol=1e-5)
    np.testing.assert_allclose(bal["prob_mean"][0].cpu().numpy(), 1 / E, rtol=1e-4)  # 2^21 terms in fp32, in 1024 parts
    dl = torch.tensor([float(T), 0.0], device="cuda")
    grad = ops.moe_route_backward(logits, ids, balance=bal, dlosses=dl, seg_offsets=off)
    p = torch.softmax(logits[-100:].double(), 1)
    want = T * E / (2 * 100) * p * ((torch.arange(E, device="cuda") == 0).double() - p[:, :1])
    assert ((grad[-100:].double() - want).abs() <= (2.0 ** -8 + 1e-4) * want.abs() + 1e-5 * T * E / 200 * p).all()

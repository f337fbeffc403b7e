"""fp4_quantize, fp4_dequantize and nvfp4_tensor_scale against their definition in 64 bits.

With bf16 values and a power-of-two tensor scale x / d is a quotient of 8 by 4 bits: fp32 rounds it without passing a
border between codes, so codes and scales are equal, ties included. Otherwise fp32's quotient is within 2^-24 of x / d
and may fall on the other side of a border that near: such codes are one step off at most."""

import numpy as np
import pytest
import torch

import oracle
from mxfp4_block_scaled_amd import ops
from tests import train_exact as ex

pytestmark = pytest.mark.gpu


def _x(rows, cols, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * torch.exp(2 * torch.randn((1, cols), generator=g))
    x[:, 3] = 0.0
    x[rows // 2] *= 0.0
    x[0, 5] = -0.0
    if rows > 2:
        x[1] *= 2.0 ** -20
    return x.to(dtype)


def _host(t):
    return t.cpu().numpy()


def _near(v):
    mid = (ex.E2M1[1:] + ex.E2M1[:-1]) / 2
    return (abs(v[..., None] - mid) <= 2.0 ** -22 * mid).any(-1)


def _compare(q, s, x, fmt, g, rnd, exact):
    codes, byte, v = ex.quantise(x, fmt, g, rnd)
    got = ex.unpack(_host(q))
    assert np.array_equal(_host(s), byte)
    off = got != codes
    if exact:
        assert not off.any()
    elif rnd is None:
        assert (_near(v) | ~off).all() and (abs((got & 7) - (codes & 7)) <= 1).all()
    else:
        assert off.mean() < 1e-4 and (abs((got & 7) - (codes & 7)) <= 1).all()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (5, 96), (127, 160), (128, 128), (129, 2080), (300, 416)])
@pytest.mark.parametrize("stochastic", [False, True])
def test_both_directions(fmt, dtype, rows, cols, stochastic):
    x = _x(rows, cols, dtype, rows + cols)
    rnd = torch.randint(0, 256, (rows, cols), dtype=torch.uint8, generator=torch.Generator().manual_seed(1))
    nv = fmt == "nvfp4"
    g = ops.nvfp4_tensor_scale(x.cuda()) if nv else None
    gv = float(g) if nv else 1.0
    xd = x.double().numpy()
    if nv:
        assert gv == ex.tensor_scale(xd)
    r = rnd if stochastic else None
    dr = rnd.cuda() if stochastic else None
    d = ops.fp4_quantize(x.cuda(), fmt, g, dr, transposed=True)
    exact = dtype == torch.bfloat16
    rn = None if r is None else r.numpy()
    _compare(d["q"], d["q_scale"], xd, fmt, gv, rn, exact)
    _compare(d["qt"], d["qt_scale"], ex.transposed(xd), fmt, gv, None if r is None else ex.transposed(rn), exact)
    alone = ops.fp4_quantize(x.cuda(), fmt, g, dr)
    assert torch.equal(alone["q"], d["q"]) and torch.equal(alone["q_scale"], d["q_scale"]) and alone["qt"] is None
    other = ops.fp4_quantize(x.cuda(), fmt, g, dr, rows=False, transposed=True)
    assert torch.equal(other["qt"], d["qt"]) and torch.equal(other["qt_scale"], d["qt_scale"]) and other["q"] is None
    for a, b in (("q", "q_scale"), ("qt", "qt_scale")):
        want = ex.values(_host(d[a]), _host(d[b]), fmt, gv)
        for dt in (torch.float32, torch.bfloat16):
            got = ops.fp4_dequantize(d[a], d[b], fmt, g, dt)
            assert got.dtype == dt and np.array_equal(got.double().cpu().numpy(), want)


def test_mxfp4_rows_are_those_of_the_activations():
    x = _x(70, 320, torch.bfloat16, 3).cuda()
    q, s = ops.mxfp4_quantize_act(x, "e2m1")
    d = ops.fp4_quantize(x, "mxfp4")
    assert torch.equal(d["q"], q) and torch.equal(d["q_scale"], s)
    codes, byte = oracle.mx_quantize(x.double().cpu().numpy(), "e2m1")
    assert np.array_equal(ex.unpack(_host(d["q"])), codes) and np.array_equal(_host(s), byte)


@pytest.mark.parametrize("g", [1.0, 0.37, 3.0e-3])
def test_any_tensor_scale(g):
    x = _x(33, 256, torch.float32, 4)
    gt = torch.tensor([g])
    d = ops.fp4_quantize(x.cuda(), "nvfp4", gt.cuda())
    _compare(d["q"], d["q_scale"], x.double().numpy(), "nvfp4", float(gt), None, False)
    got = ops.fp4_dequantize(d["q"], d["q_scale"], "nvfp4", gt.cuda())
    want = ex.values(_host(d["q"]), _host(d["q_scale"]), "nvfp4", float(gt))
    assert (abs(got.double().cpu().numpy() - want) <= 2.0 ** -8 * 1.001 * abs(want)).all()


def test_ties_of_codes_and_scales():
    """Every midpoint of the code grid at every scale mantissa, and block maxima halfway between two scales."""
    mid = (ex.E2M1[1:] + ex.E2M1[:-1]) / 2
    rows = []
    for m in range(8, 16):  # a block whose largest value sets the scale m / 8
        block = np.concatenate([[6.0], mid, -mid, [0.25]])[:16] * (m / 8)
        rows.append(block)
    x = torch.tensor(np.stack([np.concatenate([r, 2 * r]) for r in rows]), dtype=torch.float32)
    assert torch.equal(x.bfloat16().float(), x)
    for dt in (torch.float32, torch.bfloat16):
        d = ops.fp4_quantize(x.to(dt).cuda(), "nvfp4")
        _compare(d["q"], d["q_scale"], x.double().numpy(), "nvfp4", 1.0, None, True)
    s = np.repeat([6 * (a + b) / 2 for a, b in zip(ex.E4M3[8:-1], ex.E4M3[9:])], 16).reshape(-1, 16)
    s = s[: len(s) // 2 * 2].reshape(-1, 32)
    t = torch.tensor(s, dtype=torch.float32)
    d = ops.fp4_quantize(t.cuda(), "nvfp4")
    _compare(d["q"], d["q_scale"], t.double().numpy(), "nvfp4", 1.0, None, False)


@pytest.mark.parametrize("n", [32, 2048 * 16, 65_536, 65_568, 131_072, 131_104, 4_000_000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tensor_scale(n, dtype):
    for amax in (0.0, 1e-44, 2.0 ** -126, 2688.0, 2688.0 * 2 ** 7, 2704.0, 5e-7, 3e38):
        x = torch.full((n,), min(amax, 1e-6) / 3, dtype=torch.float32).to(dtype)
        x[n - 7] = -amax
        x = x.view(-1, 32).cuda()
        assert float(ops.nvfp4_tensor_scale(x)) == ex.tensor_scale(x.double().cpu().numpy()), amax


def test_extremes():
    """Blocks too small for a scale are zeros with their signs; a tensor scale of no use leaves zeros and no NaN."""
    x = torch.zeros((4, 32))
    x[0, 0], x[0, 20] = 1e-9, -1e-9  # far below 2^-10 of the scales: E4M3(amax / 6) = 0
    x[1, :] = 3e38
    x[2, 1], x[2, 17] = 448 * 6, -1e30
    d = ops.fp4_quantize(x.cuda(), "nvfp4")
    _compare(d["q"], d["q_scale"], x.double().numpy(), "nvfp4", 1.0, None, True)
    assert (d["q"][0] & 0x77).eq(0).all() and int(d["q"][0, 10]) == 8
    for bad in (0.0, -1.0, float("inf"), float("nan"), 1e-44):
        d = ops.fp4_quantize(x.cuda(), "nvfp4", torch.tensor([bad]).cuda())
        assert (d["q_scale"] < 127).all() and d["q"][d["q_scale"].eq(0).repeat_interleave(8, 1)].bitwise_and(0x77).eq(0).all()
    y = torch.randn((3, 64))
    clean = ops.fp4_quantize(y.cuda(), "nvfp4", transposed=True)
    y[1, 2], y[2, 40] = torch.nan, torch.inf
    d = ops.fp4_quantize(y.cuda(), "nvfp4", transposed=True)
    assert int(d["q_scale"][2, 2]) == 0x7E and (d["q_scale"] < 0x7F).all()
    keep = torch.ones(3, 32, dtype=torch.bool)
    keep[1, :8] = keep[2, 16:24] = False
    assert torch.equal(d["q"].cpu()[keep], clean["q"].cpu()[keep])
    cols = [c for c in range(64) if c not in (2, 40)]
    assert torch.equal(d["qt"].cpu()[cols], clean["qt"].cpu()[cols])


def test_stochastic_rounding_has_the_values_mean():
    """Over all 256 random bytes a value is rounded up as often as its part above the lower neighbour says."""
    v = torch.linspace(0, 6, 256)[None].repeat(256, 1)
    x = torch.cat([v, v], 1)
    x[:, ::16] = 6.0  # each block's scale is one
    rnd = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 512)
    d = ops.fp4_quantize(x.cuda(), "nvfp4", rnd=rnd.cuda())
    assert d["q_scale"].eq(0x38).all()
    mean = ops.fp4_dequantize(d["q"], d["q_scale"], "nvfp4", out_dtype=torch.float32).mean(0).cpu()
    assert ((mean - x[0]).abs() <= 2.0 / 512 + 1e-6).all()  # half of 1/256 of the widest step


def test_nothing_to_do():
    for n in (0,):
        d = ops.fp4_quantize(torch.empty((n, 64), dtype=torch.bfloat16).cuda(), transposed=True)
        assert d["q"].shape == (0, 32) and d["qt"].shape == (64, 0)
        assert ops.fp4_dequantize(d["q"], d["q_scale"]).shape == (0, 64)
    x = torch.zeros((4, 64)).cuda()
    for bad in (dict(fmt="fp4"), dict(fmt="mxfp4", tensor_scale=torch.ones(1).cuda()), dict(rows=False)):
        with pytest.raises(RuntimeError):
            ops.fp4_quantize(x, **bad)

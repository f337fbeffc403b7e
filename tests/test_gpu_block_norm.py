"""GPU parity of moe_block_norm against the formulas in 64 bits.

Tolerance, from arithmetic (u = 2^-24, half a step of fp32; every fp32 operation rounds by u):
the combine of k rows: (k + 1) u sum |g y|. A mean of squares of H terms summed in fp32: at most
8 C + 6 + waves additions in a row, so its relative error is under 64 u with the division and the
added eps; the reciprocal root halves it and is itself good to 2 u, and two products follow:
p is off by 40 u |p| plus what b's error brings, which the norm divides by rms(b) like b itself
(db also moves the mean: at most max(db) again). Gate, residual: 3 u more on each term. n likewise from r.
So dr = 64 u (|alpha x| + |gate p|) + |gate| (db and its mean's share) and
dn = |w| / rms(r) (dr + |r| / rms(r) max dr) + 40 u |n|. Results in bf16 round by 2^-8 of the value."""

import numpy as np
import pytest
import torch

from mxfp4_block_scaled_amd import ops

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5


def rms_norm(v, dv, w):
    """n = w v / rms(v) and its bound, from v off by dv."""
    rms = torch.sqrt(v.square().mean(1, keepdim=True) + EPS)
    n = v / rms * w
    dn = w.abs() / rms * (dv + v.abs() / rms * dv.amax(1, keepdim=True)) + 40 * U * n.abs()
    return n, dn


def reference(y, x, post, gate, alpha, pre, gates, pair):
    if gates is not None:
        T, k = gates.shape
        rows = pair.long().view(T, k)
        ok = (rows >= 0) & (rows < y.shape[0])
        terms = torch.where(ok[..., None], y.double()[rows.clamp(0, y.shape[0] - 1)], 0.0) * gates.double()[..., None]
        b, db = terms.sum(1), (k + 1) * U * terms.abs().sum(1)
    else:
        b = y.double()
        db = torch.zeros_like(b)
    if post is not None:
        b, db = rms_norm(b, db, post.double())
    g = 1.0 if gate is None else gate.double()
    p, dp = g * b, abs(g) * db
    ax = 0.0 if x is None else alpha * x.double()
    r = ax + p
    dr = dp + 64 * U * (abs(ax) + p.abs())
    n, dn = rms_norm(r, dr, 1.0 * torch.ones_like(r) if pre is None else pre.double())
    return r, dr, n, dn


def close(got, want, d, what):
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else U
    err, lim = (got.cpu().double() - want).abs(), d + half * (want.abs() + d) + 1e-40
    assert (err <= lim).all(), f"{what}: {float((err / lim).max()):.3g} of its bound"


def inputs(T, H, topk, post, gate, x_dtype, y_dtype, w_dtype, seed):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    y = rn(T * topk if topk else T, H).to(y_dtype)
    x = None if x_dtype is None else (2 * rn(T, H)).to(x_dtype)
    shape = {None: None, "channel": (H,), "token": (T, 1), "full": (T, H)}[gate]
    return dict(y=y, x=x, post=(1 + 0.1 * rn(H)).to(w_dtype) if post else None,
                gate=rn(*shape).to(y_dtype) if shape else None, pre=(1 + 0.1 * rn(H)).to(w_dtype),
                gates=torch.softmax(rn(T, topk), 1) if topk else None,
                pair=torch.randperm(T * topk, generator=g).to(torch.int32) if topk else None)


def cu(t):
    return None if t is None else t.cuda()


BF, F32 = torch.bfloat16, torch.float32
CASES = [
    (1, 8, 0, False, None, BF, BF, F32),
    (1, 7168, 0, True, None, BF, BF, F32),
    (5, 512, 0, True, "channel", F32, BF, BF),
    (3, 520, 2, True, "token", BF, F32, F32),
    (9, 1544, 6, False, "full", BF, BF, F32),
    (64, 7168, 6, True, "channel", F32, BF, F32),
    (17, 2048, 8, True, "full", BF, BF, BF),
    (33, 96, 1, False, "token", None, F32, F32),
    (2, 16384, 0, True, None, BF, BF, F32),
    (2, 30000, 3, True, "channel", F32, F32, F32),
    (3, 65536, 6, True, "full", BF, BF, BF),
    (300, 64, 0, False, None, F32, BF, F32),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v).replace("torch.", "") for v in c))
def test_against_64_bits(case):
    T, H, topk, post, gate, xd, yd, wd = case
    i = inputs(T, H, topk, post, gate, xd, yd, wd, T * H)
    alpha = 0.75
    got = ops.moe_block_norm(cu(i["y"]), x=cu(i["x"]), post_weight=cu(i["post"]), gate=cu(i["gate"]),
                             residual_scale=alpha, pre_weight=cu(i["pre"]), eps=EPS, n_dtype=F32 if T % 2 else BF,
                             expert_gates=cu(i["gates"]), pair_row=cu(i["pair"]))
    r, dr, n, dn = reference(i["y"], i["x"], i["post"], i["gate"], alpha, i["pre"], i["gates"], i["pair"])
    assert got["r"].dtype == (xd or yd)
    close(got["r"], r, dr, "r")
    close(got["n"], n, dn, "n")


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("T,H,topk", [(1, 32, 0), (7, 7168, 6), (40, 160, 2), (2, 65536, 0)])
def test_codes_are_those_of_the_quantiser(T, H, topk, fmt):
    """q and q_scale are bit for bit what mxfp4_quantize_act makes of the fp32 n of the same call."""
    i = inputs(T, H, topk, True, None, BF, BF, F32, H + T)
    got = ops.moe_block_norm(cu(i["y"]), x=cu(i["x"]), post_weight=cu(i["post"]), pre_weight=cu(i["pre"]),
                             act_fmt=fmt, n_dtype=F32, expert_gates=cu(i["gates"]), pair_row=cu(i["pair"]))
    q, qs = ops.mxfp4_quantize_act(got["n"], fmt)
    assert torch.equal(got["q"], q) and torch.equal(got["q_scale"], qs)
    only = ops.moe_block_norm(cu(i["y"]), x=cu(i["x"]), post_weight=cu(i["post"]), pre_weight=cu(i["pre"]),
                              act_fmt=fmt, want_r=False, want_n=False, expert_gates=cu(i["gates"]),
                              pair_row=cu(i["pair"]))
    assert only["r"] is None and only["n"] is None
    assert torch.equal(only["q"], q) and torch.equal(only["q_scale"], qs)


def test_combine_is_that_of_unpermute_combine():
    """Without norms, gate and residual, r is moe_unpermute_combine's result bit for bit."""
    T, H, topk = 19, 1024, 6
    i = inputs(T, H, topk, False, None, None, BF, F32, 3)
    got = ops.moe_block_norm(cu(i["y"]), want_n=False, expert_gates=cu(i["gates"]), pair_row=cu(i["pair"]))
    want = ops.moe_unpermute_combine(cu(i["y"]), cu(i["gates"]), cu(i["pair"]), T, topk)
    assert torch.equal(got["r"], want)


@pytest.mark.parametrize("topk", [2, 6])
def test_dropped_pairs_and_zero_rows(topk):
    T, H = 6, 256
    i = inputs(T, H, topk, True, None, BF, BF, F32, 11)
    pair = i["pair"].clone()
    pair[0], pair[topk], pair[2 * topk:3 * topk] = -1, T * topk, -7  # token 2 has no expert row at all
    i["x"][2] = 0
    got = ops.moe_block_norm(cu(i["y"]), x=cu(i["x"]), post_weight=cu(i["post"]), pre_weight=cu(i["pre"]), eps=EPS,
                             expert_gates=cu(i["gates"]), pair_row=cu(pair))
    r, dr, n, dn = reference(i["y"], i["x"], i["post"], None, 1.0, i["pre"], i["gates"], pair)
    close(got["r"], r, dr, "r")
    close(got["n"], n, dn, "n")
    assert (got["r"][2] == 0).all() and (got["n"][2] == 0).all()


def test_in_place_and_bad_rows_stay_apart():
    T, H = 12, 1544
    i = inputs(T, H, 0, True, "channel", BF, BF, F32, 12)
    args = dict(post_weight=cu(i["post"]), gate=cu(i["gate"]), pre_weight=cu(i["pre"]), residual_scale=0.5)
    want = ops.moe_block_norm(cu(i["y"]), x=cu(i["x"]), **args)
    x = cu(i["x"])
    got = ops.moe_block_norm(cu(i["y"]), x=x, r=x, **args)
    assert got["r"] is x and torch.equal(x, want["r"]) and torch.equal(got["n"], want["n"])
    y = cu(i["y"])
    y[3, 5], y[7] = float("nan"), float("inf")
    bad = ops.moe_block_norm(y, x=cu(i["x"]), **args)
    keep = [t for t in range(T) if t not in (3, 7)]
    assert torch.equal(bad["n"][keep], want["n"][keep]) and torch.isnan(bad["n"][3]).all()


@pytest.mark.parametrize("topk,xd,fmt", [(0, F32, None), (6, BF, "e4m3"), (2, BF, "e2m1")])
def test_large_batches_are_their_parts(topk, xd, fmt):
    """A batch that passes the caches by gives each of its rows the bits that it has in a smaller one."""
    T, H, part = 4224, 8064, 528
    i = inputs(T, H, topk, True, "full", xd, BF, BF, 21)
    t = {k: cu(v) for k, v in i.items()}
    want_fmt = dict(act_fmt=fmt, eps=EPS, residual_scale=0.75)
    whole = ops.moe_block_norm(t["y"], x=t["x"], post_weight=t["post"], gate=t["gate"], pre_weight=t["pre"],
                               expert_gates=t["gates"], pair_row=t["pair"], **want_fmt)
    for at in range(0, T, part):
        rows = slice(at, at + part)
        got = ops.moe_block_norm(t["y"] if topk else t["y"][rows], x=t["x"][rows], post_weight=t["post"],
                                 gate=t["gate"][rows], pre_weight=t["pre"],
                                 expert_gates=t["gates"][rows].contiguous() if topk else None,
                                 pair_row=t["pair"][at * topk:(at + part) * topk] if topk else None, **want_fmt)
        for k, v in got.items():
            assert v is None or torch.equal(v, whole[k][rows]), k
    few = slice(100, 140)
    pairs = i["pair"][100 * topk:140 * topk] if topk else None
    r, dr, n, dn = reference(i["y"] if topk else i["y"][few], i["x"][few], i["post"], i["gate"][few], 0.75, i["pre"],
                             i["gates"][few] if topk else None, pairs)
    close(whole["r"][few], r, dr, "r")
    close(whole["n"][few], n, dn, "n")


def test_without_weights():
    """No pre-norm weight is a weight of ones; without x and post-norm r is the gated block output."""
    i = inputs(7, 264, 0, False, "channel", None, BF, BF, 22)
    got = ops.moe_block_norm(cu(i["y"]), gate=cu(i["gate"]), eps=EPS, r_dtype=F32, n_dtype=F32)
    ones = ops.moe_block_norm(cu(i["y"]), gate=cu(i["gate"]), eps=EPS, r_dtype=F32, n_dtype=F32,
                              pre_weight=torch.ones(264, device="cuda"))
    r, dr, n, dn = reference(i["y"], None, None, i["gate"], 1.0, None, None, None)
    close(got["r"], r, dr, "r")
    close(got["n"], n, dn, "n")
    assert torch.equal(got["n"], ones["n"])


def test_no_rows():
    got = ops.moe_block_norm(torch.empty(0, 64, dtype=BF, device="cuda"))
    assert got["r"].shape == (0, 64) and got["n"].shape == (0, 64)


@pytest.mark.parametrize("H", [512, 2048, 7168, 16416, 40000])  # one, two, four and eight chunks a thread
@pytest.mark.parametrize("yd", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("topk", range(1, 9))
def test_every_number_of_combined_rows(topk, yd, H):
    """1 to 8 expert rows a token, a dropped pair and a token without any row among them; the combine alone has the
    bits of moe_unpermute_combine."""
    T = 300 if H < 7168 else 5
    i = inputs(T, H, topk, True, "channel", BF, yd, F32, topk * H)
    pair = i["pair"].clone()
    pair[topk - 1], pair[2 * topk:3 * topk] = -1, T * topk
    got = ops.moe_block_norm(cu(i["y"]), x=cu(i["x"]), post_weight=cu(i["post"]), gate=cu(i["gate"]),
                             residual_scale=0.75, pre_weight=cu(i["pre"]), eps=EPS, n_dtype=F32,
                             expert_gates=cu(i["gates"]), pair_row=cu(pair))
    r, dr, n, dn = reference(i["y"], i["x"], i["post"], i["gate"], 0.75, i["pre"], i["gates"], pair)
    close(got["r"], r, dr, "r")
    close(got["n"], n, dn, "n")
    alone = ops.moe_block_norm(cu(i["y"]), want_n=False, r_dtype=F32, expert_gates=cu(i["gates"]), pair_row=cu(i["pair"]))
    want = ops.moe_unpermute_combine(cu(i["y"]), cu(i["gates"]), cu(i["pair"]), T, topk, F32)
    assert torch.equal(alone["r"], want)


@pytest.mark.parametrize("topk,yd", [(3, BF), (8, BF), (7, F32)], ids=["3-bf16", "8-bf16", "7-fp32"])
def test_large_combined_batches_are_their_parts(topk, yd):
    T, H = 4224, 8064
    i = {k: cu(v) for k, v in inputs(T, H, topk, True, None, BF, yd, F32, 31).items()}
    whole = ops.moe_block_norm(i["y"], x=i["x"], post_weight=i["post"], pre_weight=i["pre"], act_fmt="e4m3",
                               expert_gates=i["gates"], pair_row=i["pair"])
    for at in range(0, T, 1056):
        rows = slice(at, at + 1056)
        got = ops.moe_block_norm(i["y"], x=i["x"][rows], post_weight=i["post"], pre_weight=i["pre"], act_fmt="e4m3",
                                 expert_gates=i["gates"][rows].contiguous(),
                                 pair_row=i["pair"][at * topk:(at + 1056) * topk])
        for k, v in got.items():
            assert torch.equal(v, whole[k][rows]), k


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("topk", [1, 2, 6, 8])
def test_dropped_pairs_take_nothing_from_any_row(topk, bad):
    """A dropped pair adds nothing, whatever its gate and the rows of y hold."""
    T, H = 4, 512
    i = inputs(T, H, topk, False, None, BF, BF, F32, 40 + topk)
    pair = i["pair"].clone()
    pair[::topk] = torch.tensor([-1, T * topk, -5, 2 ** 31 - 1], dtype=torch.int32)
    used = {int(p) for p in pair if 0 <= p < T * topk}
    free = [r for r in range(T * topk) if r not in used]
    i["y"][free] = bad
    i["gates"][:, 0] = bad
    got = ops.moe_block_norm(cu(i["y"]), x=cu(i["x"]), pre_weight=cu(i["pre"]), eps=EPS, expert_gates=cu(i["gates"]),
                             pair_row=cu(pair))
    clean_y, clean_g = i["y"].clone(), i["gates"].clone()
    clean_y[free], clean_g[:, 0] = 0, 0
    r, dr, n, dn = reference(clean_y, i["x"], None, None, 1.0, i["pre"], clean_g, pair)
    close(got["r"], r, dr, "r")
    close(got["n"], n, dn, "n")


@pytest.mark.parametrize("T", [2 ** 26 - 1, 2 ** 26, 2 ** 26 + 3])
def test_more_threads_than_32_bits(T):
    """A wave a token: up to 2^32 threads and more in one call. Every row, operand and result of it is the row's own."""
    H = 32
    y = torch.randn(7, H, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    t = torch.arange(T, device="cuda")
    args = dict(x=((t % 11).to(BF)[:, None] + torch.arange(H, device="cuda").to(BF)).contiguous(),
                gate=(1 + t % 3).to(BF)[:, None].contiguous(), expert_gates=(1 + t % 5).float().view(T, 1),
                pair_row=(t % 7).to(torch.int32))
    r = torch.full((T, H), float("nan"), dtype=BF, device="cuda")
    got = ops.moe_block_norm(y, act_fmt="e2m1", r=r, **args)
    for rows in (slice(0, 5000), slice(2 ** 26 - 5000, 2 ** 26), slice(T - 5000, T)):
        want = ops.moe_block_norm(y, act_fmt="e2m1", **{k: v[rows].clone() for k, v in args.items()})
        for k, v in want.items():
            assert torch.equal(got[k][rows], v), k
    assert torch.isfinite(r[::4096]).all()

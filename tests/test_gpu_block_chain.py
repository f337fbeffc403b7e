"""The block operators together, as a decoder block around 4-bit experts uses them: block norm -> FP4 projection with
adapters -> routing -> grouped W4A16 experts (moe_layer with bf16 activations) -> combine, post-norm, residual, next
pre-norm and its quantisation. Each stage against 64 bits on the stage's own inputs (the tolerances of the operators'
tests), captured graphs and other streams against the eager run bit for bit, guards around every buffer."""

import numpy as np
import pytest
import torch

import oracle
from mxfp4_block_scaled_amd import datagen as dg
from mxfp4_block_scaled_amd import ops
from tests import test_gpu_block_norm as bn
from tests import test_gpu_lora as lr
from tests import test_gpu_w4a16_grouped as gr
from tests.test_gpu_canary import Guarded

pytestmark = pytest.mark.gpu

H, I, E, TOPK = 1024, 512, 12, 3


class Block:
    """A small block's weights and one batch of T tokens of `S` requests."""

    def __init__(self, T, S, seed, fmt="mxfp4"):
        g = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.T, self.fmt = T, fmt
        self.x, self.y = (2 * rn(T, H)).to(torch.bfloat16).cuda(), rn(T, H).to(torch.bfloat16).cuda()
        self.post, self.pre = (1 + 0.1 * rn(H)).cuda(), (1 + 0.1 * rn(H)).cuda()
        self.gate = rn(H).to(torch.bfloat16).cuda()
        (self.wp, self.sp, self.hp), (self.w1, self.s1, self.h1), (self.w2, self.s2, self.h2) = (
            gr.weights(1, H, H, fmt, seed), gr.weights(E, 2 * I, H, fmt, seed + 1), gr.weights(E, H, I, fmt, seed + 2))
        if fmt == "mxfp4":  # scales of 2^-9 .. 2^4: bring the products back to about 1
            for s in (self.sp, self.s1, self.s2):
                s -= 7
            self.hp, self.h1, self.h2 = self.hp / 128, self.h1 / 128, self.h2 / 128
        self.la, self.lb, self.scaling = lr.adapters(3, 16, H, H, seed)
        cuts = sorted(torch.randperm(T - 1, generator=g)[:S - 1].tolist()) if S > 1 else []
        self.offs = [0] + [c + 1 for c in cuts] + [T]
        self.adapter = [i % 4 - 1 for i in range(S)]
        i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
        self.seg = (i32(self.offs), i32(self.adapter), self.la.cuda(), self.lb.cuda(), self.scaling.cuda())
        self.logits = torch.from_numpy(dg.logits(seed, T, E)).cuda()

    def run(self):
        a = ops.moe_block_norm(self.y, x=self.x, post_weight=self.post, gate=self.gate, residual_scale=0.5,
                               pre_weight=self.pre)
        c = ops.fp4_gemm_w4a16_lora(a["n"], self.wp[0], self.sp[0], *self.seg, self.fmt, out_dtype=torch.bfloat16)
        m = ops.moe_layer(c, self.logits, self.w1, self.s1, self.w2, self.s2, TOPK, act_fmt="bf16",
                          w_fmt=self.fmt)
        z = ops.moe_block_norm(m["y"], x=a["r"], post_weight=self.post, pre_weight=self.pre, act_fmt="e4m3",
                               expert_gates=m["gates"], pair_row=m["pair_row"])
        return dict(r=a["r"], n=a["n"], c=c, h=m["h"], y=m["y"], out=m["out"], gates=m["gates"],
                    offs=m["expert_offsets"], sp=m["sorted_pair"], pr=m["pair_row"], r2=z["r"], n2=z["n"], q=z["q"],
                    qs=z["q_scale"])


@pytest.mark.parametrize("T,S", [(1, 1), (7, 4), (130, 9), (700, 3)])
def test_stages_against_64_bits(T, S):
    b = Block(T, S, 40 + T)
    o = {k: v.cpu() for k, v in b.run().items()}
    cpu = lambda t: t.cpu()  # noqa: E731
    saved, bn.EPS = bn.EPS, 1e-6
    try:
        r, dr, n, dn = bn.reference(cpu(b.y), cpu(b.x), cpu(b.post), cpu(b.gate), 0.5, cpu(b.pre), None, None)
        bn.close(o["r"], r, dr, "r")
        bn.close(o["n"], n, dn, "n")
        c, dc = lr.reference(o["n"], b.hp[0], b.offs, b.adapter, b.la, b.lb, b.scaling)
        lr.close(o["c"], c, dc)
        ids, gates = oracle.route_topk(cpu(b.logits).numpy(), TOPK)
        offs, sp, pr = oracle.permute(ids, E)
        for got, want in ((o["offs"], offs), (o["sp"], sp), (o["pr"], pr)):
            assert np.array_equal(got.numpy(), want)
        src = o["sp"].long() // TOPK
        h, dh = gr.reference(o["c"], src, offs.tolist(), b.h1, True)
        gr.assert_close(o["h"], h, dh, "h")
        y, dy = gr.reference(o["h"], torch.arange(T * TOPK), offs.tolist(), b.h2, False)
        gr.assert_close(o["y"], y, dy, "y")
        r, dr, n, dn = bn.reference(o["y"], o["r"], cpu(b.post), None, 1.0, cpu(b.pre), o["gates"], o["pr"])
        bn.close(o["r2"], r, dr, "r2")
        bn.close(o["n2"], n, dn, "n2")
    finally:
        bn.EPS = saved


def test_bf16_layer_beside_the_quantised_one():
    """The same weights and routing: the bf16 layer's output is nearer the exact layer of the bf16 activations than
    the one that quantises them (E4M3), as for the dense products."""
    b = Block(96, 1, 5)
    x = b.x
    exact = torch.zeros(b.T, H, dtype=torch.float64)
    r = {f: ops.moe_layer(x, b.logits, b.w1, b.s1, b.w2, b.s2, TOPK, act_fmt=f) for f in ("bf16", "e4m3")}
    ids, gates, xd = r["bf16"]["topk_ids"].cpu(), r["bf16"]["gates"].cpu().double(), x.cpu().double()
    for t in range(b.T):
        for j in range(TOPK):
            e = int(ids[t, j])
            a = b.h1[e] @ xd[t]
            exact[t] += gates[t, j] * (b.h2[e] @ (a[:I] * torch.sigmoid(a[:I]) * a[I:]))
    err = {f: float((v["out"].cpu().double() - exact).norm() / exact.norm()) for f, v in r.items()}
    # h and y and out are rounded to bf16 (2^-8 each at most, on average far less); E4M3 rounds by 2^-4
    assert err["bf16"] < 3 * 2.0 ** -8 < err["e4m3"], err
    assert r["bf16"]["q"] is None and r["bf16"]["h"].dtype == torch.bfloat16


def same(got, want):
    for k in want:
        assert torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("T,S,fmt", [(1, 1, "mxfp4"), (8, 8, "mxfp4"), (300, 20, "nvfp4"), (900, 2, "mxfp4")])
def test_graph_replays_match_eager(T, S, fmt):
    b, other = Block(T, S, 60 + T, fmt), Block(T, S, 61 + T, fmt)
    want = {k: v.clone() for k, v in b.run().items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = b.run()
    with torch.cuda.graph(g2):  # a second captured run: its own workspaces
        out2 = b.run()
    mine = [b.x.clone(), b.y.clone(), b.logits.clone()]
    for rep in range(3):
        want_other = None
        if rep == 1:  # other inputs in the captured buffers
            for t, u in zip((b.x, b.y, b.logits), (other.x, other.y, other.logits)):
                t.copy_(u)
            want_other = {k: v.clone() for k, v in b.run().items()}
        other.run()  # eager work between the replays
        torch.cuda.synchronize()
        g.replay()
        g2.replay()
        torch.cuda.synchronize()
        same(out, want_other or want)
        same(out2, want_other or want)
        for t, u in zip((b.x, b.y, b.logits), mine):
            t.copy_(u)


def test_other_streams():
    """Two runs at once on streams of their own (each call its own workspace) give the eager run's bits."""
    b, c = Block(40, 10, 70), Block(260, 5, 71)
    wb, wc = ({k: v.clone() for k, v in x.run().items()} for x in (b, c))
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(3):
        with torch.cuda.stream(s1):
            ob = b.run()
        with torch.cuda.stream(s2):
            oc = c.run()
        got.append((ob, oc))
    torch.cuda.synchronize()
    for ob, oc in got:
        same(ob, wb)
        same(oc, wc)


@pytest.mark.parametrize("counts,N,K,fmt,swiglu,dt", [
    ([5, 0, 16, 2], 96, 640, "nvfp4", True, torch.bfloat16),
    ([40, 70, 3], 272, 128, "mxfp4", False, torch.float32),
    ([130, 63, 500], 4128, 128, "mxfp4", True, torch.bfloat16),
    ([17, 300, 129, 4, 256], 4112, 256, "nvfp4", False, torch.float32),
])
def test_grouped_writes_stay_inside(counts, N, K, fmt, swiglu, dt):
    R, E_ = sum(counts), len(counts)
    w, s, _ = gr.weights(E_, N, K, fmt, 80)
    offs = torch.tensor(np.cumsum([0] + counts), dtype=torch.int32).cuda()
    a = torch.randn(R, K).to(torch.bfloat16).cuda()
    y = Guarded((R, N // 2 if swiglu else N), dt, 81)
    want = ops.moe_grouped_gemm_w4a16(a, offs, w, s, fmt, swiglu=swiglu, out_dtype=dt)
    ops.moe_grouped_gemm_w4a16(a, offs, w, s, fmt, swiglu=swiglu, out=y.t)
    torch.cuda.synchronize()
    y.check("y")
    assert torch.equal(y.t, want)


@pytest.mark.parametrize("M,N,K,rank,S,dt", [
    (1, 16, 512, 8, 1, torch.bfloat16),
    (37, 272, 1536, 24, 30, torch.float32),
    (64, 1040, 512, 128, 2, torch.bfloat16),
    (65, 144, 512, 40, 65, torch.float32),
    (333, 528, 2048, 64, 3, torch.bfloat16),
    (4100, 4112, 512, 16, 4, torch.float32),  # large tiles
])
def test_lora_writes_stay_inside(M, N, K, rank, S, dt):
    w, s, _ = gr.weights(1, N, K, "mxfp4", 82)
    la, lb, scaling = (t.cuda() for t in lr.adapters(3, rank, N, K, 83))
    cuts = sorted(np.random.default_rng(M).permutation(M - 1)[:S - 1] + 1) if S > 1 else []
    offs = torch.tensor([0, *map(int, cuts), M], dtype=torch.int32).cuda()
    ad = torch.tensor([i % 4 - 1 for i in range(S)], dtype=torch.int32).cuda()
    a = torch.randn(M, K).to(torch.bfloat16).cuda()
    need = ops.load().fp4_w4a16_lora_workspace_bytes(M, N, K, rank)
    c, ws = Guarded((M, N), dt, 84), Guarded((need,), torch.uint8, 85)
    want = ops.fp4_gemm_w4a16_lora(a, w[0], s[0], offs, ad, la, lb, scaling, out_dtype=dt)
    ops.fp4_gemm_w4a16_lora(a, w[0], s[0], offs, ad, la, lb, scaling, out=c.t, workspace=ws.t)
    torch.cuda.synchronize()
    c.check("c")
    ws.check("workspace")
    assert torch.equal(c.t, want)


@pytest.mark.parametrize("T,H_,topk,fmt", [(3, 40, 0, None), (5, 1056, 2, "e2m1"), (2, 16416, 6, "e4m3"), (1, 32, 1, "e4m3")])
def test_block_norm_writes_stay_inside(T, H_, topk, fmt):
    i = bn.inputs(T, H_, topk, True, "full", torch.bfloat16, torch.bfloat16, torch.float32, 86)
    fp4 = fmt == "e2m1"
    r, n = Guarded((T, H_), torch.bfloat16, 87), Guarded((T, H_), torch.float32, 88)
    q = Guarded((T, H_ // 2 if fp4 else H_), torch.uint8, 89) if fmt else None
    qs = Guarded((T, H_ // 32), torch.uint8, 90) if fmt else None
    t = {k: bn.cu(v) for k, v in i.items()}
    at = ops._at
    ops._call("moe_block_norm", 0, at(t["y"]), 1, t["y"].shape[0], at(t["gates"]), at(t["pair"]), topk, T, H_,
              at(t["x"]), 1, 1.0, at(t["post"]), at(t["pre"]), 0, 1e-6, at(t["gate"]), 1, 3, at(r.t), at(n.t), 0,
              ops.FMTS[fmt] if fmt else 0, at(q.t) if q else None, at(qs.t) if qs else None)
    torch.cuda.synchronize()
    for name, v in (("r", r), ("n", n), ("q", q), ("q_scale", qs)):
        if v:
            v.check(name)
    assert torch.isfinite(n.t).all()


def test_binding_checks():
    """Wrong dtypes, shapes and layouts are named in the error; nothing is launched."""
    b = Block(4, 2, 90)
    with pytest.raises(RuntimeError, match="expert_offsets"):
        ops.moe_grouped_gemm_w4a16(b.x, torch.zeros(E, dtype=torch.int32, device="cuda"), b.w1, b.s1)
    with pytest.raises(RuntimeError, match="w_scale"):
        ops.moe_grouped_gemm_w4a16(b.x, torch.zeros(E + 1, dtype=torch.int32, device="cuda"), b.w1, b.s1, "nvfp4")
    with pytest.raises(RuntimeError, match="contiguous"):
        ops.moe_grouped_gemm_w4a16(b.x.t(), torch.zeros(E + 1, dtype=torch.int32, device="cuda"), b.w1, b.s1)
    with pytest.raises(RuntimeError, match="a: dtype"):
        ops.moe_grouped_gemm_w4a16(b.x.float(), torch.zeros(E + 1, dtype=torch.int32, device="cuda"), b.w1, b.s1)
    with pytest.raises(RuntimeError, match="MXF_ERR_SHAPE"):
        ops.moe_grouped_gemm_w4a16(b.x[:, :64].contiguous(), torch.zeros(2, dtype=torch.int32, device="cuda"),
                                   b.w1[:1, :, :32].contiguous(), b.s1[:1, :, :2].contiguous())
    with pytest.raises(RuntimeError, match="seg_offsets"):
        ops.fp4_gemm_w4a16_lora(b.x, b.wp[0], b.sp[0], b.seg[0][:-1], *b.seg[1:])
    with pytest.raises(RuntimeError, match="workspace"):
        ops.fp4_gemm_w4a16_lora(b.x, b.wp[0], b.sp[0], *b.seg, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(RuntimeError, match="x is on|x: "):
        ops.moe_block_norm(b.y, x=b.x[:2])
    with pytest.raises(RuntimeError, match="one dtype"):
        ops.moe_block_norm(b.y, post_weight=b.post, pre_weight=b.pre.bfloat16())
    with pytest.raises(RuntimeError, match="go together"):
        ops.moe_block_norm(b.y, pair_row=torch.zeros(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(RuntimeError, match="act_fmt"):
        ops.moe_block_norm(b.y, act_fmt="e5m2")


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_layer_of_no_tokens(fmt):
    b = Block(1, 1, 95, fmt)
    m = ops.moe_layer(b.x[:0], b.logits[:0], b.w1, b.s1, b.w2, b.s2, TOPK, act_fmt="bf16", w_fmt=fmt)
    assert m["out"].shape == (0, H) and m["h"].shape == (0, I) and m["y"].shape == (0, H)
    assert (m["expert_offsets"] == 0).all()
    z = ops.moe_block_norm(m["y"], x=b.x[:0], pre_weight=b.pre, act_fmt="e4m3", expert_gates=m["gates"],
                           pair_row=m["pair_row"])
    assert z["r"].shape == (0, H) and z["q_scale"].shape == (0, H // 32)

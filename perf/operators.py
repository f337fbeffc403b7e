"""The operators of a decoder block around 4-bit experts: cases, inputs, plain forms and exact values.

Three operators: `grouped` (ragged products by expert, FP4 weights x bf16 activations, optionally SwiGLU),
`norm` (post-norm, gate, residual and pre-norm of a block in one pass, optionally after the expert combine and
before the activation quantisation) and `lora` (a shared FP4 projection with low-rank adapters of many requests).
"""

import math

import torch

own = False

# E2M1 code -> value
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ---- cases ----------------------------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 8 tokens, top-6 of 256 experts: gate and up projections with SwiGLU
        dict(name="grouped decode fc1", op="grouped", T=8, topk=6, E=256, N=4096, K=7168, fmt="mxfp4", swiglu=True,
             gather=True, f32=False, zipf=False),
        # the skewed 2048-token prompt: the second projection of all its pairs, experts from none to hundreds of rows
        dict(name="grouped zipf fc2", op="grouped", T=2048, topk=6, E=256, N=7168, K=2048, fmt="mxfp4", swiglu=False,
             gather=False, f32=False, zipf=True),
        # one GPU's 32 of 256 experts in a 16384-token prompt spread over eight GPUs: 12288 rows, 384 an expert
        dict(name="grouped prefill share fc1", op="grouped", T=2048, topk=6, E=32, N=4096, K=7168, fmt="mxfp4",
             swiglu=True, gather=True, f32=False, zipf=False),
        # NVFP4 experts of odd sizes, a handful of tokens, fp32 results
        dict(name="grouped nvfp4 small", op="grouped", T=33, topk=2, E=6, N=528, K=1152, fmt="nvfp4", swiglu=False,
             gather=True, f32=True, zipf=False),
        # a single token through post-norm, residual and the next pre-norm: one launch's latency
        dict(name="norm one token", op="norm", T=1, H=7168, topk=0, post=True, gate="none", quant=False, f32=False),
        # the end of a 64-token expert layer: combine, post-norm, channel gate, residual, pre-norm, quantisation
        dict(name="norm combine 64", op="norm", T=64, H=7168, topk=6, post=True, gate="channel", quant=True, f32=False),
        # the same at the 16384-token prompt
        dict(name="norm combine 16384", op="norm", T=16384, H=7168, topk=6, post=True, gate="none", quant=True,
             f32=False),
        # fp32 residual stream, a gate for each token and channel, a width that is no multiple of the block
        dict(name="norm fp32 odd", op="norm", T=1999, H=1544, topk=0, post=False, gate="full", quant=False, f32=True),
        # decode: 64 requests of one token, 24 adapters among them
        dict(name="lora decode 64", op="lora", M=64, N=4096, K=7168, rank=16, L=24, S=64, fmt="mxfp4", f32=True),
        # one request, one token, an NVFP4 projection
        dict(name="lora one token", op="lora", M=1, N=2048, K=2048, rank=32, L=4, S=1, fmt="nvfp4", f32=False),
        # prompts of 16 requests together
        dict(name="lora prefill 4096", op="lora", M=4096, N=4096, K=7168, rank=64, L=8, S=16, fmt="mxfp4", f32=False),
        # chunks and single tokens mixed, odd sizes, fp32 result
        dict(name="lora mixed 777", op="lora", M=777, N=1520, K=2048, rank=24, L=16, S=101, fmt="mxfp4", f32=True),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    op = rng.choice(["grouped", "norm", "lora"])
    fmt = rng.choice(["mxfp4", "mxfp4", "nvfp4"])
    if op == "grouped":
        E = _log(rng, 2, 64)
        swiglu = rng.random() < 0.5
        return dict(op=op, T=_log(rng, 1, 1500), topk=rng.randint(1, min(6, E)), E=E,
                    N=_log(rng, 64, 4096, 32 if swiglu else 16), K=_log(rng, 128, 7168, 128), fmt=fmt, swiglu=swiglu,
                    gather=rng.random() < 0.6, f32=rng.random() < 0.3, zipf=rng.random() < 0.5)
    if op == "norm":
        quant = rng.random() < 0.4
        f32 = rng.random() < 0.3
        H = _log(rng, 64, 7168, 32 if quant else 8)
        return dict(op=op, T=_log(rng, 1, 8000), H=H, topk=rng.choice([0, 0, 1, 2, 6]), post=rng.random() < 0.6,
                    gate=rng.choice(["none", "channel", "token", "full"]), quant=quant, f32=f32)
    M = _log(rng, 1, 3000)
    return dict(op=op, M=M, N=_log(rng, 16, 4096, 16), K=_log(rng, 512, 7168, 512), rank=rng.randint(1, 16) * 8,
                L=rng.randint(1, 32), S=_log(rng, 1, min(M, 200)), fmt=fmt, f32=rng.random() < 0.5)


# ---- inputs ---------------------------------------------------------------------------------------------------

def _fp4_weights(shape, K, fmt, gen):
    """Codes uniform over the 16 values and scales of a few binades, about 0.03 in size."""
    w = torch.randint(0, 256, (*shape, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    if fmt == "nvfp4":  # UE4M3 bytes: 2^-7 .. 2^-5, every mantissa
        s = torch.randint(0, 24, (*shape, K // 16), dtype=torch.uint8, device="cuda", generator=gen)
    else:  # UE8M0 bytes: 2^-9 .. 2^-5
        s = torch.randint(118, 123, (*shape, K // 32), dtype=torch.uint8, device="cuda", generator=gen)
    return w, s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return (torch.randn(shape, device="cuda", generator=gen) * std).to(dtype)

    st = dict(case)
    if case["op"] == "grouped":
        T, topk, E, N, K = (case[k] for k in ("T", "topk", "E", "N", "K"))
        logits = torch.randn((T, E), device="cuda", generator=gen)
        if case["zipf"]:
            logits -= 1.1 * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
        ids = torch.topk(logits, topk, dim=1).indices.reshape(-1)
        st["sorted_pair"] = torch.argsort(ids, stable=True).to(torch.int32)
        counts = torch.bincount(ids, minlength=E)
        st["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        st["counts"] = counts.tolist()  # the plain form's loop goes by it
        st["a"] = normal(T if case["gather"] else T * topk, K)
        st["w"], st["ws"] = _fp4_weights((E, N), K, case["fmt"], gen)
        st["dtype"] = torch.float32 if case["f32"] else torch.bfloat16
    elif case["op"] == "norm":
        T, H, topk = case["T"], case["H"], case["topk"]
        dt = torch.float32 if case["f32"] else torch.bfloat16
        st["y"] = normal(T * topk if topk else T, H)
        if topk:
            st["expert_gates"] = torch.softmax(torch.randn((T, topk), device="cuda", generator=gen), 1)
            st["pair_row"] = torch.randperm(T * topk, device="cuda", generator=gen).to(torch.int32)
        st["x"] = normal(T, H, dtype=dt, std=2.0)
        st["post_weight"] = normal(H, dtype=torch.float32, std=0.1) + 1 if case["post"] else None
        st["pre_weight"] = normal(H, dtype=torch.float32, std=0.1) + 1
        shape = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[case["gate"]]
        st["gate"] = normal(*shape, std=0.5) if shape else None
        st["residual_scale"] = 0.875
    else:
        M, N, K, rank, L, S = (case[k] for k in ("M", "N", "K", "rank", "L", "S"))
        # S requests of at least one token; the last in four rows' places have no adapter
        cuts = torch.randperm(M - 1, device="cuda", generator=gen)[:S - 1] + 1 if S > 1 else None
        ends = torch.tensor([M], device="cuda")
        offs = torch.cat([torch.zeros_like(ends), cuts.sort().values, ends]) if S > 1 else torch.cat([0 * ends, ends])
        st["seg_offsets"] = offs.to(torch.int32)
        st["seg_adapter"] = torch.randint(-1 if L > 1 else 0, L, (S,), device="cuda", generator=gen).to(torch.int32)
        st["a"] = normal(M, K)
        st["w"], st["ws"] = _fp4_weights((N,), K, case["fmt"], gen)
        st["lora_a"] = normal(L, rank, K, std=K ** -0.5)
        st["lora_b"] = normal(L, N, rank, std=0.05)
        st["scaling"] = torch.rand((L,), device="cuda", generator=gen) + 0.5
        st["dtype"] = torch.float32 if case["f32"] else torch.bfloat16
    return st


# ---- one pass -------------------------------------------------------------------------------------------------

def run(st):
    if own:
        return _own(st)
    return {"grouped": _plain_grouped, "norm": _plain_norm, "lora": _plain_lora}[st["op"]](st)


def _own(st):
    from mxfp4_block_scaled_amd import ops

    if st["op"] == "grouped":
        return ops.moe_grouped_gemm_w4a16(st["a"], st["offsets"], st["w"], st["ws"], st["fmt"],
                                          sorted_pair=st["sorted_pair"] if st["gather"] else None,
                                          topk=st["topk"] if st["gather"] else 1, swiglu=st["swiglu"],
                                          out_dtype=st["dtype"])
    if st["op"] == "norm":
        d = ops.moe_block_norm(st["y"], x=st["x"], post_weight=st["post_weight"], gate=st["gate"],
                               residual_scale=st["residual_scale"], pre_weight=st["pre_weight"],
                               act_fmt="e4m3" if st["quant"] else None, want_n=not st["quant"],
                               expert_gates=st.get("expert_gates"), pair_row=st.get("pair_row"))
        if st["quant"]:
            return d["r"], d["q"].view(torch.float8_e4m3fn), d["q_scale"].view(torch.float8_e8m0fnu)
        return d["r"], d["n"]
    return ops.fp4_gemm_w4a16_lora(st["a"], st["w"], st["ws"], st["seg_offsets"], st["seg_adapter"], st["lora_a"],
                                   st["lora_b"], st["scaling"], st["fmt"], out_dtype=st["dtype"])


def _dequant(w, ws, fmt):
    """[N][K/2] codes and block scales -> [N][K] fp32 (exact)."""
    table = torch.tensor(E2M1, device=w.device)
    v = table[torch.stack((w & 15, w >> 4), -1).flatten(-2).int()]
    if fmt == "nvfp4":
        return (v.unflatten(-1, (-1, 16)) * ws.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * torch.exp2(ws.float() - 127)[..., None]).flatten(-2)


def _plain_grouped(st):
    rows = (st["sorted_pair"] // st["topk"]).long() if st["gather"] else None
    a = st["a"][rows] if st["gather"] else st["a"]
    R, N = a.shape[0], st["N"]
    y = torch.empty((R, N // 2 if st["swiglu"] else N), dtype=st["dtype"], device=a.device)
    at = 0
    for e, count in enumerate(st["counts"]):  # the products of an expert's rows: nothing to batch, sizes differ
        if count:
            acc = a[at:at + count].float() @ _dequant(st["w"][e], st["ws"][e], st["fmt"]).t()
            if st["swiglu"]:
                g, u = acc.chunk(2, dim=1)
                acc = g / (1 + torch.exp(-g)) * u
            y[at:at + count] = acc.to(y.dtype)
            at += count
    return y


def _rms(v, weight, eps=1e-6):
    return v / torch.sqrt(v.square().mean(1, keepdim=True) + eps) * weight


def _quantise_e4m3(n):
    """MX blocks of 32: E4M3 values and UE8M0 scales."""
    b = n.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    ex = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - 8, -127).clamp(min=-127)
    v = torch.ldexp(b, -ex)
    # the step of E4M3 at |v|: three bits below the leading one, 2^-9 under 2^-6
    step = torch.exp2((torch.frexp(v).exponent - 1).clamp(min=-6).float() - 3)
    v = (torch.round(v / step) * step).clamp(-448, 448)
    return (v.flatten(-2).to(torch.float8_e4m3fn), (ex.squeeze(-1) + 127).to(torch.uint8).view(torch.float8_e8m0fnu))


def _plain_norm(st):
    if st["topk"]:
        T, topk = st["expert_gates"].shape
        b = (st["y"].float()[st["pair_row"].long()].view(T, topk, -1) * st["expert_gates"][..., None]).sum(1)
    else:
        b = st["y"].float()
    if st["post_weight"] is not None:
        b = _rms(b, st["post_weight"])
    if st["gate"] is not None:
        b = b * st["gate"].float()
    r = st["residual_scale"] * st["x"].float() + b
    n = _rms(r, st["pre_weight"])
    r = r.to(st["x"].dtype)
    if st["quant"]:
        return (r, *_quantise_e4m3(n))
    return r, n.to(torch.bfloat16)


def _plain_lora(st):
    a = st["a"].float()
    M, N, L, rank = a.shape[0], st["N"], st["L"], st["rank"]
    seg = torch.bucketize(torch.arange(M, device=a.device, dtype=torch.int32), st["seg_offsets"], right=True) - 1
    adapter = st["seg_adapter"].long()[seg]
    low = a @ st["lora_a"].float().flatten(0, 1).t()  # every adapter's, [M][L * rank]; the others' are masked
    mine = adapter[:, None] == torch.arange(L, device=a.device)
    low = low.view(M, L, rank) * (mine * st["scaling"])[..., None]
    c = a @ _dequant(st["w"], st["ws"], st["fmt"]).t()
    c = c + low.flatten(1) @ st["lora_b"].float().transpose(1, 2).flatten(0, 1)
    return c.to(st["dtype"])


# ---- what a pass cannot do without ----------------------------------------------------------------------------

def _weight_bytes(N, K, fmt):
    return N * K // 2 + N * K // (16 if fmt == "nvfp4" else 32)


def work(case):
    if case["op"] == "grouped":
        T, topk, E, N, K = (case[k] for k in ("T", "topk", "E", "N", "K"))
        R = T * topk
        if case["zipf"]:  # experts expected to hold a row, by the share each expert has of a token's picks
            share = [(e + 1) ** -1.1 for e in range(E)]
            total = sum(share)
            touched = sum(1 - (1 - min(1.0, topk * s / total)) ** T for s in share)
        else:
            touched = E * (1 - (1 - topk / E) ** T)
        out = R * (N // 2 if case["swiglu"] else N) * (4 if case["f32"] else 2)
        return {"bytes": touched * _weight_bytes(N, K, case["fmt"]) + (T if case["gather"] else R) * K * 2 + out,
                "flops": 2.0 * R * N * K}
    if case["op"] == "norm":
        T, H, topk = case["T"], case["H"], case["topk"]
        res = 4 if case["f32"] else 2
        gate = {"none": 0, "channel": 2 * H, "token": 2 * T, "full": 2 * T * H}[case["gate"]]
        per = 2 * max(topk, 1) + 2 * res + (1 + 1 / 32 if case["quant"] else 2)
        return {"bytes": T * H * per + gate + 4 * H * (1 + case["post"]) + 8 * T * topk, "flops": 0}
    M, N, K, rank, L, S = (case[k] for k in ("M", "N", "K", "rank", "L", "S"))
    used = L * (1 - (1 - 1 / L) ** S)
    return {"bytes": _weight_bytes(N, K, case["fmt"]) + 2 * M * K + used * 2 * rank * (K + N)
            + M * N * (4 if case["f32"] else 2), "flops": 2.0 * M * N * K + 2.0 * M * rank * (K + N)}


# ---- the same from the definitions, in 64 bits ----------------------------------------------------------------

def _decode64(w, ws, fmt):
    """Weights by the bits of their codes: sign, exponent (bias 1), one mantissa bit; UE8M0 or UE4M3 scales."""
    code = torch.stack([w % 16, torch.div(w, 16, rounding_mode="floor")], dim=-1).reshape(*w.shape[:-1], -1).to(torch.int32)
    sign = 1.0 - 2.0 * (code >= 8).double()
    e, m = (code % 8) // 2, (code % 2).double()
    v = sign * torch.where(e == 0, 0.5 * m, torch.ldexp(1 + 0.5 * m, e - 1))
    s = ws.to(torch.int32)
    if fmt == "nvfp4":
        ex, ma = s // 8, (s % 8).double()
        scale = torch.where(ex == 0, ma / 512, torch.ldexp(1 + ma / 8, ex - 7))
        return v * scale.repeat_interleave(16, dim=-1)
    return v * torch.ldexp(torch.ones_like(s, dtype=torch.float64), s - 127).repeat_interleave(32, dim=-1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "grouped":
        rows = st["sorted_pair"].long()
        src = torch.div(rows, case["topk"], rounding_mode="floor") if case["gather"] else torch.arange(rows.numel(), device="cuda")
        a = st["a"].double()
        offs, parts = st["offsets"].tolist(), []
        for e in range(case["E"]):
            if offs[e + 1] > offs[e]:
                c = torch.mm(a[src[offs[e]:offs[e + 1]]], _decode64(st["w"][e], st["ws"][e], case["fmt"]).T.contiguous())
                if case["swiglu"]:
                    half = case["N"] // 2
                    c = c[:, :half] * torch.sigmoid(c[:, :half]) * c[:, half:]
                parts.append(c)
        return torch.cat(parts)
    if case["op"] == "norm":
        y, x = st["y"].double(), st["x"].double()
        T, H, topk = case["T"], case["H"], case["topk"]
        if topk:
            b = torch.zeros((T, H), dtype=torch.float64, device="cuda")
            for j in range(topk):
                b += st["expert_gates"][:, j:j + 1].double() * y[st["pair_row"][j::topk].long()]
        else:
            b = y
        if case["post"]:
            b = st["post_weight"].double() * b * torch.rsqrt((b * b).sum(1, keepdim=True) / H + 1e-6)
        if case["gate"] != "none":
            b = b * st["gate"].double()
        r = x * st["residual_scale"] + b
        n = st["pre_weight"].double() * r * torch.rsqrt((r * r).sum(1, keepdim=True) / H + 1e-6)
        if not case["quant"]:
            return r, n
        return r, None, None  # codes: values next to a border may fall on either side
    a, offs = st["a"].double(), st["seg_offsets"].tolist()
    c = torch.mm(a, _decode64(st["w"], st["ws"], case["fmt"]).T.contiguous())
    for s, l in enumerate(st["seg_adapter"].tolist()):
        if l >= 0:
            rows = slice(offs[s], offs[s + 1])
            low = torch.mm(a[rows], st["lora_a"][l].double().T.contiguous())
            c[rows] += st["scaling"][l].double() * torch.mm(low, st["lora_b"][l].double().T.contiguous())
    return c

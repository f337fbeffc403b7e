"""The operators of training with routed experts and 4-bit products: cases, inputs, plain forms and exact values.

Four operators: `balance` (per-expert counts, the load-balance and z losses of a router, and the router's gradient
from them and from its gates), `combine` (the backward pass of the gate-weighted combine), `quant` (quantisation to
MXFP4 or NVFP4 along rows, columns or both, and back) and `gemm` (the product of two quantised operands). `linear`
runs the last two together: a training step of a 4-bit linear layer.
"""

import math

import torch

own = False

# E2M1 code -> value
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
TINY = 2.0 ** -126


def _pow2(e):
    """2^e exactly, in 64 bits (torch's powers are off by an ulp on a GPU)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


# ---- cases ----------------------------------------------------------------------------------------------------

def listed():
    return [
        # one short sequence through a router of 256 experts: the launches' latency
        dict(name="balance 64 tokens", op="balance", T=64, E=256, topk=6, S=1, bf16=False, mask=False, limited=False),
        # a batch of 16 packed sequences, 16384 tokens, a tenth of them padding
        dict(name="balance 16384", op="balance", T=16384, E=256, topk=6, S=16, bf16=False, mask=True, limited=False),
        # bf16 logits of an odd number of experts, half of them ruled out for each token, many ragged sequences
        dict(name="balance bf16 odd", op="balance", T=5003, E=60, topk=4, S=37, bf16=True, mask=True, limited=True),
        # the smallest combine: one token
        dict(name="combine one token", op="combine", T=1, H=7168, topk=6, drop=0.0, f32=False),
        # the backward pass of a 16384-token expert layer's combine
        dict(name="combine 16384", op="combine", T=16384, H=7168, topk=6, drop=0.0, f32=False),
        # fp32, odd sizes, experts of limited capacity: a fifth of the pairs dropped
        dict(name="combine fp32 odd", op="combine", T=1999, H=1544, topk=3, drop=0.2, f32=True),
        # a gradient of 4096 tokens, both directions, stochastic rounding, the tensor's scale taken first
        dict(name="quant nvfp4 4096 x 7168", op="quant", rows=4096, cols=7168, fmt="nvfp4", f32=False, both=True,
             stochastic=True),
        # fp32 rows of odd number, MXFP4, along rows
        dict(name="quant mxfp4 odd", op="quant", rows=333, cols=2080, fmt="mxfp4", f32=True, both=False,
             stochastic=False),
        # a projection of 4096 tokens
        dict(name="gemm nvfp4 4096", op="gemm", M=4096, N=4096, K=7168, fmt="nvfp4", f32=False),
        # a weight gradient over 16384 tokens
        dict(name="gemm mxfp4 wgrad", op="gemm", M=4096, N=7168, K=16384, fmt="mxfp4", f32=True),
        # a handful of tokens, odd sizes
        dict(name="gemm nvfp4 small", op="gemm", M=24, N=528, K=1152, fmt="nvfp4", f32=True),
        # a training step of a linear layer: inputs, weights and gradients quantised both ways, three products
        dict(name="linear nvfp4 2000", op="linear", T=2000, O=4096, I=2048, fmt="nvfp4"),
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    op = rng.choice(["balance", "combine", "quant", "gemm", "linear"])
    fmt = rng.choice(["mxfp4", "nvfp4"])
    if op == "balance":
        T = _log(rng, 1, 16384)
        E = _log(rng, 4, 512 if T < 8000 else 256)
        return dict(op=op, T=T, E=E, topk=rng.randint(1, min(8, E // 2)), S=_log(rng, 1, min(T, 64)),
                    bf16=rng.random() < 0.4, mask=rng.random() < 0.5, limited=rng.random() < 0.3)
    if op == "combine":
        return dict(op=op, T=_log(rng, 1, 8000), H=_log(rng, 64, 7168, 8), topk=rng.randint(1, 8),
                    drop=rng.choice([0.0, 0.0, 0.1, 0.5]), f32=rng.random() < 0.3)
    if op == "quant":
        return dict(op=op, rows=_log(rng, 1, 4096), cols=_log(rng, 32, 7168, 32), fmt=fmt, f32=rng.random() < 0.3,
                    both=rng.random() < 0.6, stochastic=rng.random() < 0.4)
    if op == "gemm":
        return dict(op=op, M=_log(rng, 1, 4096), N=_log(rng, 16, 7168, 16), K=_log(rng, 128, 16384, 128), fmt=fmt,
                    f32=rng.random() < 0.5)
    return dict(op=op, T=_log(rng, 16, 4096), O=_log(rng, 128, 4096, 128), I=_log(rng, 128, 4096, 128), fmt=fmt)


# ---- inputs ---------------------------------------------------------------------------------------------------

def _fp4(rows, K, fmt, gen):
    """Codes uniform over the 16 values, scales of a few binades around one."""
    q = torch.randint(0, 256, (rows, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    if fmt == "nvfp4":  # UE4M3 bytes: 1/4 .. 4, every mantissa; and a scale of the whole tensor
        s = torch.randint(40, 72, (rows, K // 16), dtype=torch.uint8, device="cuda", generator=gen)
        return q, s, torch.rand((1,), device="cuda", generator=gen) * 0.01 + 0.01
    s = torch.randint(119, 124, (rows, K // 32), dtype=torch.uint8, device="cuda", generator=gen)
    return q, s, None


def _random_bytes(shape, gen):
    return torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=gen)


def _rows(case):
    return max(1, round(case["T"] * case["topk"] * (1 - case["drop"])))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return (torch.randn(shape, device="cuda", generator=gen) * std).to(dtype)

    st = dict(case)
    if case["op"] == "balance":
        T, E, topk, S = (case[k] for k in ("T", "E", "topk", "S"))
        logits = normal(T, E, dtype=torch.float32) + normal(E, dtype=torch.float32, std=0.5)  # some experts are liked
        if case["limited"]:  # half of the experts stay, in each token's own choice
            keep = torch.rand((T, E), device="cuda", generator=gen).argsort(1).argsort(1) < (E + 1) // 2
            logits = logits.masked_fill(~keep, -math.inf)
        logits = logits.to(torch.bfloat16 if case["bf16"] else torch.float32)
        st["logits"] = logits
        top = torch.sort(logits.float(), dim=1, descending=True, stable=True)
        st["topk_ids"] = top.indices[:, :topk].to(torch.int32).contiguous()
        st["gates"] = torch.softmax(top.values[:, :topk], 1)
        st["dgates"] = normal(T, topk, dtype=torch.float32, std=0.01)
        st["token_mask"] = (torch.rand((T,), device="cuda", generator=gen) >= 0.1).to(torch.uint8) if case["mask"] else None
        cuts = (torch.randperm(T - 1, device="cuda", generator=gen)[:S - 1] + 1).sort().values if S > 1 else None
        ends = torch.tensor([0, T], device="cuda")
        st["seg_offsets"] = (torch.cat([ends[:1], cuts, ends[1:]]) if S > 1 else ends).to(torch.int32)
        st["dlosses"] = torch.tensor([0.01, 0.001], device="cuda") * (1 + torch.rand((2,), device="cuda", generator=gen))
    elif case["op"] == "combine":
        T, H, topk = case["T"], case["H"], case["topk"]
        dt = torch.float32 if case["f32"] else torch.bfloat16
        st["gates"] = torch.softmax(torch.randn((T, topk), device="cuda", generator=gen), 1)
        st["dout"] = normal(T, H, dtype=dt, std=0.1)
        rows = _rows(case)  # of the pairs that found room
        pair_row = torch.full((T * topk,), -1, dtype=torch.int64, device="cuda")
        kept = torch.randperm(T * topk, device="cuda", generator=gen)[:rows]
        pair_row[kept] = torch.arange(rows, device="cuda")
        st["pair_row"] = pair_row.to(torch.int32)
        st["y"] = normal(rows, H, dtype=dt)
    elif case["op"] == "quant":
        rows, cols = case["rows"], case["cols"]
        x = torch.randn((rows, cols), device="cuda", generator=gen)
        x = x * torch.exp(torch.randn((1, cols), device="cuda", generator=gen))  # columns of different size
        st["x"] = (x * 0.01).to(torch.float32 if case["f32"] else torch.bfloat16)
        st["rnd"] = _random_bytes((rows, cols), gen) if case["stochastic"] else None
    elif case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        st["a"], st["a_scale"], st["a_ts"] = _fp4(M, K, case["fmt"], gen)
        st["b"], st["b_scale"], st["b_ts"] = _fp4(N, K, case["fmt"], gen)
        st["dtype"] = torch.float32 if case["f32"] else torch.bfloat16
    else:
        T, O, I = case["T"], case["O"], case["I"]
        st["x"] = normal(T, I)
        st["w"] = normal(O, I, std=I ** -0.5)
        st["dy"] = normal(T, O, std=0.01)
        st["rnd"] = _random_bytes((T, O), gen)
    return st


# ---- one pass -------------------------------------------------------------------------------------------------

def run(st):
    if own:
        return _own(st)
    return {"balance": _plain_balance, "combine": _plain_combine, "quant": _plain_quant, "gemm": _plain_gemm,
            "linear": _plain_linear}[st["op"]](st)


def _own(st):
    from mxfp4_block_scaled_amd import ops

    if st["op"] == "balance":
        d = ops.moe_balance_loss(st["logits"], st["topk_ids"], st["token_mask"], st["seg_offsets"])
        dlogits = ops.moe_route_backward(st["logits"], st["topk_ids"], st["gates"], st["dgates"], d, st["dlosses"],
                                         st["seg_offsets"])
        return d["losses"], d["counts"], d["prob_mean"], dlogits
    if st["op"] == "combine":
        return ops.moe_combine_backward(st["dout"], st["y"], st["gates"], st["pair_row"])
    fmt = st["fmt"]
    nv = fmt == "nvfp4"
    if st["op"] == "quant":
        g = ops.nvfp4_tensor_scale(st["x"]) if nv else None
        d = ops.fp4_quantize(st["x"], fmt, g, rnd=st["rnd"], transposed=st["both"])
        out = [ops.fp4_dequantize(d["q"], d["q_scale"], fmt, g), _as_float(d["q_scale"], nv)]
        if st["both"]:
            out += [ops.fp4_dequantize(d["qt"], d["qt_scale"], fmt, g), _as_float(d["qt_scale"], nv)]
        return out
    if st["op"] == "gemm":
        return ops.fp4_gemm(st["a"], st["a_scale"], st["b"], st["b_scale"], fmt, st["a_ts"], st["b_ts"],
                            out_dtype=st["dtype"])
    gx, gw, gy = (ops.nvfp4_tensor_scale(st[k]) if nv else None for k in ("x", "w", "dy"))
    x = ops.fp4_quantize(st["x"], fmt, gx, transposed=True)
    w = ops.fp4_quantize(st["w"], fmt, gw, transposed=True)
    dy = ops.fp4_quantize(st["dy"], fmt, gy, rnd=st["rnd"], transposed=True)
    y = ops.fp4_gemm(x["q"], x["q_scale"], w["q"], w["q_scale"], fmt, gx, gw, out_dtype=torch.bfloat16)
    dx = ops.fp4_gemm(dy["q"], dy["q_scale"], w["qt"], w["qt_scale"], fmt, gy, gw, out_dtype=torch.bfloat16)
    dw = ops.fp4_gemm(dy["qt"], dy["qt_scale"], x["qt"], x["qt_scale"], fmt, gy, gx, out_dtype=torch.float32)
    return y, dx, dw


def _as_float(scale, nv):
    return scale.view(torch.float8_e4m3fn if nv else torch.float8_e8m0fnu)


def _plain_balance(st):
    x, topk = st["logits"].float(), st["topk"]
    T, E = x.shape
    top = x.amax(1, keepdim=True)
    lse = top + torch.log(torch.exp(x - top).sum(1, keepdim=True))
    p = torch.exp(x - lse)
    ids = torch.arange(E, device=x.device, dtype=torch.int32)
    picks = (st["topk_ids"][..., None] == ids)  # [T][topk][E]
    chosen = picks.sum(1).float()
    offs = st["seg_offsets"]
    t = torch.arange(T, device=x.device)
    seg = ((t >= offs[:-1, None]) & (t < offs[1:, None])).float()  # [S][T]
    if st["token_mask"] is not None:
        seg = seg * st["token_mask"]
    n = seg.sum(1, keepdim=True)
    held = (n > 0).sum()
    counts = seg @ chosen
    per = 1 / n.clamp(min=1)
    mean = (seg @ p) * per
    scale = E / topk / held.clamp(min=1)
    balance = (counts * per * mean).sum() * scale
    total = n.sum().clamp(min=1)
    each = seg.sum(0)[:, None]
    z = (each * lse.square()).sum() / total
    # gradient
    c = seg.t() @ (counts * (per * per))  # [T][E], by the token's sequence
    g = st["dlosses"]
    d = g[0] * scale * p * (c - (p * c).sum(1, keepdim=True)) + g[1] * 2 / total * each * lse * p
    gates, dgates = st["gates"], st["dgates"]
    dsel = gates * (dgates - (gates * dgates).sum(1, keepdim=True))
    d = d + (picks * dsel[..., None]).sum(1)
    return torch.stack([balance, z]), counts.to(torch.int32), mean, d.to(st["logits"].dtype)


def _plain_combine(st):
    T, topk = st["gates"].shape
    row = st["pair_row"].long()
    at = row.clamp(min=0)
    dout = st["dout"].float()
    y = st["y"].float()[at].view(T, topk, -1)
    dgates = (y * dout[:, None]).sum(2) * (row >= 0).view(T, topk)
    dy = torch.empty_like(st["y"])
    pairs = torch.nonzero(row >= 0).squeeze(1)
    dy[row[pairs]] = (st["gates"].view(-1)[pairs, None] * dout[pairs // topk]).to(dy.dtype)
    return dy, dgates


def _tensor_scale(x):
    """The smallest power of two that takes the largest value to at most 6 x 448 (2688 = 21/16 x 2^11)."""
    amax = x.abs().amax()
    m, e = torch.frexp(amax)
    g = _pow2((e - 12 + (m > 21 / 32)).clamp(min=-126)).float()
    return torch.where(amax > 0, g, 1.0).reshape(1)


def _plain_values(x, fmt, g, rnd):
    """x [rows][cols] fp32, cols in blocks: the values that the codes stand for (without the tensor's scale), the
    block scales."""
    B = 16 if fmt == "nvfp4" else 32
    b = x.unflatten(-1, (-1, B))
    amax = b.abs().amax(-1, keepdim=True)
    if fmt == "nvfp4":
        s = (amax / (6 * g)).clamp(max=448).to(torch.float8_e4m3fn).float()
        s = torch.where(s * g >= TINY, s, 0.0)
        d = s * g
    else:
        s = _pow2(torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(min=-127)).float()
        d = s
    v = torch.where(d > 0, b / d, 0.0).abs()
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))
    u = v / step
    if rnd is None:
        u = torch.round(u)
    else:
        low = torch.floor(u)
        u = low + ((u - low) * 256 > rnd.unflatten(-1, (-1, B)) + 0.5)
    v = torch.copysign((u * step).clamp(max=6), b)
    return (v * s).flatten(-2), s.squeeze(-1)


def _padded_t(x):
    """x^T with its rows' length filled up to a multiple of 128."""
    return torch.nn.functional.pad(x.t(), (0, -x.shape[0] % 128)).contiguous()


def _plain_quant(st):
    x, fmt, rnd = st["x"].float(), st["fmt"], st["rnd"]
    g = _tensor_scale(x) if fmt == "nvfp4" else 1.0
    kind = torch.float8_e4m3fn if fmt == "nvfp4" else torch.float8_e8m0fnu
    v, s = _plain_values(x, fmt, g, rnd)
    out = [(v * g).to(torch.bfloat16), s.to(kind)]
    if st["both"]:
        v, s = _plain_values(_padded_t(x), fmt, g, None if rnd is None else _padded_t(rnd))
        out += [(v * g).to(torch.bfloat16), s.to(kind)]
    return out


def _decode(q, s, fmt):
    """[rows][K/2] codes and block scales -> [rows][K] fp32 (exact)."""
    table = torch.tensor(E2M1, device=q.device)
    v = table[torch.stack((q & 15, q >> 4), -1).flatten(-2).int()]
    if fmt == "nvfp4":
        return (v.unflatten(-1, (-1, 16)) * s.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)
    return (v.unflatten(-1, (-1, 32)) * _pow2(s.int() - 127).float()[..., None]).flatten(-2)


def _plain_gemm(st):
    c = _decode(st["a"], st["a_scale"], st["fmt"]) @ _decode(st["b"], st["b_scale"], st["fmt"]).t()
    if st["fmt"] == "nvfp4":
        c = c * (st["a_ts"] * st["b_ts"])
    return c.to(st["dtype"])


def _plain_linear(st):
    fmt = st["fmt"]
    x, w, dy, rnd = st["x"].float(), st["w"].float(), st["dy"].float(), st["rnd"]
    gx, gw, gy = (_tensor_scale(v) if fmt == "nvfp4" else 1.0 for v in (x, w, dy))
    y = _plain_values(x, fmt, gx, None)[0] @ _plain_values(w, fmt, gw, None)[0].t()
    dx = _plain_values(dy, fmt, gy, rnd)[0] @ _plain_values(_padded_t(w), fmt, gw, None)[0].t()
    dw = (_plain_values(_padded_t(dy), fmt, gy, _padded_t(rnd))[0]
          @ _plain_values(_padded_t(x), fmt, gx, None)[0].t())
    return (y * (gx * gw)).to(torch.bfloat16), (dx * (gy * gw)).to(torch.bfloat16), dw * (gy * gx)


# ---- what a pass cannot do without ----------------------------------------------------------------------------

def _coded(fmt):
    """Bytes of an element, its block's scale with it."""
    return 0.5 + 1 / (16 if fmt == "nvfp4" else 32)


def work(case):
    if case["op"] == "balance":
        T, E, topk, S = (case[k] for k in ("T", "E", "topk", "S"))
        e = 2 if case["bf16"] else 4
        return {"bytes": 2 * T * E * e + 12 * T * topk + T * case["mask"] + 4 * (S + 1) + 8 * S * E + 16, "flops": 0}
    if case["op"] == "combine":
        T, H, topk = case["T"], case["H"], case["topk"]
        e = 4 if case["f32"] else 2
        return {"bytes": T * H * e + 2 * _rows(case) * H * e + 12 * T * topk, "flops": 0}
    if case["op"] == "quant":
        n, padded = case["rows"] * case["cols"], -(-case["rows"] // 128) * 128 * case["cols"]
        out = 2 + _coded(case["fmt"]) - 0.5
        return {"bytes": n * ((4 if case["f32"] else 2) + case["stochastic"] + out) + case["both"] * padded * out,
                "flops": 0}
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * K * _coded(case["fmt"]) + M * N * (4 if case["f32"] else 2), "flops": 2.0 * M * N * K}
    T, O, I = case["T"], case["O"], case["I"]
    return {"bytes": 2 * (T * I + O * I + T * O) + T * O + 2 * (T * O + T * I) + 4 * O * I, "flops": 6.0 * T * O * I}


# ---- the same from the definitions, in 64 bits ----------------------------------------------------------------

def _e4m3(v):
    """Nearest E4M3 value (ties to even), at most 448, of v >= 0."""
    grid = _pow2((torch.frexp(v).exponent - 1).clamp(min=-6) - 3)
    return torch.minimum(torch.round(v / grid) * grid, torch.full_like(v, 448.0))


def _exact_values(x, fmt, g, rnd):
    rows, cols = x.shape
    B = 16 if fmt == "nvfp4" else 32
    blocks = x.reshape(rows, cols // B, B)
    amax = blocks.abs().max(dim=2).values
    if fmt == "nvfp4":
        s = _e4m3(amax / (6 * g))
    else:
        s = torch.where(amax > 0, _pow2((torch.frexp(amax).exponent - 3).clamp(min=-127)), 2.0 ** -127)
    unit = (s * g).unsqueeze(2).expand_as(blocks)
    v = torch.where(unit > 0, blocks.abs() / torch.where(unit > 0, unit, 1.0), 0.0)
    grid = torch.tensor(E2M1[:8], dtype=torch.float64, device=x.device)
    low = (torch.searchsorted(grid, v.contiguous(), right=True) - 1).clamp(0, 7)
    high = (low + 1).clamp(max=7)
    below, above = grid[low], grid[high]
    part = torch.where(above > below, (v - below) / torch.where(above > below, above - below, 1.0), 0.0)
    if rnd is None:
        up = (part > 0.5) | ((part == 0.5) & (low % 2 == 1))
    else:
        up = part > (rnd.reshape(blocks.shape).double() + 0.5) / 256
    out = torch.where(up, above, below) * torch.sign(blocks) * s.unsqueeze(2)
    return out.reshape(rows, cols) * g, s


def _exact_scale(x, fmt):
    if fmt != "nvfp4":
        return 1.0
    amax = float(x.abs().max())
    if amax == 0:
        return 1.0
    g = 2.0 ** -126
    while g * 2688 < amax:
        g *= 2
    return g


def _turned(x):
    rows, cols = x.shape
    out = torch.zeros((cols, -(-rows // 128) * 128), dtype=x.dtype, device=x.device)
    out[:, :rows] = x.T
    return out


def _exact_balance(st):
    x = st["logits"].double()
    T, E = x.shape
    topk, offs = st["topk"], st["seg_offsets"].tolist()
    S = len(offs) - 1
    p, lse = torch.softmax(x, 1), torch.logsumexp(x, 1)
    ids = st["topk_ids"].long()
    use = torch.ones(T, dtype=torch.bool, device="cuda") if st["token_mask"] is None else st["token_mask"].bool()
    counts = torch.zeros((S, E), dtype=torch.int64, device="cuda")
    mean = torch.zeros((S, E), dtype=torch.float64, device="cuda")
    sizes = [int(use[offs[s]:offs[s + 1]].sum()) for s in range(S)]
    held, total = max(1, sum(v > 0 for v in sizes)), max(1, sum(sizes))
    g = st["dlosses"].double()
    d, balance = torch.zeros_like(x), 0.0
    for s, size in enumerate(sizes):
        if size:
            at = torch.nonzero(use[offs[s]:offs[s + 1]]).squeeze(1) + offs[s]
            counts[s] = torch.bincount(ids[at].reshape(-1), minlength=E)
            mean[s] = p[at].sum(0) / size
            f = counts[s].double() * E / (topk * size)
            balance = balance + (f * mean[s]).sum() / held
            d[at] += g[0] / held / size * p[at] * (f - (p[at] * f).sum(1, keepdim=True))
    z = (lse[use] ** 2).sum() / total
    d[use] += g[1] / total * 2 * lse[use][:, None] * p[use]
    gates, dgates = st["gates"].double(), st["dgates"].double()
    d.scatter_add_(1, ids, gates * dgates - gates * (gates * dgates).sum(1, keepdim=True))
    return torch.stack([balance + 0 * z, z]), counts.to(torch.int32), mean, d


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "balance":
        return _exact_balance(st)
    if case["op"] == "combine":
        T, topk = st["gates"].shape
        row, gates = st["pair_row"].long().reshape(T, topk), st["gates"].double()
        dy = torch.zeros(st["y"].shape, dtype=torch.float64, device="cuda")
        dgates = torch.zeros_like(gates)
        for j in range(topk):
            t = torch.nonzero(row[:, j] >= 0).squeeze(1)
            dout = st["dout"][t].double()
            dy[row[t, j]] = gates[t, j:j + 1] * dout
            dgates[t, j] = (dout * st["y"][row[t, j]].double()).sum(1)
        return dy, dgates
    fmt = case["fmt"]
    if case["op"] == "quant":
        x = st["x"].double()
        g = _exact_scale(x, fmt)
        out = list(_exact_values(x, fmt, g, st["rnd"]))
        if case["both"]:
            out += _exact_values(_turned(x), fmt, g, None if st["rnd"] is None else _turned(st["rnd"]))
        return out
    if case["op"] == "gemm":
        def values(q, s, ts):
            code = torch.stack([q % 16, torch.div(q, 16, rounding_mode="floor")], dim=-1).reshape(q.shape[0], -1).int()
            e, m = (code % 8) // 2, (code % 2).double()
            v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * _pow2(e - 1)) * (1.0 - 2.0 * (code >= 8).double())
            b = s.int()
            if fmt == "nvfp4":
                k = torch.where(b // 8 == 0, (b % 8).double() / 512, (1 + (b % 8).double() / 8) * _pow2(b // 8 - 7))
                return v * k.repeat_interleave(16, dim=1) * ts.double()
            return v * _pow2(b - 127).repeat_interleave(32, dim=1)
        return torch.mm(values(st["a"], st["a_scale"], st["a_ts"]), values(st["b"], st["b_scale"], st["b_ts"]).T.contiguous())
    x, w, dy = st["x"].double(), st["w"].double(), st["dy"].double()
    gx, gw, gy = (_exact_scale(v, fmt) for v in (x, w, dy))

    def product(a, b):
        return torch.mm(a[0], b[0].T.contiguous())
    return (product(_exact_values(x, fmt, gx, None), _exact_values(w, fmt, gw, None)),
            product(_exact_values(dy, fmt, gy, st["rnd"]), _exact_values(_turned(w), fmt, gw, None)),
            product(_exact_values(_turned(dy), fmt, gy, _turned(st["rnd"])), _exact_values(_turned(x), fmt, gx, None)))

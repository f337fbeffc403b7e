"""Products of bf16 activations with FP4 weights in 64 bits on the GPU, from the formats' definitions, with the bounds
that the arithmetic gives; and which kernels a call of given sizes runs, from the library's own rule."""

import ctypes

import torch

from mxfp4_block_scaled_amd import ops

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
i32, i64 = ctypes.c_int32, ctypes.c_int64


def grouped_paths(R, E, N, K, fmt, swiglu):
    """[(rows, weight rows of a workgroup, experts of more than, up to so many rows)] of each launch."""
    fn = ops.load().mxf_w16_grouped_plan
    fn.argtypes = [i64, i32, i64, i64, i32, i32, ctypes.c_void_p]
    out = (i64 * 15)()
    n = fn(R, E, N, K, ops.WEIGHT_FMTS[fmt], int(swiglu), out)
    return [tuple(out[5 * i:5 * i + 4]) for i in range(n)]


def lora_path(M, N, K, rank, S):
    """(K slices of the projection, of the first product, rows of its workgroups, their share, tile rows, columns)"""
    fn = ops.load().mxf_w16_lora_plan
    fn.argtypes = [i64, i64, i64, i32, i64, ctypes.c_void_p]
    out = (i32 * 6)()
    fn(M, N, K, rank, S, out)
    return tuple(out)


def weights(shape, K, fmt, gen, scales=None):
    """Random codes and scale bytes [*shape][..] on the GPU; scales: the bytes' range (end excluded)."""
    lo, hi = scales or ((0, 0x50) if fmt == "nvfp4" else (118, 131))
    w = torch.randint(0, 256, (*shape, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    s = torch.randint(lo, hi, (*shape, K // (16 if fmt == "nvfp4" else 32)), dtype=torch.uint8, device="cuda", generator=gen)
    return w, s


def decode(w, s, fmt):
    """[N][K/2] codes and [N][..] scale bytes -> [N][K] doubles."""
    table = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=w.device)
    v = table[torch.stack((w & 15, w >> 4), -1).flatten(-2).long()]
    if fmt == "nvfp4":
        e, m = (s >> 3).long(), (s & 7).double()
        scale = torch.where(e == 0, m / 512, (1 + m / 8) * torch.exp2(e.double() - 7))
        return v * scale.repeat_interleave(16, -1)
    return v * torch.exp2(s.double() - 127).repeat_interleave(32, -1)


def product(x, w, s, fmt):
    """x W^T and the sum of |x| |W| in 64 bits."""
    hat = decode(w, s, fmt).t().contiguous()
    return x.double() @ hat, x.double().abs() @ hat.abs()


def silu_mul(acc, mag):
    """SwiGLU of (value, bound) halves: sup |silu'| < 1.1, and 2^-19 of the result for exponential and reciprocal."""
    (g, u), (dg, du) = acc.chunk(2, 1), mag.chunk(2, 1)
    silu = g * torch.sigmoid(g)
    return silu * u, 1.1 * dg * (u.abs() + du) + silu.abs() * du + 2.0 ** -19 * (silu * u).abs()


def close(got, want, d, what="result"):
    """|got - want| within d and the half step of got's type."""
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    err, lim = (got.double() - want).abs(), d + half * (want.abs() + d) + 1e-38
    assert (err <= lim).all(), f"{what}: error {float((err / lim).max()):.3g} of its bound"

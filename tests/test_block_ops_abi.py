"""Refusals of the block operators (grouped W4A16, adapters, block norm) on the CPU: every bad argument returns its
status before any device call, and the binding's own checks raise."""

import ctypes
import os

import pytest
import torch

from mxfp4_block_scaled_amd import ops

OK, NULL, SHAPE, ALIGN, FORMAT, UNSUPPORTED, LAUNCH, WORKSPACE = range(8)
P = ctypes.c_void_p
A, U = 4096, 4096 + 4  # never dereferenced: validation fails first


def _lib():
    if not os.path.exists(ops.lib_path()):
        pytest.skip("library not built (run __graft_entry__.build())")
    return ops.load()


def call(fn, good, **change):
    return fn(*{**good, **change}.values())


def test_grouped_w4a16_errors():
    fn = _lib().moe_grouped_gemm_w4a16
    good = dict(a=A, a_rows=8, R=16, pair=A, topk=2, offs=A, E=4, N=64, K=256, fmt=0, w=A, ws=A, swiglu=0, y=A, yd=1,
                stream=None)
    assert call(fn, good, R=0) == OK
    for change, want in [
        (dict(fmt=2), FORMAT), (dict(yd=2), FORMAT), (dict(R=-1), SHAPE), (dict(a_rows=-1), SHAPE),
        (dict(E=0), SHAPE), (dict(N=24), SHAPE), (dict(N=48, swiglu=1), SHAPE), (dict(N=0), SHAPE),
        (dict(K=192), SHAPE), (dict(K=0), SHAPE), (dict(topk=0), SHAPE), (dict(a_rows=0), SHAPE),
        (dict(pair=None), SHAPE), (dict(swiglu=2), SHAPE), (dict(E=1025), UNSUPPORTED),
        (dict(R=2 ** 31, a_rows=2 ** 30), UNSUPPORTED), (dict(K=2 ** 22), UNSUPPORTED),
        (dict(N=2 ** 17, K=2 ** 16), UNSUPPORTED), (dict(a_rows=2 ** 23, K=256), UNSUPPORTED),
        (dict(R=2 ** 31 - 1, a_rows=2 ** 20, N=2 ** 20), UNSUPPORTED),
        (dict(a=None), NULL), (dict(offs=None), NULL), (dict(w=None), NULL), (dict(ws=None), NULL), (dict(y=None), NULL),
        (dict(a=U), ALIGN), (dict(pair=U), ALIGN), (dict(offs=U), ALIGN), (dict(w=U), ALIGN), (dict(ws=U), ALIGN),
        (dict(y=U), ALIGN),
    ]:
        assert call(fn, good, **change) == want, change
    assert call(fn, good, pair=None, a_rows=16, w=None) == NULL  # ungathered: a has R rows


def test_lora_errors():
    lib = _lib()
    fn = lib.fp4_gemm_w4a16_lora
    need = lib.fp4_w4a16_lora_workspace_bytes(40, 64, 4096, 16)
    assert need >= (2 * 40 * 64 + 40 * 16) * 4  # K slices of the projection and the low-rank rows
    assert lib.fp4_w4a16_lora_workspace_bytes(0, 64, 4096, 16) == 0
    assert lib.fp4_w4a16_lora_workspace_bytes(100, 64, 4096, 16) >= 100 * 16 * 4
    good = dict(a=A, M=40, N=64, K=4096, fmt=0, w=A, ws=A, so=A, sa=A, S=3, la=A, lb=A, sc=A, L=2, rank=16, c=A, cd=0,
                wk=A, wb=need, stream=None)
    assert call(fn, good, M=0) == OK
    for change, want in [
        (dict(fmt=-1), FORMAT), (dict(cd=3), FORMAT), (dict(M=-1), SHAPE), (dict(N=40), SHAPE), (dict(K=4096 + 128), SHAPE),
        (dict(S=-1), SHAPE), (dict(L=-1), SHAPE), (dict(rank=0), SHAPE), (dict(rank=12), SHAPE), (dict(rank=136), SHAPE),
        (dict(K=2 ** 22), UNSUPPORTED), (dict(N=2 ** 17, K=2 ** 16), UNSUPPORTED),
        (dict(M=2 ** 31 - 1, N=2 ** 13), UNSUPPORTED), (dict(N=2 ** 24, K=512, rank=128), UNSUPPORTED),
        (dict(a=None), NULL), (dict(w=None), NULL), (dict(ws=None), NULL),
        (dict(c=None), NULL), (dict(so=None), NULL), (dict(sa=None), NULL), (dict(la=None), NULL), (dict(lb=None), NULL),
        (dict(sc=None), NULL), (dict(a=U), ALIGN), (dict(so=U), ALIGN), (dict(sa=U), ALIGN), (dict(la=U), ALIGN),
        (dict(lb=U), ALIGN), (dict(sc=U), ALIGN), (dict(c=U), ALIGN), (dict(wk=U), ALIGN),
        (dict(wk=None), WORKSPACE), (dict(wb=need - 1), WORKSPACE),
    ]:
        assert call(fn, good, **change) == want, change


def test_block_norm_errors():
    fn = _lib().moe_block_norm
    good = dict(y=A, yd=1, rows=24, eg=A, pr=A, topk=3, T=8, H=64, x=A, xd=1, alpha=1.0, post=A, pre=A, wd=0, eps=1e-6,
                gate=A, gd=1, gm=1, r=A, n=A, nd=1, fmt=0, q=A, qs=A, stream=None)
    assert call(fn, good, T=0) == OK
    for change, want in [
        (dict(yd=2), FORMAT), (dict(xd=-1), FORMAT), (dict(wd=2), FORMAT), (dict(gd=2), FORMAT), (dict(nd=2), FORMAT),
        (dict(fmt=2), FORMAT), (dict(gm=4), FORMAT), (dict(gm=-1), FORMAT), (dict(T=-1), SHAPE), (dict(H=0), SHAPE),
        (dict(H=40), SHAPE), (dict(H=12, q=None, qs=None), SHAPE), (dict(topk=9), SHAPE), (dict(topk=-1), SHAPE),
        (dict(rows=-1), SHAPE), (dict(topk=0), SHAPE), (dict(eps=0.0), SHAPE), (dict(eps=float("nan")), SHAPE),
        (dict(H=65568), UNSUPPORTED), (dict(T=2 ** 31, rows=8), UNSUPPORTED), (dict(y=None), NULL), (dict(eg=None), NULL),
        (dict(pr=None), NULL), (dict(gate=None), NULL), (dict(q=None), NULL), (dict(qs=None), NULL),
        (dict(r=None, n=None, q=None, qs=None), NULL), (dict(y=U), ALIGN), (dict(x=U), ALIGN), (dict(post=U), ALIGN),
        (dict(pre=U), ALIGN), (dict(gate=U), ALIGN), (dict(r=U), ALIGN), (dict(n=U), ALIGN), (dict(q=U), ALIGN),
        (dict(qs=U), ALIGN), (dict(pr=U), ALIGN), (dict(eg=U), ALIGN),
    ]:
        assert call(fn, good, **change) == want, change


def test_block_norm_combine_needs_rows():
    """The combine of dropped pairs only still reads a row of y beside them: there has to be one."""
    fn = _lib().moe_block_norm
    good = dict(y=A, yd=1, rows=0, eg=A, pr=A, topk=2, T=0, H=64, x=None, xd=1, alpha=1.0, post=None, pre=None, wd=0,
                eps=1e-6, gate=None, gd=1, gm=0, r=A, n=A, nd=1, fmt=0, q=None, qs=None, stream=None)
    assert call(fn, good) == OK
    assert call(fn, good, T=5) == SHAPE


def test_binding_refuses_host_tensors():
    z = torch.zeros
    a, off = z(4, 128, dtype=torch.bfloat16), z(3, dtype=torch.int32)
    w, s = z(2, 16, 64, dtype=torch.uint8), z(2, 16, 4, dtype=torch.uint8)
    with pytest.raises(RuntimeError, match="GPU"):
        ops.moe_grouped_gemm_w4a16(a, off, w, s)
    with pytest.raises(RuntimeError, match="GPU"):
        ops.moe_block_norm(a)
    with pytest.raises(RuntimeError, match="GPU"):
        ops.fp4_gemm_w4a16_lora(a, w[0], s[0], off, off[:2], z(1, 8, 128), z(1, 16, 8), z(1))


def test_bf16_layer_has_no_fused_form():
    x = torch.zeros(2, 512, dtype=torch.bfloat16)
    with pytest.raises(RuntimeError, match="fused"):
        ops.moe_layer(x, None, None, None, None, None, 2, act_fmt="bf16", fused=True)
    with pytest.raises(RuntimeError, match="w_fmt"):
        ops.moe_layer(x, None, None, None, None, None, 2, act_fmt="e4m3", w_fmt="nvfp4")


def test_launches_of_too_many_threads_are_refused():
    """A launch of 2^32 threads or more would run modulo 2^32: sizes that need one are UNSUPPORTED, those below are not."""
    fn = _lib().moe_grouped_gemm_w4a16
    good = dict(a=None, a_rows=128, R=128, pair=None, topk=1, offs=A, E=8, N=2 ** 26 - 512, K=128, fmt=0, w=A, ws=A, swiglu=0,
                y=A, yd=1, stream=None)
    assert call(fn, good, E=48) == NULL  # 56 units of 16 rows, each with 2^18 - 2 workgroups of 256 threads
    assert call(fn, good, E=64) == UNSUPPORTED  # 72
    assert call(fn, good, E=1024, N=2 ** 22, R=2 ** 16, a_rows=2 ** 16) == UNSUPPORTED
    assert call(fn, good, E=1024, N=2 ** 21, R=2 ** 16, a_rows=2 ** 16) == NULL
    fn = _lib().fp4_gemm_w4a16_lora
    good = dict(a=None, M=2 ** 28 - 256, N=64, K=512, fmt=0, w=A, ws=A, so=A, sa=A, S=2 ** 28, la=A, lb=A, sc=A, L=2, rank=16,
                c=A, cd=0, wk=A, wb=0, stream=None)
    assert call(fn, good) == NULL
    assert call(fn, good, M=2 ** 28) == UNSUPPORTED
    assert call(fn, good, M=2 ** 25, N=2 ** 14) == UNSUPPORTED
    out = (ctypes.c_int32 * 6)()
    plan = _lib().mxf_w16_lora_plan
    plan.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p]
    for M, rows in ((2 ** 26 - 1, 16), (2 ** 26, 32)):  # 16 rows take 1024 threads, 32 take 512
        plan(M, 64, 512, 16, M, out)
        assert out[2] == rows


def test_a_combine_of_too_many_threads_is_refused():
    fn = _lib().moe_unpermute_combine
    good = dict(y=None, yd=1, gates=A, pr=A, T=2 ** 25 - 2, topk=1, H=1024, out=A, od=1, stream=None)
    assert call(fn, good) == NULL
    assert call(fn, good, T=2 ** 25) == UNSUPPORTED
    assert call(fn, good, T=2 ** 19, H=65536) == UNSUPPORTED

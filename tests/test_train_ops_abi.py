"""Refusals of the operators of training on the CPU: every bad argument returns its status before any device call, and
the binding's own checks raise."""

import ctypes
import os

import pytest
import torch

from mxfp4_block_scaled_amd import ops

OK, NULL, SHAPE, ALIGN, FORMAT, UNSUPPORTED, LAUNCH, WORKSPACE = range(8)
A, U = 4096, 4096 + 4  # never dereferenced: validation fails first
U2 = 4096 + 2


def _lib():
    if not os.path.exists(ops.lib_path()):
        pytest.skip("library not built (run __graft_entry__.build())")
    return ops.load()


def call(fn, good, **change):
    return fn(*{**good, **change}.values())


def test_balance_loss_errors():
    lib = _lib()
    fn = lib.moe_balance_loss
    need = lib.moe_balance_loss_workspace_bytes(300, 60, 3)
    assert need >= 8 * 60 * 8  # five workgroups and three sequences: slots of counts and sums
    good = dict(lg=A, ld=0, ids=A, mask=A + 1, so=A, S=3, T=300, E=60, topk=4, c=A, n=A, p=A, lse=A, loss=A, ws=A, wb=need,
                stream=None)
    for change, want in [
        (dict(ld=2), FORMAT), (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(topk=0), SHAPE), (dict(topk=9), SHAPE),
        (dict(E=3), SHAPE), (dict(S=0), SHAPE), (dict(E=1025), UNSUPPORTED), (dict(T=2 ** 29), UNSUPPORTED),
        (dict(T=2 ** 26), UNSUPPORTED), (dict(S=2 ** 23), UNSUPPORTED), (dict(so=None), NULL), (dict(lg=None), NULL),
        (dict(ids=None), NULL), (dict(c=None), NULL), (dict(n=None), NULL), (dict(p=None), NULL), (dict(lse=None), NULL),
        (dict(loss=None), NULL), (dict(lg=U), ALIGN), (dict(ids=U), ALIGN), (dict(so=U), ALIGN), (dict(c=U), ALIGN),
        (dict(n=U), ALIGN), (dict(p=U), ALIGN), (dict(lse=U), ALIGN), (dict(loss=U), ALIGN), (dict(ws=U), ALIGN),
        (dict(ws=None), WORKSPACE), (dict(wb=need - 1), WORKSPACE),
    ]:
        assert call(fn, good, **change) == want, change


def test_route_backward_errors():
    fn = _lib().moe_route_backward
    good = dict(lg=A, ld=0, ids=A, g=A, dg=A, dl=A, lse=A, c=A, n=A, so=A, S=3, T=300, E=60, topk=4, out=A, stream=None)
    assert call(fn, good, T=0) == OK
    for change, want in [
        (dict(ld=-1), FORMAT), (dict(T=-1), SHAPE), (dict(topk=61, E=60), SHAPE), (dict(S=0), SHAPE),
        (dict(E=1025), UNSUPPORTED), (dict(T=2 ** 26), UNSUPPORTED), (dict(out=None), NULL), (dict(dg=None, dl=None), NULL),
        (dict(g=None), NULL), (dict(ids=None), NULL), (dict(lg=None), NULL), (dict(lse=None), NULL), (dict(c=None), NULL),
        (dict(n=None), NULL), (dict(so=None), NULL), (dict(lg=U), ALIGN), (dict(ids=U), ALIGN), (dict(g=U), ALIGN),
        (dict(dg=U), ALIGN), (dict(dl=U2), ALIGN), (dict(lse=U), ALIGN), (dict(c=U), ALIGN), (dict(n=U), ALIGN),
        (dict(so=U), ALIGN), (dict(out=U), ALIGN),
    ]:
        assert call(fn, good, **change) == want, change


def test_combine_backward_errors():
    fn = _lib().moe_combine_backward
    good = dict(do=A, dd=1, y=A, yd=1, rows=24, g=A, pr=A, T=8, topk=3, H=64, dy=A, dg=A, stream=None)
    assert call(fn, good, T=0) == OK
    for change, want in [
        (dict(dd=2), FORMAT), (dict(yd=2), FORMAT), (dict(T=-1), SHAPE), (dict(rows=-1), SHAPE), (dict(topk=0), SHAPE),
        (dict(topk=9), SHAPE), (dict(H=0), SHAPE), (dict(H=12), SHAPE), (dict(T=2 ** 30), UNSUPPORTED),
        (dict(T=2 ** 26, H=1024), UNSUPPORTED), (dict(T=2 ** 24, H=7168), UNSUPPORTED), (dict(do=None), NULL),
        (dict(y=None), NULL), (dict(g=None), NULL), (dict(pr=None), NULL), (dict(dy=None, dg=None), NULL), (dict(do=U), ALIGN),
        (dict(y=U), ALIGN), (dict(g=U), ALIGN), (dict(pr=U), ALIGN), (dict(dy=U), ALIGN), (dict(dg=U), ALIGN),
    ]:
        assert call(fn, good, **change) == want, change


def test_workspace_without_tokens():
    """No tokens in many sequences: one workgroup's slots beside the sequences', as for any few tokens."""
    fn = _lib().moe_balance_loss_workspace_bytes
    assert fn(0, 60, 1) == fn(64, 60, 1) == 0
    assert fn(0, 60, 5000) == fn(1, 60, 5000) >= 5000 * 60 * 8


def test_token_counts_whose_products_pass_64_bits():
    """T * topk of 2^64 is 0 in 64 bits; so are the threads of such a call."""
    lib = _lib()
    for T in (2 ** 61, 2 ** 62, 2 ** 63 - 1):
        assert lib.moe_balance_loss(A, 0, A, None, None, 1, T, 60, 8, A, A, A, A, A, A, 2 ** 62, None) == UNSUPPORTED
        assert lib.moe_route_backward(A, 0, A, A, A, A, A, A, A, None, 1, T, 60, 8, A, None) == UNSUPPORTED
        assert lib.moe_combine_backward(A, 0, A, 0, 64, A, A, T, 8, 64, A, A, None) == UNSUPPORTED


def test_quantise_errors():
    lib = _lib()
    fn = lib.nvfp4_tensor_scale
    n = 2 ** 20
    need = lib.nvfp4_tensor_scale_workspace_bytes(n, 1)
    assert need > 0 and lib.nvfp4_tensor_scale_workspace_bytes(64, 1) == 0  # small: one workgroup
    good = dict(x=A, xd=1, n=n, out=A, ws=A, wb=need, stream=None)
    for change, want in [
        (dict(xd=2), FORMAT), (dict(n=0), SHAPE), (dict(n=48), SHAPE), (dict(x=None), NULL), (dict(out=None), NULL),
        (dict(x=U), ALIGN), (dict(out=U2), ALIGN), (dict(ws=U), ALIGN), (dict(ws=None), WORKSPACE), (dict(wb=need - 1), WORKSPACE),
    ]:
        assert call(fn, good, **change) == want, change
    fn = lib.fp4_quantize
    good = dict(x=A, xd=1, rows=10, cols=64, fmt=1, g=U, rnd=A, q=A, qs=A, qt=A, qts=A, stream=None)
    assert call(fn, good, rows=0) == OK
    for change, want in [
        (dict(xd=2), FORMAT), (dict(fmt=2), FORMAT), (dict(rows=-1), SHAPE), (dict(cols=0), SHAPE), (dict(cols=48), SHAPE),
        (dict(fmt=0), SHAPE), (dict(rows=2 ** 31), UNSUPPORTED), (dict(cols=2 ** 31), UNSUPPORTED),
        (dict(rows=2 ** 30, cols=2 ** 14), UNSUPPORTED), (dict(cols=2 ** 22), UNSUPPORTED), (dict(rows=2 ** 28, cols=1024, qt=None, qts=None), UNSUPPORTED),
        (dict(x=None), NULL), (dict(q=None), NULL), (dict(qs=None), NULL), (dict(qt=None), NULL), (dict(qts=None), NULL),
        (dict(q=None, qs=None, qt=None, qts=None), NULL), (dict(x=U), ALIGN), (dict(g=U2), ALIGN), (dict(rnd=U), ALIGN),
        (dict(q=U), ALIGN), (dict(qs=U), ALIGN), (dict(qt=U), ALIGN), (dict(qts=U), ALIGN),
    ]:
        assert call(fn, good, **change) == want, change
    fn = lib.fp4_dequantize
    good = dict(q=A, qs=A, rows=10, cols=64, fmt=1, g=U, out=A, od=1, stream=None)
    assert call(fn, good, rows=0) == OK
    for change, want in [
        (dict(od=2), FORMAT), (dict(fmt=-1), FORMAT), (dict(rows=-1), SHAPE), (dict(cols=16), SHAPE), (dict(fmt=0), SHAPE),
        (dict(rows=2 ** 31), UNSUPPORTED), (dict(rows=2 ** 27, cols=1024), UNSUPPORTED), (dict(q=None), NULL),
        (dict(qs=None), NULL), (dict(out=None), NULL), (dict(q=U), ALIGN), (dict(qs=U), ALIGN), (dict(g=U2), ALIGN),
        (dict(out=U), ALIGN),
    ]:
        assert call(fn, good, **change) == want, change


def test_fp4_gemm_errors():
    lib = _lib()
    fn = lib.fp4_gemm
    M, N, K = 100, 272, 16256
    need = lib.fp4_gemm_workspace_bytes(M, N, K, 1)
    assert need >= 2 * M * N * 4 and lib.fp4_gemm_workspace_bytes(0, N, K, 1) == 0  # few tiles: K slices
    assert lib.fp4_gemm_workspace_bytes(8192, 8192, K, 0) == 0
    good = dict(a=A, sa=A, M=M, b=A, sb=A, N=N, K=K, fmt=1, ga=U, gb=U, c=A, cd=1, ws=A, wb=need, stream=None)
    assert call(fn, good, M=0) == OK
    for change, want in [
        (dict(fmt=2), FORMAT), (dict(cd=2), FORMAT), (dict(M=-1), SHAPE), (dict(N=0), SHAPE), (dict(N=24), SHAPE),
        (dict(K=0), SHAPE), (dict(K=192), SHAPE), (dict(fmt=0), SHAPE), (dict(fmt=0, ga=None), SHAPE),
        (dict(M=2 ** 31), UNSUPPORTED), (dict(N=2 ** 31), UNSUPPORTED), (dict(K=2 ** 24), UNSUPPORTED),
        (dict(M=2 ** 20, N=2 ** 14), UNSUPPORTED), (dict(M=2 ** 30, N=16), UNSUPPORTED), (dict(a=None), NULL),
        (dict(sa=None), NULL), (dict(b=None), NULL), (dict(sb=None), NULL), (dict(c=None), NULL), (dict(a=U), ALIGN),
        (dict(sa=U), ALIGN), (dict(b=U), ALIGN), (dict(sb=U), ALIGN), (dict(c=U), ALIGN), (dict(ws=U), ALIGN),
        (dict(ga=U2), ALIGN), (dict(gb=U2), ALIGN), (dict(ws=None), WORKSPACE), (dict(wb=need - 1), WORKSPACE),
    ]:
        assert call(fn, good, **change) == want, change


def test_every_launch_of_the_product_fits():
    """Sizes at the call's limits: fewer than 2^32 threads whatever tile is chosen, no more K slices than stages."""
    lib = _lib()
    plan, out = lib.mxf_fp4_pair_plan, (ctypes.c_int32 * 3)()
    plan.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int, ctypes.c_void_p]
    good = dict(a=None, sa=A, M=1, b=A, sb=A, N=16, K=128, fmt=1, ga=None, gb=None, c=A, cd=1, ws=A, wb=2 ** 62, stream=None)
    edge = 2 ** 21 * 128
    for M, N in [(1, edge), (edge, 16), (edge, 128), (2 ** 17, 2 ** 17 - 16), (128, edge), (4096 * 32, 32), (4096 * 32 + 1, 32),
                 (1, 2 ** 30), (2 ** 18, 2 ** 15)]:
        for K in (128, 256, 7168, 2 ** 24 - 128):
            for fmt in (0, 1):
                rc = call(lib.fp4_gemm, good, M=M, N=N, K=K, fmt=fmt)
                tiles = -(-M // 128) * -(-N // 128)
                assert rc == (UNSUPPORTED if tiles > 2 ** 21 or M * N >= 2 ** 34 else NULL)
                if rc == UNSUPPORTED:
                    continue
                plan(M, N, K, fmt, out)
                bm, bn, slices = out
                groups = -(-M // bm) * -(-N // bn)
                assert 8 * -(-groups // 8) * slices * (512 if bm in (32, 256) else 256) < 2 ** 32
                assert slices == 1 or (slices <= -(-K // 256) and M * N < 2 ** 30)


def test_binding_refuses_host_tensors():
    z = torch.zeros
    f, i = z(4, 64), z(4, 2, dtype=torch.int32)
    for fn, args in [(ops.moe_balance_loss, (f, i)), (ops.moe_route_backward, (f, i, z(4, 2), z(4, 2))),
                     (ops.moe_combine_backward, (f, z(8, 64), z(4, 2), i.view(-1))), (ops.nvfp4_tensor_scale, (f,)),
                     (ops.fp4_quantize, (f,)), (ops.fp4_dequantize, (z(4, 32, dtype=torch.uint8), z(4, 4, dtype=torch.uint8)))]:
        with pytest.raises(RuntimeError, match="GPU"):
            fn(*args)

"""Python binding of the C ABI in include/mxfp4_moe.h (argument marshalling only).

torch supplies device memory and the current HIP stream; every step of the
computation runs in the HIP kernels of libmxfp4moe.so. There is no fallback:
if the library is missing, or a call returns a non-zero status, a
RuntimeError is raised.
"""

import ctypes
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmxfp4moe.so")
_lib = None

MXF_E4M3, MXF_E2M1 = 0, 1
MXF_F32, MXF_BF16 = 0, 1
FMTS = {"e4m3": MXF_E4M3, "e2m1": MXF_E2M1}
WEIGHT_FMTS = {"mxfp4": 0, "nvfp4": 1}
DTYPES = {torch.float32: MXF_F32, torch.bfloat16: MXF_BF16}

_c_i64, _c_i32, _c_int, _p, _sz = ctypes.c_int64, ctypes.c_int32, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t

SIGNATURES = {
    "mxf_status_str": (ctypes.c_char_p, [_c_int]),
    "mxf_abi_version": (_c_int, []),
    "mxfp4_quantize_act": (_c_int, [_p, _c_int, _c_i64, _c_i64, _c_int, _p, _p, _p]),
    "mxfp4_gemm_workspace_bytes": (_sz, [_c_i64, _c_i64, _c_i64, _c_int]),
    "mxfp4_gemm": (_c_int, [_p, _c_i64, _c_i64, _c_i64, _c_int, _p, _p, _p, _p, _sz, _p]),
    "mxfp4_noalloc_scratch_bytes": (_sz, []),
    "mxfp4_gemm_noalloc": (_c_int, [_p, _c_i64, _c_i64, _c_i64, _c_int, _p, _p, _p, _p]),
    "fp4_w4a16_workspace_bytes": (_sz, [_c_i64, _c_i64, _c_i64]),
    "mxfp4_gemm_w4a16": (_c_int, [_p, _c_i64, _c_i64, _c_i64, _p, _p, _p, _p, _sz, _p]),
    "nvfp4_gemm_w4a16": (_c_int, [_p, _c_i64, _c_i64, _c_i64, _p, _p, _p, _p, _sz, _p]),
    "q8_quantize_act": (_c_int, [_p, _c_i64, _c_i64, _p, _p, _p]),
    "mxfp4_gemm_q8_workspace_bytes": (_sz, [_c_i64, _c_i64, _c_i64]),
    "mxfp4_gemm_q8": (_c_int, [_p, _p, _c_i64, _c_i64, _c_i64, _p, _p, _p, _p, _sz, _p]),
    "moe_route_permute": (_c_int, [_p, _c_i64, _c_i32, _c_i32, _p, _p, _p, _p, _p, _p]),
    "moe_grouped_mxfp4_gemm": (_c_int, [_p, _p, _c_int, _c_i64, _c_i32, _c_i64, _c_i64, _c_i32,
                                        _p, _p, _p, _p, _p, _p, _p, _p, _p, _c_int, _p]),
    "moe_unpermute_combine": (_c_int, [_p, _c_int, _p, _p, _c_i64, _c_i32, _c_i64, _p, _c_int, _p]),
    "moe_quantize_route": (_c_int, [_p, _c_int, _p, _c_i64, _c_i64, _c_i32, _c_i32, _c_int, _p, _p, _p, _p, _p, _p,
                                    _p, _p]),
    "moe_grouped_mxfp4_gemm_combine": (_c_int, [_p, _p, _c_int, _c_i64, _c_i32, _c_i64, _c_i64, _c_i32, _p, _p,
                                                _p, _p, _p, _p, _p, _p, _p, _p, _p, _p, _c_int, _p]),
    "moe_grouped_gemm_w4a16": (_c_int, [_p, _c_i64, _c_i64, _p, _c_i32, _p, _c_i32, _c_i64, _c_i64, _c_int, _p, _p,
                                        _c_int, _p, _c_int, _p]),
    "fp4_w4a16_lora_workspace_bytes": (_sz, [_c_i64, _c_i64, _c_i64, _c_i32]),
    "fp4_gemm_w4a16_lora": (_c_int, [_p, _c_i64, _c_i64, _c_i64, _c_int, _p, _p, _p, _p, _c_i32, _p, _p, _p, _c_i32,
                                     _c_i32, _p, _c_int, _p, _sz, _p]),
    "moe_block_norm": (_c_int, [_p, _c_int, _c_i64, _p, _p, _c_i32, _c_i64, _c_i64, _p, _c_int, ctypes.c_float, _p, _p,
                                _c_int, ctypes.c_float, _p, _c_int, _c_int, _p, _p, _c_int, _c_int, _p, _p, _p]),
    # include/mxf_ceilings.h: achievable-rate probes (measurement helpers)
    "mxf_ceiling_mfma_flops": (_c_i64, [_c_int]),
    "mxf_ceiling_mfma": (_c_int, [_c_int, _p, _c_i64, _c_int, _c_int, _p, _p]),
    "mxf_ceiling_read": (_c_int, [_p, _c_i64, _p, _p]),
    "mxf_ceiling_lds_copy_bytes": (_c_i64, [_c_int, _c_int]),
    "mxf_ceiling_lds_copy": (_c_int, [_p, _c_i64, _c_int, _c_int, _p, _p]),
    "moe_balance_loss_workspace_bytes": (_sz, [_c_i64, _c_i32, _c_i32]),
    "moe_balance_loss": (_c_int, [_p, _c_int, _p, _p, _p, _c_i32, _c_i64, _c_i32, _c_i32, _p, _p, _p, _p, _p, _p, _sz,
                                  _p]),
    "moe_route_backward": (_c_int, [_p, _c_int, _p, _p, _p, _p, _p, _p, _p, _p, _c_i32, _c_i64, _c_i32, _c_i32, _p, _p]),
    "moe_combine_backward": (_c_int, [_p, _c_int, _p, _c_int, _c_i64, _p, _p, _c_i64, _c_i32, _c_i64, _p, _p, _p]),
    "nvfp4_tensor_scale_workspace_bytes": (_sz, [_c_i64, _c_int]),
    "nvfp4_tensor_scale": (_c_int, [_p, _c_int, _c_i64, _p, _p, _sz, _p]),
    "fp4_quantize": (_c_int, [_p, _c_int, _c_i64, _c_i64, _c_int, _p, _p, _p, _p, _p, _p, _p]),
    "fp4_dequantize": (_c_int, [_p, _p, _c_i64, _c_i64, _c_int, _p, _p, _c_int, _p]),
    "fp4_gemm_workspace_bytes": (_sz, [_c_i64, _c_i64, _c_i64, _c_int]),
    "fp4_gemm": (_c_int, [_p, _p, _c_i64, _p, _p, _c_i64, _c_i64, _c_int, _p, _p, _p, _c_int, _p, _sz, _p]),
}

CEILING_MFMA_GROUPS = 512
CEILING_MFMA_WORDS = 64 * 6 * 64 * 8


def lib_path():
    return _LIB_PATH


def load():
    """Load libmxfp4moe.so (built in-tree by build.py); raise if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is not built: run mxfp4_block_scaled_amd/build.py "
                               "(or __graft_entry__.build()) first")
        lib = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _check(rc, what):
    if rc != 0:
        msg = load().mxf_status_str(rc).decode()
        raise RuntimeError(f"{what} failed with status {rc}: {msg}")


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _dev(t):
    if not t.is_cuda:
        raise RuntimeError("tensors must be on the GPU")
    if not t.is_contiguous():
        raise RuntimeError("tensors must be contiguous")
    return t.device


def _need(t, name, dtypes, shape):
    """Raise unless t has one of `dtypes` and the given shape; a shape entry given
    as (">=", n) only bounds that dimension from below."""
    if not isinstance(dtypes, tuple):
        dtypes = (dtypes,)
    if t.dtype not in dtypes:
        raise RuntimeError(f"{name}: dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if t.dim() != len(shape):
        raise RuntimeError(f"{name}: {t.dim()}-d, expected {len(shape)}-d {shape}")
    for i, (got, want) in enumerate(zip(t.shape, shape)):
        ok = got >= want[1] if isinstance(want, tuple) else got == want
        if not ok:
            raise RuntimeError(f"{name}: shape {tuple(t.shape)}, expected {shape} (dimension {i})")


# The current stream's handle without the Stream object around it (2 us of a 10 us call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)


def _is(t, name, dtype, shape, i):
    """_dev and _need in one: t is on GPU i, contiguous, of `dtype` (or one of a tuple) and `shape`."""
    if t.dtype != dtype or t.shape != shape or t.get_device() != i or not t.is_contiguous():
        _dev(t)
        _need(t, name, dtype, shape)
        if t.get_device() != i:
            raise RuntimeError(f"{name} is on {t.device}, expected GPU {i}")


def _gpu(t):
    """The index of contiguous t's GPU: _dev without the device object (0.5 us of a 9 us call)."""
    i = t.get_device()
    if i < 0 or not t.is_contiguous():
        _dev(t)
    return i


def _call(name, i, *args):
    """The C function `name` with the tensors' GPU i current and its current stream as the last argument."""
    fn = getattr(_lib or load(), name)
    if torch._C._cuda_getDevice() == i:
        rc = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(i):
            rc = fn(*args, _raw_stream(i))
    if rc:
        _check(rc, name)


def _new(like, dtype, shape):
    """An uninitialised tensor beside `like`; of its own dtype and shape the quicker way."""
    if like.dtype == dtype:
        return torch.empty_like(like) if like.shape == shape else like.new_empty(shape)
    return torch.empty(shape, dtype=dtype, device=like.device)


def _at(t):
    return t.data_ptr() if t is not None else None


def _one_of(value, table, name):
    if value not in table:
        raise RuntimeError(f"{name}: {value!r}, expected {' or '.join(str(k) for k in table)}")
    return table[value]


def mxfp4_quantize_act(x, fmt="e4m3"):
    """x [rows][K] bf16/fp32 -> (q [rows][K] or [rows][K/2] uint8, q_scale [rows][K/32] uint8)."""
    dev = _dev(x)
    if x.dim() != 2:
        raise RuntimeError("x must be 2-d [rows][K]")
    rows, K = x.shape
    _need(x, "x", (torch.bfloat16, torch.float32), (rows, K))
    f = FMTS[fmt]
    q = torch.empty((rows, K // 2 if f == MXF_E2M1 else K), dtype=torch.uint8, device=dev)
    qs = torch.empty((rows, K // 32), dtype=torch.uint8, device=dev)
    _check(load().mxfp4_quantize_act(_ptr(x), DTYPES[x.dtype], rows, K, f, _ptr(q), _ptr(qs), _stream(dev)),
           "mxfp4_quantize_act")
    return q, qs


def mxfp4_gemm(a, w, w_scale, act_fmt="e4m3", out=None, workspace=None):
    """a [M][K] bf16, w [N][K/2] uint8, w_scale [N][K/32] uint8 -> c [M][N] fp32."""
    dev = _dev(a)
    _dev(w), _dev(w_scale)
    if a.dim() != 2 or w.dim() != 2:
        raise RuntimeError("a must be [M][K] and w [N][K/2]")
    M, K = a.shape
    N = w.shape[0]
    _need(a, "a", torch.bfloat16, (M, K))
    _need(w, "w", torch.uint8, (N, K // 2))
    _need(w_scale, "w_scale", torch.uint8, (N, K // 32))
    f = FMTS[act_fmt]
    lib = load()
    need = lib.mxfp4_gemm_workspace_bytes(M, N, K, f)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _dev(workspace)
    _need(workspace, "workspace", torch.uint8, ((">=", need),))
    c = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=dev)
    _dev(c)
    _need(c, "out", torch.float32, (M, N))
    _check(lib.mxfp4_gemm(_ptr(a), M, N, K, f, _ptr(w), _ptr(w_scale), _ptr(c), _ptr(workspace),
                          workspace.numel(), _stream(dev)), "mxfp4_gemm")
    return c


def mxfp4_gemm_noalloc(a, w, w_scale, out, act_fmt="e4m3"):
    """mxfp4_gemm with the library's own fixed workspace (no allocation in the call):
    a [M][K] bf16, w [N][K/2] uint8, w_scale [N][K/32] uint8 -> out [M][N] fp32."""
    dev = _dev(a)
    _dev(w), _dev(w_scale), _dev(out)
    if a.dim() != 2 or w.dim() != 2:
        raise RuntimeError("a must be [M][K] and w [N][K/2]")
    M, K = a.shape
    N = w.shape[0]
    _need(a, "a", torch.bfloat16, (M, K))
    _need(w, "w", torch.uint8, (N, K // 2))
    _need(w_scale, "w_scale", torch.uint8, (N, K // 32))
    _need(out, "out", torch.float32, (M, N))
    _check(load().mxfp4_gemm_noalloc(_ptr(a), M, N, K, FMTS[act_fmt], _ptr(w), _ptr(w_scale), _ptr(out),
                                     _stream(dev)), "mxfp4_gemm_noalloc")
    return out


def fp4_gemm_w4a16(a, w, w_scale, fmt="mxfp4", out=None, workspace=None):
    """FP4 weights x bf16 activations: a [M][K] bf16, w [N][K/2] uint8, w_scale [N][K/32]
    (fmt "mxfp4", UE8M0) or [N][K/16] (fmt "nvfp4", UE4M3) uint8 -> c [M][N] fp32."""
    dev = _dev(a)
    _dev(w), _dev(w_scale)
    if a.dim() != 2 or w.dim() != 2:
        raise RuntimeError("a must be [M][K] and w [N][K/2]")
    M, K = a.shape
    N = w.shape[0]
    if fmt not in ("mxfp4", "nvfp4"):
        raise RuntimeError(f"unknown weight format {fmt!r}")
    _need(a, "a", torch.bfloat16, (M, K))
    _need(w, "w", torch.uint8, (N, K // 2))
    _need(w_scale, "w_scale", torch.uint8, (N, K // (16 if fmt == "nvfp4" else 32)))
    lib = load()
    need = lib.fp4_w4a16_workspace_bytes(M, N, K)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _dev(workspace)
    _need(workspace, "workspace", torch.uint8, ((">=", need),))
    c = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=dev)
    _dev(c)
    _need(c, "out", torch.float32, (M, N))
    fn = lib.nvfp4_gemm_w4a16 if fmt == "nvfp4" else lib.mxfp4_gemm_w4a16
    _check(fn(_ptr(a), M, N, K, _ptr(w), _ptr(w_scale), _ptr(c), _ptr(workspace), workspace.numel(), _stream(dev)),
           f"{fmt}_gemm_w4a16")
    return c


def q8_quantize_act(x):
    """x [rows][K] bf16 -> (q [rows][K] int8, d [rows][K/32] fp16): Q8 blocks of 32."""
    dev = _dev(x)
    if x.dim() != 2:
        raise RuntimeError("x must be [rows][K]")
    rows, K = x.shape
    _need(x, "x", torch.bfloat16, (rows, K))
    q = torch.empty((rows, K), dtype=torch.int8, device=dev)
    d = torch.empty((rows, K // 32), dtype=torch.float16, device=dev)
    _check(load().q8_quantize_act(_ptr(x), rows, K, _ptr(q), _ptr(d), _stream(dev)), "q8_quantize_act")
    return q, d


def mxfp4_gemm_q8(q, d, w, w_scale, out=None, workspace=None):
    """The lookup-table route: q [M][K] int8, d [M][K/32] fp16 (from q8_quantize_act),
    w [N][K/2] uint8, w_scale [N][K/32] uint8 -> c [M][N] fp32."""
    dev = _dev(q)
    for t in (d, w, w_scale):
        _dev(t)
    if q.dim() != 2 or w.dim() != 2:
        raise RuntimeError("q must be [M][K] and w [N][K/2]")
    M, K = q.shape
    N = w.shape[0]
    _need(q, "q", torch.int8, (M, K))
    _need(d, "d", torch.float16, (M, K // 32))
    _need(w, "w", torch.uint8, (N, K // 2))
    _need(w_scale, "w_scale", torch.uint8, (N, K // 32))
    lib = load()
    need = lib.mxfp4_gemm_q8_workspace_bytes(M, N, K)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _dev(workspace)
    _need(workspace, "workspace", torch.uint8, ((">=", need),))
    c = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=dev)
    _dev(c)
    _need(c, "out", torch.float32, (M, N))
    _check(lib.mxfp4_gemm_q8(_ptr(q), _ptr(d), M, N, K, _ptr(w), _ptr(w_scale), _ptr(c), _ptr(workspace),
                             workspace.numel(), _stream(dev)), "mxfp4_gemm_q8")
    return c


def moe_route_permute(logits, topk):
    """logits [T][E] fp32 -> (topk_ids, gates, expert_offsets, sorted_pair, pair_row)."""
    dev = _dev(logits)
    if logits.dim() != 2:
        raise RuntimeError("logits must be [T][E]")
    T, E = logits.shape
    _need(logits, "logits", torch.float32, (T, E))
    ids = torch.empty((T, topk), dtype=torch.int32, device=dev)
    gates = torch.empty((T, topk), dtype=torch.float32, device=dev)
    offs = torch.empty((E + 1,), dtype=torch.int32, device=dev)
    sp = torch.empty((max(T * topk, 1),), dtype=torch.int32, device=dev)
    pr = torch.empty((max(T * topk, 1),), dtype=torch.int32, device=dev)
    _check(load().moe_route_permute(_ptr(logits), T, E, topk, _ptr(ids), _ptr(gates), _ptr(offs), _ptr(sp),
                                    _ptr(pr), _stream(dev)), "moe_route_permute")
    return ids, gates, offs, sp[:T * topk], pr[:T * topk]


def moe_grouped_mxfp4_gemm(q, q_scale, act_fmt, T, topk, expert_offsets, sorted_pair, w1, w1_scale, w2,
                           w2_scale, y_dtype=torch.bfloat16, h=None, h_scale=None, y=None):
    """Both expert FCs. Returns (h, h_scale, y) with y [T*topk][H] in permuted row order."""
    dev = _dev(q)
    for t in (q_scale, expert_offsets, sorted_pair, w1, w1_scale, w2, w2_scale):
        _dev(t)
    if w1.dim() != 3:
        raise RuntimeError("w1 must be [E][2I][H/2]")
    E, twoI, Hh = w1.shape
    I = twoI // 2
    H = Hh * 2
    f = FMTS[act_fmt]
    R = T * topk
    fp4 = f == MXF_E2M1
    _need(q, "q", torch.uint8, (T, H // 2 if fp4 else H))
    _need(q_scale, "q_scale", torch.uint8, (T, H // 32))
    _need(expert_offsets, "expert_offsets", torch.int32, (E + 1,))
    _need(sorted_pair, "sorted_pair", torch.int32, ((">=", R),))
    _need(w1, "w1", torch.uint8, (E, 2 * I, H // 2))
    _need(w1_scale, "w1_scale", torch.uint8, (E, 2 * I, H // 32))
    _need(w2, "w2", torch.uint8, (E, H, I // 2))
    _need(w2_scale, "w2_scale", torch.uint8, (E, H, I // 32))
    if h is None:
        h = torch.empty((max(R, 1), I // 2 if fp4 else I), dtype=torch.uint8, device=dev)
    if h_scale is None:
        h_scale = torch.empty((max(R, 1), I // 32), dtype=torch.uint8, device=dev)
    if y is None:
        y = torch.empty((max(R, 1), H), dtype=y_dtype, device=dev)
    for t in (h, h_scale, y):
        _dev(t)
    _need(h, "h", torch.uint8, ((">=", R), I // 2 if fp4 else I))
    _need(h_scale, "h_scale", torch.uint8, ((">=", R), I // 32))
    _need(y, "y", (torch.float32, torch.bfloat16), ((">=", R), H))
    _check(load().moe_grouped_mxfp4_gemm(
        _ptr(q), _ptr(q_scale), f, T, topk, H, I, E, _ptr(expert_offsets), _ptr(sorted_pair), _ptr(w1),
        _ptr(w1_scale), _ptr(w2), _ptr(w2_scale), _ptr(h), _ptr(h_scale), _ptr(y), DTYPES[y.dtype],
        _stream(dev)), "moe_grouped_mxfp4_gemm")
    return h[:R], h_scale[:R], y[:R]


def moe_unpermute_combine(y, gates, pair_row, T, topk, out_dtype=torch.bfloat16, out=None):
    """out [T][H] = sum_j gates[t, j] * y[pair_row[t*topk + j]]."""
    dev = _dev(y)
    _dev(gates), _dev(pair_row)
    if y.dim() != 2:
        raise RuntimeError("y must be [T*topk][H]")
    H = y.shape[1]
    _need(y, "y", (torch.float32, torch.bfloat16), ((">=", T * topk), H))
    _need(gates, "gates", torch.float32, (T, topk))
    _need(pair_row, "pair_row", torch.int32, ((">=", T * topk),))
    if out is None:
        out = torch.empty((T, H), dtype=out_dtype, device=dev)
    _dev(out)
    _need(out, "out", (torch.float32, torch.bfloat16), (T, H))
    _check(load().moe_unpermute_combine(_ptr(y), DTYPES[y.dtype], _ptr(gates), _ptr(pair_row), T, topk, H,
                                        _ptr(out), DTYPES[out.dtype], _stream(dev)), "moe_unpermute_combine")
    return out


def moe_quantize_route(x, logits, topk, act_fmt="e4m3"):
    """mxfp4_quantize_act(x) and moe_route_permute(logits) in one launch (T <= 64,
    E <= 256). Returns (q, q_scale, topk_ids, gates, expert_offsets, sorted_pair, pair_row)."""
    dev = _dev(x)
    _dev(logits)
    if x.dim() != 2 or logits.dim() != 2:
        raise RuntimeError("x must be [T][H] and logits [T][E]")
    T, H = x.shape
    E = logits.shape[1]
    _need(x, "x", (torch.bfloat16, torch.float32), (T, H))
    _need(logits, "logits", torch.float32, (T, E))
    f = FMTS[act_fmt]
    fp4 = f == MXF_E2M1
    R = T * topk
    q = torch.empty((T, H // 2 if fp4 else H), dtype=torch.uint8, device=dev)
    qs = torch.empty((T, H // 32), dtype=torch.uint8, device=dev)
    ids = torch.empty((T, topk), dtype=torch.int32, device=dev)
    gates = torch.empty((T, topk), dtype=torch.float32, device=dev)
    offs = torch.empty((E + 1,), dtype=torch.int32, device=dev)
    sp = torch.empty((max(R, 1),), dtype=torch.int32, device=dev)
    pr = torch.empty((max(R, 1),), dtype=torch.int32, device=dev)
    _check(load().moe_quantize_route(_ptr(x), DTYPES[x.dtype], _ptr(logits), T, H, E, topk, f, _ptr(q), _ptr(qs),
                                     _ptr(ids), _ptr(gates), _ptr(offs), _ptr(sp), _ptr(pr), _stream(dev)),
           "moe_quantize_route")
    return q, qs, ids, gates, offs, sp[:R], pr[:R]


def moe_grouped_mxfp4_gemm_combine(q, q_scale, act_fmt, T, topk, expert_offsets, sorted_pair, topk_ids, pair_row,
                                   gates, w1, w1_scale, w2, w2_scale, out_dtype=torch.bfloat16, h=None,
                                   h_scale=None, out=None):
    """Both expert FCs with FC2 fused into the gate-weighted combine (T <= 64).
    Returns (h, h_scale, out) with out [T][H]."""
    dev = _dev(q)
    for t in (q_scale, expert_offsets, sorted_pair, topk_ids, pair_row, gates, w1, w1_scale, w2, w2_scale):
        _dev(t)
    if w1.dim() != 3:
        raise RuntimeError("w1 must be [E][2I][H/2]")
    E, twoI, Hh = w1.shape
    I = twoI // 2
    H = Hh * 2
    f = FMTS[act_fmt]
    R = T * topk
    fp4 = f == MXF_E2M1
    _need(q, "q", torch.uint8, (T, H // 2 if fp4 else H))
    _need(q_scale, "q_scale", torch.uint8, (T, H // 32))
    _need(expert_offsets, "expert_offsets", torch.int32, (E + 1,))
    _need(sorted_pair, "sorted_pair", torch.int32, ((">=", R),))
    _need(topk_ids, "topk_ids", torch.int32, (T, topk))
    _need(pair_row, "pair_row", torch.int32, ((">=", R),))
    _need(gates, "gates", torch.float32, (T, topk))
    _need(w1, "w1", torch.uint8, (E, 2 * I, H // 2))
    _need(w1_scale, "w1_scale", torch.uint8, (E, 2 * I, H // 32))
    _need(w2, "w2", torch.uint8, (E, H, I // 2))
    _need(w2_scale, "w2_scale", torch.uint8, (E, H, I // 32))
    if h is None:
        h = torch.empty((max(R, 1), I // 2 if fp4 else I), dtype=torch.uint8, device=dev)
    if h_scale is None:
        h_scale = torch.empty((max(R, 1), I // 32), dtype=torch.uint8, device=dev)
    if out is None:
        out = torch.empty((max(T, 1), H), dtype=out_dtype, device=dev)
    for t in (h, h_scale, out):
        _dev(t)
    _need(h, "h", torch.uint8, ((">=", R), I // 2 if fp4 else I))
    _need(h_scale, "h_scale", torch.uint8, ((">=", R), I // 32))
    _need(out, "out", (torch.float32, torch.bfloat16), ((">=", T), H))
    _check(load().moe_grouped_mxfp4_gemm_combine(
        _ptr(q), _ptr(q_scale), f, T, topk, H, I, E, _ptr(expert_offsets), _ptr(sorted_pair), _ptr(topk_ids),
        _ptr(pair_row), _ptr(gates), _ptr(w1), _ptr(w1_scale), _ptr(w2), _ptr(w2_scale), _ptr(h), _ptr(h_scale), _ptr(out),
        DTYPES[out.dtype], _stream(dev)), "moe_grouped_mxfp4_gemm_combine")
    return h[:R], h_scale[:R], out[:T]


def moe_grouped_gemm_w4a16(a, expert_offsets, w, w_scale, fmt="mxfp4", sorted_pair=None, topk=1, swiglu=False,
                           out_dtype=torch.bfloat16, out=None):
    """Ragged grouped GEMM of bf16 activations with FP4 expert weights: rows expert_offsets[e] ..
    expert_offsets[e + 1] of the result are a's rows times expert e's weights. w [E][N][K/2] uint8, w_scale
    [E][N][K/32] (fmt "mxfp4") or [E][N][K/16] (fmt "nvfp4") uint8. a [R][K], or with sorted_pair [R] (from
    moe_route_permute: all pairs, or those of the experts at hand) a [rows][K] and row r reads
    a[sorted_pair[r] // topk]. swiglu: the first N/2 weight rows are gate rows and the result is silu(gate) * up.
    Returns y [R][N] or [R][N/2]; with `out` given, rows outside every expert keep what it holds (in a new tensor
    they are uninitialised)."""
    _dev(a)
    i = a.get_device()
    if a.dim() != 2 or w.dim() != 3:
        raise RuntimeError("a must be [rows][K] and w [E][N][K/2]")
    rows, K = a.shape
    E, N, _ = w.shape
    f = _one_of(fmt, WEIGHT_FMTS, "fmt")
    R = rows if sorted_pair is None else sorted_pair.numel()
    _is(a, "a", torch.bfloat16, (rows, K), i)
    _is(expert_offsets, "expert_offsets", torch.int32, (E + 1,), i)
    _is(w, "w", torch.uint8, (E, N, K // 2), i)
    _is(w_scale, "w_scale", torch.uint8, (E, N, K // (16 if f else 32)), i)
    pairs = None
    if sorted_pair is not None:
        _is(sorted_pair, "sorted_pair", torch.int32, (R,), i)
        pairs = sorted_pair.data_ptr() or expert_offsets.data_ptr()  # no pairs: a tensor without an address
        if R > rows * topk:
            raise RuntimeError(f"sorted_pair: {R} pairs, expected at most a's {rows} rows x topk {topk}")
    shape = (R, N // 2 if swiglu else N)
    if out is None:
        _one_of(out_dtype, DTYPES, "out_dtype")
        out = _new(a, out_dtype, shape)
    else:
        _is(out, "out", (torch.float32, torch.bfloat16), shape, i)
    _call("moe_grouped_gemm_w4a16", i, a.data_ptr(), rows, R, pairs, topk, expert_offsets.data_ptr(), E, N, K, f,
          w.data_ptr(), w_scale.data_ptr(), int(swiglu), out.data_ptr(), DTYPES[out.dtype])
    return out


def fp4_gemm_w4a16_lora(a, w, w_scale, seg_offsets, seg_adapter, lora_a, lora_b, scaling, fmt="mxfp4",
                        out_dtype=torch.float32, out=None, workspace=None):
    """A shared FP4 projection with low-rank adapters of many requests: a [M][K] bf16, w and w_scale as for
    fp4_gemm_w4a16, segment s (rows seg_offsets[s] .. seg_offsets[s + 1]) adds
    scaling[l] * (a lora_a[l]^T) lora_b[l]^T of its adapter l = seg_adapter[s]; a negative l, and rows in no
    segment, get the projection alone. seg_offsets [S+1], seg_adapter [S] int32; lora_a [L][rank][K], lora_b
    [L][N][rank] bf16; scaling [L] fp32. Returns c [M][N] in out_dtype (fp32 or bf16)."""
    _dev(a)
    i = a.get_device()
    if a.dim() != 2 or w.dim() != 2 or lora_a.dim() != 3 or seg_adapter.dim() != 1:
        raise RuntimeError("a must be [M][K], w [N][K/2], lora_a [L][rank][K] and seg_adapter [S]")
    M, K = a.shape
    N = w.shape[0]
    L, rank, _ = lora_a.shape
    S = seg_adapter.shape[0]
    f = _one_of(fmt, WEIGHT_FMTS, "fmt")
    _is(a, "a", torch.bfloat16, (M, K), i)
    _is(w, "w", torch.uint8, (N, K // 2), i)
    _is(w_scale, "w_scale", torch.uint8, (N, K // (16 if f else 32)), i)
    _is(seg_offsets, "seg_offsets", torch.int32, (S + 1,), i)
    _is(seg_adapter, "seg_adapter", torch.int32, (S,), i)
    _is(lora_a, "lora_a", torch.bfloat16, (L, rank, K), i)
    _is(lora_b, "lora_b", torch.bfloat16, (L, N, rank), i)
    _is(scaling, "scaling", torch.float32, (L,), i)
    if out is None:
        _one_of(out_dtype, DTYPES, "out_dtype")
        out = _new(a, out_dtype, (M, N))
    else:
        _is(out, "out", (torch.float32, torch.bfloat16), (M, N), i)
    need = load().fp4_w4a16_lora_workspace_bytes(M, N, K, rank)
    if workspace is None:
        workspace = w.new_empty(max(need, 1))
    elif _dev(workspace) != a.device:
        raise RuntimeError(f"workspace is on {workspace.device}, expected {a.device}")
    else:
        _need(workspace, "workspace", torch.uint8, ((">=", need),))
    _call("fp4_gemm_w4a16_lora", i, a.data_ptr(), M, N, K, f, w.data_ptr(), w_scale.data_ptr(), _at(seg_offsets),
          _at(seg_adapter), S, _at(lora_a), _at(lora_b), _at(scaling), L, rank, out.data_ptr(), DTYPES[out.dtype],
          workspace.data_ptr(), workspace.numel())
    return out


def moe_block_norm(y, x=None, post_weight=None, gate=None, residual_scale=1.0, pre_weight=None, eps=1e-6, act_fmt=None,
                   want_r=True, want_n=True, n_dtype=torch.bfloat16, expert_gates=None, pair_row=None, r_dtype=None,
                   r=None):
    """The step between two blocks: r = residual_scale * x + gate * postnorm(y), n = prenorm(r), optionally its MX
    quantisation. y [T][H] bf16/fp32, or with expert_gates [T][topk] fp32 and pair_row [T*topk] int32 the expert
    rows [rows][H] that moe_unpermute_combine would sum (entries of pair_row outside them add nothing). x [T][H]
    bf16/fp32 (None: no residual); post_weight [H] (None: no post-norm), pre_weight [H] (None: ones), fp32 or
    bf16, both alike; gate [H], [T][1] or [T][H] bf16/fp32. RMS norms: v / sqrt(mean(v^2) + eps) * weight.
    act_fmt "e4m3" / "e2m1" also quantises n (from fp32) as mxfp4_quantize_act. `r` may be given as the output
    (x itself: updated in place). Returns a dict of r (x's dtype, without x r_dtype or y's), n (n_dtype), q and
    q_scale; what is not wanted is None."""
    _dev(y)
    i = y.get_device()
    if y.dim() != 2:
        raise RuntimeError("y must be 2-d [rows][H]")
    y_rows, H = y.shape
    _one_of(y.dtype, DTYPES, "y")
    topk = 0
    T = y_rows
    if (expert_gates is None) != (pair_row is None):
        raise RuntimeError("expert_gates and pair_row go together")
    if expert_gates is not None:
        if expert_gates.dim() != 2 or expert_gates.shape[1] < 1:
            raise RuntimeError("expert_gates must be [T][topk]")
        T, topk = expert_gates.shape
        _is(expert_gates, "expert_gates", torch.float32, (T, topk), i)
        _is(pair_row, "pair_row", torch.int32, (T * topk,), i)
    if x is not None:
        r_dtype = x.dtype
        _is(x, "x", r_dtype, (T, H), i)
    elif r_dtype is None:
        r_dtype = y.dtype if r is None else r.dtype
    x_dtype = _one_of(r_dtype, DTYPES, "the residual's dtype")
    w_dtype = torch.float32
    for name, t in (("post_weight", post_weight), ("pre_weight", pre_weight)):
        if t is not None:
            w_dtype = t.dtype
            _one_of(w_dtype, DTYPES, name)
            _is(t, name, w_dtype, (H,), i)
    if post_weight is not None and post_weight.dtype != w_dtype:
        raise RuntimeError(f"post_weight is {post_weight.dtype} and pre_weight {w_dtype}, expected one dtype")
    mode, g_dtype = 0, torch.float32
    if gate is not None:
        g_dtype = gate.dtype
        mode = 1 if gate.dim() == 1 else 2 if gate.dim() == 2 and gate.shape[1] == 1 else 3
        _one_of(g_dtype, DTYPES, "gate")
        _is(gate, "gate", g_dtype, {1: (H,), 2: (T, 1), 3: (T, H)}[mode], i)
    fmt = None if act_fmt is None else _one_of(act_fmt, FMTS, "act_fmt")
    if r is not None:
        _is(r, "r", r_dtype, (T, H), i)
    elif want_r:
        r = _new(y if x is None else x, r_dtype, (T, H))
    n_code = _one_of(n_dtype, DTYPES, "n_dtype")
    n = _new(y if x is None else x, n_dtype, (T, H)) if want_n else None
    q = qs = None
    if fmt is not None:
        q = torch.empty((T, H // 2 if fmt == MXF_E2M1 else H), dtype=torch.uint8, device=y.device)
        qs = q.new_empty((T, H // 32))
    _call("moe_block_norm", i, y.data_ptr(), DTYPES[y.dtype], y_rows, _at(expert_gates), _at(pair_row), topk, T, H,
          _at(x), x_dtype, residual_scale, _at(post_weight), _at(pre_weight), DTYPES[w_dtype], eps, _at(gate),
          DTYPES[g_dtype], mode, _at(r), _at(n), n_code, fmt or 0, _at(q), _at(qs))
    return dict(r=r, n=n, q=q, q_scale=qs)


def moe_balance_loss(logits, topk_ids, token_mask=None, seg_offsets=None, workspace=None):
    """Load-balance and z losses of a router, with per-expert counts. logits [T][E] fp32 or bf16, topk_ids [T][topk]
    int32 (moe_route_permute's; an id outside the experts is a dropped pair), token_mask [T] uint8 or bool (0: the
    token does not count), seg_offsets [S+1] int32 (sequences; None: one of all tokens). Returns a dict of losses [2]
    fp32 (balance, averaged over the sequences that hold a token; z), counts [S][E] int32, prob_mean [S][E] fp32,
    tokens [S+2] int32 (by sequence, in all, sequences that hold any) and lse [T] fp32: what moe_route_backward takes."""
    i = _gpu(logits)
    if logits.dim() != 2 or topk_ids.dim() != 2:
        raise RuntimeError("logits must be [T][E] and topk_ids [T][topk]")
    T, E = logits.shape
    topk = topk_ids.shape[1]
    dt = _one_of(logits.dtype, DTYPES, "logits")
    _is(topk_ids, "topk_ids", torch.int32, (T, topk), i)
    if token_mask is not None:
        _is(token_mask, "token_mask", (torch.uint8, torch.bool), (T,), i)
    S = _segments(seg_offsets, i) if seg_offsets is not None else 1
    need = (_lib or load()).moe_balance_loss_workspace_bytes(T, E, S)
    if need or workspace is not None:
        workspace = _workspace(workspace, need, topk_ids)
    counts = topk_ids.new_empty((S, E))
    tokens = topk_ids.new_empty((S + 2,))
    mean = topk_ids.new_empty((S, E), dtype=torch.float32)
    lse = mean.new_empty((T,))
    losses = mean.new_empty((2,))
    _call("moe_balance_loss", i, logits.data_ptr(), dt, topk_ids.data_ptr(), _at(token_mask), _at(seg_offsets), S, T, E,
          topk, counts.data_ptr(), tokens.data_ptr(), mean.data_ptr(), lse.data_ptr(), losses.data_ptr(),
          _at(workspace), need)
    return dict(losses=losses, counts=counts, prob_mean=mean, tokens=tokens, lse=lse)


def _segments(seg_offsets, i):
    """The number of sequences of seg_offsets [S+1] int32 on GPU i."""
    if seg_offsets.dim() != 1 or seg_offsets.shape[0] < 2:
        raise RuntimeError("seg_offsets must be [S+1] of one sequence at least")
    n = seg_offsets.shape[0]
    _is(seg_offsets, "seg_offsets", torch.int32, (n,), i)
    return n - 1


def _workspace(workspace, need, like):
    """A byte workspace of at least `need` bytes beside `like`: the given one, checked, or a new one."""
    if workspace is None:
        return like.new_empty((max(need, 1),), dtype=torch.uint8)
    if _dev(workspace) != like.device:
        raise RuntimeError(f"workspace is on {workspace.device}, expected {like.device}")
    _need(workspace, "workspace", torch.uint8, ((">=", need),))
    return workspace


def moe_route_backward(logits, topk_ids, gates=None, dgates=None, balance=None, dlosses=None, seg_offsets=None):
    """The gradient of the router's logits [T][E]: of the gates (the softmax over the selected logits) with gates and
    dgates [T][topk] fp32, and of the losses with `balance`, moe_balance_loss's dict for these seg_offsets, and dlosses
    [2] fp32 (the losses' own gradients, on the GPU). Either part may be left out. Returns dlogits, of logits' dtype.
    Where each sequence's tokens lie on several GPUs, `balance` holds counts and tokens added up over them, except its
    last, the number of sequences that then hold a token."""
    i = _gpu(logits)
    if logits.dim() != 2 or topk_ids.dim() != 2:
        raise RuntimeError("logits must be [T][E] and topk_ids [T][topk]")
    T, E = logits.shape
    topk = topk_ids.shape[1]
    dt = _one_of(logits.dtype, DTYPES, "logits")
    _is(topk_ids, "topk_ids", torch.int32, (T, topk), i)
    if (gates is None) != (dgates is None):
        raise RuntimeError("gates and dgates go together")
    if (balance is None) != (dlosses is None):
        raise RuntimeError("balance and dlosses go together")
    if gates is None and balance is None:
        raise RuntimeError("neither dgates nor dlosses: nothing to compute")
    S = _segments(seg_offsets, i) if seg_offsets is not None else 1
    lse = counts = tokens = None
    if gates is not None:
        _is(gates, "gates", torch.float32, (T, topk), i)
        _is(dgates, "dgates", torch.float32, (T, topk), i)
    if balance is not None:
        lse, counts, tokens = balance["lse"], balance["counts"], balance["tokens"]
        _is(dlosses, "dlosses", torch.float32, (2,), i)
        _is(lse, "lse", torch.float32, (T,), i)
        _is(counts, "counts", torch.int32, (S, E), i)
        _is(tokens, "tokens", torch.int32, (S + 2,), i)
    dlogits = torch.empty_like(logits)
    _call("moe_route_backward", i, logits.data_ptr(), dt, topk_ids.data_ptr(), _at(gates), _at(dgates), _at(dlosses),
          _at(lse), _at(counts), _at(tokens), _at(seg_offsets), S, T, E, topk, dlogits.data_ptr())
    return dlogits


def moe_combine_backward(dout, y, gates, pair_row, want_dy=True, want_dgates=True, dy=None):
    """The gradient of moe_unpermute_combine: dout [T][H] bf16/fp32, y [rows][H] bf16/fp32, gates [T][topk] fp32,
    pair_row [T*topk] int32 (an entry outside y's rows is a dropped pair; no row twice). Returns (dy [rows][H] of y's
    dtype, dgates [T][topk] fp32); what is not wanted is None. Rows of dy that no pair names keep what a given `dy`
    holds (in a new tensor they are uninitialised)."""
    i = _gpu(dout)
    if dout.dim() != 2 or y.dim() != 2 or gates.dim() != 2:
        raise RuntimeError("dout must be [T][H], y [rows][H] and gates [T][topk]")
    T, H = dout.shape
    rows = y.shape[0]
    topk = gates.shape[1]
    d_code, y_code = _one_of(dout.dtype, DTYPES, "dout"), _one_of(y.dtype, DTYPES, "y")
    _is(y, "y", y.dtype, (rows, H), i)
    _is(gates, "gates", torch.float32, (T, topk), i)
    _is(pair_row, "pair_row", torch.int32, (T * topk,), i)
    if dy is not None:
        _is(dy, "dy", y.dtype, (rows, H), i)
    elif want_dy:
        dy = torch.empty_like(y)
    dgates = torch.empty_like(gates) if want_dgates else None
    _call("moe_combine_backward", i, dout.data_ptr(), d_code, _at(y), y_code, rows, gates.data_ptr(), pair_row.data_ptr(),
          T, topk, H, _at(dy), _at(dgates))
    return dy, dgates


def nvfp4_tensor_scale(x, workspace=None):
    """x [rows][cols] bf16/fp32 -> [1] fp32: the smallest power of two that takes max |x| to at most 6 * 448, for
    fp4_quantize (1 for zeros and for no rows)."""
    i = _gpu(x)
    dt = _one_of(x.dtype, DTYPES, "x")
    n = x.numel()
    if n == 0:
        return x.new_ones((1,), dtype=torch.float32)
    out = x.new_empty((1,), dtype=torch.float32)
    need = (_lib or load()).nvfp4_tensor_scale_workspace_bytes(n, dt)
    if need or workspace is not None:
        workspace = _workspace(workspace, need, x)
    _call("nvfp4_tensor_scale", i, x.data_ptr(), dt, n, out.data_ptr(), _at(workspace), need)
    return out


def _tensor_scale(t, fmt, i, name="tensor_scale"):
    if t is not None:
        if not fmt:
            raise RuntimeError(f"{name}: MXFP4 has none")
        _is(t, name, torch.float32, (1,), i)


def fp4_quantize(x, fmt="nvfp4", tensor_scale=None, rnd=None, rows=True, transposed=False):
    """x [rows][cols] bf16/fp32 to 4-bit blocks: fmt "nvfp4" (16 elements, UE4M3 scales, times tensor_scale [1] fp32 if
    given) or "mxfp4" (32 elements, UE8M0). To nearest, or stochastically with rnd [rows][cols] uint8 random bytes.
    Returns a dict of q [rows][cols/2] and q_scale [rows][cols/B] (rows=True), and of qt [cols][R/2] and qt_scale
    [cols][R/B] (transposed=True): the codes of x^T, R = rows rounded up to 128 with zeros; else None. uint8, as fp4_gemm
    takes them, q where cols % 128 == 0: fill x up with columns of zeros first where it is not."""
    i = _gpu(x)
    if x.dim() != 2:
        raise RuntimeError("x must be 2-d [rows][cols]")
    n, cols = x.shape
    dt = _one_of(x.dtype, DTYPES, "x")
    f = _one_of(fmt, WEIGHT_FMTS, "fmt")
    B = 16 if f else 32
    _tensor_scale(tensor_scale, f, i)
    if rnd is not None:
        _is(rnd, "rnd", torch.uint8, (n, cols), i)
    if not rows and not transposed:
        raise RuntimeError("neither rows nor transposed: nothing to compute")
    q = qs = qt = qts = None
    if rows:
        q = x.new_empty((n, cols // 2), dtype=torch.uint8)
        qs = q.new_empty((n, cols // B))
    if transposed:
        padded = (n + 127) // 128 * 128
        qt = x.new_empty((cols, padded // 2), dtype=torch.uint8)
        qts = qt.new_empty((cols, padded // B))
    _call("fp4_quantize", i, x.data_ptr(), dt, n, cols, f, _at(tensor_scale), _at(rnd), _at(q), _at(qs), _at(qt), _at(qts))
    return dict(q=q, q_scale=qs, qt=qt, qt_scale=qts)


def fp4_dequantize(q, q_scale, fmt="nvfp4", tensor_scale=None, out_dtype=torch.bfloat16):
    """q [rows][cols/2], q_scale [rows][cols/B] uint8 (as fp4_quantize writes them) -> [rows][cols] bf16 or fp32."""
    i = _gpu(q)
    if q.dim() != 2:
        raise RuntimeError("q must be [rows][cols/2]")
    n, half = q.shape
    f = _one_of(fmt, WEIGHT_FMTS, "fmt")
    _is(q, "q", torch.uint8, (n, half), i)
    _is(q_scale, "q_scale", torch.uint8, (n, half * 2 // (16 if f else 32)), i)
    _tensor_scale(tensor_scale, f, i)
    dt = _one_of(out_dtype, DTYPES, "out_dtype")
    out = q.new_empty((n, 2 * half), dtype=out_dtype)
    if half:
        _call("fp4_dequantize", i, q.data_ptr(), q_scale.data_ptr(), n, 2 * half, f, _at(tensor_scale), out.data_ptr(), dt)
    return out


def fp4_gemm(a, a_scale, b, b_scale, fmt="nvfp4", a_tensor_scale=None, b_tensor_scale=None, out_dtype=torch.bfloat16,
             out=None, workspace=None):
    """The product of two quantised matrices (as fp4_quantize writes them): a [M][K/2], b [N][K/2] uint8 codes with
    their scales [.][K/16] (fmt "nvfp4") or [.][K/32] ("mxfp4"), tensor scales [1] fp32 of NVFP4 (None: 1) ->
    c [M][N] bf16 or fp32. K % 128 == 0 and N % 16 == 0; K = 0 (the weight gradient of no tokens) gives zeros."""
    i = _gpu(a)
    if a.dim() != 2 or b.dim() != 2:
        raise RuntimeError("a must be [M][K/2] and b [N][K/2]")
    M, half = a.shape
    N = b.shape[0]
    f = _one_of(fmt, WEIGHT_FMTS, "fmt")
    blocks = half * 2 // (16 if f else 32)
    _is(a, "a", torch.uint8, (M, half), i)
    _is(a_scale, "a_scale", torch.uint8, (M, blocks), i)
    _is(b, "b", torch.uint8, (N, half), i)
    _is(b_scale, "b_scale", torch.uint8, (N, blocks), i)
    _tensor_scale(a_tensor_scale, f, i, "a_tensor_scale")
    _tensor_scale(b_tensor_scale, f, i, "b_tensor_scale")
    if out is None:
        _one_of(out_dtype, DTYPES, "out_dtype")
        out = a.new_empty((M, N), dtype=out_dtype)
    else:
        _is(out, "out", (torch.float32, torch.bfloat16), (M, N), i)
    if half == 0 and N > 0 and N % 16 == 0:
        return out.zero_()
    need = (_lib or load()).fp4_gemm_workspace_bytes(M, N, 2 * half, f)
    if need or workspace is not None:
        workspace = _workspace(workspace, need, a)
    _call("fp4_gemm", i, a.data_ptr(), a_scale.data_ptr(), M, b.data_ptr(), b_scale.data_ptr(), N, 2 * half, f,
          _at(a_tensor_scale), _at(b_tensor_scale), out.data_ptr(), DTYPES[out.dtype], _at(workspace), need)
    return out


def moe_layer(x, logits, w1, w1_scale, w2, w2_scale, topk, act_fmt="e4m3", y_dtype=torch.bfloat16,
              out_dtype=torch.bfloat16, fused=False, w_fmt="mxfp4"):
    """The whole expert layer through the C-ABI calls (one stream, no host sync).
    fused=True (T <= 64): quantisation and routing in one launch (E <= 256), FC2 and
    the combine in one kernel; y is not formed (None).
    act_fmt="bf16": the activations enter the expert products as they are (no
    quantisation: q, q_scale and h_scale are None, h is bf16); then the weights may be
    NVFP4 (w_fmt="nvfp4") too."""
    T = x.shape[0]
    if act_fmt != "bf16" and w_fmt != "mxfp4":
        raise RuntimeError("w_fmt: NVFP4 weights need act_fmt=\"bf16\"")
    if act_fmt == "bf16":
        if fused:
            raise RuntimeError("fused: the bf16 layer has no fused form")
        ids, gates, offs, sp, pr = moe_route_permute(logits, topk)
        h = moe_grouped_gemm_w4a16(x, offs, w1, w1_scale, w_fmt, sorted_pair=sp, topk=topk, swiglu=True)
        y = moe_grouped_gemm_w4a16(h, offs, w2, w2_scale, w_fmt, out_dtype=y_dtype)
        out = moe_unpermute_combine(y, gates, pr, T, topk, out_dtype)
        return dict(q=None, q_scale=None, topk_ids=ids, gates=gates, expert_offsets=offs, sorted_pair=sp, pair_row=pr,
                    h=h, h_scale=None, y=y, out=out)
    if fused and logits.shape[1] <= 256:
        q, qs, ids, gates, offs, sp, pr = moe_quantize_route(x, logits, topk, act_fmt)
    else:
        q, qs = mxfp4_quantize_act(x, act_fmt)
        ids, gates, offs, sp, pr = moe_route_permute(logits, topk)
    if fused:
        h, hs, out = moe_grouped_mxfp4_gemm_combine(q, qs, act_fmt, T, topk, offs, sp, ids, pr, gates, w1, w1_scale,
                                                    w2, w2_scale, out_dtype)
        y = None
    else:
        h, hs, y = moe_grouped_mxfp4_gemm(q, qs, act_fmt, T, topk, offs, sp, w1, w1_scale, w2, w2_scale, y_dtype)
        out = moe_unpermute_combine(y, gates, pr, T, topk, out_dtype)
    return dict(q=q, q_scale=qs, topk_ids=ids, gates=gates, expert_offsets=offs, sorted_pair=sp, pair_row=pr,
                h=h, h_scale=hs, y=y, out=out)


def ceiling_mfma(operands, act_fmt="e2m1", scale=127, iters=2000, sink=None):
    """Register-only scaled-MFMA loop (include/mxf_ceilings.h); returns (sink, flops).
    operands: int32 device tensor of >= CEILING_MFMA_WORDS words."""
    dev = _dev(operands)
    if operands.dtype != torch.int32:
        raise RuntimeError("operands must be int32")
    if sink is None:
        sink = torch.empty(CEILING_MFMA_GROUPS, dtype=torch.float32, device=dev)
    lib = load()
    _check(lib.mxf_ceiling_mfma(FMTS[act_fmt], _ptr(operands), operands.numel(), scale, iters, _ptr(sink),
                                _stream(dev)), "mxf_ceiling_mfma")
    return sink, lib.mxf_ceiling_mfma_flops(iters)


def ceiling_read(buf, xor_out=None):
    """Streaming non-temporal read of a device buffer; returns the int32 tensor holding
    the XOR of all its 32-bit words (accumulated into xor_out when given)."""
    dev = _dev(buf)
    if xor_out is None:
        xor_out = torch.zeros(1, dtype=torch.int32, device=dev)
    nbytes = buf.numel() * buf.element_size()
    _check(load().mxf_ceiling_read(_ptr(buf), nbytes, _ptr(xor_out), _stream(dev)), "mxf_ceiling_read")
    return xor_out


CEILING_COPY_STAGES = 28
CEILING_COPY_REGION = CEILING_COPY_STAGES * 32768


def ceiling_lds_copy(buf, pattern, groups, sum_out=None):
    """HBM -> LDS copy-path probe (include/mxf_ceilings.h): `groups` workgroups each fill
    28 stages of 64 KB from their two regions of buf (pattern 0: their own; pattern 1:
    shared as in the grouped FC1 launch). Returns the int32 tensor holding the sum, mod
    2^32, of every 32-bit word read (accumulated into sum_out when given)."""
    dev = _dev(buf)
    if sum_out is None:
        sum_out = torch.zeros(1, dtype=torch.int32, device=dev)
    nbytes = buf.numel() * buf.element_size()
    _check(load().mxf_ceiling_lds_copy(_ptr(buf), nbytes, pattern, groups, _ptr(sum_out), _stream(dev)),
           "mxf_ceiling_lds_copy")
    return sum_out

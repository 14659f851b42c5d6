"""epilogue_chains_gb300 -- vertical fusion of dependent operator chains on one GB300 (sm_103a).

Thin Python binding of the C ABI in ``include/fusechain.h`` (``libfusechain.so``): the functions
below have the C names and only marshal arguments (torch tensors -> device pointers, the current
torch stream -> ``cudaStream_t``, status codes -> ``FuseError``).  Every step of every chain runs
in the library's CUDA kernels; there is no fallback: if the library cannot be built or loaded, the
first call raises.

PyTorch is used for device memory and streams only.
"""
from __future__ import annotations

import ctypes
import functools
import threading

FUSE_OK, FUSE_EINVAL, FUSE_EALIGN, FUSE_EUNSUPPORTED = 0, -1, -2, -3
FUSE_ECUDA, FUSE_ETIMEOUT, FUSE_EWORKSPACE, FUSE_EINDEX = -4, -5, -6, -7
FUSE_F32, FUSE_F16, FUSE_BF16 = 0, 1, 2
FUSE_FUSED, FUSE_UNFUSED, FUSE_FAT = 0, 1, 2
FUSE_OP_AFFINE, FUSE_OP_AFFINE_RELU = 0, 1
FUSE_MAX_STAGES = 32
FUSE_FAT_TEMPS = 48
FUSE_ROPE_INTERLEAVED = 1


class FuseError(RuntimeError):
    def __init__(self, status: int, where: str):
        lib = _load()
        msg = lib.fuse_strerror(status).decode()
        extra = lib.fuse_last_cuda_error().decode() if status == FUSE_ECUDA else ""
        super().__init__(f"{where}: {msg} ({status}) {extra}".strip())
        self.status = status


class fuse_stage(ctypes.Structure):
    _fields_ = [("op", ctypes.c_int32), ("a", ctypes.c_float), ("b", ctypes.c_float),
                ("writes", ctypes.c_int64), ("ext_reads", ctypes.c_int64),
                ("flops", ctypes.c_int64), ("live_regs", ctypes.c_int32)]


class fuse_ledger_t(ctypes.Structure):
    _fields_ = [("bytes", ctypes.c_int64), ("launches", ctypes.c_int64),
                ("reg_peak", ctypes.c_int64), ("flops", ctypes.c_int64)]


class fuse_cost_model(ctypes.Structure):
    _fields_ = [("hbm_bytes_per_s", ctypes.c_double), ("flops_per_s", ctypes.c_double),
                ("launch_s", ctypes.c_double), ("spill_penalty", ctypes.c_double),
                ("reg_limit", ctypes.c_int32)]


class fuse_kernel_record(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 64), ("regs_per_thread", ctypes.c_int32),
                ("local_bytes_per_thread", ctypes.c_int32), ("static_smem_bytes", ctypes.c_int32),
                ("dynamic_smem_bytes", ctypes.c_int32), ("block_threads", ctypes.c_int32),
                ("blocks_per_sm", ctypes.c_int32), ("max_threads_per_block", ctypes.c_int32),
                ("cluster_size", ctypes.c_int32), ("max_active_clusters", ctypes.c_int32),
                ("blocks_per_sm_api", ctypes.c_int32), ("tmem_cols", ctypes.c_int32),
                ("ptxas_registers", ctypes.c_int32), ("stack_bytes", ctypes.c_int32),
                ("spill_store_bytes", ctypes.c_int32), ("spill_load_bytes", ctypes.c_int32),
                ("symbol", ctypes.c_char * 256)]


class fuse_ptxas_record(ctypes.Structure):
    _fields_ = [("symbol", ctypes.c_char * 256), ("registers", ctypes.c_int32),
                ("stack_bytes", ctypes.c_int32), ("spill_store_bytes", ctypes.c_int32),
                ("spill_load_bytes", ctypes.c_int32)]


_P, _I32, _I64, _U32, _F32, _SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint32,
                                   ctypes.c_float, ctypes.c_size_t)
# every symbol the header declares, with its C signature
SIGNATURES = {
    "fuse_chain_run": ([ctypes.POINTER(fuse_stage), _I32, _P, _P, _I64, _I32, _I32, _P], _I32),
    "fuse_chain_run_host": ([ctypes.POINTER(fuse_stage), _I32, _P, _P, _I64, _I32, _I32, _P, _P, _I32, _P], _I32),
    "fuse_rmsnorm": ([_P, _P, _P, _I64, _I64, _F32, _I32, _P, _SZ, _P], _I32),
    "fuse_rmsnorm_workspace_bytes": ([_I64, _I64, _I32], _SZ),
    "fuse_rmsnorm_unfused_static": ([_P, _P, _P, _I64, _I64, _F32, _P], _I32),
    "fuse_causal_softmax": ([_P, _P, _I64, _I64, _F32, _I32, _I32, _I32, _P, _SZ, _P], _I32),
    "fuse_causal_softmax_workspace_bytes": ([_I64, _I64, _I32], _SZ),
    "fuse_gemm_epilogue": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _P], _I32),
    "fuse_gemm_epilogue_plan": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _U32, _P], _I32),
    "fuse_gemm_epilogue_ws": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _U32, _P, _SZ, _P], _I32),
    "fuse_gemm_workspace_bytes": ([_I64, _I64, _I64], _SZ),
    "fuse_gemm_bytes": ([_I64, _I64, _I64, _U32], _I64),
    "fuse_attention_schedule": ([_I64, _I64, _I32, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)], _I64),
    "fuse_ledger": ([ctypes.POINTER(fuse_stage), _I32, _U32, _I32, ctypes.POINTER(fuse_ledger_t)], _I32),
    "fuse_plan_time": ([ctypes.POINTER(fuse_stage), _I32, _U32, _I32, ctypes.POINTER(fuse_cost_model),
                        ctypes.POINTER(ctypes.c_double)], _I32),
    "fuse_best_plan": ([ctypes.POINTER(fuse_stage), _I32, _I32, ctypes.POINTER(fuse_cost_model),
                        ctypes.POINTER(ctypes.c_uint32), ctypes.POINTER(ctypes.c_double)], _I32),
    "fuse_launch_model": ([_I64, ctypes.c_double, ctypes.c_double, ctypes.c_double,
                           ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double),
                           ctypes.POINTER(ctypes.c_double)], _I32),
    "fuse_add_rmsnorm": ([_P, _P, _P, _P, _P, _I64, _I64, _F32, _I32, _P, _SZ, _P], _I32),
    "fuse_silu_mul": ([_P, _P, _I64, _P, _I64, _I64, _I32, _I32, _P], _I32),
    "fuse_add_rmsnorm_bytes": ([_I64, _I64, _I32], _I64),
    "fuse_attention": ([_P, _P, _P, _P, _I64, _I64, _I64, _F32, _P], _I32),
    "fuse_attention_bytes": ([_I64, _I64, _I64], _I64),
    "fuse_attention_flops": ([_I64, _I64, _I64], _I64),
    "fuse_silu_mul_bytes": ([_I64, _I64, _I32, _I32], _I64),
    "fuse_chain_bytes": ([_I32, _I64, _I32, _I32], _I64),
    "fuse_rmsnorm_bytes": ([_I64, _I64, _I32], _I64),
    "fuse_causal_softmax_bytes": ([_I64, _I64, _I32, _I32, _I32], _I64),
    "fuse_rope_append": ([_P, _I64, _P, _I64, _I64, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I64, _I64, _I32,
                          _U32, _P], _I32),
    "fuse_rope_append_bytes": ([_I64, _I64, _I64, _I64, _I64, _I64], _I64),
    "fuse_paged_attention": ([_P, _P, _P, _P, _I64, _P, _P, _I64, _P, _I64, _I64, _I64, _I64, _I64, _I64, _F32,
                              _I32, _P, _SZ, _P], _I32),
    "fuse_paged_attention_workspace_bytes": ([_I64, _I64, _I64, _I64, _I64], _SZ),
    "fuse_paged_attention_bytes": ([_I64, _I64, _I64, _I64, _I64, _I64], _I64),
    "fuse_paged_attention_flops": ([_I64, _I64, _I64, _I64, _I64], _I64),
    "fuse_w4_gemv": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I32, _I32, _P], _I32),
    "fuse_w4_gemv_bytes": ([_I64, _I64, _I64, _I64, _I32, _I32, _I32], _I64),
    "fuse_kernel_count": ([], _I32),
    "fuse_kernel_report": ([_I32, ctypes.POINTER(fuse_kernel_record)], _I32),
    "fuse_ptxas_count": ([], _I32),
    "fuse_ptxas_entry": ([_I32, ctypes.POINTER(fuse_ptxas_record)], _I32),
    "fuse_strerror": ([_I32], ctypes.c_char_p),
    "fuse_last_cuda_error": ([], ctypes.c_char_p),
    "fuse_check": ([_P], _I32),
    "fuse_debug_expire_wait": ([_I64, _P], _I32),
    "fuse_debug_split_window": ([_I64], _I32),
    "fuse_graph_begin": ([_P], _I32),
    "fuse_graph_end": ([_P, ctypes.POINTER(ctypes.c_void_p)], _I32),
    "fuse_graph_launch": ([_P, _P], _I32),
    "fuse_graph_kernel_count": ([_P], _I32),
    "fuse_graph_destroy": ([_P], None),
    "fuse_version": ([], _I32),
}

_lock = threading.Lock()
_lib = None


def _load():
    """Build (if needed) and load libfusechain.so; raises if either fails."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            from . import _build
            path = _build.build()
            lib = ctypes.CDLL(path)
            for name, (args, res) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.argtypes = args
                fn.restype = res
            _lib = lib
    return _lib


def library_path() -> str:
    from . import _build
    return _build.LIB


def _check(status: int, where: str) -> None:
    if status != FUSE_OK:
        raise FuseError(status, where)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_torch = None         # the torch module, and its calls for the current device's index and stream handle
_current_device = None
_current_handle = None


def _bind_torch():
    """torch, imported at the first call that needs it (an import statement or a Stream object at every
    call costs the host more than the launch of a small kernel)."""
    global _torch, _current_device, _current_handle
    import torch
    if not torch.cuda.is_available():
        raise ValueError("no CUDA device")
    torch.cuda.current_stream()        # initialises CUDA
    _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _current_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    _torch = torch
    return torch


def _stream(stream) -> int | None:
    if stream is None:
        if _torch is None:
            _bind_torch()
        return _current_handle(_current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dtype_code(t) -> int:
    import torch
    return {torch.float32: FUSE_F32, torch.float16: FUSE_F16, torch.bfloat16: FUSE_BF16}[t.dtype]


def _stages(stages) -> ctypes.Array:
    """Accept fuse_stage objects, (op, a, b) tuples or dicts with the struct's field names."""
    arr = (fuse_stage * len(stages))()
    for i, s in enumerate(stages):
        if isinstance(s, fuse_stage):
            arr[i] = s
        elif isinstance(s, dict):
            arr[i] = fuse_stage(**s)
        else:
            op, a, b = s
            arr[i] = fuse_stage(int(op), float(a), float(b), 0, 0, 0, 0)
    return arr


def _need_device(*ts):
    for t in ts:
        if t is not None and not isinstance(t, int):
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError("tensors must be contiguous CUDA tensors")


# ------------------------------------------------------------------------------- chains
def fuse_chain_run(stages, x, y, mode: int = FUSE_FUSED, stream=None) -> None:
    """y <- f_{K-1}(...f_0(x)) with f_s(v) = [ReLU](a_s v + b_s); see fusechain.h."""
    _need_device(x, y)
    if x.dtype != y.dtype or x.numel() != y.numel():
        raise ValueError("x and y must have the same dtype and element count")
    st = _stages(stages)
    _check(_load().fuse_chain_run(st, len(st), _ptr(x), _ptr(y), x.numel(), _dtype_code(x), mode,
                                  _stream(stream)), "fuse_chain_run")


def fuse_chain_run_host(stages, x_host, y_host, x_dev, y_dev, mode: int = FUSE_FUSED, slices: int = 8,
                        stream=None) -> None:
    """The chain on host tensors (x_host in, y_host out; pinned for asynchronous copies) through
    the caller's device scratch x_dev, y_dev (same dtype and element count); see fusechain.h.
    y_host is valid after the stream is synchronized."""
    _need_device(x_dev, y_dev)
    for t in (x_host, y_host):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("x_host and y_host must be contiguous host tensors")
    n = x_host.numel()
    if any(t.numel() != n or t.dtype != x_host.dtype for t in (y_host, x_dev, y_dev)):
        raise ValueError("all four tensors must have the same dtype and element count")
    st = _stages(stages)
    _check(_load().fuse_chain_run_host(st, len(st), _ptr(x_host), _ptr(y_host), n, _dtype_code(x_host),
                                       mode, _ptr(x_dev), _ptr(y_dev), int(slices), _stream(stream)),
           "fuse_chain_run_host")


def fuse_rmsnorm(x, w, y, eps: float, mode: int = FUSE_FUSED, workspace=None, stream=None) -> None:
    """y = x * rsqrt(mean(x^2, -1) + eps) * w over rows of a [rows, hidden] fp32 tensor."""
    import torch
    _need_device(x, w, y)
    rows, hidden = x.shape
    lib = _load()
    ws_bytes = lib.fuse_rmsnorm_workspace_bytes(rows, hidden, mode)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    ws_size = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.fuse_rmsnorm(_ptr(x), _ptr(w), _ptr(y), rows, hidden, float(eps), mode,
                            _ptr(workspace), ws_size, _stream(stream)), "fuse_rmsnorm")


def fuse_add_rmsnorm(x, r, w, h, y, eps: float, mode: int = FUSE_FUSED, workspace=None,
                     stream=None) -> None:
    """h = x + r; y = h * rsqrt(mean(h^2, -1) + eps) * w over rows of [rows, hidden] fp32."""
    import torch
    _need_device(x, r, w, h, y)
    rows, hidden = x.shape
    lib = _load()
    ws_bytes = lib.fuse_rmsnorm_workspace_bytes(rows, hidden, mode)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    ws_size = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.fuse_add_rmsnorm(_ptr(x), _ptr(r), _ptr(w), _ptr(h), _ptr(y), rows, hidden,
                                float(eps), mode, _ptr(workspace), ws_size, _stream(stream)),
           "fuse_add_rmsnorm")


def fuse_silu_mul(g, u, y, mode: int = FUSE_FUSED, stream=None) -> None:
    """y = SiLU(g) * u.  g and u: [rows, cols] tensors (possibly the two column halves of one
    merged [rows, 2 cols] tensor: same row stride); y: contiguous [rows, cols]."""
    for t in (g, u, y):
        if not t.is_cuda or t.dim() != 2 or t.stride(1) != 1:
            raise ValueError("g, u, y must be 2-D CUDA tensors with unit column stride")
    if g.shape != u.shape or g.shape != y.shape or g.stride(0) != u.stride(0):
        raise ValueError("g, u, y must have one shape and g, u one row stride")
    if not y.is_contiguous() or g.dtype != u.dtype or g.dtype != y.dtype:
        raise ValueError("y must be contiguous and all three of one dtype")
    rows, cols = g.shape
    _check(_load().fuse_silu_mul(_ptr(g), _ptr(u), g.stride(0), _ptr(y), rows, cols,
                                 _dtype_code(g), mode, _stream(stream)), "fuse_silu_mul")


def fuse_attention(q, k, v, o, scale: float, stream=None) -> None:
    """o = causal softmax(scale q k^T) v over bf16 [bh, S, D] tensors, no score matrix."""
    _need_device(q, k, v, o)
    if q.shape != k.shape or q.shape != v.shape or q.shape != o.shape or q.dim() != 3:
        raise ValueError("q, k, v, o must be [bh, S, D] tensors of one shape")
    bh, S, D = q.shape
    _check(_load().fuse_attention(_ptr(q), _ptr(k), _ptr(v), _ptr(o), bh, S, D, float(scale),
                                  _stream(stream)), "fuse_attention")


def fuse_rmsnorm_unfused_static(x, w, y, eps: float, stream=None) -> None:
    """Unfused RMSNorm with its row statistics in the library's own fixed device array (no
    workspace, no allocation; rows <= FUSE_RMSNORM_STATIC_MAX_ROWS)."""
    _need_device(x, w, y)
    rows, hidden = x.shape
    _check(_load().fuse_rmsnorm_unfused_static(_ptr(x), _ptr(w), _ptr(y), rows, hidden, float(eps),
                                               _stream(stream)), "fuse_rmsnorm_unfused_static")


FUSE_RMSNORM_STATIC_MAX_ROWS = 65536
FUSE_GEMM_STATIC_B = 0x100


def fuse_causal_softmax(s, p, scale: float, skip_tile: int = 0, mode: int = FUSE_FUSED,
                        workspace=None, stream=None) -> None:
    """p = causal softmax(scale * s) over the last axis of a bf16 [..., S, S] tensor."""
    import torch
    _need_device(s, p)
    S = s.shape[-1]
    bh = s.numel() // (S * S)
    lib = _load()
    ws_bytes = lib.fuse_causal_softmax_workspace_bytes(bh, S, mode)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=s.device)
    ws_size = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib.fuse_causal_softmax(_ptr(s), _ptr(p), bh, S, float(scale), int(skip_tile),
                                   _dtype_code(p), mode, _ptr(workspace), ws_size,
                                   _stream(stream)), "fuse_causal_softmax")


# split-K workspaces handed out by fuse_gemm_epilogue(workspace=None): one zero-filled buffer per
# (device, stream), reused (every completed call leaves it zero-filled), never freed
_GEMM_WS = {}


def _gemm_workspace(M: int, N: int, K: int, dev, stream_handle):
    import torch
    need = fuse_gemm_workspace_bytes(M, N, K)
    if need == 0:
        return None
    key = (dev.index, stream_handle)
    ws = _GEMM_WS.get(key)
    if ws is not None and ws.numel() >= need:
        return ws
    # allocate only on torch's current stream and outside graph capture; otherwise the call
    # runs unsplit
    if torch.cuda.is_current_stream_capturing() or stream_handle != torch.cuda.current_stream(dev).cuda_stream:
        return None
    ws = torch.zeros(need, dtype=torch.uint8, device=dev)
    torch.cuda.current_stream(dev).synchronize()   # zero-filled before any stream uses it
    _GEMM_WS[key] = ws
    return ws


def fuse_gemm_epilogue(A, B, bias, R, Y, cut_mask: int = 0, workspace=None, stream=None) -> None:
    """Y = fp16(GELU(A @ B + bias) + R) for fp16 A [M,K], B [K,N], bias [N], R, Y [M,N]; cut_mask
    selects the plan (0 = fully fused [4]; 7 = [1,1,1,1]).  workspace: a zero-filled device tensor
    of fuse_gemm_workspace_bytes(M, N, K) bytes (see fuse_gemm_epilogue_ws in the header), reused
    across calls on one stream; None: a buffer of that kind kept by this module per device and
    stream; False: none (the last wave of tiles is not split over K)."""
    _need_device(A, B, bias, R, Y)
    M, K = A.shape
    K2, N = B.shape
    if K != K2 or tuple(R.shape) != (M, N) or tuple(Y.shape) != (M, N) or bias.numel() != N:
        raise ValueError("shape mismatch")
    sh = _stream(stream)
    if workspace is None:
        workspace = _gemm_workspace(M, N, K, A.device, sh)
    elif workspace is False:
        workspace = None
    ws_size = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_load().fuse_gemm_epilogue_ws(_ptr(A), _ptr(B), _ptr(bias), _ptr(R), _ptr(Y), M, N, K,
                                         int(cut_mask), _ptr(workspace), ws_size, sh),
           "fuse_gemm_epilogue")


def fuse_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return _load().fuse_gemm_workspace_bytes(M, N, K)


def fuse_attention_schedule(bh: int, S: int, clusters: int):
    """Per-cluster item lists of the persistent attention kernel: (first [clusters + 1], items)."""
    n = bh * S // 256
    first = (ctypes.c_int32 * (clusters + 1))()
    items = (ctypes.c_int32 * max(1, n))()
    rc = _load().fuse_attention_schedule(bh, S, clusters, first, items)
    _check(rc if rc < 0 else 0, "fuse_attention_schedule")
    return list(first), list(items[:rc])


def fuse_gemm_bytes(M: int, N: int, K: int, cut_mask: int) -> int:
    return _load().fuse_gemm_bytes(M, N, K, cut_mask)


# ------------------------------------------------------------------------------- single-token decode
def _decode_operands(dt, ts, others) -> int:
    """The device index of the tensors: contiguous, of dtype dt (fp16 or bf16; `others`: pairs of a tensor
    or None and its dtype), all on torch's current device (the library launches there)."""
    torch = _torch
    if dt is not torch.bfloat16 and dt is not torch.float16:
        raise ValueError(f"fp16 or bf16 tensors expected, not {dt}")
    dev = ts[0].get_device()
    if dev != _current_device():
        raise ValueError("the tensors must be on the current CUDA device")
    for t in ts:
        if t is not None and (t.dtype is not dt or t.get_device() != dev or not t.is_contiguous()):
            raise ValueError(f"{tuple(t.shape)} {t.dtype} on {t.device}: contiguous {dt} on one device expected")
    for t, want in others:
        if t is not None and (t.dtype is not want or t.get_device() != dev or not t.is_contiguous()):
            raise ValueError(f"{tuple(t.shape)} {t.dtype} on {t.device}: contiguous {want} on one device expected")
    return dev


def fuse_rope_append(qkv, cos_sin, positions, slots, q_out, k_cache, v_cache, interleaved: bool = False,
                     stream=None) -> None:
    """Rotate the queries and keys of qkv [tokens, (q_heads + 2 kv_heads) D] (rows may be strided) by
    their positions, write the queries to q_out [tokens, q_heads, D] and append keys and values to
    k_cache, v_cache [num_pages, kv_heads, page_size, D] at slots (int32; negative: append nothing).
    cos_sin: fp32 [max_pos, rot], the cosines then the sines of a position's rot / 2 pairs."""
    torch = _torch or _bind_torch()
    dt = qkv.dtype
    dev = _decode_operands(dt, (q_out, k_cache, v_cache), ((positions, torch.int32), (slots, torch.int32),
                                                           (cos_sin, torch.float32)))
    tokens, q_heads, D = q_out.shape
    pages, kv_heads, page_size, D2 = k_cache.shape
    if qkv.get_device() != dev or qkv.dim() != 2 or qkv.stride(1) != 1:
        raise ValueError("qkv must be a 2-D tensor with unit column stride on the device of the others")
    if (D2 != D or v_cache.shape != k_cache.shape or qkv.shape != (tokens, (q_heads + 2 * kv_heads) * D)
            or positions.shape != (tokens,) or slots.shape != (tokens,) or cos_sin.dim() != 2):
        raise ValueError("shape mismatch")
    ld = qkv.stride(0) if tokens > 1 else qkv.shape[1]
    _check(_load().fuse_rope_append(qkv.data_ptr(), ld, cos_sin.data_ptr(), cos_sin.shape[0], cos_sin.shape[1],
                                    positions.data_ptr(), slots.data_ptr(), q_out.data_ptr(), k_cache.data_ptr(),
                                    v_cache.data_ptr(), tokens, q_heads, kv_heads, D, pages, page_size,
                                    FUSE_F16 if dt is torch.float16 else FUSE_BF16,
                                    FUSE_ROPE_INTERLEAVED if interleaved else 0, _stream(stream)),
           "fuse_rope_append")


# workspaces of fuse_paged_attention(workspace=None): one zero-filled buffer per (device, stream), grown
# as needed; every completed call leaves its counters zero, and fuse_check() drops them after a timeout
# (their memory is the stream's they were allocated and used on, so work still queued there keeps it)
_PAGED_WS = {}
_PAGED_LOCK = threading.Lock()


def _paged_workspace(need: int, dev: int, stream_handle):
    torch = _torch
    if stream_handle != _current_handle(dev) or torch.cuda.is_current_stream_capturing():
        raise ValueError("pass a zero-filled workspace of fuse_paged_attention_workspace_bytes() bytes: this module's "
                         "own ones serve calls on torch's current stream outside a graph capture only (a captured "
                         "graph may be replayed next to other calls)")
    ws = _PAGED_WS.get((dev, stream_handle))
    if ws is None or ws.numel() < need:
        ws = torch.zeros(need, dtype=torch.uint8, device=torch.device("cuda", dev))   # on the current stream
        _PAGED_WS[dev, stream_handle] = ws
    return ws


def fuse_paged_attention(q, k_cache, v_cache, block_table, seq_lens, o, scale: float, prefix_table=None,
                         prefix_len: int = 0, workspace=None, stream=None) -> None:
    """o = softmax(scale q k^T) v for one query per sequence (q, o [batch, q_heads, D]) over the first
    prefix_len keys of prefix_table's pages, which all sequences share, and the first seq_lens[b] keys of
    block_table[b]'s; k_cache, v_cache [num_pages, kv_heads, page_size, D].  workspace: a zero-filled
    device tensor (see fuse_paged_attention in the header); None: a buffer kept by this module for the
    current stream."""
    torch = _torch or _bind_torch()
    dt, i32 = q.dtype, torch.int32
    dev = _decode_operands(dt, (q, k_cache, v_cache, o), ((block_table, i32), (seq_lens, i32), (prefix_table, i32)))
    batch, q_heads, D = q.shape
    pages, kv_heads, page_size, D2 = k_cache.shape
    if (D2 != D or o.shape != q.shape or v_cache.shape != k_cache.shape or block_table.dim() != 2
            or block_table.shape[0] != batch or seq_lens.shape != (batch,)):
        raise ValueError("shape mismatch")
    if prefix_len and (prefix_table is None or prefix_table.numel() * page_size < prefix_len):
        raise ValueError("prefix_table does not hold prefix_len keys")
    lib, sh = _load(), _stream(stream)
    own = workspace is None
    if not own and (workspace.get_device() != dev or not workspace.is_contiguous()):
        raise ValueError("the workspace must be a contiguous tensor on the device of the others")
    if own:      # a call is several launches: those of two threads on one stream must not mix over one workspace
        _PAGED_LOCK.acquire()
    try:
        if own:
            workspace = _paged_workspace(fuse_paged_attention_workspace_bytes(batch, q_heads, kv_heads, D, prefix_len), dev, sh)
        status = lib.fuse_paged_attention(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
                                          block_table.shape[1], seq_lens.data_ptr(), _ptr(prefix_table), prefix_len,
                                          o.data_ptr(), batch, q_heads, kv_heads, D, pages, page_size, scale,
                                          FUSE_F16 if dt is torch.float16 else FUSE_BF16, workspace.data_ptr(),
                                          workspace.nbytes, sh)
    finally:
        if own:
            _PAGED_LOCK.release()
    _check(status, "fuse_paged_attention")


@functools.lru_cache(maxsize=256)
def fuse_paged_attention_workspace_bytes(batch: int, q_heads: int, kv_heads: int, D: int, prefix_len: int = 0) -> int:
    return _load().fuse_paged_attention_workspace_bytes(batch, q_heads, kv_heads, D, prefix_len)


def fuse_w4_gemv(x, wq, scales, y, zeros=None, bias=None, residual=None, gelu: bool = False, stream=None) -> None:
    """y = GELU(x W^T + bias) + residual for x [M, K], M <= 64, and W [N, K] in 4 bits: wq uint8 [N, K / 2]
    (input 2j in a byte's low half), scales [N, K / group] and zeros uint8 [N, K / group] (None: 8),
    W = (q - zero) scale.  bias [N], residual [M, N] and the GELU are optional."""
    torch = _torch or _bind_torch()
    dt = x.dtype
    _decode_operands(dt, (x, scales, y, bias, residual), ((wq, torch.uint8), (zeros, torch.uint8)))
    M, K = x.shape
    N, half = wq.shape
    groups = scales.shape[1] if scales.dim() == 2 else 0
    if (2 * half != K or groups < 1 or K % groups or scales.shape[0] != N or y.shape != (M, N)
            or (zeros is not None and zeros.shape != scales.shape) or (bias is not None and bias.shape != (N,))
            or (residual is not None and residual.shape != y.shape)):
        raise ValueError("shape mismatch")
    _check(_load().fuse_w4_gemv(x.data_ptr(), wq.data_ptr(), scales.data_ptr(), _ptr(zeros), _ptr(bias), _ptr(residual),
                                y.data_ptr(), M, N, K, K // groups, 1 if gelu else 0,
                                FUSE_F16 if dt is torch.float16 else FUSE_BF16, _stream(stream)), "fuse_w4_gemv")


def fuse_rope_append_bytes(tokens: int, appended: int, q_heads: int, kv_heads: int, D: int, rot: int) -> int:
    return _load().fuse_rope_append_bytes(tokens, appended, q_heads, kv_heads, D, rot)


def fuse_paged_attention_bytes(batch: int, q_heads: int, kv_heads: int, D: int, prefix_len: int, keys: int) -> int:
    return _load().fuse_paged_attention_bytes(batch, q_heads, kv_heads, D, prefix_len, keys)


def fuse_paged_attention_flops(batch: int, q_heads: int, D: int, prefix_len: int, keys: int) -> int:
    return _load().fuse_paged_attention_flops(batch, q_heads, D, prefix_len, keys)


def fuse_w4_gemv_bytes(M: int, N: int, K: int, group: int, zeros: bool = False, bias: bool = False,
                       residual: bool = False) -> int:
    return _load().fuse_w4_gemv_bytes(M, N, K, group, int(zeros), int(bias), int(residual))


# ------------------------------------------------------------------------------- ledgers
def fuse_ledger(stages, cut_mask: int, elem_bytes: int) -> dict:
    st = _stages(stages)
    out = fuse_ledger_t()
    _check(_load().fuse_ledger(st, len(st), cut_mask, elem_bytes, ctypes.byref(out)), "fuse_ledger")
    return {"bytes": out.bytes, "launches": out.launches, "reg_peak": out.reg_peak,
            "flops": out.flops}


def _model(model) -> fuse_cost_model:
    if isinstance(model, fuse_cost_model):
        return model
    return fuse_cost_model(**model)


def fuse_plan_time(stages, cut_mask: int, elem_bytes: int, model) -> float:
    """[K4] time_estimate of one cut plan, seconds."""
    st = _stages(stages)
    out = ctypes.c_double()
    _check(_load().fuse_plan_time(st, len(st), cut_mask, elem_bytes, ctypes.byref(_model(model)),
                                  ctypes.byref(out)), "fuse_plan_time")
    return out.value


def fuse_best_plan(stages, elem_bytes: int, model) -> tuple:
    """[K4] best_plan: (cut_mask, seconds) of the cheapest of the 2^(K-1) plans."""
    st = _stages(stages)
    mask, sec = ctypes.c_uint32(), ctypes.c_double()
    _check(_load().fuse_best_plan(st, len(st), elem_bytes, ctypes.byref(_model(model)),
                                  ctypes.byref(mask), ctypes.byref(sec)), "fuse_best_plan")
    return mask.value, sec.value


def fuse_add_rmsnorm_bytes(rows: int, hidden: int, mode: int) -> int:
    return _load().fuse_add_rmsnorm_bytes(rows, hidden, mode)


def fuse_silu_mul_bytes(rows: int, cols: int, dtype: int, mode: int) -> int:
    return _load().fuse_silu_mul_bytes(rows, cols, dtype, mode)


def fuse_attention_bytes(bh: int, S: int, D: int) -> int:
    return _load().fuse_attention_bytes(bh, S, D)


def fuse_attention_flops(bh: int, S: int, D: int) -> int:
    return _load().fuse_attention_flops(bh, S, D)


def fuse_launch_model(n_kernels: int, t_launch: float, t_exec: float, t_dispatch: float) -> dict:
    """Eager vs CUDA-graph timeline of n_kernels kernels; see fusechain.h."""
    e, i, g = ctypes.c_double(), ctypes.c_double(), ctypes.c_double()
    _check(_load().fuse_launch_model(n_kernels, t_launch, t_exec, t_dispatch, ctypes.byref(e),
                                     ctypes.byref(i), ctypes.byref(g)), "fuse_launch_model")
    return {"eager": e.value, "eager_idle": i.value, "graph": g.value}


def fuse_chain_bytes(K: int, n: int, dtype: int, mode: int) -> int:
    return _load().fuse_chain_bytes(K, n, dtype, mode)


def fuse_rmsnorm_bytes(rows: int, hidden: int, mode: int) -> int:
    return _load().fuse_rmsnorm_bytes(rows, hidden, mode)


def fuse_causal_softmax_bytes(bh: int, S: int, skip_tile: int, out_dtype: int, mode: int) -> int:
    return _load().fuse_causal_softmax_bytes(bh, S, skip_tile, out_dtype, mode)


def fuse_rmsnorm_workspace_bytes(rows: int, hidden: int, mode: int) -> int:
    return _load().fuse_rmsnorm_workspace_bytes(rows, hidden, mode)


def fuse_causal_softmax_workspace_bytes(bh: int, S: int, mode: int) -> int:
    return _load().fuse_causal_softmax_workspace_bytes(bh, S, mode)


# ------------------------------------------------------------------------------- status
def fuse_kernel_count() -> int:
    return _load().fuse_kernel_count()


def fuse_kernel_report(index: int) -> dict:
    rec = fuse_kernel_record()
    _check(_load().fuse_kernel_report(index, ctypes.byref(rec)), "fuse_kernel_report")
    return {f: (getattr(rec, f).decode() if f in ("name", "symbol") else getattr(rec, f))
            for f, _ in fuse_kernel_record._fields_}


def fuse_ptxas_table() -> list[dict]:
    """The ptxas -v record of every kernel compiled into the library (host only)."""
    lib = _load()
    out = []
    for i in range(lib.fuse_ptxas_count()):
        rec = fuse_ptxas_record()
        _check(lib.fuse_ptxas_entry(i, ctypes.byref(rec)), "fuse_ptxas_entry")
        out.append({f: (getattr(rec, f).decode() if f == "symbol" else getattr(rec, f))
                    for f, _ in fuse_ptxas_record._fields_})
    return out


def fuse_check(stream=None) -> int:
    """Synchronize `stream`; FUSE_ETIMEOUT, FUSE_EINDEX or FUSE_ECUDA if a call since the last check met one,
    else FUSE_OK.  After a timeout the workspaces that this module keeps for fuse_paged_attention() are dropped
    (a call that was given up leaves arrival counts in them); one that the caller passed is the caller's to zero."""
    status = _load().fuse_check(_stream(stream))
    if status == FUSE_ETIMEOUT:
        with _PAGED_LOCK:
            _PAGED_WS.clear()
    return status


def fuse_debug_expire_wait(budget_cycles: int, stream=None) -> None:
    _check(_load().fuse_debug_expire_wait(int(budget_cycles), _stream(stream)),
           "fuse_debug_expire_wait")


# ------------------------------------------------------------------------------- graphs
def fuse_graph_begin(stream=None) -> None:
    """Start capturing this library's calls on `stream` (a non-default stream)."""
    _check(_load().fuse_graph_begin(_stream(stream)), "fuse_graph_begin")


def fuse_graph_end(stream=None) -> int:
    """End the capture; returns the executable graph's handle (free with fuse_graph_destroy)."""
    g = ctypes.c_void_p()
    _check(_load().fuse_graph_end(_stream(stream), ctypes.byref(g)), "fuse_graph_end")
    return g.value


def fuse_graph_launch(graph: int, stream=None) -> None:
    _check(_load().fuse_graph_launch(graph, _stream(stream)), "fuse_graph_launch")


def fuse_graph_kernel_count(graph: int) -> int:
    n = _load().fuse_graph_kernel_count(graph)
    _check(min(n, 0), "fuse_graph_kernel_count")
    return n


def fuse_graph_destroy(graph: int) -> None:
    _load().fuse_graph_destroy(graph)


def fuse_strerror(status: int) -> str:
    return _load().fuse_strerror(status).decode()


def fuse_version() -> int:
    return _load().fuse_version()

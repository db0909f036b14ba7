"""Python binding of the xq C ABI (include/xq.h): argument marshalling only.

Every computation happens in libxq.so's CUDA kernels. Tensors are torch CUDA
tensors (torch supplies device memory and streams); the binding passes their
device pointers and the current stream to the C entry points of the same
name. A missing library is an error: there is no CPU or library fallback.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct

from . import synth

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libxq.so")

XQ_TYPE_F32 = 0
XQ_TYPE_F16 = 1
XQ_TYPE_Q4_0 = 2
XQ_TYPE_Q8_0 = 8
XQ_TYPE_Q4_K = 12
XQ_TYPE_Q6_K = 14
XQ_TYPE_IQ4_XS = 23
XQ_TYPE_BF16 = 30

STATUS = {0: "XQ_OK", 1: "XQ_ERR_ARG", 2: "XQ_ERR_SHAPE", 3: "XQ_ERR_ALIGN",
          4: "XQ_ERR_WORKSPACE", 5: "XQ_ERR_CUDA", 6: "XQ_ERR_UNSUPPORTED"}

# Every symbol include/xq.h declares.
SYMBOLS = ("xq_status_str", "xq_q8_bytes", "xq_weight_bytes", "xq_quantize_q8",
           "xq_matmul_q4k_q8", "xq_matmul_q6k_q8", "xq_layer_workspace_bytes",
           "xq_layer_mixed", "xq_debug_isums_q4k", "xq_debug_isums_q6k", "xq_layer_mixed_static",
           "xq_q8_bytes_invariant", "xq_quantize_q8_invariant", "xq_matmul_invariant",
           "xq_matmul_q8_0_q8", "xq_debug_isums_q8_0", "xq_silu_mul_quantize_q8",
           "xq_layer_ffn_workspace_bytes", "xq_layer_mixed_ffn", "xq_matmul_iq4xs_q8",
           "xq_debug_isums_iq4xs", "xq_device_error", "xq_debug_stalled_matmul_q4k", "xq_debug_tile_sums",
           "xq_debug_layer_matmuls", "xq_debug_check_probe", "xq_debug_stalled_ffn_layer",
           "xq_kv_bytes", "xq_kv_write", "xq_kv_read", "xq_kv_attn_workspace_bytes", "xq_kv_attn",
           "xq_kv_attn_shared", "xq_lora_add", "xq_qk_norm_rope", "xq_prompt_attn_workspace_bytes", "xq_prompt_attn",
           "xq_debug_stalled_prompt_attn")


class XQError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)} ({lib().xq_status_str(code).decode()})")
        self.code = code


class xq_proj(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int),
                ("W", ctypes.c_void_p), ("y", ctypes.c_void_p), ("input", ctypes.c_int),
                ("codebook", ctypes.c_void_p)]


class xq_kv_cache(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int), ("n_pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("heads", ctypes.c_int), ("dim", ctypes.c_int), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p)]


class xq_kv_query(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int), ("batch", ctypes.c_int), ("n_q", ctypes.c_int), ("heads", ctypes.c_int),
                ("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("pages", ctypes.c_void_p),
                ("page_stride", ctypes.c_int), ("max_pages", ctypes.c_int), ("lens", ctypes.c_void_p),
                ("scale", ctypes.c_float), ("window", ctypes.c_int), ("prefix_pages", ctypes.c_void_p),
                ("prefix_len", ctypes.c_int)]


class xq_adapters(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int), ("n", ctypes.c_int), ("rank", ctypes.c_int), ("K", ctypes.c_int), ("N", ctypes.c_int),
                ("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("input", ctypes.c_int)]


class xq_qk_rows(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int), ("y_type", ctypes.c_int), ("tokens", ctypes.c_int), ("heads", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("dim", ctypes.c_int), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("q_stride", ctypes.c_longlong), ("k_stride", ctypes.c_longlong), ("q_out", ctypes.c_void_p),
                ("k_out", ctypes.c_void_p), ("q_out_stride", ctypes.c_longlong), ("k_out_stride", ctypes.c_longlong),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("positions", ctypes.c_void_p), ("turns", ctypes.c_void_p), ("rot", ctypes.c_int), ("pairs", ctypes.c_int),
                ("magnitude", ctypes.c_float)]


class xq_prompts(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int), ("tokens", ctypes.c_int), ("batch", ctypes.c_int), ("heads", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("dim", ctypes.c_int), ("q", ctypes.c_void_p), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("q_stride", ctypes.c_longlong), ("k_stride", ctypes.c_longlong),
                ("v_stride", ctypes.c_longlong), ("out", ctypes.c_void_p), ("starts", ctypes.c_void_p), ("scale", ctypes.c_float),
                ("window", ctypes.c_int)]


_lib = None


def lib(path: str | None = None):
    """Open libxq.so (built in-tree by gguf_quant_integer_gb300.build)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libxq.so not found at {p}; build it with "
                           f"`python -m gguf_quant_integer_gb300.build` (no fallback exists)")
    L = ctypes.CDLL(p)
    P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.xq_status_str.argtypes = [I]
    L.xq_status_str.restype = ctypes.c_char_p
    L.xq_q8_bytes.argtypes = [I, I]
    L.xq_q8_bytes.restype = S
    L.xq_weight_bytes.argtypes = [I, I, I]
    L.xq_weight_bytes.restype = S
    L.xq_quantize_q8.argtypes = [P, I, I, P, P]
    L.xq_silu_mul_quantize_q8.argtypes = [P, P, I, I, P, P, P]
    L.xq_silu_mul_quantize_q8.restype = I
    L.xq_layer_ffn_workspace_bytes.argtypes = [ctypes.POINTER(xq_proj), I, I, I, I, I, I]
    L.xq_layer_ffn_workspace_bytes.restype = S
    L.xq_layer_mixed_ffn.argtypes = [ctypes.POINTER(xq_proj), I, I, I, I, ctypes.POINTER(ctypes.c_void_p), I, I,
                                     P, S, P]
    L.xq_layer_mixed_ffn.restype = I
    L.xq_debug_stalled_ffn_layer.argtypes = L.xq_layer_mixed_ffn.argtypes
    L.xq_debug_stalled_ffn_layer.restype = I
    L.xq_q8_bytes_invariant.argtypes = [I, I]
    L.xq_q8_bytes_invariant.restype = S
    L.xq_quantize_q8_invariant.argtypes = [P, I, I, P, P]
    L.xq_quantize_q8_invariant.restype = I
    L.xq_matmul_invariant.argtypes = [I, P, P, I, I, I, P, P]
    L.xq_matmul_invariant.restype = I
    for fn in ("xq_matmul_q4k_q8", "xq_matmul_q6k_q8", "xq_matmul_q8_0_q8"):
        getattr(L, fn).argtypes = [P, P, I, I, I, P, P]
    for fn in ("xq_debug_isums_q4k", "xq_debug_isums_q6k", "xq_debug_isums_q8_0"):
        getattr(L, fn).argtypes = [P, P, I, I, I, P, P, P]
    L.xq_matmul_iq4xs_q8.argtypes = [P, P, P, I, I, I, P, P]
    L.xq_matmul_iq4xs_q8.restype = I
    L.xq_debug_isums_iq4xs.argtypes = [P, P, P, I, I, I, P, P, P]
    L.xq_debug_isums_iq4xs.restype = I
    L.xq_device_error.argtypes = [P, ctypes.POINTER(ctypes.c_uint)]
    L.xq_device_error.restype = I
    L.xq_debug_stalled_matmul_q4k.argtypes = [P, P, I, I, I, P, P]
    L.xq_debug_stalled_matmul_q4k.restype = I
    L.xq_debug_tile_sums.argtypes = [I, P, P, P, I, I, I, P, P, P]
    L.xq_debug_tile_sums.restype = I
    L.xq_layer_workspace_bytes.argtypes = [ctypes.POINTER(xq_proj), I, I, I]
    L.xq_layer_workspace_bytes.restype = S
    L.xq_layer_mixed.argtypes = [ctypes.POINTER(xq_proj), I, ctypes.POINTER(ctypes.c_void_p), I, I, P, S, P]
    L.xq_layer_mixed_static.argtypes = [ctypes.POINTER(xq_proj), I, ctypes.POINTER(ctypes.c_void_p), I, I, P]
    L.xq_debug_layer_matmuls.argtypes = [ctypes.POINTER(xq_proj), I, I, I, P, S, P]
    L.xq_debug_check_probe.argtypes = [P, P, I, I, I, P, P]
    C, Q, LL = ctypes.POINTER(xq_kv_cache), ctypes.POINTER(xq_kv_query), ctypes.c_longlong
    L.xq_kv_bytes.argtypes = [I, I, I, I, I]
    L.xq_kv_bytes.restype = S
    L.xq_kv_write.argtypes = [C, I, P, LL, P, LL, P, I, P]
    L.xq_kv_read.argtypes = [C, P, I, I, P, P, P]
    L.xq_kv_attn_workspace_bytes.argtypes = [C, Q]
    L.xq_kv_attn_workspace_bytes.restype = S
    for fn in ("xq_kv_attn", "xq_kv_attn_shared"):
        getattr(L, fn).argtypes = [C, Q, P, S, P]
    for fn in ("xq_kv_write", "xq_kv_read", "xq_kv_attn", "xq_kv_attn_shared"):
        getattr(L, fn).restype = I
    # structures as bytes, or by reference
    L.xq_lora_add.argtypes = [P, I, P, I, I, P, P]
    L.xq_qk_norm_rope.argtypes = [P, P]
    L.xq_prompt_attn_workspace_bytes.argtypes = [P]
    L.xq_prompt_attn_workspace_bytes.restype = S
    L.xq_prompt_attn.argtypes = [P, P, S, P]
    L.xq_debug_stalled_prompt_attn.argtypes = [P, P, S, ctypes.c_longlong, I, P]
    for fn in ("xq_lora_add", "xq_qk_norm_rope", "xq_prompt_attn", "xq_debug_stalled_prompt_attn"):
        getattr(L, fn).restype = I
    for fn in ("xq_quantize_q8", "xq_matmul_q4k_q8", "xq_matmul_q6k_q8", "xq_debug_isums_q4k",
               "xq_debug_isums_q6k", "xq_layer_mixed", "xq_layer_mixed_static", "xq_matmul_q8_0_q8",
               "xq_debug_isums_q8_0", "xq_debug_layer_matmuls", "xq_debug_check_probe"):
        getattr(L, fn).restype = I
    if path is None:
        _lib = L
    return L


def _check(fn: str, rc: int):
    if rc != 0:
        raise XQError(fn, rc)


def _stream(stream):
    import torch
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def q8_bytes(M: int, K: int) -> int:
    return lib().xq_q8_bytes(M, K)


def weight_bytes(qtype: int, N: int, K: int) -> int:
    return lib().xq_weight_bytes(qtype, N, K)


def quantize_q8(x, out=None, stream=None):
    """Q8-quantize fp32 x [M, K] (CUDA) into a uint8 buffer of q8_bytes(M, K)."""
    import torch
    M, K = x.shape
    if out is None:
        out = torch.empty(q8_bytes(M, K), dtype=torch.uint8, device=x.device)
    _check("xq_quantize_q8", lib().xq_quantize_q8(_ptr(x), M, K, _ptr(out), _stream(stream)))
    return out


def q8_views(xq, M: int, K: int):
    """(qs int8 [M,K], d8 fp32 [M,K/32], s8 fp32 [M,K/32]) views into an xq buffer."""
    import torch
    mk = M * K
    qs = xq[:mk].view(torch.int8).view(M, K)
    d8 = xq[mk:mk + 4 * (mk // 32)].view(torch.float32).view(M, K // 32)
    s8 = xq[mk + 4 * (mk // 32):mk + 8 * (mk // 32)].view(torch.float32).view(M, K // 32)
    return qs, d8, s8


def matmul(qtype: int, W, xq, M: int, N: int, K: int, y=None, stream=None):
    """y [M, N] fp32 = x W^T from Q8 activations xq and GGUF weight bytes W (CUDA)."""
    import torch
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=W.device)
    fn = {XQ_TYPE_Q4_K: "xq_matmul_q4k_q8", XQ_TYPE_Q6_K: "xq_matmul_q6k_q8", XQ_TYPE_Q8_0: "xq_matmul_q8_0_q8"}[qtype]
    _check(fn, getattr(lib(), fn)(_ptr(W), _ptr(xq), M, N, K, _ptr(y), _stream(stream)))
    return y


def matmul_q4k_q8(W, xq, M, N, K, y=None, stream=None):
    return matmul(XQ_TYPE_Q4_K, W, xq, M, N, K, y, stream)


def matmul_q6k_q8(W, xq, M, N, K, y=None, stream=None):
    return matmul(XQ_TYPE_Q6_K, W, xq, M, N, K, y, stream)


def _codebook(codebook):
    """16 int8 codebook values as a host buffer (read by the C call)."""
    import numpy as np
    cb = np.ascontiguousarray(codebook, dtype=np.int8)
    if cb.shape != (16,):
        raise ValueError("an IQ4_XS codebook is 16 int8 values")
    return cb


def matmul_iq4xs_q8(W, codebook, xq, M: int, N: int, K: int, y=None, stream=None):
    """y [M, N] fp32 = x W^T for IQ4_XS weight bytes W and its 16-value int8
    codebook (host array), M <= 8."""
    import torch
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=W.device)
    cb = _codebook(codebook)
    _check("xq_matmul_iq4xs_q8", lib().xq_matmul_iq4xs_q8(_ptr(W), cb.ctypes.data, _ptr(xq), M, N, K, _ptr(y),
                                                         _stream(stream)))
    return y


def debug_isums_iq4xs(W, codebook, xq, M: int, N: int, K: int, y=None, isum=None, stream=None):
    """IQ4_XS matmul that also writes the exact int32 sub-block sums [M, N, K/32]."""
    import torch
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=W.device)
    if isum is None:
        isum = torch.empty((M, N, K // 32), dtype=torch.int32, device=W.device)
    cb = _codebook(codebook)
    _check("xq_debug_isums_iq4xs", lib().xq_debug_isums_iq4xs(_ptr(W), cb.ctypes.data, _ptr(xq), M, N, K, _ptr(y),
                                                             _ptr(isum), _stream(stream)))
    return y, isum


def q8_bytes_invariant(M: int, K: int) -> int:
    return lib().xq_q8_bytes_invariant(M, K)


def quantize_q8_invariant(x, out=None, stream=None):
    """Q8-quantize fp32 x [M, K] into the 8-token GEMV image for any M (the
    batch-invariant layout)."""
    import torch
    M, K = x.shape
    if out is None:
        out = torch.empty(q8_bytes_invariant(M, K), dtype=torch.uint8, device=x.device)
    _check("xq_quantize_q8_invariant", lib().xq_quantize_q8_invariant(_ptr(x), M, K, _ptr(out), _stream(stream)))
    return out


def matmul_invariant(qtype: int, W, xq, M: int, N: int, K: int, y=None, stream=None):
    """y [M, N] = x W^T with row m independent of M (batch-invariant mode)."""
    import torch
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=W.device)
    _check("xq_matmul_invariant",
           lib().xq_matmul_invariant(qtype, _ptr(W), _ptr(xq), M, N, K, _ptr(y), _stream(stream)))
    return y


def debug_isums(qtype: int, W, xq, M: int, N: int, K: int, y=None, isum=None, stream=None):
    """Matmul that also writes the exact int32 sub-block sums (test hook)."""
    import torch
    per = K // 16 if qtype == XQ_TYPE_Q6_K else K // 32
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=W.device)
    if isum is None:
        isum = torch.empty((M, N, per), dtype=torch.int32, device=W.device)
    fn = {XQ_TYPE_Q4_K: "xq_debug_isums_q4k", XQ_TYPE_Q6_K: "xq_debug_isums_q6k",
          XQ_TYPE_Q8_0: "xq_debug_isums_q8_0"}[qtype]
    _check(fn, getattr(lib(), fn)(_ptr(W), _ptr(xq), M, N, K, _ptr(y), _ptr(isum), _stream(stream)))
    return y, isum


def device_error(stream=None) -> int:
    """Read and clear the kernels' timed-out-wait record (xq_device_error):
    0 if no bounded device wait ran out since the last read, else
    (kernel << 8) | wait."""
    code = ctypes.c_uint(0)
    _check("xq_device_error", lib().xq_device_error(_stream(stream), ctypes.byref(code)))
    return code.value


def debug_stalled_matmul_q4k(W, xq, M: int, N: int, K: int, y, stream=None):
    """Test hook: the Q4_K warp-level MMA GEMV with no stage issued and short
    waits, so that its waits run out (y stays unwritten)."""
    _check("xq_debug_stalled_matmul_q4k",
           lib().xq_debug_stalled_matmul_q4k(_ptr(W), _ptr(xq), M, N, K, _ptr(y), _stream(stream)))


def debug_tile_sums(qtype: int, W, xq, M: int, N: int, K: int, codebook=None, y=None, sums=None, stream=None):
    """Tile-kernel matmul (M > 64) that also writes each 32-block's exact
    integer as the kernel accumulates it, int32 [M, N, K/32] (test hook)."""
    import torch
    if y is None:
        y = torch.empty((M, N), dtype=torch.float32, device=W.device)
    if sums is None:
        sums = torch.empty((M, N, K // 32), dtype=torch.int32, device=W.device)
    cb = _codebook(codebook) if codebook is not None else None
    _check("xq_debug_tile_sums", lib().xq_debug_tile_sums(qtype, _ptr(W), cb.ctypes.data if cb is not None else None,
                                                         _ptr(xq), M, N, K, _ptr(y), _ptr(sums), _stream(stream)))
    return y, sums


def _proj_array(projs):
    """projs: (type, N, K, W, y, input[, codebook]) tuples; an IQ4_XS entry
    carries its 16-value int8 codebook (host array) as the 7th element."""
    arr = (xq_proj * max(1, len(projs)))()
    keep = []
    for i, p in enumerate(projs):
        arr[i].type, arr[i].N, arr[i].K = int(p[0]), int(p[1]), int(p[2])
        arr[i].W = p[3].data_ptr() if p[3] is not None else None
        arr[i].y = p[4].data_ptr() if p[4] is not None else None
        arr[i].input = int(p[5])
        cb = p[6] if len(p) > 6 else None
        if cb is not None:
            cb = _codebook(cb)
            keep.append(cb)
            arr[i].codebook = cb.ctypes.data
    arr._codebooks = keep  # host codebooks live as long as the array
    return arr


def layer_workspace_bytes(projs, n_inputs: int, M: int) -> int:
    """projs: sequence of (type, N, K, W, y, input)."""
    return lib().xq_layer_workspace_bytes(_proj_array(projs), len(projs), n_inputs, M)


def layer_mixed(projs, inputs, M: int, workspace, stream=None):
    """Run one layer's projections. projs: (type, N, K, W, y, input) tuples;
    inputs: fp32 CUDA tensors [M, K_i]; workspace: uint8 CUDA tensor."""
    arr = _proj_array(projs)
    ins = (ctypes.c_void_p * max(1, len(inputs)))(*[t.data_ptr() for t in inputs])
    rc = lib().xq_layer_mixed(arr, len(projs), ins, len(inputs), M, _ptr(workspace),
                              workspace.numel() if workspace is not None else 0, _stream(stream))
    _check("xq_layer_mixed", rc)


def debug_layer_matmuls(projs, n_inputs: int, M: int, workspace, stream=None):
    """The matmul launches of layer_mixed alone, on the Q8 activations the last
    layer_mixed call with the same projs, input count and M left in workspace."""
    arr = _proj_array(projs)
    rc = lib().xq_debug_layer_matmuls(arr, len(projs), n_inputs, M, _ptr(workspace),
                                      workspace.numel() if workspace is not None else 0, _stream(stream))
    _check("xq_debug_layer_matmuls", rc)


def silu_mul_quantize_q8(gate, up, out=None, h_out=None, stream=None):
    """Q8 of h = silu(gate) * up (fp32 CUDA tensors [M, K]); h_out optional."""
    import torch
    M, K = gate.shape
    if out is None:
        out = torch.empty(q8_bytes(M, K), dtype=torch.uint8, device=gate.device)
    _check("xq_silu_mul_quantize_q8",
           lib().xq_silu_mul_quantize_q8(_ptr(gate), _ptr(up), M, K, _ptr(out), _ptr(h_out), _stream(stream)))
    return out


def layer_ffn_workspace_bytes(projs, n_inputs: int, M: int, gate: int, up: int, down: int) -> int:
    return lib().xq_layer_ffn_workspace_bytes(_proj_array(projs), len(projs), n_inputs, M, gate, up, down)


def layer_mixed_ffn(projs, gate: int, up: int, down: int, inputs, M: int, workspace, stream=None, _fn="xq_layer_mixed_ffn"):
    """layer_mixed with projs[down] fed by silu(y_gate) * y_up of the same call."""
    arr = _proj_array(projs)
    ins = (ctypes.c_void_p * max(1, len(inputs)))(*[t.data_ptr() for t in inputs])
    rc = getattr(lib(), _fn)(arr, len(projs), gate, up, down, ins, len(inputs), M, _ptr(workspace),
                             workspace.numel() if workspace is not None else 0, _stream(stream))
    _check(_fn, rc)


def debug_stalled_ffn_layer(projs, gate: int, up: int, down: int, inputs, M: int, workspace, stream=None):
    """Test hook: layer_mixed_ffn's fused form with h never counted ready."""
    layer_mixed_ffn(projs, gate, up, down, inputs, M, workspace, stream, _fn="xq_debug_stalled_ffn_layer")


def layer_mixed_static(projs, inputs, M: int, stream=None):
    """layer_mixed without a workspace: the library's fixed per-device array
    (XQ_LAYER_STATIC_SCRATCH_BYTES) stands in for it; nothing is allocated."""
    arr = _proj_array(projs)
    ins = (ctypes.c_void_p * max(1, len(inputs)))(*[t.data_ptr() for t in inputs])
    _check("xq_layer_mixed_static", lib().xq_layer_mixed_static(arr, len(projs), ins, len(inputs), M, _stream(stream)))


class Layer:
    """Device-resident weights of one layer plus its outputs and workspace.

    Weights are uploaded once (the raw GGUF bytes stay resident; nothing is
    dequantized) and `forward` runs xq_layer_mixed on the current stream.
    adapters: {index of a projection: (a, b, scales)} of its low-rank adapters
    (see Adapters); forward's ids then name each row's.
    """

    def __init__(self, projs, weights, M: int, device="cuda", codebooks=None, adapters=None):
        import torch
        self.projs = projs
        self.M = M
        self.W = [torch.from_numpy(w.reshape(-1)).to(device) for w in weights]
        self.y = [torch.empty((M, p.N), dtype=torch.float32, device=device) for p in projs]
        n_in = 1 + max(p.input for p in projs)
        self.n_inputs = n_in
        cbs = codebooks or [None] * len(projs)  # per projection; IQ4_XS needs one
        self.desc = [(p.qtype, p.N, p.K, self.W[i], self.y[i], p.input, cbs[i]) for i, p in enumerate(projs)]
        nb = layer_workspace_bytes(self.desc, n_in, M)
        self.workspace = torch.empty(max(nb, 256), dtype=torch.uint8, device=device)
        self.adapters = None
        if adapters:
            at = sorted(adapters)
            for i in at:
                if adapters[i][0].shape[2:] != (projs[i].K,) or adapters[i][1].shape[1:2] != (projs[i].N,):
                    raise ValueError(f"adapters of projection {i}: K = {projs[i].K} and N = {projs[i].N} expected")
            self.adapters = Adapters([(*adapters[i], projs[i].input) for i in at])
            self.adapted = [self.y[i] for i in at]

    def forward(self, inputs, stream=None, ids=None):
        """The projections' outputs; with ids int32 [M], each row's adapter (negative: none) added to them."""
        if ids is not None and self.adapters is None:
            raise ValueError("the layer has no adapters")
        # refused or not, before the projections write y
        call = None if ids is None else self.adapters._call(inputs, self.adapted, ids, stream)
        layer_mixed(self.desc, inputs, self.M, self.workspace, stream)
        if call is not None:
            self.adapters._launch(call)
        return self.y

    def weight_bytes(self) -> int:
        return sum(synth.weight_bytes(p.qtype, p.N, p.K) for p in self.projs)


def kv_bytes(qtype: int, n_pages: int, page_size: int, heads: int, dim: int) -> int:
    return lib().xq_kv_bytes(qtype, n_pages, page_size, heads, dim)


_FLOAT_TYPES = {}


def _float_type(dtype):
    if not _FLOAT_TYPES:
        import torch
        _FLOAT_TYPES.update({torch.float32: XQ_TYPE_F32, torch.float16: XQ_TYPE_F16, torch.bfloat16: XQ_TYPE_BF16})
    try:
        return _FLOAT_TYPES[dtype]
    except KeyError:
        raise ValueError(f"float32, float16 or bfloat16 expected, got {dtype}") from None


class KVCache:
    """Paged K and V of one layer, quantized as they are written.

    qtype is XQ_TYPE_Q8_0 or XQ_TYPE_Q4_0. The pools are uint8 tensors of
    kv_bytes(...) bytes each (k, v: existing ones; otherwise zeroed ones are
    made). Token slot s is row s % page_size of page s // page_size; which
    pages belong to which sequence is the caller's: attn takes a page table.
    The pools' device has to be the current one when a call is made.

    A call that needs a workspace uses one that the object keeps for each
    stream; one that is captured into a CUDA graph takes its own from the
    graph's memory. Pass `workspace` (uint8, at least attn_workspace_bytes)
    to use another. Results and workspaces that a call makes belong to the
    stream that the call runs on, the current one or `stream`.
    """

    def __init__(self, qtype: int, n_pages: int, page_size: int, heads: int, dim: int, device="cuda", k=None, v=None):
        import torch
        self._torch = torch
        nb = kv_bytes(qtype, n_pages, page_size, heads, dim)
        if nb == 0 and n_pages != 0:
            raise XQError("xq_kv_bytes", 2)
        self.k = torch.zeros(nb, dtype=torch.uint8, device=device) if k is None else k
        self.v = torch.zeros(nb, dtype=torch.uint8, device=device) if v is None else v
        for pool in (self.k, self.v):
            if pool.dtype != torch.uint8 or pool.numel() < nb or not pool.is_contiguous():
                raise ValueError(f"a pool is a contiguous uint8 tensor of {nb} bytes")
        self.device = self.k.device
        if self.v.device != self.device:
            raise ValueError("both pools have to be on one device")
        self.qtype, self.n_pages, self.page_size, self.heads, self.dim = qtype, n_pages, page_size, heads, dim
        self._desc = xq_kv_cache(qtype, n_pages, page_size, heads, dim, self.k.data_ptr(), self.v.data_ptr())
        self._ref = ctypes.byref(self._desc)
        self._inner = (dim, 1)
        L = self._lib = lib()
        self._write, self._read = L.xq_kv_write, L.xq_kv_read
        self._empty, self._int32, self._int64 = torch.empty, torch.int32, torch.int64
        self._device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        self._current = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self._capturing = torch.cuda.is_current_stream_capturing
        self._ws = {}   # stream -> (workspace, bytes, address)
        self._need = {}  # sizes of a call -> workspace bytes

    def _stream(self, stream):
        # kernels go to the current device, whatever device the pointers are of
        if self._device() != self.device.index:
            raise ValueError(f"the cache is on {self.device}: make that the current device (torch.cuda.device)")
        # the current stream's handle: torch's accessor of the bare handle costs a fortieth of building a Stream object
        if stream is None:
            return self._current(self.device.index) if self._current else self._torch.cuda.current_stream(self.device).cuda_stream
        return stream if isinstance(stream, int) else stream.cuda_stream

    def write(self, k, v, slots, stream=None):
        """Quantize rows k, v [tokens, heads, dim] into slots int64 [tokens]
        (negative ones are skipped). A token's row is contiguous; rows may be
        a part of longer ones (k.stride(0))."""
        n, dev = slots.shape[0], self.device
        shape, ks, vs = (n, self.heads, self.dim), k.stride(), v.stride()
        rows = ks[1:] == self._inner == vs[1:] or (self.heads == 1 and ks[2:] == (1,) == vs[2:])  # (one head's stride says nothing)
        if k.shape != shape or v.shape != shape or k.dtype != v.dtype or not rows:
            raise ValueError(f"k and v: {shape} of one dtype, each token's row contiguous")
        if slots.dtype != self._int64 or slots.dim() != 1 or not slots.is_contiguous():
            raise ValueError("slots: contiguous int64 [tokens]")
        if k.device != dev or v.device != dev or slots.device != dev:
            raise ValueError(f"k, v and slots have to be on {dev}")
        rc = self._write(self._ref, _float_type(k.dtype), k.data_ptr(), ks[0], v.data_ptr(), vs[0], slots.data_ptr(), n,
                         self._stream(stream))
        if rc:
            raise XQError("xq_kv_write", rc)

    def read(self, slots, dtype=None, k=None, v=None, stream=None):
        """The rows of slots int64 [tokens] as floats: (k, v), each
        [tokens, heads, dim] of dtype (float32)."""
        if stream is not None and (k is None or v is None):
            on = self._on(stream)
            if on:
                with on:
                    return self.read(slots, dtype, k, v)
        if slots.dtype != self._int64 or slots.dim() != 1 or not slots.is_contiguous():
            raise ValueError("slots: contiguous int64 [tokens]")
        n, dev = slots.shape[0], self.device
        if slots.device != dev:
            raise ValueError(f"slots have to be on {dev}")
        shape = (n, self.heads, self.dim)
        if dtype is None:
            dtype = self._torch.float32 if k is None else k.dtype
        kind = _float_type(dtype)
        if k is None:
            k = self._empty(shape, dtype=dtype, device=dev)
        elif k.shape != shape or k.dtype != dtype or not k.is_contiguous() or k.device != dev:
            raise ValueError(f"k: contiguous {shape} of {dtype} on {dev}")
        if v is None:
            v = self._empty(shape, dtype=dtype, device=dev)
        elif v.shape != shape or v.dtype != dtype or not v.is_contiguous() or v.device != dev:
            raise ValueError(f"v: contiguous {shape} of {dtype} on {dev}")
        rc = self._read(self._ref, slots.data_ptr(), n, kind, k.data_ptr(), v.data_ptr(), self._stream(stream))
        if rc:
            raise XQError("xq_kv_read", rc)
        return k, v

    def attn_workspace_bytes(self, dtype, batch: int, n_q: int, heads: int, max_pages: int, prefix_len: int = 0) -> int:
        q = xq_kv_query(type=_float_type(dtype), batch=batch, n_q=n_q, heads=heads, max_pages=max_pages,
                        page_stride=max_pages, prefix_len=prefix_len)
        nb = self._lib.xq_kv_attn_workspace_bytes(self._ref, ctypes.byref(q))
        if nb == 0:
            raise XQError("xq_kv_attn_workspace_bytes", 2)
        return nb

    def _on(self, stream):
        """Context that makes `stream` the current one, for a call that makes memory: the allocator hands a stream's freed
        memory to the same stream without waiting, so it has to be the stream that writes it. None if it is the current one."""
        handle = self._stream(stream)
        if handle == self._stream(None):
            return None
        cuda = self._torch.cuda
        return cuda.stream(cuda.ExternalStream(handle, device=self.device) if isinstance(stream, int) else stream)

    def _workspace(self, key, handle):
        """(tensor, bytes, address) of a workspace of at least what calls of these sizes (the arguments of
        attn_workspace_bytes) need on the current stream: its own, kept from call to call and replaced by a larger one, or,
        while the stream is captured, a new one. A graph keeps the address it was captured with: its memory must be the graph's (it
        stays the graph's when the tensor is dropped), and not the next graph's too."""
        need = self._need.get(key)
        if need is None:
            if len(self._need) >= 1024:  # a prefix that grows gives new sizes without end
                self._need.clear()
            need = self._need[key] = self.attn_workspace_bytes(*key)
        capturing = self._capturing()
        ws = None if capturing else self._ws.get(handle)
        if ws is None or ws[1] < need:
            t = self._empty(need, dtype=self._torch.uint8, device=self.device)
            ws = (t, need, t.data_ptr())
            if not capturing:
                self._ws[handle] = ws
        return ws

    def _attn(self, fn, q, pages, lens, scale, window, prefix_pages, prefix_len, out, workspace, stream):
        if stream is not None and (out is None or workspace is None):
            on = self._on(stream)
            if on:
                with on:
                    return self._attn(fn, q, pages, lens, scale, window, prefix_pages, prefix_len, out, workspace, None)
        dev, int32, shape = self.device, self._int32, q.shape
        if len(shape) != 4 or shape[3] != self.dim or not q.is_contiguous():
            raise ValueError(f"q: contiguous [batch, n_q, heads, {self.dim}]")
        batch, n_q, heads, dim = shape
        ps, pshape = pages.stride(), pages.shape
        if pages.dtype != int32 or len(pshape) != 2 or pshape[0] != batch or (ps[1] != 1 and pshape[1] > 1):
            raise ValueError("pages: int32 [batch, pages], each row contiguous")
        if lens.dtype != int32 or lens.shape != (batch,) or not lens.is_contiguous():
            raise ValueError("lens: contiguous int32 [batch]")
        if q.device != dev or pages.device != dev or lens.device != dev:
            raise ValueError(f"q, pages and lens have to be on {dev}")
        if out is None:
            out = self._empty(shape, dtype=q.dtype, device=dev)
        elif out.shape != shape or out.dtype != q.dtype or not out.is_contiguous() or out.device != dev:
            raise ValueError("out: a contiguous tensor like q")
        prefix = None
        if prefix_pages is not None:
            if (prefix_pages.dtype != int32 or prefix_pages.dim() != 1 or not prefix_pages.is_contiguous()
                    or prefix_pages.shape[0] * self.page_size < prefix_len or prefix_pages.device != dev):
                raise ValueError(f"prefix_pages: contiguous int32 ids of the prefix's pages, on {dev}")
            prefix = prefix_pages.data_ptr()
        s, width, dtype = self._stream(stream), pshape[1], q.dtype
        if workspace is None:
            held, ws_bytes, ws = self._workspace((dtype, batch, n_q, heads, width, prefix_len), s)
        else:
            ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
            if workspace.device != dev or not workspace.is_contiguous():
                raise ValueError(f"workspace: contiguous, on {dev}")
        # ctypes keeps the low 32 bits of an int: a larger window would become another one
        window = window if window < 0x7FFFFFFF else 0x7FFFFFFF
        if prefix_len > 0x7FFFFFFF or window < -0x80000000:
            raise XQError(fn.__name__, 2)
        query = xq_kv_query(_float_type(dtype), batch, n_q, heads, q.data_ptr(), out.data_ptr(), pages.data_ptr(),
                            ps[0] if batch > 1 else width, width, lens.data_ptr(), dim ** -0.5 if scale is None else scale, window,
                            prefix, prefix_len)
        rc = fn(self._ref, query, ws, ws_bytes, s)
        if rc:
            raise XQError(fn.__name__, rc)
        return out

    def attn(self, q, pages, lens, scale=None, window: int = 0, out=None, workspace=None, stream=None):
        """Attention of q [batch, n_q, heads, dim], the last n_q tokens of
        each sequence, over lens int32 [batch] tokens (those n_q among them)
        in the pages int32 [batch, max_pages]. scale: 1 / sqrt(dim). window:
        how many keys a query sees at most, 0 for all."""
        return self._attn(self._lib.xq_kv_attn, q, pages, lens, scale, window, None, 0, out, workspace, stream)

    def attn_shared(self, q, prefix_pages, prefix_len: int, pages, lens, scale=None, out=None, workspace=None, stream=None):
        """attn for sequences that all begin with the prefix_len tokens in
        prefix_pages int32 [pages]; pages and lens are of the tokens after it."""
        return self._attn(self._lib.xq_kv_attn_shared, q, pages, lens, scale, 0, prefix_pages, prefix_len, out, workspace,
                          stream)


_torch_calls = None


def _calls():
    """(torch, current device, raw stream of a device) accessors: the bare handle's costs a fortieth of building a Stream object."""
    global _torch_calls
    if _torch_calls is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _torch_calls = (torch, getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device),
                        raw or (lambda d: torch.cuda.current_stream(d).cuda_stream))
    return _torch_calls


def _handle(device, stream):
    """The stream's handle, for tensors on CUDA device number `device` (get_device; -1: none). Kernels go to the current device,
    whatever device the pointers are of."""
    _, current, raw = _torch_calls or _calls()
    if device < 0 or current() != device:
        raise ValueError("CUDA tensors on the current device expected (torch.cuda.device)")
    if stream is None:
        return raw(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _other_stream(device, stream):
    """Context that makes `stream` the current one, for a call that makes memory: the allocator hands a stream's freed memory
    to the same stream without waiting, so it has to be the stream that writes it. None if it is the current one."""
    handle = _handle(device, stream)
    if handle == _handle(device, None):
        return None
    cuda = _calls()[0].cuda
    return cuda.stream(cuda.ExternalStream(handle, device=device) if isinstance(stream, int) else stream)


# Structures of the C ABI as bytes: packing them costs a third of filling ctypes fields.
_ADAPTERS = "iiiii4xPPPPi4x"
_pack_rows = struct.Struct("@iiiiiiPPqqPPqqPPf4xPPiif4x").pack
_pack_prompts = struct.Struct("@iiiiiiPPPqqqPPfi").pack


class Adapters:
    """Low-rank adapters of projections that run together.

    projs: (a, b, scales, input) of each projection: a [n, rank, K] and b
    [n, N, rank] of one dtype (float32, float16 or bfloat16), scales fp32 [n]
    or None, and which of `add`'s inputs it takes. The tensors are kept.
    """

    def __init__(self, projs):
        torch = _calls()[0]
        if not 1 <= len(projs) <= 16:
            raise ValueError("1 to 16 projections a call")
        self._device = dev = projs[0][0].get_device()
        self._keep, self._shapes, self._args, self._aligned = [], [], [], True
        for a, b, scales, inp in projs:
            if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2] or a.dtype != b.dtype:
                raise ValueError("a: [n, rank, K], b: [n, N, rank], of one dtype")
            if not a.is_contiguous() or not b.is_contiguous() or dev < 0 or a.get_device() != dev or b.get_device() != dev:
                raise ValueError("a and b have to be contiguous, on one CUDA device")
            n, rank, K = a.shape
            if scales is not None and (scales.dtype != torch.float32 or scales.shape != (n,) or not scales.is_contiguous()
                                       or scales.get_device() != dev):
                raise ValueError(f"scales: contiguous float32 [{n}], on the adapters' device")
            if rank % 8 or not 8 <= rank <= 256 or K % 32 or K == 0:
                raise ValueError(f"rank a multiple of 8 up to 256 and K a multiple of 32 expected, got {rank} and {K}")
            if not 0 <= inp < 64 or n > 8192:
                raise ValueError("an input's index is 0 to 63, and there are at most 8192 adapters")
            self._args += [_float_type(a.dtype), n, rank, K, b.shape[1], a.data_ptr(), b.data_ptr(),
                           0 if scales is None else scales.data_ptr(), 0, inp]
            self._aligned &= b.shape[1] == 0 or (a.data_ptr() | b.data_ptr()) % 16 == 0
            self._keep.append((a, b, scales))
            self._shapes.append(((b.shape[1],), (K,), inp))
        self._pack = struct.Struct("@" + _ADAPTERS * len(projs)).pack
        self._n_inputs = 1 + max(p[3] for p in projs)
        self._pack_inputs = struct.Struct(f"@{self._n_inputs}P").pack
        self._add = lib().xq_lora_add
        self._float32, self._int32 = torch.float32, torch.int32

    def add(self, inputs, ys, ids, stream=None):
        """Add to each row of the projections' outputs ys (fp32 [M, N] each) what the adapter that ids int32 [M] names gives
        for the row of its input (fp32 [M, K]); rows of a negative id are left as they are. Returns ys."""
        self._launch(self._call(inputs, ys, ids, stream))
        return ys

    def _call(self, inputs, ys, ids, stream):
        """The arguments of a call that nothing is wrong with."""
        dev, f32, rows = self._device, self._float32, tuple(ids.shape)
        if len(rows) != 1 or ids.dtype != self._int32 or not ids.is_contiguous() or ids.get_device() != dev:
            raise ValueError("ids: contiguous int32 [M], on the adapters' device")
        if len(ys) != len(self._shapes) or len(inputs) < self._n_inputs:
            raise ValueError(f"{len(self._shapes)} outputs and {self._n_inputs} inputs expected, got {len(ys)} and {len(inputs)}")
        args, ins, at, odd = self._args.copy(), [0] * self._n_inputs, 8, 0  # a call's own: calls may run side by side
        for y, (N, K, inp) in zip(ys, self._shapes):
            x = inputs[inp]
            if x.shape != rows + K or x.dtype != f32 or not x.is_contiguous() or x.get_device() != dev:
                raise ValueError(f"input {inp}: contiguous float32 {[*rows, *K]}, on the adapters' device")
            if y.shape != rows + N or y.dtype != f32 or not y.is_contiguous() or y.get_device() != dev:
                raise ValueError(f"an output: contiguous float32 {[*rows, *N]}, on the adapters' device")
            args[at], ins[inp] = y.data_ptr(), x.data_ptr()
            at += 10
            odd |= x.data_ptr() & 15 if N[0] else 0
        if rows[0] and (odd or not self._aligned):
            raise XQError("xq_lora_add", 3)  # not on a 16-byte boundary
        return (self._pack(*args), len(ys), self._pack_inputs(*ins), self._n_inputs, rows[0], ids.data_ptr(), _handle(dev, stream))

    def _launch(self, call):
        rc = self._add(*call)
        if rc:
            raise XQError("xq_lora_add", rc)


def _turns(base, rot, factors):
    """base^(-2i / rot) / factors[i] radians as parts of a full turn in units of 2^-64, to the nearest one. With 64-bit floats they had
    53 bits, and an angle at position 2^40 was off by 1.6e-4."""
    import decimal

    import numpy as np
    with np.errstate(all="ignore"):
        freq = np.float64(base) ** (np.arange(0, rot, 2, dtype=np.float64) / -max(rot, 1))
        if factors is not None:
            freq = freq / factors
    if not np.isfinite(freq).all():
        raise ValueError("base and factors have to give finite frequencies")
    # 64 bits behind the point, whatever is before it
    digits = 45 + max([0, *(math.frexp(f)[1] * 3 // 10 + 1 for f in freq.tolist())])
    with decimal.localcontext(decimal.Context(prec=digits, Emin=decimal.MIN_EMIN, Emax=decimal.MAX_EMAX)) as ctx:
        D = decimal.Decimal

        def arctan(n):  # of 1 / n
            total = term = D(1) / n
            k = 1
            while abs(term) > D(10) ** -ctx.prec:
                term /= -n * n
                k += 2
                total += term / k
            return total

        over_turn = D(2) ** 64 / (8 * (4 * arctan(5) - arctan(239)))  # 2^64 / (2 pi), Machin's formula
        # base^(-2 / rot), and its powers one from the other: they lose three digits of 25 that are not needed
        step = (-2 * D(float(base)).ln() / rot).exp() if rot and math.isfinite(base) else D(0)
        turns, power = [], D(1)
        for i, f in enumerate(freq.tolist()):
            exact = D(0) if f == 0.0 else power / (D(1) if factors is None else D(float(factors[i]))) * over_turn
            turns.append(int(exact.to_integral_value(decimal.ROUND_HALF_EVEN)) % (1 << 64))
            power *= step
    return turns


class Rope:
    """Position rotation: the first `rot` elements of a head turn in rot / 2 pairs, pair i by base^(-2i / rot) radians a
    position, divided by factors[i] if given. pairs: neighbouring elements (2i, 2i + 1) make a pair, otherwise (i, i + rot / 2).
    magnitude: factor of the rotated elements. The table's angles are rounded to 2^-64 of a turn a position, which is all that is
    lost at far positions."""

    def __init__(self, rot: int, base: float = 10000.0, factors=None, pairs: bool = False, magnitude: float = 1.0, device="cuda"):
        import numpy as np
        torch = _calls()[0]
        if rot < 0 or rot % 16:
            raise ValueError("rot: a multiple of 16")
        if factors is not None:
            factors = np.asarray(factors.cpu() if hasattr(factors, "cpu") else factors, dtype=np.float64)
            if factors.shape != (rot // 2,):
                raise ValueError(f"{rot // 2} factors expected")
        self.rot, self.pairs, self.magnitude = rot, bool(pairs), float(magnitude)
        turns = [(t + (1 << 63)) % (1 << 64) - (1 << 63) for t in _turns(float(base), rot, factors)]
        self.turns = torch.tensor(turns, dtype=torch.int64, device=device)
        self._device, self._at = self.turns.get_device(), self.turns.data_ptr()


def _rows_of(x, shape, dtype, device):
    """The stride between tokens of x [tokens, heads, dim], each token's rows contiguous."""
    st = x.stride()
    if x.shape != shape or x.dtype != dtype or x.get_device() != device or st[2] != 1 or (st[1] != shape[2] and shape[1] > 1):
        raise ValueError(f"{tuple(shape)} of {dtype} expected on the call's device, each token's rows contiguous")
    return st[0]


def qk_norm_rope(q, k, positions, rope, q_weight=None, k_weight=None, eps: float = 1e-6, dtype=None, q_out=None, k_out=None,
                 stream=None):
    """Each head's row of q [tokens, heads, dim] and k [tokens, kv_heads, dim] normalized (x * weight / sqrt(mean(x^2) + eps);
    not without a weight) and rotated to its position (int64 [tokens]). A token's rows are contiguous; tokens may be parts of
    longer rows. Returns (q_out, k_out) of `dtype` (the inputs'); an output may be its input."""
    dev = q.get_device()
    if stream is not None and (q_out is None or k_out is None):
        on = _other_stream(dev, stream)
        if on:
            with on:
                return qk_norm_rope(q, k, positions, rope, q_weight, k_weight, eps, dtype, q_out, k_out)
    torch, kind, qs, ks = _calls()[0], q.dtype, q.shape, k.shape
    if len(qs) != 3 or len(ks) != 3 or ks[0] != qs[0] or ks[2] != qs[2]:
        raise ValueError("q: [tokens, heads, dim], k: [tokens, kv_heads, dim]")
    T, H, D = qs
    q_stride, k_stride = _rows_of(q, qs, kind, dev), _rows_of(k, ks, kind, dev)
    if positions.dtype != torch.int64 or positions.shape != (T,) or not positions.is_contiguous() or positions.get_device() != dev:
        raise ValueError(f"positions: contiguous int64 [{T}], on the call's device")
    for w in (q_weight, k_weight):
        if w is not None and (w.dtype != torch.float32 or w.shape != (D,) or not w.is_contiguous() or w.get_device() != dev):
            raise ValueError(f"weights: contiguous float32 [{D}], on the call's device")
    if rope._device != dev:
        raise ValueError("the rotation's table has to be on the call's device")
    handle = _handle(dev, stream)
    if dtype is None:
        dtype = kind if q_out is None else q_out.dtype
    y_type = _float_type(dtype)
    if q_out is None:
        q_out, q_out_stride = torch.empty(qs, dtype=dtype, device=q.device), H * D
    else:
        q_out_stride = _rows_of(q_out, qs, dtype, dev)
    if k_out is None:
        k_out, k_out_stride = torch.empty(ks, dtype=dtype, device=q.device), ks[1] * D
    else:
        k_out_stride = _rows_of(k_out, ks, dtype, dev)
    rc = lib().xq_qk_norm_rope(
        _pack_rows(_float_type(kind), y_type, T, H, ks[1], D, q.data_ptr(), k.data_ptr(), q_stride, k_stride, q_out.data_ptr(),
                   k_out.data_ptr(), q_out_stride, k_out_stride, 0 if q_weight is None else q_weight.data_ptr(),
                   0 if k_weight is None else k_weight.data_ptr(), eps, positions.data_ptr(), rope._at, rope.rot, rope.pairs,
                   rope.magnitude), handle)
    if rc:
        raise XQError("xq_qk_norm_rope", rc)
    return q_out, k_out


_prompt_need = {}  # sizes of a call -> workspace bytes


def prompt_attn(q, k, v, starts, scale=None, window: int = 0, out=None, workspace=None, stream=None, _hook=None):
    """Causal attention of packed prompts: q [tokens, heads, dim], k and v [tokens, kv_heads, dim]; sequence b is rows
    starts[b] .. starts[b + 1] - 1 (starts int32 [batch + 1]). A token's rows are contiguous; tokens may be parts of longer
    rows. scale: 1 / sqrt(dim). window: how many keys a query sees at most, 0 for all. Returns out [tokens, heads, dim]; its
    rows that belong to no sequence are not written."""
    dev, kind = q.get_device(), q.dtype
    if stream is not None and (out is None or workspace is None):
        on = _other_stream(dev, stream)
        if on:
            with on:
                return prompt_attn(q, k, v, starts, scale, window, out, workspace, _hook=_hook)
    torch, qs, ks = _calls()[0], q.shape, k.shape
    if len(qs) != 3 or len(ks) != 3 or ks[0] != qs[0] or ks[2] != qs[2]:
        raise ValueError("q: [tokens, heads, dim], k and v: [tokens, kv_heads, dim]")
    T, H, D = qs
    q_stride, k_stride, v_stride = _rows_of(q, qs, kind, dev), _rows_of(k, ks, kind, dev), _rows_of(v, ks, kind, dev)
    if starts.dtype != torch.int32 or starts.dim() != 1 or starts.shape[0] < 1 or not starts.is_contiguous() or starts.get_device() != dev:
        raise ValueError("starts: contiguous int32 [batch + 1], on the call's device")
    handle, x_type, batch = _handle(dev, stream), _float_type(kind), starts.shape[0] - 1
    if out is None:
        out = torch.empty(qs, dtype=kind, device=q.device)
    elif out.shape != qs or out.dtype != kind or not out.is_contiguous() or out.get_device() != dev:
        raise ValueError(f"out: contiguous {tuple(qs)} of {kind}, on the call's device")
    # a larger window than an int holds is no window
    if not 0 <= window:
        raise XQError("xq_prompt_attn", 2)
    p = _pack_prompts(x_type, T, batch, H, ks[1], D, q.data_ptr(), k.data_ptr(), v.data_ptr(), q_stride, k_stride, v_stride,
                      out.data_ptr(), starts.data_ptr(), D ** -0.5 if scale is None else scale, min(window, 0x7FFFFFFF))
    L = lib()
    if workspace is None:
        sizes = (x_type, T, batch, H, ks[1], D)
        need = _prompt_need.get(sizes)
        if need is None:
            if len(_prompt_need) >= 1024:
                _prompt_need.clear()
            need = _prompt_need[sizes] = L.xq_prompt_attn_workspace_bytes(p)
        ws = torch.empty(need, dtype=torch.uint8, device=q.device) if need > 16 else None
        at, size = (ws.data_ptr(), need) if need > 16 else (None, 0)
    else:
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace: contiguous, on the call's device")
        at, size = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    rc = L.xq_prompt_attn(p, at, size, handle) if _hook is None else L.xq_debug_stalled_prompt_attn(p, at, size, *_hook, handle)
    if rc:
        raise XQError("xq_prompt_attn", rc)
    return out


def debug_stalled_prompt_attn(q, k, v, starts, clocks: int, withhold: bool, **kw):
    """Test hook: prompt_attn with `clocks` for the 2^32 of its waits' limit, and with withhold without its first copies, so that the
    waits run out (see xq_debug_stalled_prompt_attn)."""
    return prompt_attn(q, k, v, starts, _hook=(clocks, int(withhold)), **kw)

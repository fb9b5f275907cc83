"""Python binding of libmoe_mi355x.so: the routed MoE expert-FFN hot path
and the paged key-value cache and attention beside it, on MI355X (gfx950).

Argument marshalling only. Every step of the path runs in the library's HIP
kernels; torch supplies device memory (tensors) and the current stream. The
functions carry the C names (moe_route, moe_permute, moe_quantize_act_fp8,
moe_quantize_act_mxfp8,
moe_grouped_gemm1_act, moe_grouped_gemm2_combine, moe_forward,
moe_attn_decode, moe_attn_prefill, moe_cache_append, ...), take
torch tensors for the arrays, and raise MoeError on a negative status.
There is no fallback: without the built library every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
from ctypes import POINTER, c_float, c_int, c_long, c_size_t, c_void_p
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_mi355x.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "moe_mi355x.h")

MOE_W_BF16, MOE_W_FP8_B128, MOE_W_INT4_G32, MOE_W_NVFP4, MOE_W_MXFP4 = 0, 1, 2, 3, 4
MOE_W_MXFP4_A8 = 5
_PACKED4 = (MOE_W_INT4_G32, MOE_W_NVFP4, MOE_W_MXFP4, MOE_W_MXFP4_A8)
MOE_DEVERR_GLOBAL_ID_OOB = 0x1
MOE_DEVERR_F16_RANGE = 0x2
MOE_DEVERR_W4_SCALE = 0x4
MOE_DEVERR_CACHE_PAGE = 0x8
MOE_DEVERR_CACHE_FULL = 0x10
MOE_DEVERR_CACHE_BUSY = 0x20
MOE_KV_BF16, MOE_KV_F16, MOE_KV_E4M3 = 0, 1, 2
STATUS = {0: "MOE_OK", -1: "MOE_ERR_NULL", -2: "MOE_ERR_SHAPE",
          -3: "MOE_ERR_FORMAT", -4: "MOE_ERR_LOCAL_RANGE", -5: "MOE_ERR_PARAM",
          -6: "MOE_ERR_WORKSPACE", -8: "MOE_ERR_HIP", -9: "MOE_ERR_SCRATCH"}
MOE_SCRATCH_BYTES = 32 << 20


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str, msg: str):
        super().__init__(f"{where}: {STATUS.get(status, status)} ({msg})")
        self.status = status


class MoeActParams(ctypes.Structure):
    _fields_ = [("alpha", c_float), ("beta", c_float), ("limit", c_float)]


class MoeWeights(ctypes.Structure):
    _fields_ = [("fmt", c_int), ("n_groups", c_int), ("N", c_int), ("K", c_int),
                ("q", c_void_p), ("scale", c_void_p), ("gscale", c_void_p)]


class MoeLora(ctypes.Structure):
    _fields_ = [("rank", c_int), ("n_groups", c_int), ("scale", c_float),
                ("A", c_void_p), ("B", c_void_p), ("n_adapters", c_int),
                ("adapter_ids", c_void_p)]


class MoeLayer(ctypes.Structure):
    _fields_ = [("H", c_int), ("I", c_int), ("num_experts_global", c_int),
                ("num_local_experts", c_int), ("local_expert_offset", c_int),
                ("shared_expert", c_int), ("top_k", c_int), ("n_sink", c_int),
                ("route_scale", c_float), ("global_scale", c_float),
                ("shared_w", c_float), ("w13", MoeWeights), ("w2", MoeWeights),
                ("act", MoeActParams), ("lora", POINTER(MoeLora)),
                ("lora_down", POINTER(MoeLora))]


class MoeKvCache(ctypes.Structure):
    _fields_ = [("fmt", c_int), ("n_pages", c_int), ("page_size", c_int),
                ("n_heads", c_int), ("head_dim", c_int), ("stride_page", c_long),
                ("stride_head", c_long), ("stride_tok", c_long), ("k", c_void_p),
                ("v", c_void_p), ("k_scale", c_void_p), ("v_scale", c_void_p)]


class MoeKvTable(ctypes.Structure):
    _fields_ = [("n_slots", c_int), ("max_pages", c_int), ("ld", c_long),
                ("n_pages", c_int), ("page_size", c_int), ("table", c_void_p),
                ("len", c_void_p), ("refs", c_void_p)]


class MoeAttn(ctypes.Structure):
    _fields_ = [("fmt", c_int), ("n_heads", c_int), ("q", c_void_p),
                ("q_stride_row", c_long), ("q_stride_head", c_long),
                ("out", c_void_p), ("out_stride_row", c_long),
                ("out_stride_head", c_long), ("lse", c_void_p), ("scale", c_float),
                ("window", c_int), ("n_first", c_int)]


_lib = None

_SIGS = {
    "moe_route": (c_int, [c_void_p, c_long, c_long, c_int, c_int, c_int, c_void_p,
                          c_float, c_float, c_void_p, c_void_p, c_void_p, c_void_p,
                          c_void_p]),
    "moe_gate_route_workspace_size": (c_size_t, [c_long, c_int, c_int, c_int]),
    "moe_gate_route": (c_int, [c_void_p, c_void_p, c_long, c_int, c_int, c_int, c_int,
                               c_void_p, c_float, c_float, c_void_p, c_void_p,
                               c_void_p, c_void_p, c_void_p, c_void_p, c_size_t,
                               c_void_p]),
    "moe_permute": (c_int, [c_void_p, c_long, c_int, c_int, c_int, c_int, c_int,
                            c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                            c_size_t, c_void_p]),
    "moe_permute_workspace_size": (c_size_t, [c_long, c_int, c_int]),
    "moe_quantize_act_fp8": (c_int, [c_void_p, c_long, c_int, c_void_p, c_void_p,
                                     c_void_p]),
    "moe_quantize_act_mxfp8": (c_int, [c_void_p, c_long, c_int, c_void_p, c_void_p,
                                       c_void_p]),
    "moe_grouped_gemm1_act": (c_int, [POINTER(MoeWeights), c_void_p, c_void_p,
                                      c_void_p, c_long, c_int, c_int, c_int,
                                      c_long, c_void_p, c_void_p,
                                      POINTER(MoeActParams), POINTER(MoeLora),
                                      c_void_p, c_void_p, c_void_p, c_void_p,
                                      c_void_p, c_size_t, c_void_p]),
    "moe_gemm1_workspace_size": (c_size_t, [POINTER(MoeWeights), c_long, POINTER(MoeLora)]),
    "moe_grouped_gemm2_combine": (c_int, [POINTER(MoeWeights), c_void_p, c_void_p,
                                          c_void_p, POINTER(MoeLora),
                                          c_long, c_int, c_int, c_int, c_int,
                                          c_long, c_void_p, c_void_p, c_void_p,
                                          c_void_p, c_float, c_void_p, c_void_p,
                                          c_void_p, c_size_t, c_void_p]),
    "moe_gemm2_workspace_size": (c_size_t, [POINTER(MoeWeights), c_long,
                                            POINTER(MoeLora)]),
    "moe_forward": (c_int, [POINTER(MoeLayer), c_void_p, c_void_p, c_long, c_long,
                            c_void_p, c_void_p, c_void_p, c_void_p, c_void_p,
                            c_void_p, c_size_t, c_void_p]),
    "moe_workspace_size": (c_size_t, [POINTER(MoeLayer), c_long]),
    "moe_forward_no_workspace": (c_int, [POINTER(MoeLayer), c_void_p, c_void_p, c_long,
                                         c_long, c_void_p, c_void_p, c_void_p, c_void_p,
                                         c_void_p, c_void_p]),
    "moe_scratch_error": (ctypes.c_char_p, []),
    "moe_attn_decode": (c_int, [POINTER(MoeKvCache), POINTER(MoeKvTable), c_void_p, c_long,
                                POINTER(MoeAttn), c_void_p, c_void_p, c_size_t,
                                c_void_p]),
    "moe_attn_decode_workspace_size": (c_size_t, [POINTER(MoeKvCache), c_long, c_int]),
    "moe_attn_prefill": (c_int, [POINTER(MoeKvCache), POINTER(MoeKvTable), c_void_p, c_long,
                                 c_void_p, c_long, POINTER(MoeAttn), c_void_p, c_void_p,
                                 c_size_t, c_void_p]),
    "moe_attn_prefill_workspace_size": (c_size_t, [POINTER(MoeKvCache), c_long, c_long,
                                                   c_int]),
    "moe_cache_append": (c_int, [POINTER(MoeKvCache), POINTER(MoeKvTable), c_void_p,
                                 c_void_p, c_void_p, c_long, c_long, c_int, c_void_p,
                                 c_long, c_long, c_void_p, c_long, c_long, c_void_p,
                                 c_void_p]),
    "moe_cache_grow": (c_int, [POINTER(MoeKvTable), c_void_p, c_void_p, c_long, c_void_p,
                               c_void_p, c_void_p, c_size_t, c_void_p]),
    "moe_cache_free": (c_int, [POINTER(MoeKvTable), c_void_p, c_long, c_void_p, c_void_p]),
    "moe_cache_trim": (c_int, [POINTER(MoeKvTable), c_void_p, c_long, c_int, c_int,
                               c_void_p, c_void_p]),
    "moe_cache_fork": (c_int, [POINTER(MoeKvCache), c_int, POINTER(MoeKvTable), c_void_p,
                               c_void_p, c_long, c_void_p, c_void_p, c_size_t, c_void_p]),
    "moe_cache_compact": (c_int, [POINTER(MoeKvCache), c_int, POINTER(MoeKvTable), c_void_p,
                                  c_void_p, c_void_p, c_size_t, c_void_p]),
    "moe_cache_copy_pages": (c_int, [POINTER(MoeKvCache), c_int, c_void_p, c_void_p, c_long,
                                     c_void_p, c_void_p]),
    "moe_cache_workspace_size": (c_size_t, [POINTER(MoeKvTable), c_long]),
    "moe_read_device_error": (c_int, [c_void_p, POINTER(c_int), c_void_p]),
    "moe_status_string": (ctypes.c_char_p, [c_int]),
    "moe_last_error": (ctypes.c_char_p, []),
}


def lib():
    """The loaded C library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with "
                "`python -m mixture_experts_expert_sigmoid_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream):
    """The hipStream_t to enqueue on: the current device's current stream if
    None (asked of torch directly; building a Stream object for it costs more
    than a kernel launch)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _check(status: int, where: str):
    if status != 0:
        L = lib()
        raise MoeError(status, where, L.moe_status_string(status).decode()
                       + ("; " + L.moe_last_error().decode() if status == -8 else ""))


# ---------------------------------------------------------------- descriptors

def weights(fmt: int, q: torch.Tensor, scale: Optional[torch.Tensor] = None,
            gscale: Optional[torch.Tensor] = None) -> MoeWeights:
    """Descriptor of a stacked [G][N][K] weight (4-bit formats: q is
    [G][N][K/2]). gscale: W13 [G][2] (gate, up), W2 [G] (FP4 formats)."""
    G, N, Kq = q.shape
    K = 2 * Kq if fmt in _PACKED4 else Kq
    w = MoeWeights(fmt, G, N, K, q.data_ptr(),
                   None if scale is None else scale.data_ptr(),
                   None if gscale is None else gscale.data_ptr())
    w._keep = (q, scale, gscale)
    return w


def act_params(alpha=1.0, beta=0.0, limit=math.inf) -> MoeActParams:
    return MoeActParams(alpha, beta, limit)


def lora_desc(A: torch.Tensor, B: torch.Tensor, scale=1.0,
              adapter_ids: Optional[torch.Tensor] = None) -> MoeLora:
    """A [G][r][K] (one adapter) or [n_adapters][G][r][K] (a batch, with
    per-token adapter_ids int32 [T] set here or per call)."""
    na = 1 if A.dim() == 3 else A.shape[0]
    G, r = A.shape[-3], A.shape[-2]
    d = MoeLora(r, G, scale, A.data_ptr(), B.data_ptr(), na,
                None if adapter_ids is None else adapter_ids.data_ptr())
    d._keep = (A, B, adapter_ids)
    return d


def layer_desc(H, I, num_experts_global, num_local_experts, local_expert_offset,
               shared_expert, top_k, n_sink, route_scale, global_scale, shared_w,
               w13: MoeWeights, w2: MoeWeights, act: MoeActParams,
               lora: Optional[MoeLora] = None,
               lora_down: Optional[MoeLora] = None) -> MoeLayer:
    L = MoeLayer(H, I, num_experts_global, num_local_experts, local_expert_offset,
                 shared_expert, top_k, n_sink, route_scale, global_scale,
                 shared_w, w13, w2, act, _lp(lora), _lp(lora_down))
    L._keep = (w13, w2, lora, lora_down)
    return L


# ------------------------------------------------------------ entry points

def moe_route(logits, n_routed, n_sink, top_k, route_scale, global_scale,
              topk_ids, topk_w, sink_w=None, stream=None, sel_bias=None,
              packed=None):
    T, ld = logits.shape
    _check(lib().moe_route(_p(logits), T, logits.stride(0), n_routed, n_sink,
                           top_k, _p(sel_bias), route_scale, global_scale,
                           _p(topk_ids), _p(topk_w), _p(sink_w), _p(packed),
                           _stream(stream)), "moe_route")


def moe_gate_route_workspace_size(T, H, n_routed, n_sink) -> int:
    return lib().moe_gate_route_workspace_size(T, H, n_routed, n_sink)


def moe_gate_route(x_bf16, wg_bf16, n_routed, n_sink, top_k, route_scale,
                   global_scale, topk_ids, topk_w, sink_w=None, sel_bias=None,
                   logits=None, packed=None, ws=None, stream=None):
    T, H = x_bf16.shape
    _check(lib().moe_gate_route(_p(x_bf16), _p(wg_bf16), T, H, n_routed, n_sink,
                                top_k, _p(sel_bias), route_scale, global_scale,
                                _p(logits), _p(topk_ids), _p(topk_w), _p(sink_w),
                                _p(packed), _p(ws),
                                0 if ws is None else ws.numel() * ws.element_size(),
                                _stream(stream)), "moe_gate_route")


def moe_permute_workspace_size(T, top_k, n_groups) -> int:
    return lib().moe_permute_workspace_size(T, top_k, n_groups)


def moe_permute(topk_ids, top_k, num_experts_global, local_expert_offset,
                num_local_experts, shared_expert, offsets, sorted_pair, pair_row,
                err_word, ws, stream=None):
    T = topk_ids.shape[0]
    _check(lib().moe_permute(_p(topk_ids), T, top_k, num_experts_global,
                             local_expert_offset, num_local_experts,
                             shared_expert, _p(offsets), _p(sorted_pair),
                             _p(pair_row), _p(err_word), _p(ws),
                             ws.numel() * ws.element_size(), _stream(stream)),
           "moe_permute")


def moe_quantize_act_fp8(x_bf16, xq, xs, stream=None):
    T, H = x_bf16.shape
    _check(lib().moe_quantize_act_fp8(_p(x_bf16), T, H, _p(xq), _p(xs),
                                      _stream(stream)), "moe_quantize_act_fp8")


def moe_quantize_act_mxfp8(x_bf16, xq, xe, stream=None):
    T, H = x_bf16.shape
    _check(lib().moe_quantize_act_mxfp8(_p(x_bf16), T, H, _p(xq), _p(xe),
                                        _stream(stream)), "moe_quantize_act_mxfp8")


def moe_gemm1_workspace_size(w13: MoeWeights, p_cap, lora: Optional[MoeLora] = None) -> int:
    return lib().moe_gemm1_workspace_size(
        ctypes.byref(w13), p_cap, ctypes.pointer(lora) if lora is not None else None)


def _lp(lora):
    return ctypes.pointer(lora) if lora is not None else None


def moe_grouped_gemm1_act(w13: MoeWeights, x, xs, x_bf16, T, H, I, top_k, p_cap,
                          offsets, sorted_pair, act: MoeActParams,
                          lora: Optional[MoeLora], h, hs, ws, stream=None,
                          h_lora=None, err_word=None):
    _check(lib().moe_grouped_gemm1_act(
        ctypes.byref(w13), _p(x), _p(xs), _p(x_bf16), T, H, I, top_k, p_cap,
        _p(offsets), _p(sorted_pair), ctypes.byref(act), _lp(lora), _p(h), _p(hs),
        _p(h_lora), _p(err_word), _p(ws),
        0 if ws is None else ws.numel() * ws.element_size(),
        _stream(stream)), "moe_grouped_gemm1_act")


def moe_gemm2_workspace_size(w2: MoeWeights, p_cap,
                             lora_down: Optional[MoeLora] = None) -> int:
    return lib().moe_gemm2_workspace_size(ctypes.byref(w2), p_cap, _lp(lora_down))


def moe_grouped_gemm2_combine(w2: MoeWeights, h, hs, T, H, I, top_k,
                              shared_expert, p_cap, offsets, pair_row, topk_w,
                              shared_w, out, ws, stream=None, h_lora=None,
                              lora_down: Optional[MoeLora] = None, sorted_pair=None,
                              err_word=None):
    _check(lib().moe_grouped_gemm2_combine(
        ctypes.byref(w2), _p(h), _p(hs), _p(h_lora), _lp(lora_down), T, H, I,
        top_k, shared_expert, p_cap, _p(offsets), _p(sorted_pair), _p(pair_row),
        _p(topk_w), shared_w, _p(out), _p(err_word), _p(ws),
        ws.numel() * ws.element_size(), _stream(stream)), "moe_grouped_gemm2_combine")


def moe_workspace_size(layer: MoeLayer, T_max) -> int:
    n = lib().moe_workspace_size(ctypes.byref(layer), T_max)
    if n == 0:
        raise MoeError(-2, "moe_workspace_size", "invalid layer descriptor")
    return n


def moe_forward(layer: MoeLayer, x_bf16, logits, out, topk_ids, topk_w, sink_w,
                err_word, ws, stream=None):
    T = x_bf16.shape[0]
    _check(lib().moe_forward(ctypes.byref(layer), _p(x_bf16), _p(logits), T,
                             logits.stride(0), _p(out), _p(topk_ids), _p(topk_w),
                             _p(sink_w), _p(err_word), _p(ws),
                             ws.numel() * ws.element_size(), _stream(stream)),
           "moe_forward")


def moe_forward_no_workspace(layer: MoeLayer, x_bf16, logits, out, topk_ids, topk_w,
                             sink_w, err_word, stream=None):
    """moe_forward with the library's static device scratch as workspace."""
    T = x_bf16.shape[0]
    L = lib()
    st = L.moe_forward_no_workspace(ctypes.byref(layer), _p(x_bf16), _p(logits), T,
                                    logits.stride(0), _p(out), _p(topk_ids), _p(topk_w),
                                    _p(sink_w), _p(err_word), _stream(stream))
    if st == -9:
        raise MoeError(st, "moe_forward_no_workspace", L.moe_scratch_error().decode())
    _check(st, "moe_forward_no_workspace")


def moe_read_device_error(err_word, stream=None) -> int:
    bits = c_int(0)
    _check(lib().moe_read_device_error(_p(err_word), ctypes.byref(bits),
                                       _stream(stream)), "moe_read_device_error")
    return bits.value


# ------------------------------------------------- key-value cache, attention

_KV_FMT = {torch.bfloat16: MOE_KV_BF16, torch.float16: MOE_KV_F16,
           torch.float8_e4m3fn: MOE_KV_E4M3}


_INT32 = torch.int32


def _kv_fmt(t: torch.Tensor, where: str) -> int:
    fmt = _KV_FMT.get(t.dtype)
    if fmt is None:
        raise MoeError(-3, where, f"dtype {t.dtype}")
    return fmt


def _on_gpu(where: str, *tensors: Optional[torch.Tensor]):
    """The kernels take addresses: one of host memory would fault the GPU."""
    for t in tensors:
        if t is not None and not t.is_cuda:
            raise MoeError(-5, where, f"tensor {tuple(t.shape)} is on the device {t.device}")


def _i32(t: Optional[torch.Tensor], n: int, where: str):
    """Pointer of a contiguous int32 list of at least n entries (or None)."""
    if t is None:
        return None
    if t.dtype is not _INT32 or t.numel() < n or not t.is_contiguous():
        raise MoeError(-2, where, f"wants {n} contiguous int32, got {t.dtype} "
                                  f"{tuple(t.shape)}")
    if not t.is_cuda:
        _on_gpu(where, t)
    return t.data_ptr()


def _err(t: Optional[torch.Tensor], where: str):
    """Pointer of an error word."""
    if t is not None and t.dtype is _INT32 and t.is_cuda and t.numel():
        return t.data_ptr()
    return _i32(t, 1, where)


def _work(ws: Optional[torch.Tensor], where: str):
    """Pointer and bytes of a workspace."""
    if ws is None:
        return None, 0
    if not (ws.is_cuda and ws.is_contiguous()):
        _on_gpu(where, ws)
        raise MoeError(-2, where, "the workspace is not contiguous")
    return ws.data_ptr(), ws.nbytes


def kv_cache(k: torch.Tensor, v: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
             v_scale: Optional[torch.Tensor] = None) -> MoeKvCache:
    """Descriptor of one layer's cache: k and v [pages][heads][page_size][head_dim]
    of bfloat16, float16 or float8_e4m3fn (with scales [heads] fp32), of any
    strides alike in both but with rows of head_dim contiguous; a cache laid
    out [pages][page_size][heads][head_dim] is passed as its transpose(1, 2)."""
    if k.shape != v.shape or k.dtype != v.dtype or k.dim() != 4:
        raise MoeError(-2, "kv_cache", "k and v differ in shape or type")
    P, H, ps, D = k.shape
    # a dimension of one entry has no stride of its own: one that a dense cache
    # would have stands for it
    strides = [(x.stride(0) if P > 1 else H * ps * D, x.stride(1) if H > 1 else D, x.stride(2),
                x.stride(3)) for x in (k, v)]
    if strides[0] != strides[1]:
        raise MoeError(-2, "kv_cache", "k and v differ in strides")
    if strides[0][3] != 1:
        raise MoeError(-2, "kv_cache", "rows of head_dim are not contiguous")
    for sc in (k_scale, v_scale):
        if sc is not None and (sc.dtype != torch.float32 or sc.numel() != k.shape[1]
                               or not sc.is_contiguous()):
            raise MoeError(-2, "kv_cache", "scales are fp32 [heads]")
    _on_gpu("kv_cache", k, v, k_scale, v_scale)
    c = MoeKvCache(_kv_fmt(k, "kv_cache"), P, ps, H, D, *strides[0][:3], k.data_ptr(),
                   v.data_ptr(), None if k_scale is None else k_scale.data_ptr(),
                   None if v_scale is None else v_scale.data_ptr())
    c._keep = (k, v, k_scale, v_scale)
    return c


def kv_table(table: torch.Tensor, lens: torch.Tensor, page_size: int, n_pages: int,
             refs: Optional[torch.Tensor] = None) -> MoeKvTable:
    """Descriptor of the page tables: table int32 [slots][max_pages], lens int32
    [slots], refs int32 [n_pages] (for grow, free, trim, fork, compact)."""
    if table.dtype != torch.int32 or table.dim() != 2 or table.stride(1) != 1:
        raise MoeError(-2, "kv_table", "table is int32 [slots][max_pages], rows contiguous")
    _on_gpu("kv_table", table)
    ld = table.stride(0) if table.shape[0] > 1 else table.shape[1]
    t = MoeKvTable(table.shape[0], table.shape[1], ld, n_pages, page_size, table.data_ptr(),
                   _i32(lens, table.shape[0], "kv_table"),
                   None if refs is None else _i32(refs, n_pages, "kv_table"))
    t._keep = (table, lens, refs)
    return t


def _rows(t: torch.Tensor, where: str, shape, D: int):
    """Strides (row, head) of a [rows][heads][head_dim] tensor. A dimension of
    one entry has no stride of its own."""
    st = t.stride()
    if len(st) != 3 or shape[2] != D or st[2] != 1 or t.shape != shape:
        raise MoeError(-2, where, f"wants {tuple(shape)} of [rows][heads][{D}] with contiguous "
                                  f"rows, got {tuple(t.shape)} strides {st}")
    if not t.is_cuda:
        _on_gpu(where, t)
    if shape[0] > 1 and shape[1] > 1:
        return st
    return (st[0] if shape[0] > 1 else shape[1] * D), (st[1] if shape[1] > 1 else D)


def _attn(where, cache: MoeKvCache, shape, q, out, scale, window, n_first, lse) -> MoeAttn:
    D, fmt = cache.head_dim, _KV_FMT.get(q.dtype)
    if out.dtype is not q.dtype:
        raise MoeError(-2, where, "out and q differ in type")
    if fmt is None:
        raise MoeError(-3, where, f"dtype {q.dtype}")
    qs, os_ = _rows(q, where, shape, D), _rows(out, where, shape, D)
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != shape[:2]
                            or not lse.is_contiguous() or not lse.is_cuda):
        _on_gpu(where, lse)
        raise MoeError(-2, where, "lse is fp32 [rows][heads], contiguous")
    return MoeAttn(fmt, shape[1], q.data_ptr(), qs[0], qs[1], out.data_ptr(), os_[0], os_[1],
                   None if lse is None else lse.data_ptr(), scale, window, n_first)


def moe_attn_decode_workspace_size(cache: MoeKvCache, n: int, n_heads: int) -> int:
    return lib().moe_attn_decode_workspace_size(cache, n, n_heads)


def moe_attn_decode(cache: MoeKvCache, table: MoeKvTable, q, out, scale, err_word, ws, *,
                    window=0, n_first=0, slots=None, lse=None, stream=None):
    """One new token per sequence: q and out [n][heads][head_dim], lse [n][heads]."""
    where = "moe_attn_decode"
    shape = q.shape
    a, n = _attn(where, cache, shape, q, out, scale, window, n_first, lse), shape[0]
    _check(lib().moe_attn_decode(cache, table, _i32(slots, n, where), n, a,
                                 _err(err_word, where), *_work(ws, where),
                                 _stream(stream)), where)


def moe_attn_prefill_workspace_size(cache: MoeKvCache, n: int, T: int, n_heads: int) -> int:
    return lib().moe_attn_prefill_workspace_size(cache, n, T, n_heads)


def moe_attn_prefill(cache: MoeKvCache, table: MoeKvTable, q, cu_q, out, scale, err_word, ws,
                     *, window=0, n_first=0, slots=None, lse=None, stream=None):
    """The newest tokens of n = len(cu_q) - 1 sequences: q and out
    [T][heads][head_dim], lse [T][heads]."""
    where = "moe_attn_prefill"
    shape = q.shape
    a = _attn(where, cache, shape, q, out, scale, window, n_first, lse)
    n = cu_q.numel() - 1
    _check(lib().moe_attn_prefill(cache, table, _i32(slots, n, where), n,
                                  _i32(cu_q, 1, where), shape[0], a, _err(err_word, where),
                                  *_work(ws, where), _stream(stream)), where)


def moe_cache_append(cache: MoeKvCache, table: MoeKvTable, start, cu, k, v, err_word, *,
                     slots=None, stream=None):
    """k and v [T][heads][head_dim] to positions start[i].. of the slots; cu int32
    [n + 1], or None for one token each."""
    where = "moe_cache_append"
    shape, D = k.shape, cache.head_dim
    T = shape[0]
    n = T if cu is None else cu.numel() - 1
    if v.dtype is not k.dtype or (T and shape[1] != cache.n_heads):
        raise MoeError(-2, where, "k and v differ in type, or their heads from the cache's")
    ks, vs = _rows(k, where, shape, D), _rows(v, where, shape, D)
    _check(lib().moe_cache_append(
        cache, table, _i32(slots, n, where), _i32(start, n, where), _i32(cu, 1, where), n, T,
        _kv_fmt(k, where), _p(k), ks[0], ks[1], _p(v), vs[0], vs[1], _err(err_word, where),
        _stream(stream)), where)


def moe_cache_workspace_size(table: MoeKvTable, n: int) -> int:
    return lib().moe_cache_workspace_size(table, n)


def moe_cache_grow(table: MoeKvTable, slots, n_new, start, err_word, ws, stream=None):
    where = "moe_cache_grow"
    n = n_new.numel()
    _check(lib().moe_cache_grow(table, _i32(slots, n, where),
                                _i32(n_new, n, where), n, _i32(start, n, where),
                                _err(err_word, where), *_work(ws, where),
                                _stream(stream)), where)


def moe_cache_free(table: MoeKvTable, slots, err_word, stream=None):
    where = "moe_cache_free"
    n = slots.numel()
    _check(lib().moe_cache_free(table, _i32(slots, n, where), n,
                                _err(err_word, where), _stream(stream)), where)


def moe_cache_trim(table: MoeKvTable, slots, window, n_first, err_word, stream=None):
    where = "moe_cache_trim"
    n = slots.numel()
    _check(lib().moe_cache_trim(table, _i32(slots, n, where), n, window, n_first,
                                _err(err_word, where), _stream(stream)), where)


def _layers(caches):
    return (MoeKvCache * len(caches))(*caches)


def moe_cache_fork(caches, table: MoeKvTable, src, dst, err_word, ws, stream=None):
    """caches: the MoeKvCache of every layer."""
    where = "moe_cache_fork"
    n = src.numel()
    _check(lib().moe_cache_fork(_layers(caches), len(caches), table,
                                _i32(src, n, where), _i32(dst, n, where), n,
                                _err(err_word, where), *_work(ws, where),
                                _stream(stream)), where)


def moe_cache_compact(caches, table: MoeKvTable, n_used, err_word, ws, stream=None):
    where = "moe_cache_compact"
    _check(lib().moe_cache_compact(_layers(caches), len(caches), table,
                                   _i32(n_used, 1, where), _err(err_word, where),
                                   *_work(ws, where), _stream(stream)), where)


def moe_cache_copy_pages(caches, src, dst, err_word, stream=None):
    where = "moe_cache_copy_pages"
    n = src.numel()
    _check(lib().moe_cache_copy_pages(_layers(caches), len(caches), _i32(src, n, where),
                                      _i32(dst, n, where), n, _err(err_word, where),
                                      _stream(stream)), where)


class _Workspace:
    """A workspace that grows. Every buffer handed out is kept: a graph captured
    with it goes on writing there, and so may work on another stream. Each is at
    least twice the one before it, so all of them together take at most twice
    the last."""

    def __init__(self, device):
        self.device, self.buffers = device, []

    def get(self, need: int) -> torch.Tensor:
        if not self.buffers or self.buffers[-1].numel() < need:
            last = self.buffers[-1].numel() if self.buffers else 0
            self.buffers.append(torch.empty(max(need, 2 * last, 16), dtype=torch.uint8,
                                            device=self.device))
        return self.buffers[-1]


class KvCache:
    """A paged cache of several layers with its tables: device tensors, their
    descriptors and a workspace. Slots are handed in as int32 device tensors.
    Everything is enqueued on `stream` (the current one if None); calls on
    different streams have to be ordered by the caller, as they share the
    tables and the workspace. Graphs captured through the object hold its
    addresses, so it has to outlive them; later calls, larger ones too, leave
    what they use in place. Problems found on the device are ORed into
    err_word."""

    def __init__(self, *, n_layers, n_pages, page_size, n_heads, head_dim, n_slots, max_pages,
                 dtype=torch.bfloat16, k_scale=None, v_scale=None, device="cuda"):
        shape = (n_layers, n_pages, n_heads, page_size, head_dim)
        self.k = torch.empty(shape, dtype=dtype, device=device)
        self.v = torch.empty(shape, dtype=dtype, device=device)
        i32 = dict(dtype=torch.int32, device=device)
        self.table = torch.full((n_slots, max_pages), -1, **i32)
        self.lens = torch.zeros(n_slots, **i32)
        self.refs = torch.zeros(n_pages, **i32)
        self.err_word = torch.zeros(1, **i32)
        # scales: [n_layers][n_heads], for float8_e4m3fn
        self.layers = [kv_cache(self.k[i], self.v[i], None if k_scale is None else k_scale[i],
                                None if v_scale is None else v_scale[i])
                       for i in range(n_layers)]
        self.desc = kv_table(self.table, self.lens, page_size, n_pages, self.refs)
        self._scales = [t for t in (k_scale, v_scale) if t is not None]
        self._ws = _Workspace(self.k.device)
        self._streams = {}                       # those that work was enqueued on

    def _on(self, stream):
        """Tells the allocator, once per stream, that this stream uses the
        object's tensors, so that none is given back while its work runs."""
        raw = _stream(stream)
        if raw not in self._streams:
            self._streams[raw] = s = torch.cuda.current_stream() if stream is None else stream
            for t in (self.k, self.v, self.table, self.lens, self.refs, self.err_word,
                      *self._scales, *self._ws.buffers):
                t.record_stream(s)

    def _new(self, like, stream):
        """An empty tensor like `like`, contiguous, of the stream it is used on."""
        with torch.cuda.stream(stream):
            return torch.empty_like(like, memory_format=torch.contiguous_format)

    def workspace(self, need, stream=None):
        """At least `need` bytes for work on `stream`."""
        self._on(stream)
        held = len(self._ws.buffers)
        with torch.cuda.stream(stream):
            ws = self._ws.get(need)
        if len(self._ws.buffers) > held:
            for s in self._streams.values():
                ws.record_stream(s)
        return ws

    def grow(self, slots, n_new, stream=None):
        """Room for n_new more tokens of each slot; returns their first positions
        (-1 where there was none)."""
        start = self._new(n_new, stream)
        ws = self.workspace(moe_cache_workspace_size(self.desc, n_new.numel()), stream)
        moe_cache_grow(self.desc, slots, n_new, start, self.err_word, ws, stream)
        return start

    def append(self, layer, slots, start, cu, k, v, stream=None):
        self._on(stream)
        moe_cache_append(self.layers[layer], self.desc, start, cu, k, v, self.err_word,
                         slots=slots, stream=stream)

    def decode(self, layer, slots, q, scale, out=None, window=0, n_first=0, lse=None,
               stream=None):
        out = self._new(q, stream) if out is None else out
        c = self.layers[layer]
        ws = self.workspace(moe_attn_decode_workspace_size(c, q.shape[0], q.shape[1]), stream)
        moe_attn_decode(c, self.desc, q, out, scale, self.err_word, ws, window=window,
                        n_first=n_first, slots=slots, lse=lse, stream=stream)
        return out

    def prefill(self, layer, slots, q, cu_q, scale, out=None, window=0, n_first=0, lse=None,
                stream=None):
        out = self._new(q, stream) if out is None else out
        c = self.layers[layer]
        ws = self.workspace(moe_attn_prefill_workspace_size(c, cu_q.numel() - 1, q.shape[0],
                                                            q.shape[1]), stream)
        moe_attn_prefill(c, self.desc, q, cu_q, out, scale, self.err_word, ws, window=window,
                         n_first=n_first, slots=slots, lse=lse, stream=stream)
        return out

    def free(self, slots, stream=None):
        self._on(stream)
        moe_cache_free(self.desc, slots, self.err_word, stream)

    def trim(self, slots, window, n_first=0, stream=None):
        self._on(stream)
        moe_cache_trim(self.desc, slots, window, n_first, self.err_word, stream)

    def fork(self, src, dst, stream=None):
        ws = self.workspace(moe_cache_workspace_size(self.desc, src.numel()), stream)
        moe_cache_fork(self.layers, self.desc, src, dst, self.err_word, ws, stream)

    def compact(self, n_used=None, stream=None):
        ws = self.workspace(moe_cache_workspace_size(self.desc, 0), stream)
        moe_cache_compact(self.layers, self.desc, n_used, self.err_word, ws, stream)


# ------------------------------------------------------------ layer object

class MoeModule:
    """Device tensors of one layer plus its descriptor; forward() allocates
    the outputs and a workspace with torch and calls moe_forward."""

    def __init__(self, *, fmt, H, I, num_experts_global, top_k, w13_q, w2_q,
                 w13_s=None, w2_s=None, gscale=None, gscale2=None,
                 num_local_experts=None,
                 local_expert_offset=0, shared_expert=0, n_sink=0,
                 route_scale=1.0, global_scale=1.0, shared_w=1.0, alpha=1.0,
                 beta=0.0, limit=math.inf, lora_A=None, lora_B=None,
                 lora_scale=1.0, lora_A2=None, lora_B2=None):
        self.fmt, self.H, self.I, self.top_k, self.n_sink = fmt, H, I, top_k, n_sink
        self.shared_expert = shared_expert
        E_loc = num_experts_global if num_local_experts is None else num_local_experts
        self.w13 = weights(fmt, w13_q, w13_s, gscale)
        self.w2 = weights(fmt, w2_q, w2_s, gscale2)
        self.act = act_params(alpha, beta, limit)
        self.lora = lora_desc(lora_A, lora_B, lora_scale) if lora_A is not None else None
        self.lora_down = (lora_desc(lora_A2, lora_B2, lora_scale)
                          if lora_A2 is not None else None)
        self.desc = layer_desc(H, I, num_experts_global, E_loc, local_expert_offset,
                               shared_expert, top_k, n_sink, route_scale,
                               global_scale, shared_w, self.w13, self.w2, self.act,
                               self.lora, self.lora_down)
        self._ws = None

    def workspace(self, T):
        need = moe_workspace_size(self.desc, T)
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        return self._ws

    def alloc_outputs(self, T):
        dev = "cuda"
        return dict(
            out=torch.empty(T, self.H, dtype=torch.float32, device=dev),
            topk_ids=torch.empty(T, self.top_k, dtype=torch.int32, device=dev),
            topk_w=torch.empty(T, self.top_k, dtype=torch.float32, device=dev),
            sink_w=(torch.empty(T, self.n_sink, dtype=torch.float32, device=dev)
                    if self.n_sink else None),
            err_word=torch.zeros(1, dtype=torch.int32, device=dev))

    def set_adapters(self, adapter_ids: Optional[torch.Tensor]):
        """Per-token adapter ids (int32 [T], -1 none) for a batch of adapters."""
        for d in (self.lora, self.lora_down):
            if d is not None and d.n_adapters > 1:
                d.adapter_ids = None if adapter_ids is None else adapter_ids.data_ptr()
                d._keep = d._keep[:2] + (adapter_ids,)

    def forward(self, x_bf16, logits, outs=None, stream=None, adapter_ids=None):
        T = x_bf16.shape[0]
        if adapter_ids is not None:
            self.set_adapters(adapter_ids)
        o = outs if outs is not None else self.alloc_outputs(T)
        moe_forward(self.desc, x_bf16, logits, o["out"], o["topk_ids"], o["topk_w"],
                    o["sink_w"], o["err_word"], self.workspace(T), stream)
        return o

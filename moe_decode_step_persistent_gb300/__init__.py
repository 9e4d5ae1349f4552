"""Python binding of libmsk.so: the persistent MoE verify-step kernels.

Argument marshalling only: every step of the verify computation runs in the
library's CUDA kernels.  PyTorch supplies device memory and streams.  There
is no CPU fallback: if the compiled library is missing, every call raises.

The entry points carry the C names (``msk_create``, ``msk_load_layer``,
``msk_layer_step``, ``msk_decode_step``, ...); :class:`Model` bundles them for
weights held in torch tensors.  The operators beside the step
(``msk_kv4_write``, ``msk_kv4_read``, ``msk_attention_kv4``, ``msk_linear_fp4``,
``msk_token_logprobs``) and those of a whole prompt's experts
(``msk_moe_route``, ``msk_moe_sort``, ``msk_quantize_fp4``,
``msk_dequantize_fp4``, ``msk_experts_fp4``, ``msk_moe_combine``) take torch
tensors, with :class:`Kv4Cache`, :class:`Fp4Weight` and :class:`Fp4Experts` as
the handles of a 4-bit cache, a 4-bit matrix and one matrix of each expert.
"""

from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "lib", "libmsk.so")

MSK_OK = 0
STATUS = {0: "ok", 1: "invalid argument", 2: "shape", 3: "alignment", 4: "bad scale",
          5: "unsupported device", 6: "out of memory", 7: "CUDA error", 8: "timeout",
          9: "not loaded"}
MSK_ERR_INVALID_ARG = 1
MSK_ERR_TIMEOUT = 8
MSK_ERR_NOT_LOADED = 9
TIMELINE_SLOTS = 64
PHASES = ["start", "pro_qkv", "attn", "combine", "oproj", "pool", "router", "topk", "gemm1",
          "gemm2", "mcomb", "unpool", "qkv", "end"]


class MskError(RuntimeError):
    def __init__(self, status, where):
        super().__init__(f"{where}: {STATUS.get(status, status)} ({status})")
        self.status = status


class ModelConfig(ctypes.Structure):
    _fields_ = [
        ("n_layers", ctypes.c_int32), ("hidden", ctypes.c_int32), ("n_q_heads", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("pooled", ctypes.c_int32),
        ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32), ("inter", ctypes.c_int32),
        ("verify_tokens", ctypes.c_int32), ("max_seq", ctypes.c_int32),
        ("prefetch_experts", ctypes.c_int32), ("layer_is_global", ctypes.POINTER(ctypes.c_uint8)),
        ("window", ctypes.c_int32), ("rms_eps", ctypes.c_float), ("rope_theta", ctypes.c_float),
        ("wait_budget_ns", ctypes.c_uint64),
    ]


class Bf16Desc(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("ld_elems", ctypes.c_int64)]


class Nvfp4Desc(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("tensor_scale", ctypes.c_float), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class LayerWeightsC(ctypes.Structure):
    _fields_ = [("attn_norm", Bf16Desc), ("moe_norm", Bf16Desc), ("w_qkv", Bf16Desc),
                ("w_o", Bf16Desc), ("w_pool", Bf16Desc), ("w_unpool", Bf16Desc),
                ("w_router", Bf16Desc), ("router_bias", ctypes.c_void_p),
                ("w_gate", ctypes.POINTER(Nvfp4Desc)), ("w_up", ctypes.POINTER(Nvfp4Desc)),
                ("w_down", ctypes.POINTER(Nvfp4Desc))]


class Kv4Desc(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("max_seq", ctypes.c_int32), ("k_scale", ctypes.c_float),
                ("v_scale", ctypes.c_float)]


class Fp4ExpertsC(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("tensor_scales", ctypes.c_void_p),
                ("n_experts", ctypes.c_int32), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("maps", ctypes.c_void_p)]


MSK_FP4_MAPS_BYTES = 384

#: every symbol include/msk.h declares
SYMBOLS = ["msk_create", "msk_load_layer", "msk_layer_step", "msk_decode_step", "msk_layer_step_tree",
           "msk_decode_step_tree", "msk_step_graph_capture", "msk_step_graph_launch", "msk_set_timing",
           "msk_get_timeline", "msk_set_launch_timing", "msk_get_launch_ms", "msk_set_wait_budget",
           "msk_set_fault_injection", "msk_debug_scratch", "msk_debug_dequant", "msk_debug_quantize", "msk_debug_convert",
           "msk_debug_fp4_gemm",
           "msk_attention_noalloc", "msk_kv4_write", "msk_kv4_read", "msk_attention_kv4_workspace",
           "msk_attention_kv4", "msk_linear_fp4", "msk_ops_check", "msk_token_logprobs",
           "msk_moe_route", "msk_moe_sort", "msk_quantize_fp4", "msk_dequantize_fp4", "msk_fp4_experts_maps", "msk_experts_fp4",
           "msk_debug_experts_fault",
           "msk_moe_combine", "msk_get_info", "msk_status_string", "msk_destroy"]

_lib = None


def load_library(path: str = LIB_PATH):
    """Loads libmsk.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libmsk.so not found at {path}: build it first "
                           "(python -m moe_decode_step_persistent_gb300.build)")
    L = ctypes.CDLL(path)
    vp, i32, i64, u64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64
    L.msk_create.argtypes = [ctypes.POINTER(ModelConfig), ctypes.POINTER(vp)]
    L.msk_load_layer.argtypes = [vp, i32, ctypes.POINTER(LayerWeightsC), vp]
    L.msk_layer_step.argtypes = [vp, i32, vp, vp, ctypes.POINTER(i32), vp, vp, i32, vp]
    L.msk_decode_step.argtypes = [vp, vp, vp, ctypes.POINTER(i32), vp, vp, vp]
    L.msk_layer_step_tree.argtypes = [vp, i32, vp, vp, i32, ctypes.POINTER(i32), vp, vp, i32, vp]
    L.msk_decode_step_tree.argtypes = [vp, vp, vp, i32, ctypes.POINTER(i32), vp, vp, vp]
    L.msk_step_graph_capture.argtypes = [vp, vp, vp, vp, vp]
    L.msk_step_graph_launch.argtypes = [vp, i32, ctypes.POINTER(i32), vp]
    L.msk_set_timing.argtypes = [vp, i32]
    L.msk_get_timeline.argtypes = [vp, ctypes.POINTER(ctypes.c_uint64), ctypes.c_size_t,
                                   ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(i32), ctypes.POINTER(i32)]
    L.msk_set_launch_timing.argtypes = [vp, i32]
    L.msk_get_launch_ms.argtypes = [vp, ctypes.POINTER(ctypes.c_float), i32, ctypes.POINTER(i32)]
    L.msk_set_wait_budget.argtypes = [vp, u64]
    L.msk_set_fault_injection.argtypes = [vp, i32, i32]
    L.msk_debug_scratch.argtypes = [vp, i32, vp, ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t), vp]
    L.msk_debug_dequant.argtypes = [vp, i32, i32, i32, vp, vp]
    L.msk_debug_quantize.argtypes = [vp, i64, i64, vp, vp, vp]
    L.msk_debug_convert.argtypes = [vp, i64, vp, vp, vp]
    L.msk_debug_fp4_gemm.argtypes = [vp, vp, vp, vp, i32, i32, vp, vp]
    L.msk_attention_noalloc.argtypes = [vp, vp, i32, i32, i32, i32, i32, i32, i32, vp, vp]
    f32, size, kv4 = ctypes.c_float, ctypes.c_size_t, ctypes.POINTER(Kv4Desc)
    L.msk_kv4_write.argtypes = [kv4, vp, vp, i32, i32, i64, i64, i32, vp, vp]
    L.msk_kv4_read.argtypes = [kv4, i32, i32, vp, vp, i32, i64, i64, vp]
    L.msk_attention_kv4_workspace.argtypes = [i32] * 6
    L.msk_attention_kv4.argtypes = [vp, i32, i64, kv4, i32, i32, i32, vp, ctypes.POINTER(i32), i32, f32, vp, vp,
                                    size, vp]
    L.msk_linear_fp4.argtypes = [vp, i32, i64, ctypes.POINTER(Nvfp4Desc), i32, vp, i32, i64, vp]
    L.msk_ops_check.argtypes = [vp]
    L.msk_token_logprobs.argtypes = [vp, i32, i64, i64, i64, vp, f32, i32, vp, vp, vp, vp, vp, vp]
    fp4, experts = ctypes.POINTER(Nvfp4Desc), ctypes.POINTER(Fp4ExpertsC)
    L.msk_moe_route.argtypes = [vp, i32, i64, i32, i64, vp, i32, vp, vp, vp]
    L.msk_moe_sort.argtypes = [vp, i64, i32, vp, vp, vp, vp]
    L.msk_quantize_fp4.argtypes = [vp, i32, i64, i64, i64, f32, vp, vp, vp]
    L.msk_dequantize_fp4.argtypes = [vp, vp, f32, i64, i64, vp, i32, i64, vp]
    L.msk_fp4_experts_maps.argtypes = [experts, vp]
    L.msk_experts_fp4.argtypes = [fp4, vp, i32, i64, vp, experts, experts, vp, i32, i64, vp]
    L.msk_debug_experts_fault.argtypes = [i32, u64]
    L.msk_moe_combine.argtypes = [vp, i32, i64, i64, vp, vp, i64, i32, i64, vp, i32, i64, vp]
    L.msk_get_info.argtypes = [vp, ctypes.POINTER(i32), ctypes.POINTER(i64)]
    L.msk_status_string.argtypes = [i32]
    L.msk_status_string.restype = ctypes.c_char_p
    L.msk_destroy.argtypes = [vp]
    L.msk_destroy.restype = None
    for name in SYMBOLS:
        if name.endswith("_workspace"):
            getattr(L, name).restype = size
        elif name not in ("msk_status_string", "msk_destroy"):
            getattr(L, name).restype = i32
    _lib = L
    return L


def _check(status, where):
    if status != MSK_OK:
        raise MskError(status, where)


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _int32(value, what):
    """`value` as an int that the C call takes as it is (ctypes drops the bits
    that do not fit)."""
    value = int(value)
    if not -0x80000000 <= value <= 0x7FFFFFFF:
        raise ValueError(f"{what} does not fit 32 bits: {value}")
    return value


def _positions(positions):
    return (ctypes.c_int32 * len(positions))(*[_int32(p, "a position") for p in positions])


# ----------------------------------------------------------------------------
# thin wrappers, same names as the C ABI
# ----------------------------------------------------------------------------


def msk_create(cfg: ModelConfig) -> ctypes.c_void_p:
    L = load_library()
    h = ctypes.c_void_p()
    _check(L.msk_create(ctypes.byref(cfg), ctypes.byref(h)), "msk_create")
    return h


def msk_load_layer(handle, layer, weights: LayerWeightsC, stream=None):
    _check(load_library().msk_load_layer(handle, layer, ctypes.byref(weights), _stream(stream)), "msk_load_layer")


def msk_layer_step(handle, layer, hidden, kv_cache, positions, prev_routing=None, routing_out=None,
                   run_prologue=False, stream=None):
    return load_library().msk_layer_step(handle, layer, _ptr(hidden), _ptr(kv_cache), _positions(positions),
                                         _ptr(prev_routing), _ptr(routing_out), int(run_prologue), _stream(stream))


def msk_decode_step(handle, hidden, kv_cache, positions, prev_routing=None, routing_out=None, stream=None):
    return load_library().msk_decode_step(handle, _ptr(hidden), _ptr(kv_cache), _positions(positions),
                                          _ptr(prev_routing), _ptr(routing_out), _stream(stream))


def msk_layer_step_tree(handle, layer, hidden, kv_cache, cache_len, parents, prev_routing=None, routing_out=None,
                        run_prologue=False, stream=None):
    return load_library().msk_layer_step_tree(handle, layer, _ptr(hidden), _ptr(kv_cache), int(cache_len),
                                              _positions(parents), _ptr(prev_routing), _ptr(routing_out),
                                              int(run_prologue), _stream(stream))


def msk_decode_step_tree(handle, hidden, kv_cache, cache_len, parents, prev_routing=None, routing_out=None,
                         stream=None):
    return load_library().msk_decode_step_tree(handle, _ptr(hidden), _ptr(kv_cache), int(cache_len),
                                               _positions(parents), _ptr(prev_routing), _ptr(routing_out),
                                               _stream(stream))


def msk_step_graph_capture(handle, hidden, kv_cache, prev_routing=None, routing_out=None):
    return load_library().msk_step_graph_capture(handle, _ptr(hidden), _ptr(kv_cache), _ptr(prev_routing),
                                                 _ptr(routing_out))


def msk_step_graph_launch(handle, cache_len, parents=None, stream=None):
    par = None if parents is None else _positions(parents)
    return load_library().msk_step_graph_launch(handle, int(cache_len), par, _stream(stream))


def msk_debug_dequant(handle, layer, expert, which, out, stream=None):
    _check(load_library().msk_debug_dequant(handle, layer, expert, which, _ptr(out), _stream(stream)),
           "msk_debug_dequant")


def msk_debug_quantize(x, codes, scales, stream=None):
    _check(load_library().msk_debug_quantize(_ptr(x), x.shape[0], x.shape[1], _ptr(codes), _ptr(scales),
                                             _stream(stream)), "msk_debug_quantize")


def msk_debug_convert(x, e2m1, e4m3, stream=None):
    _check(load_library().msk_debug_convert(_ptr(x), x.numel(), _ptr(e2m1), _ptr(e4m3), _stream(stream)),
           "msk_debug_convert")


def msk_debug_fp4_gemm(a_codes, a_scales, b_codes, b_scales, d, stream=None):
    """d[128][16] = A B^T on the tensor cores (block-scaled NVFP4; see
    include/msk.h).  a_codes [128][K/2], a_scales [128][K/16], b_codes
    [n][K/2], b_scales [n][K/16] uint8; d [128][16] fp32.  Returns the status."""
    return load_library().msk_debug_fp4_gemm(_ptr(a_codes), _ptr(a_scales), _ptr(b_codes), _ptr(b_scales),
                                             b_codes.shape[0], a_codes.shape[1] * 2, _ptr(d), _stream(stream))


def msk_attention_noalloc(q, kv_layer, pos0, window, out, stream=None):
    """Standalone split-KV attention that allocates no device memory (its
    scratch is a fixed array inside the library): for callers that cannot
    allocate at the point of the call.  q: [T][Hq][d] bf16; kv_layer:
    [2][Hkv][max_seq][d] bf16; out: [T][Hq*d] bf16.  Returns the status."""
    T, Hq, d = q.shape
    Hkv, max_seq = kv_layer.shape[1], kv_layer.shape[2]
    return load_library().msk_attention_noalloc(_ptr(q), _ptr(kv_layer), T, Hq, Hkv, d, max_seq, int(pos0),
                                                int(window), _ptr(out), _stream(stream))


def msk_destroy(handle):
    load_library().msk_destroy(handle)


# ----------------------------------------------------------------------------
# operators beside the step
# ----------------------------------------------------------------------------

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _need(ok, what):
    if not ok:
        raise ValueError(what)


#: the current stream's handle without the Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _enqueue(stream, *tensors):
    """The stream handle of a call on these tensors, which all live on the
    current device."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError(f"every tensor must live on the current CUDA device (cuda:{dev}), got one on {t.device}")
    return _raw_stream(dev) if stream is None else stream.cuda_stream


def _empty(stream, shape, dtype):
    """A new tensor on the current device for a call on `stream`: taken from
    that stream's memory pool, so that freeing it is ordered after the call."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device="cuda")
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device="cuda")


def _workspace(given, need, stream):
    """(tensor kept alive over the call, address, bytes)."""
    if given is None:
        if need == 0:
            return None, None, 0
        given = _empty(stream, need, torch.uint8)
        return given, given.data_ptr(), need
    _need(given.is_contiguous(), "workspace must be contiguous")
    return given, given.data_ptr(), given.numel() * given.element_size()


class Kv4Cache:
    """One layer's KV cache held in 4 bits (see msk_kv4_desc in
    include/msk.h), over the caller's tensors: codes [2][n_kv_heads][max_seq]
    [head_dim / 2] and scales [2][n_kv_heads][max_seq][head_dim / 16], uint8."""

    def __init__(self, codes, scales, k_scale=1.0, v_scale=1.0):
        _need(codes.dtype == torch.uint8 and scales.dtype == torch.uint8, "codes and scales are uint8")
        _need(codes.dim() == 4 and codes.shape[0] == 2 and codes.is_contiguous(),
              "codes: contiguous [2][n_kv_heads][max_seq][head_dim / 2]")
        self.n_kv_heads, self.max_seq, self.head_dim = codes.shape[1], codes.shape[2], 2 * codes.shape[3]
        _need(scales.shape == (2, self.n_kv_heads, self.max_seq, self.head_dim // 16) and scales.is_contiguous(),
              "scales: contiguous [2][n_kv_heads][max_seq][head_dim / 16]")
        _need(codes.is_cuda and codes.device == scales.device, "codes and scales live on one CUDA device")
        # (fixed: the descriptor holds their addresses)
        self._codes, self._scales = codes, scales
        self.desc = ctypes.pointer(Kv4Desc(codes.data_ptr(), scales.data_ptr(), self.n_kv_heads, self.head_dim,
                                           self.max_seq, k_scale, v_scale))

    codes = property(lambda self: self._codes)
    scales = property(lambda self: self._scales)

    @classmethod
    def empty(cls, n_kv_heads, max_seq, head_dim, k_scale=1.0, v_scale=1.0, device="cuda"):
        """A new cache of zeros."""
        shape = (2, n_kv_heads, max_seq)
        return cls(torch.zeros(*shape, head_dim // 2, dtype=torch.uint8, device=device),
                   torch.zeros(*shape, head_dim // 16, dtype=torch.uint8, device=device), k_scale, v_scale)


class Fp4Weight:
    """A 4-bit matrix [rows][cols] (see msk_nvfp4_desc in include/msk.h) over
    the caller's tensors: packed [rows][cols / 2] and scales
    [rows][cols / 16], uint8."""

    def __init__(self, packed, scales, tensor_scale=1.0):
        _need(packed.dtype == torch.uint8 and scales.dtype == torch.uint8, "packed and scales are uint8")
        _need(packed.dim() == 2 and packed.is_contiguous(), "packed: contiguous [rows][cols / 2]")
        self.rows, self.cols = packed.shape[0], 2 * packed.shape[1]
        _need(scales.shape == (self.rows, self.cols // 16) and scales.is_contiguous(),
              "scales: contiguous [rows][cols / 16]")
        _need(packed.is_cuda and packed.device == scales.device, "packed and scales live on one CUDA device")
        self._set(packed, scales, tensor_scale)

    def _set(self, packed, scales, tensor_scale):
        # (fixed: the descriptor holds their addresses)
        self._packed, self._scales, self._tensor_scale, self._desc = packed, scales, float(tensor_scale), None

    @classmethod
    def _new(cls, rows, cols, tensor_scale, stream):
        """A new matrix on the current device."""
        w = cls.__new__(cls)
        w.rows, w.cols = rows, cols
        w._set(_empty(stream, (rows, cols // 2), torch.uint8), _empty(stream, (rows, cols // 16), torch.uint8), tensor_scale)
        return w

    @property
    def desc(self):
        if self._desc is None:
            self._desc = ctypes.pointer(Nvfp4Desc(self._packed.data_ptr(), self._scales.data_ptr(), self._tensor_scale,
                                                  self.rows, self.cols))
        return self._desc

    packed = property(lambda self: self._packed)
    scales = property(lambda self: self._scales)
    tensor_scale = property(lambda self: self._tensor_scale)


class Fp4Experts:
    """One 4-bit matrix [rows][cols] of each expert (see msk_fp4_experts in
    include/msk.h) over the caller's tensors: packed [n_experts][rows]
    [cols / 2] and scales [n_experts][rows][cols / 16], uint8, and
    tensor_scales, fp32 [n_experts] or None for 1."""

    def __init__(self, packed, scales, tensor_scales=None):
        _need(packed.dtype == torch.uint8 and scales.dtype == torch.uint8, "packed and scales are uint8")
        _need(packed.dim() == 3 and packed.is_contiguous(), "packed: contiguous [n_experts][rows][cols / 2]")
        self.n_experts, self.rows, self.cols = packed.shape[0], packed.shape[1], 2 * packed.shape[2]
        _need(scales.shape == (self.n_experts, self.rows, self.cols // 16) and scales.is_contiguous(),
              "scales: contiguous [n_experts][rows][cols / 16]")
        _need(tensor_scales is None or (tensor_scales.dtype == torch.float32 and tensor_scales.is_contiguous() and
                                        tensor_scales.shape == (self.n_experts,)),
              "tensor_scales: contiguous fp32 [n_experts]")
        _need(packed.is_cuda and packed.device == scales.device and
              (tensor_scales is None or tensor_scales.device == packed.device),
              "packed, scales and tensor_scales live on one CUDA device")
        # (fixed: the descriptor holds their addresses)
        self._packed, self._scales, self._tensor_scales = packed, scales, tensor_scales
        self.desc = ctypes.pointer(Fp4ExpertsC(packed.data_ptr(), scales.data_ptr(),
                                               None if tensor_scales is None else tensor_scales.data_ptr(),
                                               self.n_experts, self.rows, self.cols, None))
        # (of weights that the products take: the others are refused when they are used)
        self._maps = ctypes.create_string_buffer(MSK_FP4_MAPS_BYTES + 128)
        at = ctypes.addressof(self._maps) + 127 & ~127
        with torch.cuda.device(packed.device):
            if load_library().msk_fp4_experts_maps(self.desc, at) == MSK_OK:
                self.desc.contents.maps = at

    packed = property(lambda self: self._packed)
    scales = property(lambda self: self._scales)
    tensor_scales = property(lambda self: self._tensor_scales)


def _step(t, axis):
    """Elements between neighbours of an axis; 0 where there are none (the
    stride of an axis of one is arbitrary)."""
    return t.stride(axis) if t.shape[axis] > 1 else 0


def _position(pos):
    """(host value, device address) of a position given as an int or as a
    CUDA int32 tensor of one element."""
    if isinstance(pos, torch.Tensor):
        _need(pos.dtype == torch.int32 and pos.numel() == 1 and pos.get_device() == torch.cuda.current_device(),
              "a position tensor is one int32 on the current CUDA device")
        return 0, pos.data_ptr()
    return _int32(pos, "a position"), None


def _kv_rows(cache, k, v):
    """(type, rows, steps between rows and between heads) of k and v."""
    shape, dtype = k.shape, _DTYPES.get(k.dtype)
    _need(len(shape) == 3 and shape == v.shape and dtype is not None and v.dtype == k.dtype,
          "k and v: [tokens][n_kv_heads][head_dim], one shape and floating type")
    T, H, d = shape
    _need(H == cache.n_kv_heads and d == cache.head_dim, "k and v do not fit the cache's heads")
    ts, hs, es = k.stride()
    tv, hv, ev = v.stride()
    # (the stride of an axis of one is arbitrary)
    if T == 1:
        ts = tv = 0
    if H == 1:
        hs = hv = 0
    _need(es == 1 and ev == 1 and ts == tv and hs == hv, "k and v: contiguous heads, one layout")
    return dtype, T, ts, hs


def msk_kv4_write(cache, k, v, pos0, stream=None):
    """Quantises k and v ([tokens][n_kv_heads][head_dim], any strides of the
    first two axes) into cache rows pos0, pos0 + 1, ...  pos0: an int, or a
    CUDA int32 tensor read when the kernel runs."""
    dtype, T, ts, hs = _kv_rows(cache, k, v)
    host, dev = _position(pos0)
    st = _enqueue(stream, k, v, cache._codes)
    _check(load_library().msk_kv4_write(cache.desc, k.data_ptr(), v.data_ptr(), dtype, T, ts, hs, host, dev, st),
           "msk_kv4_write")


def msk_kv4_read(cache, pos0, tokens, dtype=torch.bfloat16, out=None, stream=None):
    """Rows pos0 .. pos0 + tokens - 1 as (k, v), each
    [tokens][n_kv_heads][head_dim] of `dtype`, or into the pair `out`."""
    if out is None:
        _need(tokens >= 0 and dtype in _DTYPES, "tokens >= 0 and a floating type")
        shape = (tokens, cache.n_kv_heads, cache.head_dim)
        out = _empty(stream, shape, dtype), _empty(stream, shape, dtype)
    k, v = out
    dt, T, ts, hs = _kv_rows(cache, k, v)
    _need(T == tokens, "out does not hold `tokens` rows")
    st = _enqueue(stream, k, v, cache._codes)
    _check(load_library().msk_kv4_read(cache.desc, _int32(pos0, "a position"), tokens, k.data_ptr(), v.data_ptr(), dt,
                                       ts, hs, st), "msk_kv4_read")
    return k, v


def msk_attention_kv4_workspace(tokens, n_q_heads, n_kv_heads, head_dim, window, cache_len):
    """Workspace bytes of msk_attention_kv4 (0 for few keys)."""
    sizes = (tokens, n_q_heads, n_kv_heads, head_dim, window, cache_len)
    _need(-0x80000000 <= min(sizes) and max(sizes) <= 0x7FFFFFFF, "sizes that fit 32 bits")
    return load_library().msk_attention_kv4_workspace(tokens, n_q_heads, n_kv_heads, head_dim, window, cache_len)


def msk_attention_kv4(q, cache, cache_len, window=0, parents=None, softmax_scale=0.0, out=None, workspace=None,
                      stream=None):
    """Attention of q ([tokens][n_q_heads][head_dim] bf16 or fp16, any token
    stride) over a Kv4Cache holding `cache_len` rows and then the tokens' own;
    returns out [tokens][n_q_heads * head_dim].  cache_len: an int, or a CUDA
    int32 tensor read when the kernels run.  parents: the candidate tree as in
    msk_decode_step_tree, None for the chain.  Nothing is waited for."""
    T, Hq, d = q.shape
    ts, hs, es = q.stride()
    dtype = _DTYPES.get(q.dtype)
    _need(dtype is not None and d == cache.head_dim and es == 1 and (hs == d or Hq == 1),
          "q: [tokens][n_q_heads][head_dim] with contiguous heads")
    _need(parents is None or len(parents) == T, "parents: one for each token")
    if out is None:
        out = _empty(stream, (T, Hq * d), q.dtype)
    else:
        _need(out.dtype == q.dtype and out.numel() == q.numel() and out.is_contiguous(),
              "out: contiguous [tokens][n_q_heads * head_dim] of q's type")
    host, dev = _position(cache_len)
    window = _int32(window, "window")
    need = msk_attention_kv4_workspace(T, Hq, cache.n_kv_heads, d, window, host if dev is None else cache.max_seq - T)
    ws, addr, size = _workspace(workspace, need, stream)
    st = _enqueue(stream, q, out, cache._codes) if ws is None else _enqueue(stream, q, out, cache._codes, ws)
    _check(load_library().msk_attention_kv4(q.data_ptr(), dtype, ts if T > 1 else 0, cache.desc, T, Hq, host, dev,
                                            None if parents is None else _positions(parents), window,
                                            softmax_scale, out.data_ptr(), addr, size, st), "msk_attention_kv4")
    return out


def msk_linear_fp4(x, weight, out_dtype=None, out=None, stream=None):
    """x ([tokens][cols] bf16 or fp16, any row stride) times the transposed
    Fp4Weight: [tokens][rows] of out_dtype (x's type unless given) or into
    `out` (any row stride)."""
    shape, xt = x.shape, _DTYPES.get(x.dtype)
    _need(len(shape) == 2 and shape[1] == weight.cols and x.stride(1) == 1 and xt is not None,
          "x: [tokens][cols], contiguous rows")
    T = shape[0]
    yt = _DTYPES.get((x.dtype if out_dtype is None else out_dtype) if out is None else out.dtype)
    _need(yt is not None, "out: of a floating type")
    if out is None:
        out = _empty(stream, (T, weight.rows), x.dtype if out_dtype is None else out_dtype)
        ys = weight.rows
    else:
        _need(out.shape == (T, weight.rows) and (out.stride(1) == 1 or weight.rows <= 1),
              "out: [tokens][rows], contiguous rows")
        ys = _step(out, 0)
    st = _enqueue(stream, x, out, weight._packed)
    _check(load_library().msk_linear_fp4(x.data_ptr(), xt, _step(x, 0), weight.desc, T, out.data_ptr(), yt, ys, st),
           "msk_linear_fp4")
    return out


def msk_ops_check(stream=None):
    """Waits for the stream and raises MskError (timeout) if a bounded device
    wait of the operators ran out since the last check."""
    _check(load_library().msk_ops_check(_stream(stream)), "msk_ops_check")


def msk_token_logprobs(logits, tokens=None, top=0, temperature=1.0, stream=None):
    """Log probabilities of `tokens` (int32 [rows]; a negative one marks a
    padded row) under softmax(logits / temperature), logits [rows][vocab] of
    any floating type and row stride.  Returns (logprob, entropy, rank,
    top_ids, top_logprobs): fp32 [rows], fp32 [rows], int32 [rows], int32
    [rows][top], fp32 [rows][top]; logprob and rank are None without tokens."""
    _need(logits.dim() == 2 and logits.dtype in _DTYPES and (logits.stride(1) == 1 or logits.shape[1] <= 1),
          "logits: [rows][vocab], contiguous rows")
    R, V = logits.shape
    _need(0 <= top <= 32, "top: 0 to 32 alternatives")
    logprob = rank = tok = lp = rk = None
    if tokens is not None:
        _need(tokens.dtype == torch.int32 and tokens.shape == (R,) and tokens.is_contiguous(), "tokens: int32 [rows]")
        logprob, rank = _empty(stream, R, torch.float32), _empty(stream, R, torch.int32)
        tok, lp, rk = tokens.data_ptr(), logprob.data_ptr(), rank.data_ptr()
    entropy = _empty(stream, R, torch.float32)
    top_ids, top_logprobs = _empty(stream, (R, top), torch.int32), _empty(stream, (R, top), torch.float32)
    st = _enqueue(stream, logits, entropy) if tokens is None else _enqueue(stream, logits, tokens, entropy)
    _check(load_library().msk_token_logprobs(logits.data_ptr(), _DTYPES[logits.dtype], R, V, _step(logits, 0), tok,
                                             temperature, top, lp, rk, entropy.data_ptr(), top_ids.data_ptr(),
                                             top_logprobs.data_ptr(), st), "msk_token_logprobs")
    return logprob, entropy, rank, top_ids, top_logprobs


def msk_moe_route(logits, top_k, bias=None, stream=None):
    """Each token's top_k experts and their gates: (experts int32, gates
    fp32), both [tokens][top_k], from logits [tokens][n_experts] of any
    floating type and row stride (rows that do not overlap), with an fp32
    bias [n_experts] added.  A barred expert has a logit of -inf; ranks that find none are -1, gate 0."""
    _need(logits.dim() == 2 and logits.dtype in _DTYPES and (logits.stride(1) == 1 or logits.shape[1] <= 1),
          "logits: [tokens][n_experts], contiguous rows")
    T, E = logits.shape
    _need(1 <= top_k <= min(32, E), "top_k: 1 to 32, n_experts at most")
    _need(bias is None or (bias.dtype == torch.float32 and bias.shape == (E,) and bias.is_contiguous()),
          "bias: contiguous fp32 [n_experts]")
    st = _enqueue(stream, logits) if bias is None else _enqueue(stream, logits, bias)
    # (here and below, outputs last: an allocation waits for the launch before it to leave the
    # core, which the checks above take part of)
    experts, gates = _empty(stream, (T, top_k), torch.int32), _empty(stream, (T, top_k), torch.float32)
    _check(load_library().msk_moe_route(logits.data_ptr(), _DTYPES[logits.dtype], T, E, _step(logits, 0),
                                        None if bias is None else bias.data_ptr(), top_k, experts.data_ptr(),
                                        gates.data_ptr(), st), "msk_moe_route")
    return experts, gates


def msk_moe_sort(experts, n_experts, stream=None):
    """The slots of `experts` (int32, any shape, usually [tokens][top_k])
    sorted by expert: (offsets int32 [n_experts + 1], slots int32 [n], places
    int32 of experts' shape).  An expert outside [0, n_experts) drops its
    slot: its place is -1, and slots ends in as many -1."""
    _need(experts.dtype == torch.int32 and experts.is_contiguous(), "experts: contiguous int32")
    _need(1 <= n_experts <= 1024, "n_experts: 1 to 1024")
    n, st = experts.numel(), _enqueue(stream, experts)
    offsets, slots = _empty(stream, n_experts + 1, torch.int32), _empty(stream, n, torch.int32)
    places = _empty(stream, experts.shape, torch.int32)
    _check(load_library().msk_moe_sort(experts.data_ptr(), n, n_experts, offsets.data_ptr(), slots.data_ptr(),
                                       places.data_ptr(), st), "msk_moe_sort")
    return offsets, slots, places


def msk_quantize_fp4(x, tensor_scale=1.0, out=None, stream=None):
    """x ([rows][cols] of any floating type and row stride, cols a multiple of
    16) in 4 bits, an Fp4Weight: a new one, or `out`, whose tensor's scale is
    taken."""
    _need(x.dim() == 2 and x.dtype in _DTYPES and x.stride(1) == 1 and x.shape[1] % 16 == 0 and x.shape[1] > 0,
          "x: [rows][cols], contiguous rows of whole blocks of 16")
    R, C = x.shape
    if out is None:
        st = _enqueue(stream, x)
        out = Fp4Weight._new(R, C, tensor_scale, stream)
    else:
        _need(out.rows == R and out.cols == C, "out: [rows][cols] of x")
        st = _enqueue(stream, x, out._packed)
    _check(load_library().msk_quantize_fp4(x.data_ptr(), _DTYPES[x.dtype], R, C, _step(x, 0), out._tensor_scale,
                                           out._packed.data_ptr(), out._scales.data_ptr(), st), "msk_quantize_fp4")
    return out


def msk_dequantize_fp4(w, dtype=torch.bfloat16, out=None, stream=None):
    """The values of an Fp4Weight, [rows][cols] of `dtype`, or into `out` (any
    row stride)."""
    if out is None:
        _need(dtype in _DTYPES, "a floating type")
        st = _enqueue(stream, w._packed)
        out = _empty(stream, (w.rows, w.cols), dtype)
    else:
        _need(out.shape == (w.rows, w.cols) and out.dtype in _DTYPES and out.stride(1) == 1,
              "out: [rows][cols], contiguous rows")
        st = _enqueue(stream, out, w._packed)
    _check(load_library().msk_dequantize_fp4(w._packed.data_ptr(), w._scales.data_ptr(), w._tensor_scale, w.rows, w.cols,
                                             out.data_ptr(), _DTYPES[out.dtype], _step(out, 0), st), "msk_dequantize_fp4")
    return out


def msk_experts_fp4(x, experts, offsets, up=None, slots=None, top_k=None, out_dtype=torch.bfloat16, out=None, stream=None):
    """Products of the 4-bit rows x (an Fp4Weight) with their experts'
    matrices (Fp4Experts): places offsets[e] .. offsets[e + 1] - 1 are expert
    e's, and place p takes row p of x, or with `slots` (int32 [n], as from
    msk_moe_sort) row slots[p] // top_k (1 unless given; more slots than x has
    rows need it said).  With `up` (a second Fp4Experts of
    the same size) the result is silu(x w^T) * (x up^T).  Returns
    [n][experts.rows] of out_dtype, or `out` (any row stride); rows of places
    behind the last expert's are not written."""
    _need(offsets.dtype == torch.int32 and offsets.shape == (experts.n_experts + 1,) and offsets.is_contiguous(),
          "offsets: contiguous int32 [n_experts + 1]")
    _need(x.cols == experts.cols and x.cols % 64 == 0, "x has the weights' columns, a multiple of 64")
    _need(up is None or (up.n_experts, up.rows, up.cols) == (experts.n_experts, experts.rows, experts.cols),
          "up: of the other weights' size")
    _need(slots is None or (slots.dtype == torch.int32 and slots.dim() == 1 and slots.is_contiguous()),
          "slots: contiguous int32 [n]")
    # (rows behind x's last are taken as that one: a top_k that was forgotten would not be seen)
    _need(slots is None or top_k is not None or slots.shape[0] <= x.rows, "slots: more than x has rows, say top_k")
    top_k = 1 if top_k is None else _int32(top_k, "top_k")
    _need(slots is None or top_k >= 1, "top_k: 1 or more")
    n = x.rows if slots is None else slots.shape[0]
    if out is None:
        _need(out_dtype in _DTYPES, "out_dtype: a floating type")
    else:
        _need(out.shape == (n, experts.rows) and out.dtype in _DTYPES and (out.stride(1) == 1 or experts.rows <= 1),
              "out: [n][rows], contiguous rows")
    given = [x._packed, experts._packed, offsets]
    slot_ptr = up_desc = None
    if slots is not None:
        slot_ptr = slots.data_ptr()
        given.append(slots)
    if up is not None:
        up_desc = up.desc
        given.append(up._packed)
    if out is not None:
        given.append(out)
    st, x_desc, ptr = _enqueue(stream, *given), x.desc, offsets.data_ptr()
    if out is None:
        step, out = experts.rows, _empty(stream, (n, experts.rows), out_dtype)
    else:
        step = _step(out, 0)
    _check(load_library().msk_experts_fp4(x_desc, slot_ptr, top_k, n, ptr, experts.desc, up_desc, out.data_ptr(),
                                          _DTYPES[out.dtype], step, st), "msk_experts_fp4")
    return out


def msk_debug_experts_fault(tile=-1, wait_ns=0):
    """For tests: later calls of msk_experts_fp4 never say that a pair of
    blocks' tile number `tile` is complete, and wait for wait_ns at most; the
    defaults put an end to both (see include/msk.h)."""
    _check(load_library().msk_debug_experts_fault(_int32(tile, "tile"), int(wait_ns)), "msk_debug_experts_fault")


def msk_moe_combine(y, places, gates=None, out_dtype=None, out=None, stream=None):
    """out[t] = sum over ranks of gates[t][r] * y[places[t][r]] (gates None:
    1), y [rows][cols] of any floating type and row stride (rows that do not
    overlap), places int32 and
    gates fp32 [tokens][top_k]; a place outside y's rows is a dropped slot.
    Returns [tokens][cols] of out_dtype (y's unless given), or `out`."""
    _need(y.dim() == 2 and y.dtype in _DTYPES and (y.stride(1) == 1 or y.shape[1] <= 1), "y: [rows][cols], contiguous rows")
    _need(places.dim() == 2 and places.dtype == torch.int32 and places.is_contiguous() and places.shape[1] >= 1,
          "places: contiguous int32 [tokens][top_k]")
    _need(gates is None or (gates.dtype == torch.float32 and gates.shape == places.shape and gates.is_contiguous()),
          "gates: contiguous fp32 [tokens][top_k]")
    (T, k), C = places.shape, y.shape[1]
    if out is None:
        _need(out_dtype is None or out_dtype in _DTYPES, "out_dtype: a floating type")
    else:
        _need(out.shape == (T, C) and out.dtype in _DTYPES and (out.stride(1) == 1 or C <= 1), "out: [tokens][cols], contiguous rows")
        _enqueue(stream, out)
    st = _enqueue(stream, y, places) if gates is None else _enqueue(stream, y, places, gates)
    if out is None:
        out = _empty(stream, (T, C), y.dtype if out_dtype is None else out_dtype)
    _check(load_library().msk_moe_combine(y.data_ptr(), _DTYPES[y.dtype], y.shape[0], _step(y, 0), places.data_ptr(),
                                          None if gates is None else gates.data_ptr(), T, k, C, out.data_ptr(),
                                          _DTYPES[out.dtype], _step(out, 0), st), "msk_moe_combine")
    return out


# ----------------------------------------------------------------------------
# Model: descriptors from torch tensors
# ----------------------------------------------------------------------------


def _bf16(t):
    t2 = t if t.dim() == 2 else t.reshape(1, -1)
    assert t2.dtype == torch.bfloat16 and t2.is_cuda and t2.stride(1) == 1
    return Bf16Desc(t2.data_ptr(), t2.shape[0], t2.shape[1], t2.stride(0))


def _fp4_array(trip):
    packed, scales, ts = trip
    n = packed.shape[0]
    arr = (Nvfp4Desc * n)()
    tsh = ts.detach().float().cpu().tolist()
    for e in range(n):
        arr[e] = Nvfp4Desc(packed[e].data_ptr(), scales[e].data_ptr(), tsh[e], packed.shape[1],
                           packed.shape[2] * 2)
    return arr


class Model:
    """A loaded model.  ``dims`` is any object with the workload fields
    (hidden, n_q_heads, n_kv_heads, head_dim, pooled, n_experts, top_k,
    inter, tokens, max_seq, windows, rms_eps, rope_theta)."""

    def __init__(self, dims, prefetch_experts=14, wait_budget_ns=0):
        windows = list(dims.windows)
        self.dims = dims
        self.n_layers = len(windows)
        sliding = [w for w in windows if w > 0]
        if len(set(sliding)) > 1:
            raise ValueError("all sliding-window layers share one window size (msk_model_config.window); "
                             f"got {sorted(set(sliding))}")
        self._glob = (ctypes.c_uint8 * self.n_layers)(*[1 if w == 0 else 0 for w in windows])
        cfg = ModelConfig(self.n_layers, dims.hidden, dims.n_q_heads, dims.n_kv_heads, dims.head_dim,
                          dims.pooled, dims.n_experts, dims.top_k, dims.inter, dims.tokens, dims.max_seq,
                          prefetch_experts, self._glob, sliding[0] if sliding else 0, dims.rms_eps,
                          dims.rope_theta, wait_budget_ns)
        self.handle = msk_create(cfg)
        n = ctypes.c_int32()
        b = ctypes.c_int64()
        _check(load_library().msk_get_info(self.handle, ctypes.byref(n), ctypes.byref(b)), "msk_get_info")
        self.n_ctas = n.value

    def load_layer(self, layer, lt, stream=None):
        """lt: msk_synth.LayerTensors on the current CUDA device."""
        gate, up, down = _fp4_array(lt.gate), _fp4_array(lt.up), _fp4_array(lt.down)
        w = LayerWeightsC(_bf16(lt.attn_norm), _bf16(lt.moe_norm), _bf16(lt.w_qkv), _bf16(lt.w_o),
                          _bf16(lt.w_pool), _bf16(lt.w_unpool), _bf16(lt.w_router),
                          lt.router_bias.data_ptr(), gate, up, down)
        msk_load_layer(self.handle, layer, w, stream)

    def device_bytes(self):
        n = ctypes.c_int32()
        b = ctypes.c_int64()
        _check(load_library().msk_get_info(self.handle, ctypes.byref(n), ctypes.byref(b)), "msk_get_info")
        return b.value

    def layer_step(self, layer, hidden, kv_cache, positions, prev_routing=None, routing_out=None,
                   run_prologue=False, stream=None, check=True):
        st = msk_layer_step(self.handle, layer, hidden, kv_cache, positions, prev_routing, routing_out,
                            run_prologue, stream)
        if check:
            _check(st, "msk_layer_step")
        return st

    def decode_step(self, hidden, kv_cache, positions, prev_routing=None, routing_out=None, stream=None,
                    check=True):
        st = msk_decode_step(self.handle, hidden, kv_cache, positions, prev_routing, routing_out, stream)
        if check:
            _check(st, "msk_decode_step")
        return st

    def layer_step_tree(self, layer, hidden, kv_cache, cache_len, parents, prev_routing=None, routing_out=None,
                        run_prologue=False, stream=None, check=True):
        """One launch verifying a tree of candidates (see msk_layer_step_tree)."""
        st = msk_layer_step_tree(self.handle, layer, hidden, kv_cache, cache_len, parents, prev_routing,
                                 routing_out, run_prologue, stream)
        if check:
            _check(st, "msk_layer_step_tree")
        return st

    def decode_step_tree(self, hidden, kv_cache, cache_len, parents, prev_routing=None, routing_out=None,
                         stream=None, check=True):
        st = msk_decode_step_tree(self.handle, hidden, kv_cache, cache_len, parents, prev_routing, routing_out,
                                  stream)
        if check:
            _check(st, "msk_decode_step_tree")
        return st

    def capture_step(self, hidden, kv_cache, prev_routing=None, routing_out=None):
        """Records one whole step over these buffers as a CUDA graph (see
        msk_step_graph_capture)."""
        _check(msk_step_graph_capture(self.handle, hidden, kv_cache, prev_routing, routing_out),
               "msk_step_graph_capture")

    def replay_step(self, cache_len, parents=None, stream=None, check=True):
        st = msk_step_graph_launch(self.handle, cache_len, parents, stream)
        if check:
            _check(st, "msk_step_graph_launch")
        return st

    def set_timing(self, on):
        _check(load_library().msk_set_timing(self.handle, int(on)), "msk_set_timing")

    def timeline(self):
        """Per-launch, per-block phase timestamps (ns): int64 tensor
        [launches][ctas][TIMELINE_SLOTS] (zeros where a phase was not run)."""
        L = load_library()
        cap = self.n_layers * self.n_ctas * TIMELINE_SLOTS
        buf = (ctypes.c_uint64 * cap)()
        n = ctypes.c_size_t()
        nl = ctypes.c_int32()
        nc = ctypes.c_int32()
        _check(L.msk_get_timeline(self.handle, buf, cap, ctypes.byref(n), ctypes.byref(nl), ctypes.byref(nc)),
               "msk_get_timeline")
        t = torch.tensor(list(buf)[: n.value], dtype=torch.int64)
        return t.reshape(nl.value, nc.value, TIMELINE_SLOTS) if n.value else t

    def set_launch_timing(self, on):
        _check(load_library().msk_set_launch_timing(self.handle, int(on)), "msk_set_launch_timing")

    def launch_ms(self):
        """Durations (ms) of the last call's launches, from CUDA events
        recorded on the call's stream."""
        buf = (ctypes.c_float * self.n_layers)()
        n = ctypes.c_int32()
        _check(load_library().msk_get_launch_ms(self.handle, buf, self.n_layers, ctypes.byref(n)),
               "msk_get_launch_ms")
        return list(buf)[: n.value]

    def set_wait_budget(self, ns):
        _check(load_library().msk_set_wait_budget(self.handle, int(ns)), "msk_set_wait_budget")

    def set_fault_injection(self, barrier, cta):
        _check(load_library().msk_set_fault_injection(self.handle, int(barrier), int(cta)),
               "msk_set_fault_injection")

    def debug_scratch(self, which, out, stream=None):
        """Copies intermediate `which` of the last launch into tensor `out`."""
        n = ctypes.c_size_t()
        _check(load_library().msk_debug_scratch(self.handle, which, _ptr(out), out.numel() * out.element_size(),
                                                ctypes.byref(n), _stream(stream)), "msk_debug_scratch")
        return n.value

    def debug_dequant(self, layer, expert, which, out, stream=None):
        msk_debug_dequant(self.handle, layer, expert, which, out, stream)

    def close(self):
        if getattr(self, "handle", None):
            msk_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

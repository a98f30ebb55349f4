"""Python binding of the hybrid decode-attention C ABI (include/hybrid_decode.h).

Argument marshalling only: every step of the path runs in the CUDA kernels of
``libhybriddecode.so``.  PyTorch provides device memory and streams; tensors
are passed as raw device pointers.  Importing this package loads the in-tree
library and raises if it has not been built -- there is no fallback.

Names follow the C entry points: ``hybrid_decode_init``, ``rope_append_kv``,
``decode_attn_sliding``, ``decode_attn_full``, ``decode_step`` (plus
``hybrid_decode_destroy`` and the helpers); over paged caches ``paged_cache``,
``paged_batch``, ``rope_append_paged``, ``attn_paged``, ``select_pages`` and
``attn_selected_pages``; for normed heads, other angles and other scores
``rope_table``, ``norm_rope_append_paged``, ``scoring``, ``attn_paged_scored``
and ``read_paged``.  Each call raises ``HDError``
carrying the hd_status when the library rejects it.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass, field

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(PKG, "libhybriddecode.so")

HD_SLIDING, HD_FULL = 0, 1
HD_LAYOUT_AUTO, HD_LAYOUT_RING, HD_LAYOUT_ROLL = 0, 1, 2
HD_CONSUMER_CUDA_CORE, HD_CONSUMER_TENSOR_CORE, HD_CONSUMER_TENSOR_MEMORY = 0, 1, 2
HD_PROFILE_SLIDING, HD_PROFILE_FULL, HD_PROFILE_FIRST_ONLY, HD_PROFILE_STEP = 1 << HD_SLIDING, 1 << HD_FULL, 4, 8
HD_PROFILE_KIND_STEP = 2
HD_KV_BF16, HD_KV_FP8_E4M3 = 0, 1
HD_STATIC_SCRATCH_BYTES = 64 << 20   # the allocation-free entry point's scratch array
STATUS = {0: "HD_OK", 1: "HD_ERR_INVALID_ARG", 2: "HD_ERR_UNSUPPORTED", 3: "HD_ERR_CAPACITY",
          4: "HD_ERR_CUDA", 5: "HD_ERR_STATE"}
DEVERR = {1: "HD_DEVERR_CONTEXT_NEGATIVE", 2: "HD_DEVERR_CONTEXT_CAPACITY",
          4: "HD_DEVERR_CONTEXT_PLAN", 8: "HD_DEVERR_WAIT_TIMEOUT", 16: "HD_DEVERR_TOKEN_OFFSETS",
          32: "HD_DEVERR_PAGE", 64: "HD_DEVERR_SPAN"}
HD_ROPE_HALVES, HD_ROPE_NEIGHBOURS = 0, 1
HD_ROPE_PLAIN, HD_ROPE_LINEAR, HD_ROPE_RAMP, HD_ROPE_BANDS = 0, 1, 2, 3

if not os.path.exists(LIBRARY):
    raise ImportError(f"{LIBRARY} is missing: build it with full_gqa_decode_gb300.build.build() "
                      "(or __graft_entry__.build()); there is no non-CUDA fallback")
_lib = ctypes.CDLL(LIBRARY)


class HDError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)}")
        self.status = status


class hd_config(ctypes.Structure):
    _fields_ = [("num_layers", ctypes.c_int32), ("layer_types", ctypes.POINTER(ctypes.c_int32)),
                ("num_q_heads", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("sliding_window", ctypes.c_int32),
                ("rotary_dim_sliding", ctypes.c_int32), ("rotary_dim_full", ctypes.c_int32),
                ("rope_theta_sliding", ctypes.c_double), ("rope_theta_full", ctypes.c_double),
                ("cache_layout", ctypes.c_int32), ("max_batch", ctypes.c_int32),
                ("max_context", ctypes.c_int32), ("kv_dtype", ctypes.c_int32)]


class hd_kv_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("seq_stride", ctypes.c_int64),
                ("capacity", ctypes.c_int32), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class hd_layer_io(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("cache", hd_kv_cache), ("sink", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("lse", ctypes.c_void_p), ("gate", ctypes.c_void_p)]


class hd_paged_cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("bounds", ctypes.c_void_p)]


class hd_paged_batch(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("context", ctypes.c_void_p), ("token_offsets", ctypes.c_void_p),
                ("table_stride", ctypes.c_int32), ("max_blocks", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("num_tokens", ctypes.c_int32), ("max_tokens", ctypes.c_int32), ("max_context", ctypes.c_int32)]


class hd_rope_params(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int32), ("scaling", ctypes.c_int32), ("theta", ctypes.c_double),
                ("factor", ctypes.c_double), ("original_context", ctypes.c_double), ("slow", ctypes.c_double),
                ("fast", ctypes.c_double), ("amplitude", ctypes.c_double)]


class hd_rope_table(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("positions", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("layout", ctypes.c_int32)]


class hd_head_norm(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("f32_weights", ctypes.c_int32),
                ("per_head", ctypes.c_int32), ("offset", ctypes.c_float), ("eps", ctypes.c_float)]


class hd_scoring(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("slopes", ctypes.c_void_p),
                ("first", ctypes.c_void_p), ("last", ctypes.c_void_p)]


_c = ctypes
_P = _c.c_void_p
_i32, _i64 = _c.c_int32, _c.c_int64
_SIGS = {
    "hd_validate_config": [_c.POINTER(hd_config)],
    "hd_plan_split": [_i32, _i32, _i32, _i32, _c.POINTER(_i32), _c.POINTER(_i32)],
    "hd_plan_step_split": [_i32, _c.POINTER(_i32), _c.POINTER(_c.c_uint8), _i32, _i32, _i32, _i32, _i32, _i32,
                           _c.POINTER(_i32)],
    "hybrid_decode_init": [_c.POINTER(hd_config), _c.POINTER(_P)],
    "hybrid_decode_destroy": [_P],
    "rope_append_kv": [_P, _i32, _i32, _P, _P, _P, _P, _P, hd_kv_cache, _P],
    "decode_attn_sliding": [_P, _i32, _i32, _P, _P, hd_kv_cache, _P, _P, _P, _P, _P],
    "decode_attn_full": [_P, _i32, _i32, _P, _i32, _P, hd_kv_cache, _P, _P, _P, _P, _P],
    "decode_step": [_P, _i32, _P, _i32, _c.POINTER(hd_layer_io), _P],
    "decode_step_tokens": [_P, _i32, _i32, _P, _i32, _c.POINTER(hd_layer_io), _P],
    "hybrid_decode_device_errors": [_P, _c.POINTER(_i32), _P],
    "hybrid_decode_launch_count": [_P, _c.POINTER(_i64)],
    "hybrid_decode_set_profiling": [_P, _i32],
    "hybrid_decode_profile": [_P, _i32, _c.POINTER(_c.c_double), _c.POINTER(_i64)],
    "hybrid_decode_set_consumer": [_P, _i32],
    "decode_attn_full_static_scratch": [_i32, _i32, _i32, _P, _i32, _P, hd_kv_cache, _P, _P, _P, _P],
    "decode_attn_full_static_scratch_plan": [_i32, _i32, _i32, _i32, _i32, _c.POINTER(_i64), _c.POINTER(_i32),
                                             _c.POINTER(_i32)],
    "hybrid_decode_read_probe": [_P, _i64, _P],
    "hybrid_decode_inject_lost_copy": [_P, _i32],
    "hybrid_decode_set_layer_overlap": [_P, _i32],
    "hybrid_decode_set_step_fusion": [_P, _i32],
    "hybrid_decode_set_cluster_combine": [_P, _i32],
    "hd_validate_paged": [_c.POINTER(hd_config), _c.POINTER(hd_paged_batch), _c.POINTER(hd_paged_cache)],
    "rope_append_paged": [_P, _i32, _c.POINTER(hd_paged_batch), _P, _i64, _P, _i64, _P, _i64, _P,
                          _c.POINTER(hd_paged_cache), _P],
    "attn_paged": [_P, _i32, _c.POINTER(hd_paged_batch), _P, _c.POINTER(hd_paged_cache), _P, _P, _P, _P, _P],
    "select_pages": [_P, _i32, _c.POINTER(hd_paged_batch), _P, _c.POINTER(hd_paged_cache), _i32, _i32, _i32, _P, _P],
    "attn_selected_pages": [_P, _i32, _c.POINTER(hd_paged_batch), _P, _c.POINTER(hd_paged_cache), _P, _i32, _P, _P, _P,
                            _P, _P],
    "hd_rope_frequencies": [_c.POINTER(hd_rope_params), _c.POINTER(_c.c_double), _c.POINTER(_c.c_double)],
    "hd_rope_fill": [_c.POINTER(hd_rope_params), _i32, _P, _P],
    "norm_rope_append_paged": [_P, _i32, _c.POINTER(hd_paged_batch), _c.POINTER(hd_head_norm), _c.POINTER(hd_rope_table), _P,
                               _P, _i64, _P, _i64, _P, _i64, _P, _c.POINTER(hd_paged_cache), _P],
    "attn_paged_scored": [_P, _i32, _c.POINTER(hd_paged_batch), _c.POINTER(hd_scoring), _P, _c.POINTER(hd_paged_cache), _P,
                          _P, _P, _P, _P],
    "read_paged": [_P, _c.POINTER(hd_paged_batch), _c.POINTER(hd_paged_cache), _P, _i64, _P, _i64, _P],
}
for _name, _args in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _c.c_int
_lib.hd_status_string.argtypes = [_c.c_int]
_lib.hd_status_string.restype = _c.c_char_p


def _check(status: int, what: str) -> None:
    if status != 0:
        raise HDError(status, what)


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


def _check_sink(sink, num_q_heads: int, like: torch.Tensor) -> None:
    """Sink checks of vllm/models/hy_v4/nvidia/flashmla_sparse.py (`_validate_sinks`,
    `_sinks_for_query`): fp32, shape (num_q_heads,), on the query's device."""
    if sink is None:
        return
    if sink.dtype != torch.float32:
        raise ValueError(f"sink must be float32, got {sink.dtype}")
    if sink.dim() != 1 or sink.shape[0] != num_q_heads:
        raise ValueError(f"sink must have shape ({num_q_heads},), got {tuple(sink.shape)}")
    if sink.device != like.device:
        raise ValueError(f"sink and query must be on the same device ({sink.device} vs {like.device})")
    if not sink.is_contiguous():
        raise ValueError("sink must be contiguous")


def _check_gate(gate, batch: int, num_q_heads: int, like: torch.Tensor, tokens: int | None = None) -> None:
    """Output-gate logits: fp32, shape (batch, num_q_heads) -- or (batch, tokens,
    num_q_heads) for a multi-token step -- contiguous, on the query's device."""
    if gate is None:
        return
    if gate.dtype != torch.float32:
        raise ValueError(f"gate must be float32, got {gate.dtype}")
    want = (batch, num_q_heads) if tokens is None else (batch, tokens, num_q_heads)
    if tuple(gate.shape) != want:
        raise ValueError(f"gate must have shape {want}, got {tuple(gate.shape)}")
    if gate.device != like.device:
        raise ValueError(f"gate and query must be on the same device ({gate.device} vs {like.device})")
    if not gate.is_contiguous():
        raise ValueError("gate must be contiguous")


def _stream_lookup(torch_c):
    """What gives the raw handle of a device's current stream: torch's own look-up where it has
    one, as torch.cuda.current_stream() makes an object around it, 3 us on a Grace host, as much
    as a launch; else that."""
    return getattr(torch_c, "_cuda_getCurrentRawStream", None) or (
        lambda device: torch.cuda.current_stream(device).cuda_stream)


_raw_stream = _stream_lookup(torch._C)


def _stream(stream) -> int | None:
    if stream is None:
        return _raw_stream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


@dataclass
class Config:
    """Model shape; field meanings follow ``hd_config`` in include/hybrid_decode.h."""
    layer_types: list
    num_q_heads: int = 8
    num_kv_heads: int = 2
    head_dim: int = 256
    sliding_window: int = 512
    rotary_dim_sliding: int = 256
    rotary_dim_full: int = 64
    rope_theta_sliding: float = 1.0e4
    rope_theta_full: float = 5.0e6
    cache_layout: int = HD_LAYOUT_AUTO
    max_batch: int = 1
    max_context: int = 4096
    kv_dtype: int = HD_KV_BF16
    _types: object = field(default=None, repr=False)

    def to_c(self) -> hd_config:
        self._types = (ctypes.c_int32 * len(self.layer_types))(*self.layer_types)
        return hd_config(len(self.layer_types), self._types, self.num_q_heads, self.num_kv_heads,
                         self.head_dim, self.sliding_window, self.rotary_dim_sliding,
                         self.rotary_dim_full, self.rope_theta_sliding, self.rope_theta_full,
                         self.cache_layout, self.max_batch, self.max_context, self.kv_dtype)


_FP8_CACHE_TYPES = (torch.uint8, torch.float8_e4m3fn)


def kv_cache(k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor | None = None,
             v_scale: torch.Tensor | None = None) -> hd_kv_cache:
    """Describe a cache pair shaped [batch, num_kv_heads, capacity, head_dim] on CUDA:
    bf16, or E4M3 codes (uint8 or float8_e4m3fn) with fp32 ``k_scale``/``v_scale``
    of shape [num_kv_heads] on the same device (the context's kv_dtype must match)."""
    if k.shape != v.shape or k.dim() != 4 or k.stride() != v.stride():
        raise ValueError("k and v caches must share a [batch, kv_heads, capacity, head_dim] layout")
    fp8 = k.dtype in _FP8_CACHE_TYPES
    if fp8:
        if v.dtype not in _FP8_CACHE_TYPES:
            raise ValueError("k and v caches must have the same element type")
        for name, sc in (("k_scale", k_scale), ("v_scale", v_scale)):
            if sc is None or sc.dtype != torch.float32 or tuple(sc.shape) != (k.shape[1],):
                raise ValueError(f"an FP8 cache needs {name} as float32 of shape ({k.shape[1]},)")
            if sc.device != k.device or not sc.is_contiguous():
                raise ValueError(f"{name} must be contiguous and on the cache's device")
    else:
        if k.dtype != torch.bfloat16 or v.dtype != torch.bfloat16:
            raise ValueError("caches must be bf16, or E4M3 codes with scales")
        if k_scale is not None or v_scale is not None:
            raise ValueError("scales belong to FP8 caches only")
    if k.stride(3) != 1 or k.stride(2) != k.shape[3] or k.stride(1) != k.shape[2] * k.shape[3]:
        raise ValueError("each sequence's cache must be contiguous [kv_heads, capacity, head_dim]")
    if not k.is_cuda or not v.is_cuda:
        raise ValueError("caches must be CUDA tensors")
    c = hd_kv_cache(k.data_ptr(), v.data_ptr(), k.stride(0), k.shape[2],
                    k_scale.data_ptr() if fp8 else None, v_scale.data_ptr() if fp8 else None)
    c.batch = k.shape[0]  # sequences the tensors hold; calls may not pass a larger batch
    c.keep = (k_scale, v_scale)  # the scales must outlive the descriptor
    return c


def _check_batch(cache: hd_kv_cache, batch: int) -> None:
    held = getattr(cache, "batch", None)
    if held is not None and held < batch:
        raise ValueError(f"cache holds {held} sequences, call passes batch {batch}")


def hd_validate_config(cfg: Config) -> int:
    return _lib.hd_validate_config(ctypes.byref(cfg.to_c()))


def hd_plan_split(batch: int, num_kv_heads: int, max_keys: int, num_sms: int) -> tuple[int, int]:
    ck, nc = ctypes.c_int32(), ctypes.c_int32()
    _check(_lib.hd_plan_split(batch, num_kv_heads, max_keys, num_sms, ctypes.byref(ck),
                              ctypes.byref(nc)), "hd_plan_split")
    return ck.value, nc.value


def hd_plan_step_split(max_keys, batch: int, num_kv_heads: int, rows: int, num_sms: int,
                       kv_dtype: int = 0, multi_token: bool = False, one_chunk=None) -> int:
    """Chunk size decode_step's step grid uses for layers scoring at most max_keys[i] keys."""
    n = len(max_keys)
    mk = (ctypes.c_int32 * n)(*[int(x) for x in max_keys])
    oc = None if one_chunk is None else (ctypes.c_uint8 * n)(*[1 if x else 0 for x in one_chunk])
    ck = ctypes.c_int32()
    _check(_lib.hd_plan_step_split(n, mk, oc, batch, num_kv_heads, rows, int(bool(multi_token)), kv_dtype,
                                   num_sms, ctypes.byref(ck)), "hd_plan_step_split")
    return ck.value


def hd_status_string(status: int) -> str:
    return _lib.hd_status_string(status).decode()


class Context:
    """Owns one ``hd_ctx``; create it with ``hybrid_decode_init``."""

    def __init__(self, handle: int, cfg: Config):
        self.handle = handle
        self.cfg = cfg

    def close(self) -> None:
        if self.handle:
            _check(_lib.hybrid_decode_destroy(self.handle), "hybrid_decode_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def hybrid_decode_init(cfg: Config) -> Context:
    h = ctypes.c_void_p()
    _check(_lib.hybrid_decode_init(ctypes.byref(cfg.to_c()), ctypes.byref(h)), "hybrid_decode_init")
    return Context(h.value, cfg)


def hybrid_decode_destroy(ctx: Context) -> None:
    ctx.close()


def rope_append_kv(ctx: Context, layer: int, context: torch.Tensor, q, k, v, q_rot, cache: hd_kv_cache,
                   stream=None) -> None:
    _check_batch(cache, q.shape[0])
    _check(_lib.rope_append_kv(ctx.handle, layer, q.shape[0], _ptr(context), _ptr(q), _ptr(k), _ptr(v),
                               _ptr(q_rot), cache, _stream(stream)), "rope_append_kv")


def decode_attn_sliding(ctx: Context, layer: int, context, q_rot, cache: hd_kv_cache, sink, out, lse,
                        stream=None, gate=None) -> None:
    _check_sink(sink, ctx.cfg.num_q_heads, q_rot)
    _check_gate(gate, q_rot.shape[0], ctx.cfg.num_q_heads, q_rot)
    _check_batch(cache, q_rot.shape[0])
    _check(_lib.decode_attn_sliding(ctx.handle, layer, q_rot.shape[0], _ptr(context), _ptr(q_rot),
                                    cache, _ptr(sink), _ptr(gate), _ptr(out), _ptr(lse), _stream(stream)),
           "decode_attn_sliding")


def decode_attn_full(ctx: Context, layer: int, context, q_rot, cache: hd_kv_cache, sink, out, lse,
                     max_context_hint: int = 0, stream=None, gate=None) -> None:
    _check_sink(sink, ctx.cfg.num_q_heads, q_rot)
    _check_gate(gate, q_rot.shape[0], ctx.cfg.num_q_heads, q_rot)
    _check_batch(cache, q_rot.shape[0])
    _check(_lib.decode_attn_full(ctx.handle, layer, q_rot.shape[0], _ptr(context), max_context_hint,
                                 _ptr(q_rot), cache, _ptr(sink), _ptr(gate), _ptr(out), _ptr(lse),
                                 _stream(stream)), "decode_attn_full")


def layer_io(q, k, v, cache: hd_kv_cache, sink, out, lse, gate=None) -> hd_layer_io:
    """One layer's tensors for decode_step (q [B, Hq, D]) or decode_step_tokens
    (q [B, T, Hq, D]; k/v/out/lse/gate with the same token index)."""
    if sink is not None:
        _check_sink(sink, q.shape[-2], q)
    _check_gate(gate, q.shape[0], q.shape[-2], q, tokens=q.shape[1] if q.dim() == 4 else None)
    _check_batch(cache, q.shape[0])
    return hd_layer_io(_ptr(q), _ptr(k), _ptr(v), cache, _ptr(sink), _ptr(out), _ptr(lse), _ptr(gate))


def layer_array(ctx: Context, layers) -> ctypes.Array:
    """The host array of hd_layer_io decode_step reads, one entry per layer of the
    context; build it once and pass it to every step whose tensors stay the same."""
    if isinstance(layers, ctypes.Array) and layers._type_ is hd_layer_io:
        arr = layers
    else:
        arr = (hd_layer_io * len(layers))(*layers)
    if len(arr) != len(ctx.cfg.layer_types):
        raise ValueError(f"decode_step needs one hd_layer_io per layer ({len(ctx.cfg.layer_types)}), got {len(arr)}")
    return arr


def decode_step(ctx: Context, context: torch.Tensor, layers, batch: int,
                max_context_hint: int = 0, stream=None) -> None:
    """layers: a list of hd_layer_io (one per layer) or an array from layer_array()."""
    _check(_lib.decode_step(ctx.handle, batch, _ptr(context), max_context_hint, layer_array(ctx, layers),
                            _stream(stream)), "decode_step")


def decode_step_tokens(ctx: Context, context: torch.Tensor, layers: list, batch: int, num_tokens: int,
                       max_context_hint: int = 0, stream=None) -> None:
    """num_tokens new tokens per sequence (q/out [B, T, Hq, D], k/v [B, T, Hkv, D],
    lse/gate [B, T, Hq]), equal to num_tokens decode_step calls in order.  layers as
    for decode_step."""
    _check(_lib.decode_step_tokens(ctx.handle, batch, num_tokens, _ptr(context), max_context_hint,
                                   layer_array(ctx, layers), _stream(stream)), "decode_step_tokens")


def hybrid_decode_device_errors(ctx: Context, stream=None) -> int:
    f = ctypes.c_int32()
    _check(_lib.hybrid_decode_device_errors(ctx.handle, ctypes.byref(f), _stream(stream)),
           "hybrid_decode_device_errors")
    return f.value


def hybrid_decode_launch_count(ctx: Context) -> int:
    n = ctypes.c_int64()
    _check(_lib.hybrid_decode_launch_count(ctx.handle, ctypes.byref(n)), "hybrid_decode_launch_count")
    return n.value


def hybrid_decode_set_profiling(ctx: Context, mask: int) -> None:
    """mask of launches to bracket with events: HD_PROFILE_SLIDING | HD_PROFILE_FULL (layer
    kernels), HD_PROFILE_STEP (step grids), or 0; with HD_PROFILE_FIRST_ONLY only the first
    layer kernel of each type per decode_step."""
    _check(_lib.hybrid_decode_set_profiling(ctx.handle, int(mask)), "hybrid_decode_set_profiling")


def hybrid_decode_profile(ctx: Context, layer_type: int = HD_FULL) -> tuple[float, int]:
    """(summed kernel milliseconds, launches) of the given layer type (or HD_PROFILE_KIND_STEP:
    step grids) since the last read."""
    ms, n = ctypes.c_double(), ctypes.c_int64()
    _check(_lib.hybrid_decode_profile(ctx.handle, layer_type, ctypes.byref(ms), ctypes.byref(n)),
           "hybrid_decode_profile")
    return ms.value, n.value


def hybrid_decode_set_layer_overlap(ctx: Context, enable: bool) -> None:
    """Whether decode_step lets a layer start before the previous one finishes (default on)."""
    _check(_lib.hybrid_decode_set_layer_overlap(ctx.handle, int(bool(enable))), "hybrid_decode_set_layer_overlap")


def hybrid_decode_set_step_fusion(ctx: Context, enable: bool) -> None:
    """Whether decode_step runs the attention of all layers as one grid (default on)."""
    _check(_lib.hybrid_decode_set_step_fusion(ctx.handle, int(bool(enable))), "hybrid_decode_set_step_fusion")


def hybrid_decode_set_cluster_combine(ctx: Context, enable: bool) -> None:
    """Single-layer launches of small grids merge their chunks inside a
    thread-block cluster (default True), or through the workspace (False)."""
    _check(_lib.hybrid_decode_set_cluster_combine(ctx.handle, 1 if enable else 0), "hybrid_decode_set_cluster_combine")


def hybrid_decode_set_consumer(ctx: Context, consumer: int) -> None:
    """HD_CONSUMER_CUDA_CORE, HD_CONSUMER_TENSOR_CORE (the default) or
    HD_CONSUMER_TENSOR_MEMORY (tcgen05 for 16-row multi-token passes over bf16 caches)."""
    _check(_lib.hybrid_decode_set_consumer(ctx.handle, consumer), "hybrid_decode_set_consumer")


def decode_attn_full_static_scratch(num_kv_heads: int, context, max_context: int, q_rot,
                                    cache: hd_kv_cache, sink, out, lse, stream=None) -> None:
    """Full-layer attention without a context and without any allocation: for
    callers that cannot allocate device memory while running.  The scratch is a
    64 MiB array inside the library, shared by all calls: calls that overlap on
    the GPU race, so order them on one stream.  See include/hybrid_decode.h."""
    batch, num_q_heads = q_rot.shape[0], q_rot.shape[1]
    _check_sink(sink, num_q_heads, q_rot)
    _check_batch(cache, batch)
    _check(_lib.decode_attn_full_static_scratch(batch, num_q_heads, num_kv_heads, _ptr(context),
                                                max_context, _ptr(q_rot), cache, _ptr(sink), _ptr(out),
                                                _ptr(lse), _stream(stream)),
           "decode_attn_full_static_scratch")


def decode_attn_full_static_scratch_plan(batch: int, num_q_heads: int, num_kv_heads: int, max_context: int,
                                         num_sms: int) -> tuple[int, int, int, int]:
    """(scratch bytes, keys per chunk, chunks, status) of decode_attn_full_static_scratch
    for this shape (pure host function).  Status 0: the call fits the array; 3
    (HD_ERR_CAPACITY): it would be refused; 1 / 2: the shape is rejected."""
    nbytes, chunk, chunks = _i64(0), _i32(0), _i32(0)
    st = _lib.decode_attn_full_static_scratch_plan(batch, num_q_heads, num_kv_heads, max_context, num_sms,
                                                   ctypes.byref(nbytes), ctypes.byref(chunk), ctypes.byref(chunks))
    return nbytes.value, chunk.value, chunks.value, st


def hd_validate_paged(cfg: Config, batch: hd_paged_batch, cache: hd_paged_cache) -> int:
    """Status of the pure host check that every paged call makes on its descriptors."""
    return _lib.hd_validate_paged(ctypes.byref(cfg.to_c()), ctypes.byref(batch), ctypes.byref(cache))


class PagedCache:
    """A pool of K/V pages (see ``paged_cache``): the C descriptor and the tensors it points into."""

    def __init__(self, c, keep, shape, device):
        self.c, self.ref, self.keep = c, ctypes.byref(c), keep
        self.num_kv_heads, self.device = shape[1], device


class PagedBatch:
    """The sequences of a paged call (see ``paged_batch``): the C descriptor and its tensors."""

    def __init__(self, c, keep, device):
        self.c, self.ref, self.keep = c, ctypes.byref(c), keep
        self.num_tokens, self.device = c.num_tokens, device


def paged_cache(k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor | None = None,
                v_scale: torch.Tensor | None = None, bounds: torch.Tensor | None = None) -> PagedCache:
    """Describe a pool of pages shaped [num_pages, num_kv_heads, page_size, head_dim] on CUDA:
    bf16, or E4M3 codes (uint8 or float8_e4m3fn) with fp32 ``k_scale``/``v_scale`` of shape
    [num_kv_heads].  Pages may lie apart (stride 0) but each is contiguous.  ``bounds``: bf16
    [num_pages, num_kv_heads, 2, head_dim] for select_pages.  Keep it while the tensors stay."""
    if k.shape != v.shape or k.dim() != 4 or any(a != b for n, a, b in zip(k.shape, k.stride(), v.stride()) if n > 1):
        raise ValueError("k and v pages must share a [num_pages, kv_heads, page_size, head_dim] layout")
    if not k.is_cuda or v.device != k.device:
        raise ValueError("pages must be CUDA tensors on one device")
    P, H, S, D = k.shape
    fp8 = k.dtype in _FP8_CACHE_TYPES
    if v.dtype != k.dtype or not (fp8 or k.dtype == torch.bfloat16):
        raise ValueError("pages must be bf16, or E4M3 codes with scales, K and V alike")
    if (D != 256 or (H > 1 and k.stride(1) != S * D) or (S > 1 and k.stride(2) != D) or k.stride(3) != 1 or
            (P > 1 and k.stride(0) < H * S * D)):
        raise ValueError("each page must be contiguous [kv_heads, page_size, 256] and pages may not overlap")
    for name, sc in (("k_scale", k_scale), ("v_scale", v_scale)):
        if not fp8:
            if sc is not None:
                raise ValueError("scales belong to FP8 caches only")
        elif (sc is None or sc.dtype != torch.float32 or tuple(sc.shape) != (H,) or sc.device != k.device or
              not sc.is_contiguous()):
            raise ValueError(f"E4M3 pages need {name} as contiguous float32 of shape ({H},) on the pages' device")
    if bounds is not None and (bounds.dtype != torch.bfloat16 or tuple(bounds.shape) != (P, H, 2, D) or
                               bounds.device != k.device or not bounds.is_contiguous()):
        raise ValueError(f"bounds must be contiguous bf16 of shape ({P}, {H}, 2, {D}) on the pages' device")
    c = hd_paged_cache(k.data_ptr(), v.data_ptr(), k.stride(0) if P > 1 else H * S * D, P, S, _ptr(k_scale),
                       _ptr(v_scale), _ptr(bounds))
    r = PagedCache(c, (k, v, k_scale, v_scale, bounds), k.shape, k.device)
    r.fp8 = fp8
    return r


def paged_batch(block_table: torch.Tensor, context: torch.Tensor, token_offsets: torch.Tensor | None = None,
                num_tokens: int | None = None, max_tokens: int = 1, max_context: int = 0) -> PagedBatch:
    """Describe the sequences of a paged call: int32 CUDA tensors ``block_table`` [batch, max_blocks],
    ``context`` [batch] (previous tokens) and ``token_offsets`` [batch + 1] (None: one new token per
    sequence).  ``num_tokens``: rows of q / k / v / out (default: the batch); ``max_tokens`` and
    ``max_context``: bounds on a sequence's new tokens and context (0: the configuration's).  They
    pick kernels, so a call with bounds near the truth (1 for prompts from their start) is faster:
    16 tokens from a sequence's start, scored, 8.5 us with 1 and 18.7 with 0 and a table of 32768
    positions."""
    batch = context.shape[0]
    if context.dim() != 1 or block_table.dim() != 2 or block_table.shape[0] != batch:
        raise ValueError("block_table must be [batch, max_blocks] and context [batch]")
    for name, t in (("block_table", block_table), ("context", context), ("token_offsets", token_offsets)):
        if t is not None and (t.dtype != torch.int32 or t.device != context.device or not t.is_cuda or
                              (t.numel() > 0 and t.shape[-1] > 1 and t.stride(-1) != 1)):
            raise ValueError(f"{name} must be an int32 CUDA tensor with unit stride, on one device with the others")
    if token_offsets is not None and (token_offsets.dim() != 1 or token_offsets.shape[0] != batch + 1):
        raise ValueError(f"token_offsets must have shape ({batch + 1},)")
    if batch > 1 and block_table.stride(0) < block_table.shape[1]:
        raise ValueError("rows of the block table may not overlap")
    c = hd_paged_batch(block_table.data_ptr(), context.data_ptr(), _ptr(token_offsets),
                       block_table.stride(0) if batch > 1 else block_table.shape[1], block_table.shape[1], batch,
                       batch if num_tokens is None else num_tokens, max_tokens, max_context)
    return PagedBatch(c, (block_table, context, token_offsets), context.device)


def _check_rows(name: str, t: torch.Tensor, shape: tuple, dtype, device, strided: bool = False) -> int:
    """A tensor of a paged call: its shape, type and device; contiguous, or (strided) contiguous rows, of which
    it returns the stride."""
    if t.shape != shape or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be {dtype} of shape {shape} on {device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    if t.is_contiguous():
        return shape[1] * shape[2] if strided else 0
    if not (strided and t.stride(2) == 1 and (shape[1] == 1 or t.stride(1) == shape[2])):
        raise ValueError(f"{name} must be contiguous" + (" within each row" if strided else ""))
    return t.stride(0) if shape[0] > 1 else shape[1] * shape[2]


def _check_paged(ctx: Context, batch: PagedBatch, cache: PagedCache) -> None:
    if cache.num_kv_heads != ctx.cfg.num_kv_heads or cache.fp8 != (ctx.cfg.kv_dtype == HD_KV_FP8_E4M3):
        raise ValueError("the pages' kv heads and element type must be the context's")
    if batch.device != cache.device or cache.device.index != torch.cuda.current_device():
        raise ValueError("the batch and the pages must be on the current device")


def _check_append(ctx: Context, batch: PagedBatch, q, k, v, q_rot, cache: PagedCache) -> tuple:
    """Row strides of q (0: none), k and v."""
    _check_paged(ctx, batch, cache)
    n, D, dev = batch.num_tokens, 256, cache.device
    kv = (n, ctx.cfg.num_kv_heads, D)
    ks = _check_rows("k", k, kv, torch.bfloat16, dev, True)
    vs = _check_rows("v", v, kv, torch.bfloat16, dev, True)
    qs = 0
    if (q is None) != (q_rot is None):
        raise ValueError("q and q_rot go together")
    if q is not None:
        qs = _check_rows("q", q, (n, ctx.cfg.num_q_heads, D), torch.bfloat16, dev, True)
        _check_rows("q_rot", q_rot, (n, ctx.cfg.num_q_heads, D), torch.bfloat16, dev)
    return qs, ks, vs


def rope_append_paged(ctx: Context, layer: int, batch: PagedBatch, q, k, v, q_rot, cache: PagedCache,
                      stream=None) -> None:
    """Rotate the new q [num_tokens, Hq, 256] into q_rot (bf16; may be q) and the new k, and store
    k / v [num_tokens, Hkv, 256] in their pages, with the pages' bounds when the cache has them.
    q, k and v may be parts of wider rows; q and q_rot may both be None."""
    qs, ks, vs = _check_append(ctx, batch, q, k, v, q_rot, cache)
    _check(_lib.rope_append_paged(ctx.handle, layer, batch.ref, _ptr(q), qs, k.data_ptr(), ks, v.data_ptr(), vs,
                                  _ptr(q_rot), cache.ref, _stream(stream)), "rope_append_paged")


def _check_attn_paged(ctx: Context, batch: PagedBatch, q_rot, cache: PagedCache, sink, gate, out, lse) -> None:
    _check_paged(ctx, batch, cache)
    n, Hq, dev = batch.num_tokens, ctx.cfg.num_q_heads, cache.device
    _check_rows("q_rot", q_rot, (n, Hq, 256), torch.bfloat16, dev)
    _check_rows("out", out, (n, Hq, 256), torch.bfloat16, dev)
    _check_rows("lse", lse, (n, Hq), torch.float32, dev)
    _check_sink(sink, Hq, q_rot)
    _check_gate(gate, n, Hq, q_rot)


def attn_paged(ctx: Context, layer: int, batch: PagedBatch, q_rot, cache: PagedCache, sink, out, lse, gate=None,
               stream=None) -> None:
    """Attention of every new token over its sequence's pages (appended before by
    rope_append_paged), one token per sequence or chunks: q_rot / out [num_tokens, Hq, 256] bf16,
    lse / gate [num_tokens, Hq] fp32."""
    _check_attn_paged(ctx, batch, q_rot, cache, sink, gate, out, lse)
    _check(_lib.attn_paged(ctx.handle, layer, batch.ref, q_rot.data_ptr(), cache.ref, _ptr(sink), _ptr(gate),
                           out.data_ptr(), lse.data_ptr(), _stream(stream)), "attn_paged")


def select_pages(ctx: Context, layer: int, batch: PagedBatch, q_rot, cache: PagedCache, selected, keep_first: int = 1,
                 keep_last: int = 1, stream=None) -> None:
    """Choose for every new token and kv head the blocks it attends to, by the pages' bounds:
    ``selected`` int32 [num_tokens, Hkv, num_selected], ascending, -1 behind the last."""
    _check_paged(ctx, batch, cache)
    _check_rows("q_rot", q_rot, (batch.num_tokens, ctx.cfg.num_q_heads, 256), torch.bfloat16, cache.device)
    _check_rows("selected", selected, (batch.num_tokens, ctx.cfg.num_kv_heads, selected.shape[-1]), torch.int32,
                cache.device)
    _check(_lib.select_pages(ctx.handle, layer, batch.ref, q_rot.data_ptr(), cache.ref, selected.shape[-1], keep_first,
                             keep_last, selected.data_ptr(), _stream(stream)), "select_pages")


def attn_selected_pages(ctx: Context, layer: int, batch: PagedBatch, q_rot, cache: PagedCache, selected, sink, out, lse,
                        gate=None, stream=None) -> None:
    """attn_paged restricted, for every token and kv head, to the blocks in ``selected``."""
    _check_attn_paged(ctx, batch, q_rot, cache, sink, gate, out, lse)
    _check_rows("selected", selected, (batch.num_tokens, ctx.cfg.num_kv_heads, selected.shape[-1]), torch.int32,
                cache.device)
    _check(_lib.attn_selected_pages(ctx.handle, layer, batch.ref, q_rot.data_ptr(), cache.ref, selected.data_ptr(),
                                    selected.shape[-1], _ptr(sink), _ptr(gate), out.data_ptr(), lse.data_ptr(),
                                    _stream(stream)), "attn_selected_pages")


def _rope_params(rotary_dim, theta, scaling, factor, original_context, slow, fast, amplitude) -> hd_rope_params:
    return hd_rope_params(rotary_dim, scaling, theta, factor, original_context, slow, fast, amplitude)


def hd_rope_frequencies(rotary_dim: int, theta: float = 1.0e4, scaling: int = HD_ROPE_PLAIN, factor: float = 1.0,
                        original_context: float = 0.0, slow: float = 1.0, fast: float = 32.0,
                        amplitude: float = 0.0) -> tuple[list, float]:
    """(frequencies of the rotary_dim / 2 pairs in radians a position, amplitude) of a table of
    angles (pure host function); the arguments are hd_rope_params' in include/hybrid_decode.h."""
    p = _rope_params(rotary_dim, theta, scaling, factor, original_context, slow, fast, amplitude)
    f, m = (ctypes.c_double * 128)(), ctypes.c_double()
    _check(_lib.hd_rope_frequencies(ctypes.byref(p), f, ctypes.byref(m)), "hd_rope_frequencies")
    return list(f[: rotary_dim // 2]), m.value


class RopeTable:
    """A table of angles (see ``rope_table``): the C descriptor and its tensor."""

    def __init__(self, c, table):
        self.c, self.ref, self.table = c, ctypes.byref(c), table


def rope_table(rotary_dim: int, positions: int, theta: float = 1.0e4, layout: int = HD_ROPE_HALVES,
               scaling: int = HD_ROPE_PLAIN, factor: float = 1.0, original_context: float = 0.0, slow: float = 1.0,
               fast: float = 32.0, amplitude: float = 0.0, table: torch.Tensor | None = None, stream=None) -> RopeTable:
    """A table of ``positions`` rows of angles for norm_rope_append_paged, made once for a model:
    HD_ROPE_PLAIN, or scaled for long contexts (LINEAR, RAMP, BANDS; include/hybrid_decode.h has the
    formulas), turning dims in HD_ROPE_HALVES or as HD_ROPE_NEIGHBOURS.  ``table``: float32
    [positions, rotary_dim / 2, 2] on the current device to fill (default: a new one, of ``stream``'s
    memory when one is given: other streams wait for that one before they use the table)."""
    p = _rope_params(rotary_dim, theta, scaling, factor, original_context, slow, fast, amplitude)
    f, m = (ctypes.c_double * 128)(), ctypes.c_double()
    _check(_lib.hd_rope_frequencies(ctypes.byref(p), f, ctypes.byref(m)), "rope_table")
    if layout not in (HD_ROPE_HALVES, HD_ROPE_NEIGHBOURS) or positions < 1:
        raise ValueError("layout must be HD_ROPE_HALVES or HD_ROPE_NEIGHBOURS, positions at least 1")
    shape = (positions, rotary_dim // 2, 2)
    if table is None:
        # Memory that the current stream gave back may still be written there: a fill elsewhere takes its own stream's.
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream))
        with torch.cuda.stream(stream):
            table = torch.empty(shape, dtype=torch.float32, device=torch.device("cuda", torch.cuda.current_device()))
    elif (tuple(table.shape) != shape or table.dtype != torch.float32 or not table.is_contiguous() or not table.is_cuda or
          table.device.index != torch.cuda.current_device()):
        raise ValueError(f"table must be contiguous float32 of shape {shape} on the current device")
    _check(_lib.hd_rope_fill(ctypes.byref(p), positions, table.data_ptr(), _stream(stream)), "rope_table")
    return RopeTable(hd_rope_table(table.data_ptr(), positions, rotary_dim, layout), table)


def _check_ints(name: str, t, n: int, device) -> None:
    if t is not None and (t.dtype != torch.int32 or tuple(t.shape) != (n,) or t.device != device or not t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous int32 of shape ({n},) on {device}")


def _check_weight(name: str, w: torch.Tensor, heads: int, device) -> tuple:
    """A norm's weight: its (type, dims)."""
    dtype, dims = w.dtype, w.dim()
    if (w.shape != ((256,) if dims == 1 else (heads, 256)) or not (dtype is torch.bfloat16 or dtype is torch.float32) or
            w.device != device or not w.is_contiguous()):
        raise ValueError(f"{name} must be contiguous bf16 or float32 of shape (256,) or ({heads}, 256) on {device}")
    return dtype, dims


def norm_rope_append_paged(ctx: Context, layer: int, batch: PagedBatch, q, k, v, q_rot, cache: PagedCache,
                           rope: RopeTable | None = None, q_weight: torch.Tensor | None = None,
                           k_weight: torch.Tensor | None = None, eps: float = 1.0e-6, weight_offset: float = 0.0,
                           positions: torch.Tensor | None = None, norm: bool = True, stream=None) -> None:
    """rope_append_paged for models that norm the heads of their queries and keys or turn them by other
    angles: y = x / rms(x) * (weight_offset + weight), rotated by ``rope`` (None: the context's own
    angles) at the rows' positions in their sequences, or at ``positions`` (int32 [num_tokens]).
    ``q_weight`` / ``k_weight``: bf16 or float32 [256], or one row a head ([Hq, 256] and [Hkv, 256]);
    None: ones.  ``norm=False``: the rotation alone."""
    qs, ks, vs = _check_append(ctx, batch, q, k, v, q_rot, cache)
    if positions is not None:
        _check_ints("positions", positions, batch.num_tokens, cache.device)
    if rope is not None and rope.table.device != cache.device:
        raise ValueError("the table of angles must be on the pages' device")
    ref = None
    if norm:
        kind, q_ptr, k_ptr = (), None, None   # (type, dims) of the weights
        if q_weight is not None:
            kind, q_ptr = _check_weight("q_weight", q_weight, ctx.cfg.num_q_heads, cache.device), q_weight.data_ptr()
        if k_weight is not None:
            other, k_ptr = _check_weight("k_weight", k_weight, ctx.cfg.num_kv_heads, cache.device), k_weight.data_ptr()
            if kind and other != kind:
                raise ValueError("q_weight and k_weight must share a type and be both per head or both shared")
            kind = other
        ref = ctypes.byref(hd_head_norm(q_ptr, k_ptr, torch.float32 in kind, 2 in kind, weight_offset, eps))
    elif q_weight is not None or k_weight is not None:
        raise ValueError("weights belong to a norm")
    _check(_lib.norm_rope_append_paged(ctx.handle, layer, batch.ref, ref, None if rope is None else rope.ref, _ptr(positions),
                                       _ptr(q), qs, k.data_ptr(), ks, v.data_ptr(), vs, _ptr(q_rot),
                                       cache.ref, _stream(stream)), "norm_rope_append_paged")


class Scoring:
    """A rule of scores and visible positions (see ``scoring``): the C descriptor and its tensors."""

    def __init__(self, c, slopes, first, last):
        self.c, self.ref, self.slopes, self.first, self.last = c, ctypes.byref(c), slopes, first, last


def scoring(softcap: float = 0.0, scale: float = 0.0, slopes: torch.Tensor | None = None, first: torch.Tensor | None = None,
            last: torch.Tensor | None = None) -> Scoring:
    """How attn_paged_scored scores and masks: scores scale * q.k (0: 1/16), capped at ``softcap`` by a
    tanh (0: not), less ``slopes[head]`` (float32 [Hq]) times the distance of query and key; row r sees
    the positions ``first[r]`` .. ``last[r]`` (int32 [num_tokens], both ascending along a sequence's rows;
    None: 0 and its own position), within a sliding layer's window and the sequence.  Few rows are
    served by the kernel that the batch's bounds (``paged_batch``) say is sooner."""
    return Scoring(hd_scoring(scale, softcap, _ptr(slopes), _ptr(first), _ptr(last)), slopes, first, last)


def attn_paged_scored(ctx: Context, layer: int, batch: PagedBatch, rule: Scoring | None, q_rot, cache: PagedCache, sink, out,
                      lse, gate=None, stream=None) -> None:
    """attn_paged with capped or biased scores and masks of documents and prefixes (``scoring``; None: attn_paged's own)."""
    if rule is None:
        return attn_paged(ctx, layer, batch, q_rot, cache, sink, out, lse, gate, stream)
    _check_attn_paged(ctx, batch, q_rot, cache, sink, gate, out, lse)
    if rule.slopes is not None and (rule.slopes.dtype != torch.float32 or tuple(rule.slopes.shape) != (ctx.cfg.num_q_heads,) or
                                    rule.slopes.device != cache.device or not rule.slopes.is_contiguous()):
        raise ValueError(f"slopes must be contiguous float32 of shape ({ctx.cfg.num_q_heads},) on {cache.device}")
    _check_ints("first", rule.first, batch.num_tokens, cache.device)
    _check_ints("last", rule.last, batch.num_tokens, cache.device)
    _check(_lib.attn_paged_scored(ctx.handle, layer, batch.ref, rule.ref, q_rot.data_ptr(), cache.ref, _ptr(sink), _ptr(gate),
                                  out.data_ptr(), lse.data_ptr(), _stream(stream)), "attn_paged_scored")


def read_paged(ctx: Context, batch: PagedBatch, cache: PagedCache, k=None, v=None, stream=None) -> None:
    """Read entries back: k / v [num_tokens, Hkv, 256] bf16 (either may be None, rows may be parts of wider
    ones) get the entries at the batch's "new" positions, context[b] onwards; E4M3 codes times their
    scale, rounded once.  Keys come as stored, rotated."""
    _check_paged(ctx, batch, cache)
    shape = (batch.num_tokens, ctx.cfg.num_kv_heads, 256)
    ks, vs = (0 if t is None else _check_rows(name, t, shape, torch.bfloat16, cache.device, True)
              for name, t in (("k", k), ("v", v)))
    _check(_lib.read_paged(ctx.handle, batch.ref, cache.ref, _ptr(k), ks, _ptr(v), vs, _stream(stream)), "read_paged")


def hybrid_decode_read_probe(buffer: torch.Tensor, stream=None) -> int:
    """One pass of a pure read stream over a device buffer; returns the bytes the
    pass covers (a whole number of 32 KiB stages per CTA).  Time it with events."""
    nbytes = buffer.numel() * buffer.element_size()
    _check(_lib.hybrid_decode_read_probe(_ptr(buffer), nbytes, _stream(stream)), "hybrid_decode_read_probe")
    ctas = 2 * torch.cuda.get_device_properties(buffer.device).multi_processor_count
    return (nbytes // (32 * 1024) // ctas) * ctas * 32 * 1024


def hybrid_decode_inject_lost_copy(ctx: Context, stage: int) -> None:
    """Test hook: attention producers stop issuing copies at `stage` (-1: off)."""
    _check(_lib.hybrid_decode_inject_lost_copy(ctx.handle, stage), "hybrid_decode_inject_lost_copy")

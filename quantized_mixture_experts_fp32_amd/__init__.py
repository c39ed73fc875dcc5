"""MI355X (gfx950) routed-expert MoE FFN with low-bit weight-only experts.

Thin Python binding of the C ABI in `include/moe_wq.h` (libmoe_wq.so).  The
functions below only marshal torch tensors into pointers and sizes; every
step of the layer runs in the library's HIP kernels.  PyTorch provides
device memory and the current HIP stream.  There is no CPU fallback: the
library must be built (`build.build()`) and a GPU present, or calls raise.

Layer = moe_route -> moe_permute -> moe_expert_ffn_wq -> moe_combine (the
first two also as one call, moe_route_permute).
"""
from __future__ import annotations

import collections
import contextlib
import ctypes
import functools
import inspect
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_wq.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = range(5)
MOE_FMT_W4_SYM, MOE_FMT_BITPLANE8 = 0, 1
MOE_BITS_NONE, MOE_BITS_PER_PAIR, MOE_BITS_PER_EXPERT, MOE_BITS_RANK_RULE = 0, 1, 2, 3
MOE_OUT_BF16, MOE_OUT_F32 = 0, 1
MOE_PATH_AUTO, MOE_PATH_DECODE, MOE_PATH_PREFILL = 0, 1, 2
MOE_GATE_NONE, MOE_GATE_TOKEN, MOE_GATE_CHANNEL = 0, 1, 2
MOE_GROUP = 128

# Every symbol the header declares (checked by the CPU tests).
EXPORTS = ("moe_status_str", "moe_last_error", "moe_route_ws_bytes", "moe_route",
           "moe_permute_ws_bytes",
           "moe_permute", "moe_route_permute_ws_bytes", "moe_route_permute",
           "moe_ffn_ws_bytes", "moe_expert_ffn_wq", "moe_combine",
           "moe_quantize_w4", "moe_quantize_bitplane8", "moe_set_ffn_events",
           "moe_layer_ws_bytes", "moe_layer_forward_wq", "moe_layer_forward_wq_noalloc",
           "moe_bp_distortion_ws_bytes",
           "moe_bp_distortion", "moe_allocate_bits", "moe_cache_create", "moe_cache_destroy",
           "moe_cache_ws_bytes", "moe_cache_forward", "moe_cache_stats", "moe_cache_slots",
           "moe_cache_reset", "moe_cache_plan", "moe_retile_w4", "moe_retile_bitplane8",
           "moe_linear_w4_ws_bytes", "moe_linear_w4_kernel", "moe_linear_w4", "moe_rmsnorm",
           "moe_rmsnorm_bwd_ws_bytes", "moe_rmsnorm_bwd", "moe_combine_residual",
           "moe_combine_residual_bwd_ws_bytes", "moe_combine_residual_bwd", "moe_dispatch",
           "moe_dispatch_bwd", "moe_combine_bwd", "moe_quantize_i8", "moe_dequantize_i8",
           "moe_rmsnorm_i8", "moe_rmsnorm_bwd_i8", "moe_linear_i8_ws_bytes",
           "moe_linear_i8_kernel", "moe_linear_i8", "moe_gated_ffn_ws_bytes",
           "moe_gated_ffn_kernel", "moe_gated_ffn", "moe_gated_ffn_bwd_ws_bytes",
           "moe_gated_ffn_bwd")


class MoeError(RuntimeError):
    def __init__(self, fn, status, detail):
        super().__init__(f"{fn} failed: {status_str(status)} ({detail})")
        self.status = status


_lib = None


def load_library():
    """Load libmoe_wq.so (and with it libmoe_wq_i8.so beside it); raise if they have
    not been built."""
    global _lib
    if _lib is not None:
        return _lib
    for path in (LIB_PATH, os.path.join(os.path.dirname(LIB_PATH), "libmoe_wq_i8.so")):
        if not os.path.exists(path):
            raise RuntimeError(f"{path} not built: run "
                               "quantized_mixture_experts_fp32_amd.build.build()")
    lib = ctypes.CDLL(LIB_PATH)
    i32, vp, sz = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    lib.moe_status_str.argtypes, lib.moe_status_str.restype = [i32], ctypes.c_char_p
    lib.moe_last_error.argtypes, lib.moe_last_error.restype = [], ctypes.c_char_p
    lib.moe_route_ws_bytes.argtypes, lib.moe_route_ws_bytes.restype = [i32, i32], sz
    lib.moe_route.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, sz, vp]
    lib.moe_permute_ws_bytes.argtypes, lib.moe_permute_ws_bytes.restype = [i32, i32, i32], sz
    lib.moe_permute.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    lib.moe_route_permute_ws_bytes.argtypes = [i32, i32, i32]
    lib.moe_route_permute_ws_bytes.restype = sz
    lib.moe_route_permute.argtypes = [vp, vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp,
                                      vp, sz, vp]
    lib.moe_ffn_ws_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.moe_ffn_ws_bytes.restype = sz
    lib.moe_expert_ffn_wq.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, i32, i32,
                                      vp, vp, vp, vp, vp, i32, vp, vp, sz, i32, vp]
    lib.moe_combine.argtypes = [vp, vp, vp, i32, i32, i32, vp, i32, vp]
    lib.moe_quantize_w4.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp]
    lib.moe_quantize_bitplane8.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp]
    lib.moe_set_ffn_events.argtypes = [vp, vp, vp, vp]
    lib.moe_layer_ws_bytes.argtypes = [i32, i32, i32, i32, i32, i32]
    lib.moe_layer_ws_bytes.restype = sz
    lib.moe_layer_forward_wq.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, i32, i32,
                                         vp, vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp,
                                         vp, i32, vp, sz, i32, vp]
    lib.moe_layer_forward_wq_noalloc.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, i32,
                                                 i32, vp, vp, vp, vp, vp, i32, vp, vp, vp,
                                                 vp, vp, vp, vp, i32, i32, vp]
    lib.moe_retile_w4.argtypes = [vp, i32, i32, i32, vp, vp]
    lib.moe_retile_bitplane8.argtypes = [vp, i32, i32, i32, vp, vp]
    lib.moe_bp_distortion_ws_bytes.argtypes = [i32, i32, i32]
    lib.moe_bp_distortion_ws_bytes.restype = sz
    lib.moe_bp_distortion.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, vp, sz, vp]
    lib.moe_allocate_bits.argtypes = [vp, vp, i32, i32, i32, i32, i32, ctypes.c_int64, vp,
                                      vp, vp, vp]
    lib.moe_cache_create.argtypes = [i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp,
                                     vp]
    lib.moe_cache_destroy.argtypes, lib.moe_cache_destroy.restype = [vp], None
    lib.moe_cache_ws_bytes.argtypes, lib.moe_cache_ws_bytes.restype = [vp, i32, i32], sz
    lib.moe_cache_forward.argtypes = [vp, vp, vp, vp, i32, i32, vp, i32, vp, vp, vp, vp, vp,
                                      i32, vp, sz, vp]
    lib.moe_cache_stats.argtypes = [vp, vp]
    lib.moe_cache_slots.argtypes = [vp, vp, vp]
    lib.moe_cache_reset.argtypes = [vp]
    lib.moe_cache_plan.argtypes = [i32, i32, i32, vp, vp, vp, ctypes.c_int64, vp, vp, vp, i32,
                                   vp, vp, i32, vp, vp]
    f32 = ctypes.c_float
    lib.moe_linear_w4_ws_bytes.argtypes, lib.moe_linear_w4_ws_bytes.restype = [i32] * 3, sz
    lib.moe_linear_w4_kernel.argtypes = [i32] * 3
    lib.moe_linear_w4_kernel.restype = ctypes.c_char_p
    lib.moe_linear_w4.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, vp, i32, vp, sz, vp]
    lib.moe_rmsnorm.argtypes = [vp, i32, vp, i32, i32, f32, vp, i32, vp]
    lib.moe_rmsnorm_bwd_ws_bytes.argtypes = [i32, i32]
    lib.moe_rmsnorm_bwd_ws_bytes.restype = sz
    lib.moe_rmsnorm_bwd.argtypes = [vp, i32, vp, i32, vp, vp, i32, i32, f32, vp, vp, vp, sz, vp]
    lib.moe_combine_residual.argtypes = [vp, i32, vp, vp, vp, i32, vp, vp, vp, i32, f32, f32, vp,
                                         i32, i32, vp, vp, vp]
    lib.moe_combine_residual_bwd_ws_bytes.argtypes = [i32, i32]
    lib.moe_combine_residual_bwd_ws_bytes.restype = sz
    lib.moe_combine_residual_bwd.argtypes = [vp, i32, vp, vp, vp, i32, vp, vp, vp, i32, f32, f32,
                                             i32, i32, vp, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_dispatch.argtypes = [vp, i32, vp, vp, i32, i32, i32, vp, vp]
    lib.moe_dispatch_bwd.argtypes = [vp, i32, vp, vp, vp, i32, i32, i32, vp, vp, vp]
    lib.moe_combine_bwd.argtypes = [vp, i32, vp, vp, vp, i32, i32, i32, vp, i32, vp, vp]
    lib.moe_quantize_i8.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp]
    lib.moe_dequantize_i8.argtypes = [vp, vp, i32, i32, i32, vp, i32, vp]
    lib.moe_rmsnorm_i8.argtypes = [vp, vp, vp, i32, i32, f32, vp, i32, vp]
    lib.moe_rmsnorm_bwd_i8.argtypes = [vp, i32, vp, vp, vp, vp, i32, i32, f32, vp, i32, vp, vp,
                                       sz, vp]
    lib.moe_linear_i8_kernel.argtypes = [i32] * 3
    lib.moe_linear_i8_kernel.restype = ctypes.c_char_p
    lib.moe_gated_ffn_kernel.argtypes = [i32] * 5
    lib.moe_gated_ffn_kernel.restype = ctypes.c_char_p
    lib.moe_linear_i8_ws_bytes.argtypes, lib.moe_linear_i8_ws_bytes.restype = [i32] * 4, sz
    lib.moe_linear_i8.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp, vp, i32, vp, sz, vp]
    lib.moe_gated_ffn_ws_bytes.argtypes, lib.moe_gated_ffn_ws_bytes.restype = [i32] * 3, sz
    lib.moe_gated_ffn.argtypes = [vp, vp, vp, i32, i32, i32, vp, i32, vp, vp, sz, vp]
    lib.moe_gated_ffn_bwd_ws_bytes.argtypes = [i32] * 6
    lib.moe_gated_ffn_bwd_ws_bytes.restype = sz
    lib.moe_gated_ffn_bwd.argtypes = [vp, i32, vp, vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, i32,
                                      vp, sz, vp]
    for name in ("moe_linear_w4", "moe_rmsnorm", "moe_rmsnorm_bwd", "moe_combine_residual",
                 "moe_combine_residual_bwd", "moe_dispatch", "moe_dispatch_bwd",
                 "moe_combine_bwd", "moe_quantize_i8", "moe_dequantize_i8", "moe_rmsnorm_i8",
                 "moe_rmsnorm_bwd_i8", "moe_linear_i8", "moe_gated_ffn", "moe_gated_ffn_bwd"):
        getattr(lib, name).restype = i32
    for name in ("moe_route", "moe_permute", "moe_route_permute", "moe_expert_ffn_wq",
                 "moe_combine", "moe_layer_forward_wq", "moe_layer_forward_wq_noalloc",
                 "moe_bp_distortion",
                 "moe_allocate_bits", "moe_cache_create", "moe_cache_forward",
                 "moe_cache_stats", "moe_cache_slots", "moe_cache_reset", "moe_cache_plan",
                 "moe_quantize_w4", "moe_quantize_bitplane8", "moe_set_ffn_events",
                 "moe_retile_w4", "moe_retile_bitplane8"):
        getattr(lib, name).restype = i32
    _lib = lib
    return lib


def status_str(status: int) -> str:
    return load_library().moe_status_str(int(status)).decode()


def _check(fn, rc):
    if rc != MOE_OK:
        raise MoeError(fn, rc, load_library().moe_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _empty(shape, dtype, like):
    import torch
    return torch.empty(shape, dtype=dtype, device=like.device)


@contextlib.contextmanager
def _launch_on(stream, values):
    """Makes `stream` current, so that what the call allocates comes from that
    stream's memory, and records the tensors among `values` on it, so that
    memory the caller frees meanwhile is not handed out before the call is
    through."""
    import torch
    with torch.cuda.stream(stream):
        if not torch.cuda.is_current_stream_capturing():
            for t in values:
                if isinstance(t, torch.Tensor) and t.device == stream.device:
                    t.record_stream(stream)
        yield


def _on_stream(fn):
    """For calls with an argument `stream` that create what they are not given:
    runs fn with that stream current."""
    at = list(inspect.signature(fn).parameters).index("stream")

    @functools.wraps(fn)
    def call(*args, **kw):
        stream = args[at] if len(args) > at else kw.get("stream")
        if stream is None:
            return fn(*args, **kw)
        with _launch_on(stream, (*args, *kw.values())):
            return fn(*args, **kw)

    return call


def _current_device():
    import torch
    return torch._C._cuda_getDevice()


def _launch_stream():
    """The current stream's handle, and whether it is recording a graph."""
    import torch
    return (torch._C._cuda_getCurrentRawStream(_current_device()),
            torch.cuda.is_current_stream_capturing())


class _StepBuffers:
    """Keeps a layer's buffers from step to step (_alloc makes them).

    A set serves one batch size on one stream and comes from that stream's
    memory, so that dropping it needs no wait.  A step that is recorded into a
    graph takes a set of its own from the graph's memory, which lasts as long
    as the graph does, and leaves it to no later step."""

    _held = None

    def _buffers(self, T, like):
        stream, recording = _launch_stream()
        if recording or self._held != (T, stream):
            self._held = None
            self._alloc(T, like)
            if not recording:
                self._held = (T, stream)


# ----------------------------------------------------------------- the ABI
def moe_route_ws_bytes(T, E):
    return int(load_library().moe_route_ws_bytes(T, E))


@_on_stream
def moe_route(x, wr, bias, k, topk_idx=None, topk_w=None, ws=None, stream=None):
    """x bf16 [T][d], wr bf16 [E][d], bias fp32 [E] or None -> (idx, w)."""
    import torch
    T, d = x.shape
    E = wr.shape[0]
    if topk_idx is None:
        topk_idx = _empty((T, k), torch.int32, x)
    if topk_w is None:
        topk_w = _empty((T, k), torch.float32, x)
    if ws is None:
        ws = _empty((max(moe_route_ws_bytes(T, E), 16),), torch.uint8, x)
    _check("moe_route", load_library().moe_route(
        _ptr(x), _ptr(wr), _ptr(bias), T, d, E, k, _ptr(topk_idx), _ptr(topk_w),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))
    return topk_idx, topk_w


def moe_permute_ws_bytes(T, k, E):
    return int(load_library().moe_permute_ws_bytes(T, k, E))


@_on_stream
def moe_permute(topk_idx, E, ws=None, offsets=None, sorted_pair=None,
                pair_pos=None, stream=None):
    """topk_idx int32 [T][k] -> (expert_offsets [E+1], sorted_pair, pair_pos)."""
    import torch
    T, k = topk_idx.shape
    P = T * k
    if offsets is None:
        offsets = _empty((E + 1,), torch.int32, topk_idx)
    if sorted_pair is None:
        sorted_pair = _empty((P,), torch.int32, topk_idx)
    if pair_pos is None:
        pair_pos = _empty((P,), torch.int32, topk_idx)
    need = moe_permute_ws_bytes(T, k, E)
    if ws is None:
        ws = _empty((max(need, 16),), torch.uint8, topk_idx)
    _check("moe_permute", load_library().moe_permute(
        _ptr(topk_idx), T, k, E, _ptr(offsets), _ptr(sorted_pair), _ptr(pair_pos),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))
    return offsets, sorted_pair, pair_pos


def moe_route_permute_ws_bytes(T, k, E):
    return int(load_library().moe_route_permute_ws_bytes(T, k, E))


@_on_stream
def moe_route_permute(x, wr, bias, k, ws=None, topk_idx=None, topk_w=None, offsets=None,
                      sorted_pair=None, pair_pos=None, stream=None):
    """moe_route then moe_permute in one call -> (idx, w, offsets, sorted_pair,
    pair_pos)."""
    import torch
    T, d = x.shape
    E = wr.shape[0]
    P = T * k
    if topk_idx is None:
        topk_idx = _empty((T, k), torch.int32, x)
    if topk_w is None:
        topk_w = _empty((T, k), torch.float32, x)
    if offsets is None:
        offsets = _empty((E + 1,), torch.int32, x)
    if sorted_pair is None:
        sorted_pair = _empty((P,), torch.int32, x)
    if pair_pos is None:
        pair_pos = _empty((P,), torch.int32, x)
    if ws is None:
        ws = _empty((max(moe_route_permute_ws_bytes(T, k, E), 16),), torch.uint8, x)
    _check("moe_route_permute", load_library().moe_route_permute(
        _ptr(x), _ptr(wr), _ptr(bias), T, d, E, k, _ptr(topk_idx), _ptr(topk_w),
        _ptr(offsets), _ptr(sorted_pair), _ptr(pair_pos), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))
    return topk_idx, topk_w, offsets, sorted_pair, pair_pos


def moe_ffn_ws_bytes(T, k, E, d, f, fmt=MOE_FMT_W4_SYM):
    return int(load_library().moe_ffn_ws_bytes(T, k, E, d, f, fmt))


@_on_stream
def moe_expert_ffn_wq(x, expert_offsets, sorted_pair, k, f, gate_up_codes,
                      gate_up_scales, down_codes, down_scales,
                      fmt=MOE_FMT_W4_SYM, bits=None, bits_mode=MOE_BITS_NONE,
                      y_pairs=None, ws=None, path=MOE_PATH_AUTO, stream=None):
    """Per-pair SwiGLU outputs y_pairs fp32 [T*k][d] in grouped order."""
    import torch
    T, d = x.shape
    E = expert_offsets.numel() - 1
    if y_pairs is None:
        y_pairs = _empty((T * k, d), torch.float32, x)
    need = moe_ffn_ws_bytes(T, k, E, d, f, fmt)
    if ws is None:
        ws = _empty((max(need, 256),), torch.uint8, x)
    _check("moe_expert_ffn_wq", load_library().moe_expert_ffn_wq(
        _ptr(x), _ptr(expert_offsets), _ptr(sorted_pair), T, k, E, d, f, fmt,
        MOE_GROUP, _ptr(gate_up_codes), _ptr(gate_up_scales), _ptr(down_codes),
        _ptr(down_scales), _ptr(bits), bits_mode, _ptr(y_pairs), _ptr(ws),
        ws.numel() * ws.element_size(), path, _stream(stream)))
    return y_pairs


def expert_ffn_per_expert(x, expert_offsets, sorted_pair, k, f, gate_up_codes,
                          gate_up_scales, down_codes, down_scales, y_pairs, ws,
                          fmt=MOE_FMT_W4_SYM, bits=None, bits_mode=MOE_BITS_NONE,
                          path=MOE_PATH_DECODE, stream=None, experts=None, events=None):
    """The sequential baseline of ExactMoE's ablation ("Every Expert Counts
    ...", Abstract: fused grouped execution against one launch per expert):
    the same expert FFN computed by one moe_expert_ffn_wq call per expert.
    Call e sees a one-expert problem whose expert_offsets are the pointer
    expert_offsets + e (so its slot range is [offsets[e], offsets[e+1]) of
    the shared sorted_pair / y_pairs) and whose weights are expert e's
    slices.  experts: the expert ids to launch (the activated ones, which
    the caller reads from the routing); None launches every expert, and
    those without pairs exit at once.  Writes the y_pairs rows of the
    launched experts like the grouped call.  ws must hold
    moe_ffn_ws_bytes(T, k, 1, d, f, fmt) bytes.  events: optional list with
    one 4-tuple of hipEvent_t handles per launched expert, armed with
    moe_set_ffn_events before that expert's call."""
    T, d = x.shape
    E = expert_offsets.numel() - 1
    lib = load_library()
    vp = ctypes.c_void_p
    esz = lambda t: (t.numel() // t.shape[0]) * t.element_size()
    gu_b, gus_b, dn_b, dns_b = (esz(gate_up_codes), esz(gate_up_scales),
                                esz(down_codes), esz(down_scales))
    wsb, st = ws.numel() * ws.element_size(), _stream(stream)
    for i, e in enumerate(range(E) if experts is None else experts):
        e = int(e)
        if events is not None:
            moe_set_ffn_events(*events[i])
        if not 0 <= e < E:
            raise ValueError(f"expert id {e} outside [0, {E})")
        # a per-expert bit-width array is indexed by the (one) local expert
        b = None if bits is None else vp(
            bits.data_ptr() + (e if bits_mode == MOE_BITS_PER_EXPERT else 0))
        _check("moe_expert_ffn_wq", lib.moe_expert_ffn_wq(
            _ptr(x), vp(expert_offsets.data_ptr() + 4 * e), _ptr(sorted_pair), T, k, 1, d,
            f, fmt, MOE_GROUP, vp(gate_up_codes.data_ptr() + e * gu_b),
            vp(gate_up_scales.data_ptr() + e * gus_b), vp(down_codes.data_ptr() + e * dn_b),
            vp(down_scales.data_ptr() + e * dns_b), b, bits_mode, _ptr(y_pairs),
            _ptr(ws), wsb, path, st))
    return y_pairs


def moe_layer_ws_bytes(T, k, E, d, f, fmt=MOE_FMT_W4_SYM):
    return int(load_library().moe_layer_ws_bytes(T, k, E, d, f, fmt))


def moe_layer_forward(x, wr, bias, k, f, gate_up_codes, gate_up_scales, down_codes,
                      down_scales, topk_idx, topk_w, offsets, sorted_pair, pair_pos,
                      y_pairs, out, ws, fmt=MOE_FMT_W4_SYM, bits=None,
                      bits_mode=MOE_BITS_NONE, out_dtype=MOE_OUT_BF16,
                      path=MOE_PATH_AUTO, stream=None):
    """moe_route_permute -> moe_expert_ffn_wq -> moe_combine in one ABI call
    (same outputs); every output buffer is caller-provided."""
    T, d = x.shape
    E = wr.shape[0]
    _check("moe_layer_forward_wq", load_library().moe_layer_forward_wq(
        _ptr(x), _ptr(wr), _ptr(bias), T, d, E, k, f, fmt, MOE_GROUP, _ptr(gate_up_codes),
        _ptr(gate_up_scales), _ptr(down_codes), _ptr(down_scales), _ptr(bits), bits_mode,
        _ptr(topk_idx), _ptr(topk_w), _ptr(offsets), _ptr(sorted_pair), _ptr(pair_pos),
        _ptr(y_pairs), _ptr(out), out_dtype, _ptr(ws), ws.numel() * ws.element_size(),
        path, _stream(stream)))
    return out


MOE_NOALLOC_SCRATCH_BYTES = 32 << 20


def moe_layer_forward_noalloc(x, wr, bias, k, f, gate_up_codes, gate_up_scales, down_codes,
                              down_scales, topk_idx, topk_w, offsets, sorted_pair, pair_pos,
                              y_pairs, out, fmt=MOE_FMT_W4_SYM, bits=None,
                              bits_mode=MOE_BITS_NONE, out_dtype=MOE_OUT_F32,
                              path=MOE_PATH_AUTO, stream=None):
    """moe_layer_forward_wq_noalloc: the layer step with the library's fixed
    device scratch in place of a workspace (nothing is allocated)."""
    T, d = x.shape
    E = wr.shape[0]
    _check("moe_layer_forward_wq_noalloc", load_library().moe_layer_forward_wq_noalloc(
        _ptr(x), _ptr(wr), _ptr(bias), T, d, E, k, f, fmt, MOE_GROUP, _ptr(gate_up_codes),
        _ptr(gate_up_scales), _ptr(down_codes), _ptr(down_scales), _ptr(bits), bits_mode,
        _ptr(topk_idx), _ptr(topk_w), _ptr(offsets), _ptr(sorted_pair), _ptr(pair_pos),
        _ptr(y_pairs), _ptr(out), out_dtype, path, _stream(stream)))
    return out


@_on_stream
def moe_bp_distortion(gate_up_planes, gate_up_scales, down_planes, down_scales, d, f,
                      dist=None, ws=None, stream=None):
    """Weight-space distortion [E][8] (fp64) of bitplane experts at prefix
    widths 1..8 (the offline table of the read-budget allocator)."""
    import torch
    E = gate_up_planes.shape[0]
    if dist is None:
        dist = torch.empty((E, 8), dtype=torch.float64, device=gate_up_planes.device)
    if ws is None:
        ws = torch.empty((int(load_library().moe_bp_distortion_ws_bytes(E, d, f)),),
                         dtype=torch.uint8, device=gate_up_planes.device)
    _check("moe_bp_distortion", load_library().moe_bp_distortion(
        _ptr(gate_up_planes), _ptr(gate_up_scales), _ptr(down_planes), _ptr(down_scales),
        E, d, f, _ptr(dist), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))
    return dist


@_on_stream
def moe_allocate_bits(dist, counts, d, f, b_min, b_max, budget_bytes, bits=None,
                      lam=None, read=None, stream=None):
    """Per-expert prefix widths [E] (u8) under a routing-weighted read
    budget -> (bits, lambda [1] fp64, read [1] int64), all on the device."""
    import torch
    E = dist.shape[0]
    dev = dist.device
    if bits is None:
        bits = torch.empty((E,), dtype=torch.uint8, device=dev)
    if lam is None:
        lam = torch.empty((1,), dtype=torch.float64, device=dev)
    if read is None:
        read = torch.empty((1,), dtype=torch.int64, device=dev)
    _check("moe_allocate_bits", load_library().moe_allocate_bits(
        _ptr(dist), _ptr(counts), E, d, f, b_min, b_max, int(budget_bytes), _ptr(bits),
        _ptr(lam), _ptr(read), _stream(stream)))
    return bits, lam, read


@_on_stream
def moe_combine(y_pairs, pair_pos, topk_w, out=None, out_dtype=MOE_OUT_BF16,
                stream=None):
    """Layer output [T][d] (bf16 bits in an int16 tensor, or fp32)."""
    import torch
    T, k = topk_w.shape
    d = y_pairs.shape[1]
    if out is None:
        out = _empty((T, d), torch.bfloat16 if out_dtype == MOE_OUT_BF16
                     else torch.float32, y_pairs)
    _check("moe_combine", load_library().moe_combine(
        _ptr(y_pairs), _ptr(pair_pos), _ptr(topk_w), T, k, d, _ptr(out), out_dtype,
        _stream(stream)))
    return out


@_on_stream
def moe_quantize_w4(w, codes=None, scales=None, stream=None):
    """fp32 [E][N][K] -> (codes, scales fp16-bits [E][N][K/128]).

    codes is a u8 tensor of shape [E][N][K/2] holding the tiled int4 layout
    of include/moe_wq.h (per expert [N/16][K/128][16][64] bytes); N % 16 == 0.
    """
    import torch
    E, N, K = w.shape
    if codes is None:
        codes = _empty((E, N, K // 2), torch.uint8, w)
    if scales is None:
        scales = _empty((E, N, K // 128), torch.int16, w)
    _check("moe_quantize_w4", load_library().moe_quantize_w4(
        _ptr(w), E, N, K, MOE_GROUP, _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


@_on_stream
def moe_retile_w4(codes_canonical, N, K, codes=None, stream=None):
    """Canonical row-major int4 codes u8 [E][N][K/2] -> the tiled layout
    (a u8 tensor [E][N][K/2] as moe_quantize_w4 returns)."""
    import torch
    E = codes_canonical.shape[0]
    if codes is None:
        codes = _empty((E, N, K // 2), torch.uint8, codes_canonical)
    _check("moe_retile_w4", load_library().moe_retile_w4(
        _ptr(codes_canonical), E, N, K, _ptr(codes), _stream(stream)))
    return codes


@_on_stream
def moe_retile_bitplane8(planes_canonical, N, K, planes=None, stream=None):
    """Canonical plane slabs u8 [E][8][N][K/8] -> the bitplane streaming
    layout (a u8 tensor [E][8][N][K/8] as moe_quantize_bitplane8 returns)."""
    import torch
    E = planes_canonical.shape[0]
    if planes is None:
        planes = _empty((E, 8, N, K // 8), torch.uint8, planes_canonical)
    _check("moe_retile_bitplane8", load_library().moe_retile_bitplane8(
        _ptr(planes_canonical), E, N, K, _ptr(planes), _stream(stream)))
    return planes


@_on_stream
def moe_quantize_bitplane8(w, planes=None, scales=None, stream=None):
    """fp32 [E][N][K] -> (planes, scales fp16-bits [E][N][K/128]).

    planes is a u8 tensor of shape [E][8][N][K/8] holding the bitplane layout
    of include/moe_wq.h (per expert [N/16][K/128][8][16][16] bytes);
    N % 16 == 0.
    """
    import torch
    E, N, K = w.shape
    if planes is None:
        planes = _empty((E, 8, N, K // 8), torch.uint8, w)
    if scales is None:
        scales = _empty((E, N, K // 128), torch.int16, w)
    _check("moe_quantize_bitplane8", load_library().moe_quantize_bitplane8(
        _ptr(w), E, N, K, MOE_GROUP, _ptr(planes), _ptr(scales), _stream(stream)))
    return planes, scales


def moe_set_ffn_events(gateup_begin=None, gateup_end=None, down_begin=None,
                       down_end=None):
    """Arm raw hipEvent_t handles (ints) for the next moe_expert_ffn_wq call."""
    def h(e):
        return None if e is None else ctypes.c_void_p(e)
    _check("moe_set_ffn_events", load_library().moe_set_ffn_events(
        h(gateup_begin), h(gateup_end), h(down_begin), h(down_end)))


# ------------------------------------------- around the routed experts
# These calls check shapes, types, layout and device before they touch a
# pointer (ValueError), launch on the device their tensors are on, and take
# outputs and workspaces that they create from the memory of the stream they
# launch on.
# Results carry no autograd history, whatever their inputs require: the *_bwd
# calls give the gradients.

def _on_device(fn):
    """Runs fn with its first parameter's device current and, when the keyword
    `stream` is given, with that stream current; fn launches on the current
    stream."""
    sig = inspect.signature(fn)
    lead = next(iter(sig.parameters))

    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        import torch
        if not args and lead not in kw:
            return fn(**kw)  # (a TypeError that names the parameter)
        first = args[0] if args else kw[lead]
        if not isinstance(first, torch.Tensor):
            raise ValueError(f"{fn.__name__}: a tensor is needed, got {type(first).__name__}")
        if stream is None:
            if not first.is_cuda or first.get_device() == _current_device():
                return fn(*args, **kw)
            with torch.cuda.device(first.device):
                return fn(*args, **kw)
        if first.is_cuda and stream.device != first.device:
            raise ValueError(f"{fn.__name__}: stream of {stream.device}, tensors on "
                             f"{first.device}")
        with _launch_on(stream, (*args, *kw.values())):
            return fn(*args, **kw)

    call.__signature__ = sig.replace(parameters=[
        *sig.parameters.values(),
        inspect.Parameter("stream", inspect.Parameter.KEYWORD_ONLY, default=None)])
    return call


def _raw_stream(t):
    import torch
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _addr(t):
    return None if t is None else t.data_ptr()


def _rows(fn, name, t, shape, dtypes, like=None):
    """Checks one tensor: its shape, that its dtype is one of `dtypes`, that it
    is dense, and that it is on like's device.  Without like it is the call's
    first tensor, which must be on a GPU and whose sizes (the other tensors
    have them too) the ABI's 32-bit ints must hold."""
    if t.shape == shape and t.dtype in dtypes and t.is_contiguous() and (
            t.is_cuda and max(shape) < 1 << 31 if like is None
            else t.get_device() == like.get_device()):
        return t
    if t.shape != shape:
        raise ValueError(f"{fn}: {name} has shape {tuple(t.shape)}, expected {shape}")
    if t.dtype not in dtypes:
        raise ValueError(f"{fn}: {name} is {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if not t.is_contiguous():
        raise ValueError(f"{fn}: {name} is not contiguous")
    if like is None and max(shape) >= 1 << 31:
        raise ValueError(f"{fn}: {name} has shape {tuple(shape)}, sizes must be below 2^31")
    raise ValueError(f"{fn}: {name} is on {t.device}, expected "
                     f"{'a GPU' if like is None else like.device}")


@functools.lru_cache(None)
def _types():
    """(bf16 as torch has it or as its bits, bf16 or fp32, fp32, int32)."""
    import torch
    return ((torch.bfloat16, torch.int16), (torch.bfloat16, torch.int16, torch.float32),
            (torch.float32,), (torch.int32,))


@functools.lru_cache(None)
def _i8():
    import torch
    return (torch.int8,)


def _groups(n):
    """Groups of 128 in a row of n values, the last may be shorter."""
    return -(-n // MOE_GROUP)


def _code(t):
    """The ABI's dtype code of a row tensor."""
    return MOE_OUT_F32 if t.element_size() == 4 else MOE_OUT_BF16


def _out_rows(fn, name, t, shape, code, like):
    dtypes = _types()[2 if code == MOE_OUT_F32 else 0]
    if t is None:
        if like.shape == shape:  # (a shorter call)
            import torch
            return torch.empty_like(like, dtype=dtypes[0])
        return like.new_empty(shape, dtype=dtypes[0])
    return _rows(fn, name, t, shape, dtypes, like)


def _out_f32(fn, name, t, shape, like):
    return _out_rows(fn, name, t, shape, MOE_OUT_F32, like)


def _workspace(fn, ws, need, like):
    if ws is None:  # (of like's type: the shortest call)
        return like.new_empty(-(-need // like.element_size())) if need else None
    if not ws.is_contiguous() or ws.device != like.device:
        raise ValueError(f"{fn}: ws must be contiguous and on {like.device}")
    return ws


def _ws_args(ws):
    return (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())


def moe_linear_w4_ws_bytes(T, N, K):
    return int(load_library().moe_linear_w4_ws_bytes(T, N, K))


def moe_linear_w4_kernel(T, N, K):
    """The kernel that these sizes run ("" where nothing runs)."""
    return load_library().moe_linear_w4_kernel(T, N, K).decode()


@_on_device
def moe_linear_w4(x, codes, scales, bias=None, out=None, out_dtype=MOE_OUT_BF16, ws=None):
    """x bf16 [T][K] times an int4 matrix -> [T][N] (bf16 or fp32).

    codes u8 [N][K/2] and scales fp16 (or their bits) [N][K/128] as
    moe_quantize_w4 returns them for one matrix (its leading axis of length 1
    may stay); bias fp32 [N] or None.
    """
    import torch
    fn = "moe_linear_w4"
    bf, _, f32, _ = _types()
    if x.dim() != 2 or codes.dim() not in (2, 3):
        raise ValueError(f"{fn}: x must be [T][K] and codes [N][K/2]")
    T, K = x.shape
    N = codes.shape[-2]
    if N >= 1 << 31:
        raise ValueError(f"{fn}: codes have {N} rows, sizes must be below 2^31")
    lead = (1,) * (codes.dim() - 2)
    _rows(fn, "x", x, (T, K), bf)
    _rows(fn, "codes", codes, lead + (N, K // 2), (torch.uint8,), x)
    _rows(fn, "scales", scales, (1,) * (scales.dim() - 2) + (N, K // MOE_GROUP),
          (torch.int16, torch.float16), x)
    if bias is not None:
        _rows(fn, "bias", bias, (N,), f32, x)
    out = _out_rows(fn, "out", out, (T, N), out_dtype, x)
    lib = _lib or load_library()
    if T > 64 or ws is not None:  # the query is 0 up to 64 tokens
        ws = _workspace(fn, ws, lib.moe_linear_w4_ws_bytes(T, N, K), x)
    rc = lib.moe_linear_w4(x.data_ptr(), T, N, K, MOE_GROUP, codes.data_ptr(), scales.data_ptr(),
                           _addr(bias), out.data_ptr(), out_dtype, *_ws_args(ws), _raw_stream(x))
    if rc:
        _check(fn, rc)
    return out


@_on_device
def moe_rmsnorm(x, gain=None, eps=1e-6, out=None, out_dtype=MOE_OUT_BF16, x_scales=None):
    """The norm in front of a block: x [T][d] (bf16 or fp32), gain fp32 [d].
    With x_scales [T][ceil(d/128)], x is an 8-bit checkpoint: the int8 codes
    that moe_quantize_i8 returned beside those scales."""
    fn = "moe_rmsnorm"
    _, row, f32, _ = _types()
    if x.dim() != 2:
        raise ValueError(f"{fn}: x must be [T][d]")
    T, d = x.shape
    _rows(fn, "x", x, (T, d), row if x_scales is None else _i8())
    if x_scales is not None:
        _rows(fn, "x_scales", x_scales, (T, _groups(d)), f32, x)
    if gain is not None:
        _rows(fn, "gain", gain, (d,), f32, x)
    out = _out_rows(fn, "out", out, (T, d), out_dtype, x)
    lib = _lib or load_library()
    if x_scales is None:
        rc = lib.moe_rmsnorm(x.data_ptr(), _code(x), _addr(gain), T, d, eps, out.data_ptr(),
                             out_dtype, _raw_stream(x))
    else:
        rc = lib.moe_rmsnorm_i8(x.data_ptr(), x_scales.data_ptr(), _addr(gain), T, d, eps,
                                out.data_ptr(), out_dtype, _raw_stream(x))
    if rc:
        _check(fn, rc)
    return out


@_on_device
def moe_rmsnorm_bwd(dout, x, gain=None, eps=1e-6, dres=None, dx=None, dgain=None, ws=None,
                    x_scales=None, dx_dtype=None):
    """Gradient of moe_rmsnorm, plus dres (the gradient of x past the norm)
    -> (dx in x's type, dgain fp32 [d]; None when there is no gain).
    With x_scales, x is an 8-bit checkpoint (as in moe_rmsnorm); dx and dres
    then have the type dx_dtype (bf16 unless given)."""
    fn = "moe_rmsnorm_bwd"
    _, row, f32, _ = _types()
    if dout.dim() != 2:
        raise ValueError(f"{fn}: dout must be [T][d]")
    T, d = dout.shape
    _rows(fn, "dout", dout, (T, d), row)
    if x_scales is None:
        _rows(fn, "x", x, (T, d), row, dout)
        if dx_dtype not in (None, _code(x)):
            raise ValueError(f"{fn}: dx_dtype is for 8-bit checkpoints, dx has x's type")
        dx_dtype = _code(x)
        like_x = (x.dtype,)
    else:
        _rows(fn, "x", x, (T, d), _i8(), dout)
        _rows(fn, "x_scales", x_scales, (T, _groups(d)), f32, dout)
        dx_dtype = MOE_OUT_BF16 if dx_dtype is None else dx_dtype
        like_x = _types()[2 if dx_dtype == MOE_OUT_F32 else 0]
    if dres is not None:
        _rows(fn, "dres", dres, (T, d), like_x, dout)
    dx = _out_rows(fn, "dx", dx, (T, d), dx_dtype, dout)
    if gain is not None:
        _rows(fn, "gain", gain, (d,), f32, dout)
        dgain = _out_f32(fn, "dgain", dgain, (d,), dout)
    elif dgain is not None:
        raise ValueError(f"{fn}: dgain without gain")
    lib = _lib or load_library()
    ws = _workspace(fn, ws, lib.moe_rmsnorm_bwd_ws_bytes(T, d) if dgain is not None else 0, dout)
    if x_scales is None:
        rc = lib.moe_rmsnorm_bwd(dout.data_ptr(), _code(dout), x.data_ptr(), _code(x),
                                 _addr(gain), _addr(dres), T, d, eps, dx.data_ptr(), _addr(dgain),
                                 *_ws_args(ws), _raw_stream(dout))
    else:
        rc = lib.moe_rmsnorm_bwd_i8(dout.data_ptr(), _code(dout), x.data_ptr(),
                                    x_scales.data_ptr(), _addr(gain), _addr(dres), T, d, eps,
                                    dx.data_ptr(), dx_dtype, _addr(dgain), *_ws_args(ws),
                                    _raw_stream(dout))
    if rc:
        _check(fn, rc)
    return dx, dgain


def _block_inputs(fn, rows, y_pairs, pair_pos, topk_w, add, post_gain, gate, gate_mode):
    """Checks the inputs that moe_combine_residual and its gradient share;
    rows: the residual or its gradient.  Returns (T, d, k)."""
    _, row, f32, i32 = _types()
    if rows.dim() != 2:
        raise ValueError(f"{fn}: the residual and its gradient must be [T][d]")
    T, d = rows.shape
    _rows(fn, "residual" if fn == "moe_combine_residual" else "dout", rows, (T, d), row)
    k = 0
    if y_pairs is not None:
        if pair_pos is None or topk_w is None or topk_w.dim() != 2:
            raise ValueError(f"{fn}: y_pairs needs pair_pos [T*k] and topk_w [T][k]")
        k = topk_w.shape[1]
        if k >= 1 << 31:
            raise ValueError(f"{fn}: k = {k}, sizes must be below 2^31")
        _rows(fn, "topk_w", topk_w, (T, k), f32, rows)
        _rows(fn, "y_pairs", y_pairs, (T * k, d), f32, rows)
        if pair_pos.numel() != T * k:
            raise ValueError(f"{fn}: pair_pos has {pair_pos.numel()} entries, expected {T * k}")
        _rows(fn, "pair_pos", pair_pos, tuple(pair_pos.shape), i32, rows)
    elif pair_pos is not None or topk_w is not None:
        raise ValueError(f"{fn}: pair_pos and topk_w without y_pairs")
    if add is not None:
        _rows(fn, "add", add, (T, d), (rows.dtype,), rows)
    if post_gain is not None:
        _rows(fn, "post_gain", post_gain, (d,), f32, rows)
    if gate is not None:
        shape = {MOE_GATE_TOKEN: (T,), MOE_GATE_CHANNEL: (d,)}.get(gate_mode)
        if shape is None:
            raise ValueError(f"{fn}: gate does not fit gate_mode {gate_mode}")
        _rows(fn, "gate", gate, shape, f32, rows)
    elif gate_mode != MOE_GATE_NONE:
        raise ValueError(f"{fn}: gate_mode {gate_mode} needs a gate")
    return T, d, k


@_on_device
def moe_combine_residual(residual, y_pairs=None, pair_pos=None, topk_w=None, add=None,
                         post_gain=None, gate=None, gate_mode=MOE_GATE_NONE, res_scale=1.0,
                         eps=1e-6, next_gain=None, out=None, next_out=None, next_norm=None):
    """End of a block: combine (+ add), norm after the block (with post_gain),
    gate, scaled residual and the next block's norm -> (out, next_out).

    residual [T][d] (bf16 or fp32; add and out have its type); y_pairs,
    pair_pos, topk_w as for moe_combine, or all None for a block whose output
    is `add` alone; pairs with a pair_pos of -1 are dropped.  next_out (bf16)
    is computed when next_gain or next_out is given or next_norm is true,
    otherwise it is None.  out may be residual.
    """
    fn = "moe_combine_residual"
    T, d, k = _block_inputs(fn, residual, y_pairs, pair_pos, topk_w, add, post_gain, gate,
                            gate_mode)
    code = _code(residual)
    out = _out_rows(fn, "out", out, (T, d), code, residual)
    if next_gain is not None:
        _rows(fn, "next_gain", next_gain, (d,), _types()[2], residual)
    if next_gain is not None or next_out is not None or next_norm:
        next_out = _out_rows(fn, "next_out", next_out, (T, d), MOE_OUT_BF16, residual)
    rc = (_lib or load_library()).moe_combine_residual(
        residual.data_ptr(), code, _addr(y_pairs), _addr(pair_pos), _addr(topk_w), k, _addr(add),
        _addr(post_gain), _addr(gate), gate_mode, res_scale, eps, _addr(next_gain), T, d,
        out.data_ptr(), _addr(next_out), _raw_stream(residual))
    if rc:
        _check(fn, rc)
    return out, next_out


CombineResidualGrads = collections.namedtuple(
    "CombineResidualGrads", "dy_pairs dtopk_w dadd dresidual dpost_gain dgate")


@_on_device
def moe_combine_residual_bwd(dout, y_pairs=None, pair_pos=None, topk_w=None, add=None,
                             post_gain=None, gate=None, gate_mode=MOE_GATE_NONE, res_scale=1.0,
                             eps=1e-6, dy_dtype=MOE_OUT_F32, dy_pairs=None, dtopk_w=None,
                             dadd=None, dresidual=None, dpost_gain=None, dgate=None, ws=None):
    """Gradient of moe_combine_residual's `out` against each of its inputs, as
    a CombineResidualGrads (None for inputs that are absent).

    dout [T][d] in the residual's type.  Rows of dy_pairs that no pair owns
    are not written.  dresidual may be dout.
    """
    fn = "moe_combine_residual_bwd"
    T, d, k = _block_inputs(fn, dout, y_pairs, pair_pos, topk_w, add, post_gain, gate, gate_mode)
    code = _code(dout)
    for name, g, given in (("dy_pairs", dy_pairs, y_pairs), ("dtopk_w", dtopk_w, topk_w),
                           ("dadd", dadd, add), ("dpost_gain", dpost_gain, post_gain),
                           ("dgate", dgate, gate)):
        if g is not None and given is None:
            raise ValueError(f"{fn}: {name} without its input")
    if y_pairs is not None:
        dy_pairs = _out_rows(fn, "dy_pairs", dy_pairs, (T * k, d), dy_dtype, dout)
        dtopk_w = _out_f32(fn, "dtopk_w", dtopk_w, (T, k), dout)
    if add is not None:
        dadd = _out_rows(fn, "dadd", dadd, (T, d), code, dout)
    dresidual = _out_rows(fn, "dresidual", dresidual, (T, d), code, dout)
    if post_gain is not None:
        dpost_gain = _out_f32(fn, "dpost_gain", dpost_gain, (d,), dout)
    if gate is not None:
        dgate = _out_f32(fn, "dgate", dgate, tuple(gate.shape), dout)
    lib = _lib or load_library()
    colsum = post_gain is not None or gate_mode == MOE_GATE_CHANNEL
    ws = _workspace(fn, ws, lib.moe_combine_residual_bwd_ws_bytes(T, d) if colsum else 0, dout)
    rc = lib.moe_combine_residual_bwd(
        dout.data_ptr(), code, _addr(y_pairs), _addr(pair_pos), _addr(topk_w), k, _addr(add),
        _addr(post_gain), _addr(gate), gate_mode, res_scale, eps, T, d, _addr(dy_pairs), dy_dtype,
        _addr(dtopk_w), _addr(dadd), _addr(dresidual), _addr(dpost_gain), _addr(dgate),
        *_ws_args(ws), _raw_stream(dout))
    if rc:
        _check(fn, rc)
    return CombineResidualGrads(dy_pairs, dtopk_w, dadd, dresidual, dpost_gain, dgate)


def _sort_inputs(fn, T, k, pair_pos, topk_w, like):
    _, _, f32, i32 = _types()
    if not -1 << 31 <= k < 1 << 31:
        raise ValueError(f"{fn}: k = {k}, sizes must be below 2^31")
    if pair_pos.numel() != T * k:
        raise ValueError(f"{fn}: pair_pos has {pair_pos.numel()} entries, expected {T * k}")
    _rows(fn, "pair_pos", pair_pos, tuple(pair_pos.shape), i32, like)
    if topk_w is not None:
        _rows(fn, "topk_w", topk_w, (T, k), f32, like)


@_on_device
def moe_dispatch(x, pair_pos, k, topk_w=None, out=None):
    """Tokens into expert order: row pair_pos[t*k+j] of the result [T*k][d] is
    x[t] (times topk_w[t][j] when given), in x's type.  Rows that no pair owns
    are not written."""
    fn = "moe_dispatch"
    if x.dim() != 2:
        raise ValueError(f"{fn}: x must be [T][d]")
    T, d = x.shape
    _rows(fn, "x", x, (T, d), _types()[1])
    _sort_inputs(fn, T, k, pair_pos, topk_w, x)
    out = _out_rows(fn, "out", out, (T * k, d), _code(x), x)
    rc = (_lib or load_library()).moe_dispatch(
        x.data_ptr(), _code(x), pair_pos.data_ptr(), _addr(topk_w), T, k, d, out.data_ptr(),
        _raw_stream(x))
    if rc:
        _check(fn, rc)
    return out


@_on_device
def moe_dispatch_bwd(dxs, pair_pos, k, x=None, topk_w=None, dx=None, dtopk_w=None):
    """Gradient of moe_dispatch -> (dx [T][d] in dxs's type, dtopk_w [T][k]).
    dtopk_w is computed when topk_w and x are given, otherwise it is None."""
    fn = "moe_dispatch_bwd"
    _, row, _, _ = _types()
    if dxs.dim() != 2 or k < 1 or dxs.shape[0] % k:
        raise ValueError(f"{fn}: dxs must be [T*k][d]")
    T, d = dxs.shape[0] // k, dxs.shape[1]
    _rows(fn, "dxs", dxs, (T * k, d), row)
    _sort_inputs(fn, T, k, pair_pos, topk_w, dxs)
    dx = _out_rows(fn, "dx", dx, (T, d), _code(dxs), dxs)
    if x is not None:
        _rows(fn, "x", x, (T, d), (dxs.dtype,), dxs)
    if x is not None and topk_w is not None:
        dtopk_w = _out_f32(fn, "dtopk_w", dtopk_w, (T, k), dxs)
    elif dtopk_w is not None:
        raise ValueError(f"{fn}: dtopk_w needs x and topk_w")
    rc = (_lib or load_library()).moe_dispatch_bwd(
        dxs.data_ptr(), _code(dxs), _addr(x), pair_pos.data_ptr(), _addr(topk_w), T, k, d,
        dx.data_ptr(), _addr(dtopk_w), _raw_stream(dxs))
    if rc:
        _check(fn, rc)
    return dx, dtopk_w


@_on_device
def moe_combine_bwd(dout, y_pairs, pair_pos, topk_w, dy_dtype=MOE_OUT_F32, dy_pairs=None,
                    dtopk_w=None):
    """Gradient of moe_combine for dout [T][d] (bf16 or fp32) -> (dy_pairs
    [T*k][d] of dy_dtype, dtopk_w fp32 [T][k]).  Rows of dy_pairs that no pair
    owns are not written."""
    fn = "moe_combine_bwd"
    _, row, f32, _ = _types()
    if dout.dim() != 2 or topk_w.dim() != 2:
        raise ValueError(f"{fn}: dout must be [T][d] and topk_w [T][k]")
    T, d = dout.shape
    k = topk_w.shape[1]
    _rows(fn, "dout", dout, (T, d), row)
    _rows(fn, "y_pairs", y_pairs, (T * k, d), f32, dout)
    _sort_inputs(fn, T, k, pair_pos, topk_w, dout)
    dy_pairs = _out_rows(fn, "dy_pairs", dy_pairs, (T * k, d), dy_dtype, dout)
    dtopk_w = _out_f32(fn, "dtopk_w", dtopk_w, (T, k), dout)
    rc = (_lib or load_library()).moe_combine_bwd(
        dout.data_ptr(), _code(dout), y_pairs.data_ptr(), pair_pos.data_ptr(), topk_w.data_ptr(),
        T, k, d, dy_pairs.data_ptr(), dy_dtype, dtopk_w.data_ptr(), _raw_stream(dout))
    if rc:
        _check(fn, rc)
    return dy_pairs, dtopk_w


# ------------------------------------- beside the routed experts: 8-bit rows
def _i8_inputs(fn, codes, scales, like=None):
    """Checks 8-bit rows: codes int8 [T][K] with scales fp32 [T][ceil(K/128)]
    or [T].  Returns (T, K, group size)."""
    if codes.dim() != 2 or scales.dim() not in (1, 2):
        raise ValueError(f"{fn}: codes must be [T][K], scales [T][ceil(K/128)] or [T]")
    T, K = codes.shape
    _rows(fn, "codes", codes, (T, K), _i8(), like)
    by_row = scales.dim() == 1
    _rows(fn, "scales", scales, (T,) if by_row else (T, _groups(K)), _types()[2], codes)
    return T, K, 0 if by_row else MOE_GROUP


@_on_device
def moe_quantize_i8(x, group=MOE_GROUP, codes=None, scales=None):
    """Rows x [T][K] (bf16 or fp32) in 8-bit integers -> (codes int8 [T][K],
    scales fp32).  group 128: a scale for each 128 values of a row,
    [T][ceil(K/128)], the form of activation checkpoints; group 0: one scale a
    row, [T], the form of moe_linear_i8's operands."""
    import torch
    fn = "moe_quantize_i8"
    if x.dim() != 2:
        raise ValueError(f"{fn}: x must be [T][K]")
    T, K = x.shape
    _rows(fn, "x", x, (T, K), _types()[1])
    if group not in (0, MOE_GROUP):
        raise ValueError(f"{fn}: group is {group}, expected 128 or 0 (a whole row)")
    codes = (torch.empty_like(x, dtype=torch.int8) if codes is None
             else _rows(fn, "codes", codes, (T, K), _i8(), x))
    scales = _out_f32(fn, "scales", scales, (T, _groups(K)) if group else (T,), x)
    rc = (_lib or load_library()).moe_quantize_i8(x.data_ptr(), _code(x), T, K, group,
                                                  codes.data_ptr(), scales.data_ptr(),
                                                  _raw_stream(x))
    if rc:
        _check(fn, rc)
    return codes, scales


@_on_device
def moe_dequantize_i8(codes, scales, out=None, out_dtype=MOE_OUT_BF16):
    """What moe_quantize_i8 stored: codes times scales, [T][K] bf16 or fp32."""
    fn = "moe_dequantize_i8"
    T, K, group = _i8_inputs(fn, codes, scales)
    out = _out_rows(fn, "out", out, (T, K), out_dtype, codes)
    rc = (_lib or load_library()).moe_dequantize_i8(codes.data_ptr(), scales.data_ptr(), T, K,
                                                    group, out.data_ptr(), out_dtype,
                                                    _raw_stream(codes))
    if rc:
        _check(fn, rc)
    return out


def moe_linear_i8_ws_bytes(T, N, K, x_quantized=False):
    return int(load_library().moe_linear_i8_ws_bytes(T, N, K, x_quantized))


def moe_linear_i8_kernel(T, N, K):
    """The kernel that moe_linear_i8 runs at these sizes ("" where nothing runs)."""
    return load_library().moe_linear_i8_kernel(T, N, K).decode()


@_on_device
def moe_linear_i8(x, codes, scales, bias=None, out=None, out_dtype=MOE_OUT_BF16, ws=None,
                  x_scales=None):
    """x [T][K] times a matrix in 8-bit integers -> [T][N] (bf16 or fp32).

    codes int8 [N][K] and scales fp32 [N] as moe_quantize_i8(w, group=0)
    returns them; bias fp32 [N] or None.  x is bf16, quantized by token inside
    the call, or int8 codes with x_scales fp32 [T].
    """
    fn = "moe_linear_i8"
    bf, _, f32, _ = _types()
    if x.dim() != 2 or codes.dim() != 2:
        raise ValueError(f"{fn}: x must be [T][K] and codes [N][K]")
    T, K = x.shape
    N = codes.shape[0]
    if N >= 1 << 31:
        raise ValueError(f"{fn}: codes have {N} rows, sizes must be below 2^31")
    _rows(fn, "x", x, (T, K), bf if x_scales is None else _i8())
    if x_scales is not None:
        _rows(fn, "x_scales", x_scales, (T,), f32, x)
    _rows(fn, "codes", codes, (N, K), _i8(), x)
    _rows(fn, "scales", scales, (N,), f32, x)
    if bias is not None:
        _rows(fn, "bias", bias, (N,), f32, x)
    out = _out_rows(fn, "out", out, (T, N), out_dtype, x)
    lib = _lib or load_library()
    ws = _workspace(fn, ws, lib.moe_linear_i8_ws_bytes(T, N, K, x_scales is not None), x)
    rc = lib.moe_linear_i8(x.data_ptr(), _addr(x_scales), T, N, K, codes.data_ptr(),
                           scales.data_ptr(), _addr(bias), out.data_ptr(), out_dtype,
                           *_ws_args(ws), _raw_stream(x))
    if rc:
        _check(fn, rc)
    return out


# --------------------------------- beside the routed experts: a shared expert
def _gated_weights(fn, w_gate_up, w_down, d, like):
    """Checks the block's weights; returns f."""
    bf = _types()[0]
    if w_gate_up.dim() != 2 or w_down.dim() != 2:
        raise ValueError(f"{fn}: w_gate_up must be [2f][d] and w_down [d][f]")
    f = w_down.shape[1]
    if f >= 1 << 30:
        raise ValueError(f"{fn}: f = {f}, sizes must be below 2^31")
    _rows(fn, "w_gate_up", w_gate_up, (2 * f, d), bf, like)
    _rows(fn, "w_down", w_down, (d, f), bf, like)
    return f


def moe_gated_ffn_ws_bytes(T, d, f):
    return int(load_library().moe_gated_ffn_ws_bytes(T, d, f))


GATED_PRODUCTS = ("gate_up", "down", "dh", "dx", "dw_gate_up", "dw_down")


def moe_gated_ffn_kernel(product, T, d, f, all=False):
    """The kernel that a product of the block (one of GATED_PRODUCTS) runs at these
    sizes ("" where nothing runs): by itself, or (all) in a moe_gated_ffn_bwd that
    asks for every gradient, and for gate_up and dh computes them again."""
    if product not in GATED_PRODUCTS:
        raise ValueError(f"moe_gated_ffn_kernel: product {product!r} is none of {GATED_PRODUCTS}")
    at = GATED_PRODUCTS.index(product)
    return load_library().moe_gated_ffn_kernel(at, T, d, f, all).decode()


@_on_device
def moe_gated_ffn(x, w_gate_up, w_down, out=None, out_dtype=MOE_OUT_BF16, save=False,
                  gate_up=None, ws=None):
    """A gated feed-forward block, (silu(x Wg^T) * (x Wu^T)) Wd^T -> (out,
    gate_up).

    x bf16 [T][d], w_gate_up bf16 [2f][d] (gate rows, then up rows), w_down
    bf16 [d][f], out [T][d] (bf16 or fp32).  gate_up bf16 [T][2f], the
    pre-activations that the gradient can use, is stored when `save` is true or
    a tensor for it is given, otherwise it is None.
    """
    fn = "moe_gated_ffn"
    if x.dim() != 2:
        raise ValueError(f"{fn}: x must be [T][d]")
    T, d = x.shape
    _rows(fn, "x", x, (T, d), _types()[0])
    f = _gated_weights(fn, w_gate_up, w_down, d, x)
    out = _out_rows(fn, "out", out, (T, d), out_dtype, x)
    if save or gate_up is not None:
        gate_up = _out_rows(fn, "gate_up", gate_up, (T, 2 * f), MOE_OUT_BF16, x)
    lib = _lib or load_library()
    ws = _workspace(fn, ws, lib.moe_gated_ffn_ws_bytes(T, d, f), x)
    rc = lib.moe_gated_ffn(x.data_ptr(), w_gate_up.data_ptr(), w_down.data_ptr(), T, d, f,
                           out.data_ptr(), out_dtype, _addr(gate_up), *_ws_args(ws),
                           _raw_stream(x))
    if rc:
        _check(fn, rc)
    return out, gate_up


GatedFfnGrads = collections.namedtuple("GatedFfnGrads", "dx dw_gate_up dw_down")


# (kept by size: the query goes through the choices of fewer tokens too, 2 to 150 us up
# to 16384 tokens)
@functools.lru_cache(4096)
def moe_gated_ffn_bwd_ws_bytes(T, d, f, dout_dtype=MOE_OUT_BF16, x_quantized=False,
                               gate_up_kept=False):
    """Bytes of workspace for T or fewer tokens."""
    return int(load_library().moe_gated_ffn_bwd_ws_bytes(T, d, f, dout_dtype, x_quantized,
                                                         gate_up_kept))


@_on_device
def moe_gated_ffn_bwd(dout, x, w_gate_up, w_down, x_scales=None, gate_up=None,
                      dw_dtype=MOE_OUT_BF16, dx=None, dw_gate_up=None, dw_down=None,
                      need_dx=True, need_dw=True, ws=None):
    """Gradient of moe_gated_ffn for dout [T][d] (bf16 or fp32), as a
    GatedFfnGrads (dx bf16 [T][d]; dw_gate_up [2f][d] and dw_down [d][f] of
    dw_dtype; None for what need_dx or need_dw leave out).

    x as in the forward call, or an 8-bit checkpoint of it (the codes of
    moe_quantize_i8, with its scales as x_scales).  gate_up: what the forward
    call saved; without it the pre-activations are computed again from x.
    """
    fn = "moe_gated_ffn_bwd"
    bf, row, f32, _ = _types()
    if dout.dim() != 2:
        raise ValueError(f"{fn}: dout must be [T][d]")
    T, d = dout.shape
    _rows(fn, "dout", dout, (T, d), row)
    _rows(fn, "x", x, (T, d), bf if x_scales is None else _i8(), dout)
    if x_scales is not None:
        _rows(fn, "x_scales", x_scales, (T, _groups(d)), f32, dout)
    f = _gated_weights(fn, w_gate_up, w_down, d, dout)
    if gate_up is not None:
        _rows(fn, "gate_up", gate_up, (T, 2 * f), bf, dout)
    for name, g, need in (("dx", dx, need_dx), ("dw_gate_up", dw_gate_up, need_dw),
                          ("dw_down", dw_down, need_dw)):
        if g is not None and not need:
            raise ValueError(f"{fn}: {name} given, but not needed")
    if need_dx:
        dx = _out_rows(fn, "dx", dx, (T, d), MOE_OUT_BF16, dout)
    if need_dw:
        dw_gate_up = _out_rows(fn, "dw_gate_up", dw_gate_up, (2 * f, d), dw_dtype, dout)
        dw_down = _out_rows(fn, "dw_down", dw_down, (d, f), dw_dtype, dout)
    lib = _lib or load_library()
    code = _code(dout)
    ws = _workspace(fn, ws, moe_gated_ffn_bwd_ws_bytes(T, d, f, code, x_scales is not None,
                                                       gate_up is not None), dout)
    rc = lib.moe_gated_ffn_bwd(dout.data_ptr(), code, x.data_ptr(), _addr(x_scales),
                               _addr(gate_up), w_gate_up.data_ptr(), w_down.data_ptr(), T, d, f,
                               _addr(dx), _addr(dw_gate_up), _addr(dw_down), dw_dtype,
                               *_ws_args(ws), _raw_stream(dout))
    if rc:
        _check(fn, rc)
    return GatedFfnGrads(dx, dw_gate_up, dw_down)


# ------------------------------------------------------ expert slot cache
def _np_ptr(a):
    return ctypes.c_void_p(a.ctypes.data)


def moe_cache_plan(E, slots, fmt, slot_expert, slot_bits, slot_last, step, need):
    """One step's slot assignment on host state (no device work).  The slot
    arrays (numpy int32/int32/int64 [slots]) are updated in place; returns
    dict(vmap [E], chunks [n][4], loads [n][6], V)."""
    import numpy as np
    for a, dt in ((slot_expert, np.int32), (slot_bits, np.int32), (slot_last, np.int64)):
        if a.dtype != dt or not a.flags.c_contiguous or a.shape != (slots,):
            raise ValueError("slot arrays: contiguous int32, int32, int64 of length slots")
    need = np.ascontiguousarray(need, np.int32)
    vmap = np.zeros(E, np.int32)
    max_chunks = 2 + 2 * E // max(slots // 2, 1)
    chunks = np.zeros((max_chunks, 4), np.int32)
    loads = np.zeros((2 * E + 1, 6), np.int32)
    nc, nl, V = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    ref = lambda v: ctypes.cast(ctypes.pointer(v), ctypes.c_void_p)  # noqa: E731
    _check("moe_cache_plan", load_library().moe_cache_plan(
        E, slots, fmt, _np_ptr(slot_expert), _np_ptr(slot_bits), _np_ptr(slot_last),
        int(step), _np_ptr(need), _np_ptr(vmap), _np_ptr(chunks), max_chunks, ref(nc),
        _np_ptr(loads), loads.shape[0], ref(nl), ref(V)))
    return dict(vmap=vmap, chunks=chunks[:nc.value].copy(), loads=loads[:nl.value].copy(),
                V=V.value)


class ExpertCache(_StepBuffers):
    """Expert bank in pinned host memory behind `slots` device slots
    (moe_cache_*): forward(x) runs one layer step, copying the experts (or
    bitplanes) it is missing into the slots first."""

    def __init__(self, wr, bias, k, f, gate_up_codes, gate_up_scales, down_codes,
                 down_scales, fmt, slots):
        import torch
        self.wr, self.bias, self.k, self.f, self.fmt, self.slots = wr, bias, k, f, fmt, slots
        self.E, self.d = wr.shape
        dev = wr.device
        # the whole bank, pinned host memory (the cache's backing store)
        self.host = [t.detach().to("cpu").contiguous().pin_memory()
                     for t in (gate_up_codes, gate_up_scales, down_codes, down_scales)]
        self.dev = [torch.empty((slots,) + tuple(t.shape[1:]), dtype=t.dtype, device=dev)
                    for t in self.host]
        h = ctypes.c_void_p()
        _check("moe_cache_create", load_library().moe_cache_create(
            self.E, self.d, f, fmt, slots, *[_ptr(t) for t in self.host],
            *[_ptr(t) for t in self.dev], ctypes.cast(ctypes.pointer(h), ctypes.c_void_p)))
        self.handle = h

    def _alloc(self, T, like):
        import torch
        k, d = self.k, self.d
        dev = like.device
        self.topk_idx = torch.empty((T, k), dtype=torch.int32, device=dev)
        self.topk_w = torch.empty((T, k), dtype=torch.float32, device=dev)
        self.pair_pos = torch.empty((T * k,), dtype=torch.int32, device=dev)
        self.y_pairs = torch.empty((T * k, d), dtype=torch.float32, device=dev)
        nb = int(load_library().moe_cache_ws_bytes(self.handle, T, k))
        self.ws = torch.empty((max(nb, 256),), dtype=torch.uint8, device=dev)

    def forward(self, x, out=None, out_dtype=MOE_OUT_BF16, bits=None,
                bits_mode=MOE_BITS_NONE, stream=None):
        import torch
        if stream is not None:
            with _launch_on(stream, (x, out, bits)):
                return self.forward(x, out, out_dtype, bits, bits_mode)
        T = x.shape[0]
        self._buffers(T, x)
        if out is None:
            out = _empty((T, self.d), torch.bfloat16 if out_dtype == MOE_OUT_BF16
                         else torch.float32, x)
        _check("moe_cache_forward", load_library().moe_cache_forward(
            self.handle, _ptr(x), _ptr(self.wr), _ptr(self.bias), T, self.k, _ptr(bits),
            bits_mode, _ptr(self.topk_idx), _ptr(self.topk_w), _ptr(self.pair_pos),
            _ptr(self.y_pairs), _ptr(out), out_dtype, _ptr(self.ws),
            self.ws.numel(), _stream(stream)))
        return out

    def stats(self):
        import numpy as np
        a = np.zeros(6, np.int64)
        _check("moe_cache_stats", load_library().moe_cache_stats(self.handle, _np_ptr(a)))
        keys = ("steps", "hits", "loads_full", "loads_partial", "bytes", "chunks")
        return {k: int(v) for k, v in zip(keys, a)}

    def resident(self):
        """(expert [slots], planes [slots]) of each slot; -1 = empty."""
        import numpy as np
        e = np.zeros(self.slots, np.int32)
        b = np.zeros(self.slots, np.int32)
        _check("moe_cache_slots", load_library().moe_cache_slots(self.handle, _np_ptr(e),
                                                                _np_ptr(b)))
        return e, b

    def reset(self):
        _check("moe_cache_reset", load_library().moe_cache_reset(self.handle))

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            load_library().moe_cache_destroy(self.handle)
            self.handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# --------------------------------------------------------- one whole layer
class MoeLayer(_StepBuffers):
    """Resident quantized expert weights plus the buffers of a step;
    `forward(x)` enqueues route+permute, the expert FFN and the combine on one
    stream.  The buffers (topk_idx, .., y_pairs) are those of the last step and
    stay in place while its batch size and stream do."""

    def __init__(self, wr, bias, k, f, gate_up_codes, gate_up_scales,
                 down_codes, down_scales, fmt=MOE_FMT_W4_SYM,
                 bits_mode=MOE_BITS_NONE, bits=None):
        self.wr, self.bias, self.k, self.f = wr, bias, k, f
        self.E, self.d = wr.shape
        self.gu, self.gus, self.dn, self.dns = (gate_up_codes, gate_up_scales,
                                                down_codes, down_scales)
        self.fmt, self.bits_mode, self.bits = fmt, bits_mode, bits

    def _alloc(self, T, like):
        import torch
        E, k, d, f = self.E, self.k, self.d, self.f
        P = T * k
        dev = like.device
        self.topk_idx = torch.empty((T, k), dtype=torch.int32, device=dev)
        self.topk_w = torch.empty((T, k), dtype=torch.float32, device=dev)
        self.offsets = torch.empty((E + 1,), dtype=torch.int32, device=dev)
        self.sorted_pair = torch.empty((P,), dtype=torch.int32, device=dev)
        self.pair_pos = torch.empty((P,), dtype=torch.int32, device=dev)
        self.ws_rp = torch.empty((max(moe_route_permute_ws_bytes(T, k, E), 16),),
                                 dtype=torch.uint8, device=dev)
        self.ws_ffn = torch.empty((max(moe_ffn_ws_bytes(T, k, E, d, f, self.fmt), 256),),
                                  dtype=torch.uint8, device=dev)
        self.ws_layer = torch.empty((max(moe_layer_ws_bytes(T, k, E, d, f, self.fmt), 256),),
                                    dtype=torch.uint8, device=dev)
        self.y_pairs = torch.empty((P, d), dtype=torch.float32, device=dev)

    def forward(self, x, out=None, out_dtype=MOE_OUT_BF16, path=MOE_PATH_AUTO,
                stream=None, weights=None):
        """One layer step through moe_layer_forward_wq."""
        import torch
        if stream is not None:
            with _launch_on(stream, (x, out, *(weights or ()))):
                return self.forward(x, out, out_dtype, path, None, weights)
        T = x.shape[0]
        self._buffers(T, x)
        gu, gus, dn, dns = weights if weights is not None else (
            self.gu, self.gus, self.dn, self.dns)
        if out is None:
            out = _empty((T, self.d), torch.bfloat16 if out_dtype == MOE_OUT_BF16
                         else torch.float32, x)
        return moe_layer_forward(x, self.wr, self.bias, self.k, self.f, gu, gus, dn, dns,
                                 self.topk_idx, self.topk_w, self.offsets, self.sorted_pair,
                                 self.pair_pos, self.y_pairs, out, self.ws_layer, self.fmt,
                                 self.bits, self.bits_mode, out_dtype, path, stream)

    def forward_steps(self, x, out=None, out_dtype=MOE_OUT_BF16, path=MOE_PATH_AUTO,
                      stream=None, weights=None):
        """The same step as moe_route_permute, moe_expert_ffn_wq and
        moe_combine calls (the composition the layer entry point equals)."""
        if stream is not None:
            with _launch_on(stream, (x, out, *(weights or ()))):
                return self.forward_steps(x, out, out_dtype, path, None, weights)
        T = x.shape[0]
        self._buffers(T, x)
        gu, gus, dn, dns = weights if weights is not None else (
            self.gu, self.gus, self.dn, self.dns)
        moe_route_permute(x, self.wr, self.bias, self.k, self.ws_rp, self.topk_idx,
                          self.topk_w, self.offsets, self.sorted_pair, self.pair_pos,
                          stream)
        moe_expert_ffn_wq(x, self.offsets, self.sorted_pair, self.k, self.f, gu, gus,
                          dn, dns, self.fmt, self.bits, self.bits_mode,
                          self.y_pairs, self.ws_ffn, path, stream)
        return moe_combine(self.y_pairs, self.pair_pos, self.topk_w, out, out_dtype,
                           stream)

    def forward_block(self, residual, gain=None, eps=1e-6, add=None, post_gain=None, gate=None,
                      gate_mode=MOE_GATE_NONE, res_scale=1.0, next_gain=None, out=None,
                      next_out=None, path=MOE_PATH_AUTO, stream=None, shared=None):
        """The layer as a residual block of a model: moe_rmsnorm of the
        residual stream, routing, expert FFN, and moe_combine_residual in the
        place of the combine -> (out, next_out or None), as that call.
        residual [T][d] (bf16 or fp32) on the layer's device.  shared: a
        GatedFfn that runs beside the routed experts on the same normed rows
        and takes the place of `add`."""
        if shared is not None and add is not None:
            raise ValueError("forward_block: shared and add are given, one is the other's place")
        if shared is not None and (shared.d != self.d or shared.w_down.device != self.wr.device):
            raise ValueError(f"forward_block: shared has width {shared.d} on "
                             f"{shared.w_down.device}, the layer {self.d} on {self.wr.device}")
        if residual.dim() != 2 or residual.shape[1] != self.d:
            raise ValueError(f"forward_block: residual has shape {tuple(residual.shape)}, "
                             f"expected [T][{self.d}]")
        if residual.device != self.wr.device:
            raise ValueError(f"forward_block: residual is on {residual.device}, the layer on "
                             f"{self.wr.device}")
        if stream is not None:
            if residual.is_cuda and stream.device != residual.device:
                raise ValueError(f"forward_block: stream of {stream.device}, residual on "
                                 f"{residual.device}")
            weights = () if shared is None else (shared.w_gate_up, shared.w_down)
            with _launch_on(stream, (residual, gain, add, post_gain, gate, next_gain, out,
                                     next_out, *weights)):
                return self.forward_block(residual, gain, eps, add, post_gain, gate, gate_mode,
                                          res_scale, next_gain, out, next_out, path,
                                          shared=shared)
        if residual.is_cuda and residual.get_device() != _current_device():
            import torch
            with torch.cuda.device(residual.device):
                return self.forward_block(residual, gain, eps, add, post_gain, gate, gate_mode,
                                          res_scale, next_gain, out, next_out, path,
                                          shared=shared)
        x = moe_rmsnorm(residual, gain, eps=eps)
        if shared is not None:
            add = shared.forward(x, out_dtype=_code(residual))
        self._buffers(residual.shape[0], x)
        moe_route_permute(x, self.wr, self.bias, self.k, self.ws_rp, self.topk_idx,
                          self.topk_w, self.offsets, self.sorted_pair, self.pair_pos)
        moe_expert_ffn_wq(x, self.offsets, self.sorted_pair, self.k, self.f, self.gu, self.gus,
                          self.dn, self.dns, self.fmt, self.bits, self.bits_mode,
                          self.y_pairs, self.ws_ffn, path)
        return moe_combine_residual(residual, self.y_pairs, self.pair_pos, self.topk_w, add=add,
                                    post_gain=post_gain, gate=gate, gate_mode=gate_mode,
                                    res_scale=res_scale, eps=eps, next_gain=next_gain, out=out,
                                    next_out=next_out)

    def bind(self, x, out, weights=None, path=MOE_PATH_AUTO, out_dtype=MOE_OUT_BF16,
             stream=None):
        """A step with every argument marshalled once: returns a callable that
        enqueues the same ABI call as forward(x, out, ...) for these fixed
        buffers (x, out and the weights must stay alive and in place; the
        step's own buffers are kept with the callable) on the stream that was
        current here, or `stream`.
        For decode loops, where converting arguments on every call would cost
        as much host time as the kernels take on the GPU."""
        if stream is not None:
            with _launch_on(stream, (x, out, *(weights or ()))):
                return self.bind(x, out, weights, path, out_dtype)
        T = x.shape[0]
        self._buffers(T, x)
        gu, gus, dn, dns = weights if weights is not None else (
            self.gu, self.gus, self.dn, self.dns)
        E, k, d, f = self.E, self.k, self.d, self.f
        args = (_ptr(x), _ptr(self.wr), _ptr(self.bias), T, d, E, k, f, self.fmt, MOE_GROUP,
                _ptr(gu), _ptr(gus), _ptr(dn), _ptr(dns), _ptr(self.bits), self.bits_mode,
                _ptr(self.topk_idx), _ptr(self.topk_w), _ptr(self.offsets),
                _ptr(self.sorted_pair), _ptr(self.pair_pos), _ptr(self.y_pairs), _ptr(out),
                out_dtype, _ptr(self.ws_layer),
                self.ws_layer.numel() * self.ws_layer.element_size(), path, _stream(stream))
        fn = load_library().moe_layer_forward_wq

        def step():
            rc = fn(*args)
            if rc:
                _check("moe_layer_forward_wq", rc)
            return out

        # (a later step with another batch size or stream takes other buffers)
        step.buffers = (self.topk_idx, self.topk_w, self.offsets, self.sorted_pair,
                        self.pair_pos, self.y_pairs, self.ws_layer)
        return step

    def capture(self, x, out, weights=None, path=MOE_PATH_AUTO, out_dtype=MOE_OUT_BF16):
        """One step for these fixed buffers recorded as a HIP graph (torch's
        CUDAGraph object; replay() re-runs the five kernels with one host
        call).  The library records only kernel launches (no memset or copy
        nodes), and the step's own buffers are the graph's: replays do not
        meet other steps' of this layer, eager or recorded."""
        import torch
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):  # binds to the capture stream
            self.bind(x, out, weights, path, out_dtype)()
        return g


# ------------------------------------------------------------ a shared expert
class GatedFfn:
    """Resident bf16 weights of a gated feed-forward block: a shared expert
    (`MoeLayer.forward_block(shared=...)`), or a dense block of its own in a
    model that is trained with 8-bit checkpoints (forward_block keeps one of
    the residual stream, backward_block computes the rest again from it)."""

    def __init__(self, w_gate_up, w_down):
        _rows("GatedFfn", "w_down", w_down, tuple(w_down.shape), _types()[0])
        self.f = _gated_weights("GatedFfn", w_gate_up, w_down, w_down.shape[0], w_down)
        self.d = w_down.shape[0]
        self.w_gate_up, self.w_down = w_gate_up, w_down

    def forward(self, x, out=None, out_dtype=MOE_OUT_BF16, stream=None):
        """moe_gated_ffn of x [T][d] -> out."""
        return moe_gated_ffn(x, self.w_gate_up, self.w_down, out=out, out_dtype=out_dtype,
                             stream=stream)[0]

    @contextlib.contextmanager
    def _stream_of(self, fn, first, stream, *values):
        if first.is_cuda and stream.device != first.device:
            raise ValueError(f"{fn}: stream of {stream.device}, tensors on {first.device}")
        with _launch_on(stream, (first, self.w_gate_up, self.w_down, *values)):
            yield

    def forward_block(self, residual, gain=None, eps=1e-6, keep=True, stream=None):
        """residual + block(moe_rmsnorm(residual)) -> (out, kept); residual
        [T][d] (bf16 or fp32).  kept: the residual as an 8-bit checkpoint
        (codes, scales), None if not `keep`."""
        if stream is not None:
            with self._stream_of("forward_block", residual, stream, gain):
                return self.forward_block(residual, gain, eps, keep)
        x = moe_rmsnorm(residual, gain, eps=eps)
        kept = moe_quantize_i8(residual) if keep else None
        y = self.forward(x, out_dtype=_code(residual))
        return moe_combine_residual(residual, add=y)[0], kept

    def backward_block(self, dout, kept, gain=None, eps=1e-6, dw_dtype=MOE_OUT_BF16,
                       stream=None):
        """Gradient of forward_block at the checkpointed residual, for dout
        [T][d] in the residual's type -> (dresidual in that type, dgain fp32 [d]
        or None, dw_gate_up, dw_down)."""
        if kept is None:
            raise ValueError("backward_block: kept is None (forward_block ran with keep=False)")
        codes, scales = kept
        if stream is not None:
            with self._stream_of("backward_block", dout, stream, gain, codes, scales):
                return self.backward_block(dout, kept, gain, eps, dw_dtype)
        x = moe_rmsnorm(codes, gain, eps=eps, x_scales=scales)
        g = moe_gated_ffn_bwd(dout, x, self.w_gate_up, self.w_down, dw_dtype=dw_dtype)
        dres, dgain = moe_rmsnorm_bwd(g.dx, codes, gain, eps=eps, dres=dout, x_scales=scales,
                                      dx_dtype=_code(dout))
        return dres, dgain, g.dw_gate_up, g.dw_down

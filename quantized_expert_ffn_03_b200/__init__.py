"""Python binding of libmoe: the streaming-experts MoE layer on B200.

Argument marshalling only.  Every computation of the layer runs in the CUDA
library (``libmoe.so``, built by ``python quantized_expert_ffn_03_b200/build.py``);
if the library is missing, importing this package raises ImportError.
Device arguments are torch CUDA tensors (bf16 tensors may be torch.bfloat16
or 16-bit integer views); host arguments of the host packer are numpy arrays.
Entry points keep the names of the C ABI in include/moe.h.
"""
import ctypes as C
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        "libmoe.so is not built (%s); run `python quantized_expert_ffn_03_b200/build.py`" % LIB_PATH)

_lib = C.CDLL(LIB_PATH)

MOE_OK = 0
MOE_ERR_WORKSPACE = 3
MOE_ERR_DEVICE = 8
NOALLOC_SCRATCH_BYTES = 4 << 20  # MOE_NOALLOC_SCRATCH_BYTES of moe.h
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE",
          4: "MOE_ERR_CUDA", 5: "MOE_ERR_OOM", 6: "MOE_ERR_TIMEOUT", 7: "MOE_ERR_IO",
          8: "MOE_ERR_DEVICE"}
STATUS_BY_NAME = {v: k for k, v in STATUS.items()}


class MoeError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__("%s: %s" % (STATUS.get(status, status), msg))
        self.status = status


class MoeConfig(C.Structure):
    _fields_ = [("hidden", C.c_int), ("inter", C.c_int), ("n_experts", C.c_int),
                ("top_k", C.c_int), ("bits", C.c_int), ("group", C.c_int),
                ("eps", C.c_float), ("has_shared", C.c_int)]


class MoeLayerWeights(C.Structure):
    _fields_ = [("expert_ptr", C.c_void_p), ("router_w", C.c_void_p), ("router_bias", C.c_void_p),
                ("shared_gate", C.c_void_p), ("shared_up", C.c_void_p), ("shared_down", C.c_void_p),
                ("gamma", C.c_void_p), ("shared_out_gate", C.c_void_p), ("shared_packed", C.c_void_p)]


class MoeLinearConfig(C.Structure):
    _fields_ = [("in_features", C.c_int), ("out_features", C.c_int), ("dtype", C.c_int), ("out_dtype", C.c_int),
                ("act", C.c_int), ("gated", C.c_int)]


class MoeLinearWeights(C.Structure):
    _fields_ = [("w", C.c_void_p), ("w_up", C.c_void_p), ("bias", C.c_void_p), ("bias_up", C.c_void_p),
                ("ldw", C.c_int64), ("ldw_up", C.c_int64)]


class MoeRouteConfig(C.Structure):
    _fields_ = [("n_experts", C.c_int), ("top_k", C.c_int), ("score", C.c_int), ("n_groups", C.c_int),
                ("topk_groups", C.c_int), ("group_score", C.c_int), ("renormalise", C.c_int), ("scale", C.c_float)]


EXPORTS = {
    "moe_last_error": (C.c_char_p, []),
    "moe_packed_expert_bytes": (C.c_size_t, [C.c_void_p]),
    "moe_packed_layout": (C.c_int, [C.c_void_p, C.c_void_p]),
    "moe_pack_experts": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int, C.c_int,
                                   C.c_void_p, C.c_size_t]),
    "moe_pack_experts_device": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int,
                                          C.c_void_p, C.c_size_t, C.c_void_p]),
    "moe_router_workspace_bytes": (C.c_size_t, [C.c_void_p, C.c_int]),
    "moe_router_topk": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int, C.c_void_p,
                                  C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]),
    "moe_topk_from_logits": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_void_p, C.c_void_p,
                                       C.c_void_p]),
    "moe_layer_workspace_bytes": (C.c_size_t, [C.c_void_p, C.c_int]),
    "moe_workspace_init": (C.c_int, [C.c_void_p, C.c_size_t, C.c_void_p]),
    "moe_layer_forward": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int,
                                    C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                    C.c_size_t, C.c_void_p]),
    "moe_layer_host_workspace_bytes": (C.c_size_t, [C.c_void_p, C.c_int]),
    "moe_layer_forward_host": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int,
                                         C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]),
    "moe_layer_forward_host_async": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int,
                                               C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]),
    "moe_layer_forward_host_packed": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_int, C.c_void_p,
                                                C.c_void_p, C.c_size_t, C.c_void_p]),
    "moe_layer_trace_blocks": (C.c_int, []),
    "moe_layer_forward_traced": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int,
                                           C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p,
                                           C.c_size_t, C.c_void_p]),
    "moe_layer_forward_noalloc": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int,
                                            C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]),
    "moe_layer_tokens_per_launch": (C.c_int, [C.c_void_p]),
    "moe_layer_batched_workspace_bytes": (C.c_size_t, [C.c_void_p, C.c_int]),
    "moe_layer_forward_batched": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int,
                                            C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                            C.c_size_t, C.c_void_p]),
    "moe_layer_forward_chunked": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int,
                                            C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                            C.c_size_t, C.c_void_p]),
    "moe_layer_forward_prenorm": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int,
                                            C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                            C.c_void_p, C.c_size_t, C.c_void_p]),
    "moe_layer_forward_routed": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int,
                                           C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                           C.c_size_t, C.c_void_p]),
    "moe_layer_forward_routed_batched": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int,
                                                   C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                                   C.c_size_t, C.c_void_p]),
    "moe_route_from_logits": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int, C.c_int64, C.c_void_p, C.c_int,
                                        C.c_void_p, C.c_void_p, C.c_void_p]),
    "moe_route_workspace_bytes": (C.c_size_t, [C.c_void_p, C.c_int]),
    "moe_route_topk": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int,
                                 C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]),
    "moe_linear_forward": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_int64, C.c_void_p, C.c_int64, C.c_int,
                                     C.c_void_p, C.c_int64, C.c_void_p]),
    "moe_linear_device_error": (C.c_int, [C.c_void_p, C.c_void_p]),
    "moe_linear_selftest_bounded_wait": (C.c_int, [C.c_uint64, C.c_void_p]),
    "moe_stream_create": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.c_size_t, C.c_int, C.c_void_p]),
    "moe_stream_inject_fault": (C.c_int, [C.c_void_p, C.c_int, C.c_int]),
    "moe_stream_create_file": (C.c_int, [C.c_void_p, C.c_int, C.c_char_p, C.c_int, C.c_int, C.c_int,
                                         C.c_void_p]),
    "moe_stream_file_stats": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]),
    "moe_stream_enable_copy_timing": (C.c_int, [C.c_void_p, C.c_int]),
    "moe_stream_copy_timing": (C.c_int, [C.c_void_p, C.c_void_p]),
    "moe_stream_prefetch": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.c_int, C.c_void_p]),
    "moe_stream_resolve": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.c_int, C.c_void_p, C.c_void_p]),
    "moe_stream_stats": (C.c_int, [C.c_void_p, C.c_void_p]),
    "moe_stream_resolve_device": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.c_int, C.c_void_p, C.c_void_p]),
    "moe_layer_forward_streamed": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int,
                                             C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                             C.c_int, C.c_void_p, C.c_size_t, C.c_void_p]),
    "moe_stream_destroy": (None, [C.c_void_p]),
    "moe_device_error": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p]),
    "moe_noalloc_device_error": (C.c_int, [C.c_void_p, C.c_void_p]),
    "moe_selftest_bounded_wait": (C.c_int, [C.c_void_p, C.c_size_t, C.c_uint64, C.c_void_p]),
}

for _name, (_res, _args) in EXPORTS.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args


def lib():
    return _lib


def last_error():
    return _lib.moe_last_error().decode()


def _check(status):
    if status != MOE_OK:
        raise MoeError(status, last_error())


def config(hidden, inter, n_experts, top_k, bits=4, group=64, eps=1e-6, has_shared=1):
    return MoeConfig(hidden, inter, n_experts, top_k, bits, group, eps, has_shared)


def _ptr(t):
    """Device or host address of a torch tensor / numpy array / int / None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _nbytes(t):
    """Byte size of a torch tensor / numpy array (0 for None)."""
    if t is None:
        return 0
    if isinstance(t, np.ndarray):
        return t.nbytes
    if isinstance(t, int):
        raise TypeError("a raw address needs an explicit byte count")
    return t.numel() * t.element_size()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ---- packed format -------------------------------------------------------------

def moe_packed_expert_bytes(cfg):
    return _lib.moe_packed_expert_bytes(C.byref(cfg))


def moe_packed_layout(cfg):
    off = (C.c_size_t * 6)()
    _check(_lib.moe_packed_layout(C.byref(cfg), off))
    return [int(v) for v in off]


def moe_pack_experts(cfg, w_gate, w_up, w_down, e_begin=0, e_count=None):
    """Host packer.  w_gate/w_up: float32 [n][I][H], w_down: float32 [n][H][I]
    (numpy).  Returns uint8 [e_count][bytes]."""
    wg = np.ascontiguousarray(w_gate, dtype=np.float32)
    wu = np.ascontiguousarray(w_up, dtype=np.float32)
    wd = np.ascontiguousarray(w_down, dtype=np.float32)
    if wg.ndim == 2:
        wg, wu, wd = wg[None], wu[None], wd[None]
    if e_count is None:
        e_count = wg.shape[0] - e_begin
    nb = moe_packed_expert_bytes(cfg)
    out = np.zeros((e_count, nb), dtype=np.uint8)
    _check(_lib.moe_pack_experts(C.byref(cfg), _ptr(wg), _ptr(wu), _ptr(wd), e_begin, e_count,
                                 _ptr(out), out.nbytes))
    return out


def moe_pack_experts_device(cfg, w_gate, w_up, w_down, out, stream=None):
    """Device packer: torch float32 CUDA tensors [n][I][H], [n][I][H], [n][H][I];
    out: torch uint8 CUDA tensor of n * moe_packed_expert_bytes bytes."""
    n = w_gate.shape[0]
    _check(_lib.moe_pack_experts_device(C.byref(cfg), _ptr(w_gate), _ptr(w_up), _ptr(w_down), n,
                                        _ptr(out), out.numel() * out.element_size(), _stream(stream)))
    return out


# ---- router ----------------------------------------------------------------------

def moe_router_workspace_bytes(cfg, T):
    return _lib.moe_router_workspace_bytes(C.byref(cfg), T)


def moe_router_topk(cfg, x, wr, bias, idx, w, logits_out=None, workspace=None, stream=None):
    T = x.shape[0]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.moe_router_topk(C.byref(cfg), _ptr(x), _ptr(wr), _ptr(bias), T, _ptr(idx), _ptr(w),
                                _ptr(logits_out), _ptr(workspace), ws_bytes, _stream(stream)))


def moe_topk_from_logits(cfg, logits, idx, w, stream=None):
    _check(_lib.moe_topk_from_logits(C.byref(cfg), _ptr(logits), logits.shape[0], _ptr(idx), _ptr(w),
                                     _stream(stream)))


# ---- layer -----------------------------------------------------------------------

def moe_layer_workspace_bytes(cfg, T):
    return _lib.moe_layer_workspace_bytes(C.byref(cfg), T)


def moe_layer_host_workspace_bytes(cfg, T):
    return _lib.moe_layer_host_workspace_bytes(C.byref(cfg), T)


def moe_workspace_init(workspace, stream=None):
    _check(_lib.moe_workspace_init(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                   _stream(stream)))


def layer_weights(expert_ptr, router_w, router_bias, shared_gate, shared_up, shared_down, gamma,
                  shared_out_gate=None, shared_packed=None):
    """expert_ptr: int64 CUDA tensor [E] of blob addresses; the rest CUDA tensors or None
    (shared_packed: a uint8 CUDA tensor holding one packed blob)."""
    return MoeLayerWeights(_ptr(expert_ptr), _ptr(router_w), _ptr(router_bias), _ptr(shared_gate),
                           _ptr(shared_up), _ptr(shared_down), _ptr(gamma), _ptr(shared_out_gate),
                           _ptr(shared_packed))


def moe_layer_forward(cfg, wts, x, residual, h_out, y_norm, idx_out=None, w_out=None,
                      workspace=None, stream=None):
    T = x.shape[0]
    _check(_lib.moe_layer_forward(C.byref(cfg), C.byref(wts), _ptr(x), _ptr(residual), T, _ptr(h_out),
                                  _ptr(y_norm), _ptr(idx_out), _ptr(w_out), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_layer_tokens_per_launch(cfg):
    return _lib.moe_layer_tokens_per_launch(C.byref(cfg))


def moe_layer_batched_workspace_bytes(cfg, T):
    return _lib.moe_layer_batched_workspace_bytes(C.byref(cfg), int(T))


def moe_layer_forward_batched(cfg, wts, x, residual, h_out, y_norm, idx_out=None, w_out=None,
                              workspace=None, stream=None):
    """The layer through the grouped tensor-core GEMMs (see moe.h)."""
    T = x.shape[0]
    _check(_lib.moe_layer_forward_batched(C.byref(cfg), C.byref(wts), _ptr(x), _ptr(residual), T, _ptr(h_out),
                                          _ptr(y_norm), _ptr(idx_out), _ptr(w_out), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_layer_forward_chunked(cfg, wts, x, residual, h_out, y_norm, idx_out=None, w_out=None,
                              workspace=None, stream=None):
    """The layer through the fused decode kernel on chunks of tokens (see moe.h)."""
    T = x.shape[0]
    _check(_lib.moe_layer_forward_chunked(C.byref(cfg), C.byref(wts), _ptr(x), _ptr(residual), T, _ptr(h_out),
                                          _ptr(y_norm), _ptr(idx_out), _ptr(w_out), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_layer_forward_prenorm(cfg, wts, gamma_pre, h_in, h_out, y_norm, x_out, idx_out=None, w_out=None,
                              workspace=None, stream=None):
    """The layer with the RMSNorm before it, on the residual stream h_in (see moe.h)."""
    T = h_in.shape[0]
    _check(_lib.moe_layer_forward_prenorm(C.byref(cfg), C.byref(wts), _ptr(gamma_pre), _ptr(h_in), T,
                                          _ptr(h_out), _ptr(y_norm), _ptr(idx_out), _ptr(w_out), _ptr(x_out),
                                          _ptr(workspace), workspace.numel() * workspace.element_size(),
                                          _stream(stream)))


def moe_layer_forward_routed(cfg, wts, x, residual, idx, w, h_out, y_norm, workspace, stream=None):
    """The layer with the routing given: idx int32 [T][K], w float32 [T][K] (CUDA)."""
    T = x.shape[0]
    _check(_lib.moe_layer_forward_routed(C.byref(cfg), C.byref(wts), _ptr(x), _ptr(residual), T, _ptr(idx),
                                         _ptr(w), _ptr(h_out), _ptr(y_norm), _ptr(workspace),
                                         workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_layer_forward_noalloc(cfg, wts, x, residual, h_out, y_norm, idx_out=None, w_out=None, stream=None):
    """moe_layer_forward on the library's built-in scratch (no workspace)."""
    T = x.shape[0]
    _check(_lib.moe_layer_forward_noalloc(C.byref(cfg), C.byref(wts), _ptr(x), _ptr(residual), T, _ptr(h_out),
                                          _ptr(y_norm), _ptr(idx_out), _ptr(w_out), _stream(stream)))


def moe_layer_trace_blocks():
    return _lib.moe_layer_trace_blocks()


def moe_layer_forward_traced(cfg, wts, x, residual, h_out, y_norm, trace, workspace, stream=None):
    """trace: int64 CUDA tensor of moe_layer_trace_blocks()*128 entries."""
    T = x.shape[0]
    _check(_lib.moe_layer_forward_traced(C.byref(cfg), C.byref(wts), _ptr(x), _ptr(residual), T,
                                         _ptr(h_out), _ptr(y_norm), _ptr(workspace),
                                         workspace.numel() * workspace.element_size(), _ptr(trace),
                                         trace.numel(), _stream(stream)))


def moe_layer_forward_host(cfg, wts, x, residual, h_out, y_norm, workspace, stream=None):
    """x, residual, h_out, y_norm: host arrays/tensors (pinned for async copies)."""
    T = x.shape[0]
    _check(_lib.moe_layer_forward_host(C.byref(cfg), C.byref(wts), _ptr(x), _ptr(residual), T,
                                       _ptr(h_out), _ptr(y_norm), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_layer_forward_host_async(cfg, wts, x, residual, h_out, y_norm, workspace, stream=None):
    """moe_layer_forward_host without the final synchronisation (see moe.h)."""
    T = x.shape[0]
    _check(_lib.moe_layer_forward_host_async(C.byref(cfg), C.byref(wts), _ptr(x), _ptr(residual), T,
                                             _ptr(h_out), _ptr(y_norm), _ptr(workspace),
                                             workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_layer_forward_host_packed(cfg, wts, xr, hy, workspace, stream=None):
    """xr: pinned host [2][T][H] (x, residual); hy: pinned host [2][T][H]
    (h_out, y_norm), filled once the stream reaches the end of the call."""
    T = xr.shape[1]
    _check(_lib.moe_layer_forward_host_packed(C.byref(cfg), C.byref(wts), _ptr(xr), T, _ptr(hy), _ptr(workspace),
                                              workspace.numel() * workspace.element_size(), _stream(stream)))


def moe_layer_forward_routed_batched(cfg, wts, x, residual, idx, w, h_out, y_norm, workspace, stream=None):
    """The batched path with the routing given: idx int32 [T][K], w float32 [T][K] (CUDA)."""
    T = x.shape[0]
    _check(_lib.moe_layer_forward_routed_batched(C.byref(cfg), C.byref(wts), _ptr(x), _ptr(residual), T, _ptr(idx),
                                                 _ptr(w), _ptr(h_out), _ptr(y_norm), _ptr(workspace),
                                                 workspace.numel() * workspace.element_size(), _stream(stream)))


# ---- expert choice and dense products ----------------------------------------------
# Unlike the calls above these take strided rows, so they check the tensors'
# shapes, types, strides and device and raise MoeError(MOE_ERR_INVALID_ARG).

MOE_ERR_INVALID_ARG = 1
MOE_BF16, MOE_F16, MOE_F32 = 0, 1, 2
MOE_ACT_NONE, MOE_ACT_SILU, MOE_ACT_GELU, MOE_ACT_GELU_TANH, MOE_ACT_RELU = 0, 1, 2, 3, 4
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_GROUP_MAX, MOE_GROUP_TOP2 = 0, 1

_DTYPE_NAMES = {MOE_BF16: ("bfloat16", "int16", "uint16"), MOE_F16: ("float16", "int16", "uint16"),
                MOE_F32: ("float32",)}
_dtype_sets = {}  # code -> torch types of its elements (16-bit types also as integer views)
_logit_codes = {}  # torch type -> code
_torch_c = _int32 = None


def _types():
    """Looks torch up, once; the package imports without it."""
    global _torch_c, _int32
    import torch
    torch.cuda.current_stream()  # initialises CUDA
    _dtype_sets.update({c: frozenset(getattr(torch, n) for n in names) for c, names in _DTYPE_NAMES.items()})
    _logit_codes.update({torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.float16: MOE_F16})
    _int32 = torch.int32
    _torch_c = torch._C  # last: what other threads look at


def _bad(what):
    raise MoeError(MOE_ERR_INVALID_ARG, what)


def _current():
    """(current CUDA device, raw handle of its current stream)."""
    if _torch_c is None:
        _types()
    dev = _torch_c._cuda_getDevice()
    return dev, _torch_c._cuda_getCurrentRawStream(dev)


def _rows(t, name, shape, code, dev):
    """Row stride of a 2-d CUDA tensor with adjacent columns; raises otherwise."""
    if t.shape != shape or t.dtype not in _dtype_sets[code]:
        _bad("%s must be %s of type %s, got %s %s" % (name, tuple(shape), _DTYPE_NAMES[code][0], tuple(t.shape), t.dtype))
    if t.get_device() != dev:
        _bad("%s must be on the current CUDA device" % name)
    ld, step = t.stride()
    if step != 1 and shape[1] > 1:
        _bad("%s must have adjacent columns" % name)
    return ld if shape[0] > 1 else (shape[1] + 7) & ~7  # a single row: its stride is never used


def _vec(t, name, n, dev):
    if t.shape != (n,) or t.dtype not in _dtype_sets[MOE_F32] or (n > 1 and t.stride(0) != 1):
        _bad("%s must be a contiguous float32 vector of %d" % (name, n))
    if t.get_device() != dev:
        _bad("%s must be on the current CUDA device" % name)
    return t.data_ptr()


def linear_config(in_features, out_features, act=MOE_ACT_NONE, gated=False, dtype=MOE_BF16, out_dtype=None):
    return MoeLinearConfig(in_features, out_features, dtype, dtype if out_dtype is None else out_dtype, act,
                           1 if gated else 0)


def linear_weights(cfg, w, bias=None, w_up=None, bias_up=None):
    """w, w_up: CUDA tensors [out_features][in_features]; bias, bias_up: float32 [out_features] or None.
    The result keeps the tensors alive."""
    if _torch_c is None:
        _types()
    shape, dev = (cfg.out_features, cfg.in_features), w.get_device()
    if dev < 0:
        _bad("w must be on a CUDA device")
    if (w_up is not None) != bool(cfg.gated) or (bias_up is not None and w_up is None):
        _bad("w_up goes with a gated config, bias_up with w_up")
    ld = _rows(w, "w", shape, cfg.dtype, dev)
    ld_up = 0 if w_up is None else _rows(w_up, "w_up", shape, cfg.dtype, dev)
    wts = MoeLinearWeights(w.data_ptr(), _ptr(w_up), None if bias is None else _vec(bias, "bias", shape[0], dev),
                           None if bias_up is None else _vec(bias_up, "bias_up", shape[0], dev), ld, ld_up)
    wts.kept = (w, bias, w_up, bias_up)
    wts.made_for = (shape[0], shape[1], cfg.dtype, cfg.gated, dev)
    return wts


def moe_linear_forward(cfg, wts, x, out, residual=None, stream=None):
    """out = act(x w^T + bias) [* (x w_up^T + bias_up)] [+ residual] (see moe.h).  x [T][in], out and
    residual [T][out]: CUDA tensors with adjacent columns; out may be residual itself."""
    dev, st = _current()
    N, K, code, gated, at = wts.made_for
    if cfg.in_features != K or cfg.out_features != N or cfg.dtype != code or cfg.gated != gated or at != dev:
        _bad("the weights were made for another config or device")
    T, out_code = x.shape[0], cfg.out_dtype
    ldx = _rows(x, "x", (T, K), code, dev)
    ldo = _rows(out, "out", (T, N), out_code, dev)
    if residual is None:
        res, ldr = None, 0
    else:
        res, ldr = residual.data_ptr(), _rows(residual, "residual", (T, N), out_code, dev)
    err = _lib.moe_linear_forward(C.byref(cfg), C.byref(wts), x.data_ptr(), ldx, res, ldr, T, out.data_ptr(), ldo,
                                  st if stream is None else _stream(stream))
    if err:
        _check(err)


def moe_linear_device_error(stream=None):
    """Returns (status, detail) of the dense products made on this stream and clears it."""
    detail = C.c_uint32(0)
    st = _lib.moe_linear_device_error(C.byref(detail), _stream(stream))
    return st, detail.value


def moe_linear_selftest_bounded_wait(timeout_ns, stream=None):
    _check(_lib.moe_linear_selftest_bounded_wait(int(timeout_ns), _stream(stream)))


def route_config(n_experts, top_k, score=MOE_SCORE_SOFTMAX, n_groups=1, topk_groups=1, group_score=MOE_GROUP_MAX,
                 renormalise=True, scale=1.0):
    return MoeRouteConfig(n_experts, top_k, score, n_groups, topk_groups, group_score, 1 if renormalise else 0, scale)


def _route_out(T, K, idx, w, dev):
    shape = (T, K)
    if idx.shape != shape or w.shape != shape or idx.dtype is not _int32 or w.dtype not in _dtype_sets[MOE_F32] \
            or not idx.is_contiguous() or not w.is_contiguous():
        _bad("idx and w must be contiguous int32 and float32 tensors of %s" % (shape,))
    if idx.get_device() != dev or w.get_device() != dev:
        _bad("idx and w must be on the current CUDA device")


def moe_route_from_logits(cfg, logits, idx, w, select_bias=None, stream=None):
    """Expert choice (see moe.h).  logits: float32, bfloat16 or float16 CUDA tensor [T][E] with adjacent
    columns; idx int32 [T][K], w float32 [T][K] (written)."""
    dev, st = _current()
    T, E = logits.shape[0], cfg.n_experts
    code = _logit_codes.get(logits.dtype, MOE_F32)
    ld = _rows(logits, "logits", (T, E), code, dev)
    _route_out(T, cfg.top_k, idx, w, dev)
    bias = None if select_bias is None else _vec(select_bias, "select_bias", E, dev)
    err = _lib.moe_route_from_logits(C.byref(cfg), logits.data_ptr(), code, ld, bias, T, idx.data_ptr(), w.data_ptr(),
                                     st if stream is None else _stream(stream))
    if err:
        _check(err)


def moe_route_workspace_bytes(cfg, T):
    return _lib.moe_route_workspace_bytes(C.byref(cfg), int(T))


def moe_route_topk(cfg, x, wr, idx, w, router_bias=None, select_bias=None, logits_out=None, workspace=None,
                   stream=None):
    """Router projection and expert choice (see moe.h).  x bf16 [T][H], wr bf16 [E][H], contiguous; the logits go
    to logits_out (float32 [T][E]) or to the workspace."""
    dev, st = _current()
    T, H, E = x.shape[0], x.shape[1], cfg.n_experts
    if not x.is_contiguous() or not wr.is_contiguous() or (logits_out is not None and not logits_out.is_contiguous()):
        _bad("x, wr and logits_out must be contiguous")
    _rows(x, "x", (T, H), MOE_BF16, dev)
    _rows(wr, "wr", (E, H), MOE_BF16, dev)
    if logits_out is not None:
        _rows(logits_out, "logits_out", (T, E), MOE_F32, dev)
    if workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous()):
        _bad("workspace must be contiguous, on the current CUDA device")
    _route_out(T, cfg.top_k, idx, w, dev)
    rb = None if router_bias is None else _vec(router_bias, "router_bias", E, dev)
    sb = None if select_bias is None else _vec(select_bias, "select_bias", E, dev)
    _check(_lib.moe_route_topk(C.byref(cfg), H, x.data_ptr(), wr.data_ptr(), rb, sb, T, idx.data_ptr(), w.data_ptr(),
                               _ptr(logits_out), _ptr(workspace), 0 if workspace is None else _nbytes(workspace),
                               st if stream is None else _stream(stream)))


# ---- expert-streaming tier -------------------------------------------------------

class MoeStreamCounters(C.Structure):
    _fields_ = [("hits", C.c_uint64), ("misses", C.c_uint64), ("prefetches", C.c_uint64),
                ("prefetch_hits", C.c_uint64), ("prefetch_dropped", C.c_uint64), ("bytes_h2d", C.c_uint64),
                ("device_error", C.c_uint64)]


def moe_stream_create(cfg, n_layers, host_store, n_slots, store_bytes=None):
    """host_store: pinned host tensor (or address) of n_layers*E packed blobs;
    store_bytes defaults to the tensor's size.  Returns the cache handle (an
    int)."""
    if store_bytes is None:
        store_bytes = _nbytes(host_store)
    h = C.c_void_p(0)
    _check(_lib.moe_stream_create(C.byref(cfg), int(n_layers), _ptr(host_store), int(store_bytes), int(n_slots),
                                  C.byref(h)))
    return h.value


def moe_stream_create_file(cfg, n_layers, path, n_slots, direct_io=False, n_read_threads=4):
    """A cache whose store is a file of n_layers*E packed blobs (see moe.h).
    Returns the cache handle (an int)."""
    h = C.c_void_p(0)
    _check(_lib.moe_stream_create_file(C.byref(cfg), int(n_layers), os.fsencode(path), 1 if direct_io else 0,
                                       int(n_slots), int(n_read_threads), C.byref(h)))
    return h.value


def moe_stream_file_stats(cache):
    reads, nbytes, ms = C.c_uint64(0), C.c_uint64(0), C.c_double(0.0)
    _check(_lib.moe_stream_file_stats(cache, C.byref(reads), C.byref(nbytes), C.byref(ms)))
    return {"reads": int(reads.value), "read_bytes": int(nbytes.value), "read_ms": float(ms.value)}


MOE_FAULT_NONE, MOE_FAULT_COPY, MOE_FAULT_ALLOC = 0, 1, 2


def moe_stream_inject_fault(cache, what, countdown=0):
    _check(_lib.moe_stream_inject_fault(cache, int(what), int(countdown)))


def _ids(ids):
    a = np.ascontiguousarray(np.asarray(ids, dtype=np.int32).reshape(-1))
    return a, a.size


def moe_stream_prefetch(cache, layer, expert_ids, copy_stream=None):
    a, n = _ids(expert_ids)
    _check(_lib.moe_stream_prefetch(cache, int(layer), a.ctypes.data, n, _stream(copy_stream)))


def moe_stream_resolve(cache, layer, idx, expert_ptr, stream=None):
    """idx: host ids (numpy / list); expert_ptr: int64 CUDA tensor [E] (written)."""
    a, n = _ids(idx)
    _check(_lib.moe_stream_resolve(cache, int(layer), a.ctypes.data, n, _ptr(expert_ptr), _stream(stream)))


def moe_stream_resolve_device(cache, layer, idx, expert_ptr, stream=None):
    """idx: int32 CUDA tensor of expert ids (any shape, at most 64); expert_ptr:
    int64 CUDA tensor [E] (written on the device).  Nothing is read back."""
    _check(_lib.moe_stream_resolve_device(cache, int(layer), _ptr(idx), int(idx.numel()), _ptr(expert_ptr),
                                          _stream(stream)))


def moe_layer_forward_streamed(cfg, wts, x, residual, h_out, y_norm, cache, layer, workspace, idx_out=None,
                               w_out=None, stream=None):
    """One streamed layer in one launch: the routed experts come from the
    device-resolved cache `cache` (layer `layer`); wts' expert_ptr is ignored."""
    T = x.shape[0]
    _check(_lib.moe_layer_forward_streamed(C.byref(cfg), C.byref(wts), _ptr(x), _ptr(residual), T, _ptr(h_out),
                                           _ptr(y_norm), _ptr(idx_out), _ptr(w_out), cache, int(layer),
                                           _ptr(workspace), workspace.numel() * workspace.element_size(),
                                           _stream(stream)))


def moe_stream_stats(cache):
    out = MoeStreamCounters()
    _check(_lib.moe_stream_stats(cache, C.byref(out)))
    return {f: int(getattr(out, f)) for f, _ in MoeStreamCounters._fields_}


class MoeStreamCopyTimes(C.Structure):
    _fields_ = [("busy_ms", C.c_double), ("copy_ms", C.c_double), ("copies", C.c_uint64), ("bytes", C.c_uint64)]


def moe_stream_enable_copy_timing(cache, on=True):
    _check(_lib.moe_stream_enable_copy_timing(cache, 1 if on else 0))


def moe_stream_copy_timing(cache):
    out = MoeStreamCopyTimes()
    _check(_lib.moe_stream_copy_timing(cache, C.byref(out)))
    return {f: (float(getattr(out, f)) if f.endswith("_ms") else int(getattr(out, f)))
            for f, _ in MoeStreamCopyTimes._fields_}


def moe_stream_destroy(cache):
    _lib.moe_stream_destroy(cache)


def moe_device_error(workspace, stream=None):
    """Returns (status, detail) and clears the workspace's error word."""
    detail = C.c_uint32(0)
    st = _lib.moe_device_error(_ptr(workspace), C.byref(detail), _stream(stream))
    return st, detail.value


def moe_noalloc_device_error(stream=None):
    """Returns (status, detail) of the last moe_layer_forward_noalloc call on
    the current device and clears it."""
    detail = C.c_uint32(0)
    st = _lib.moe_noalloc_device_error(C.byref(detail), _stream(stream))
    return st, detail.value


def moe_selftest_bounded_wait(workspace, timeout_ns, stream=None):
    _check(_lib.moe_selftest_bounded_wait(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                          int(timeout_ns), _stream(stream)))

"""ctypes binding of libsbp (the C ABI in include/sbp.h).

Argument marshalling only: tensors are passed as raw device pointers, the workspace is a
torch uint8 tensor, the stream is torch's current CUDA stream.  Every step of the streamed
backward runs inside libsbp's kernels; there is no CPU or PyTorch fallback -- if the library
is missing, ``load()`` raises.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import itertools
import os
from typing import Dict, Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libsbp.so")

SBP_F32, SBP_BF16 = 0, 1
STATUS = {0: "SBP_OK", 1: "SBP_ERR_INVALID_ARG", 2: "SBP_ERR_UNSUPPORTED", 3: "SBP_ERR_WORKSPACE",
          4: "SBP_ERR_CUDA", 5: "SBP_ERR_DEVICE_TIMEOUT", 6: "SBP_ERR_BAD_TARGET"}

EXPORTS = [
    "sbp_last_error", "sbp_version", "sbp_chunk_bounds", "sbp_get_device_status",
    "sbp_lmhead_ce_workspace_size", "sbp_lmhead_ce_backward_stream",
    "sbp_decoder_layer_workspace_size", "sbp_decoder_layer_backward_stream",
    "sbp_decoder_layer_forward_stream", "sbp_rmsnorm_forward",
    "sbp_rmsnorm_backward_workspace_size", "sbp_rmsnorm_backward", "sbp_embedding_forward",
    "sbp_embedding_backward_workspace_size", "sbp_embedding_backward", "sbp_debug_gemm_bf16",
    "sbp_launch_count", "sbp_profile_begin", "sbp_profile_end", "sbp_lmhead_ce_backward_noalloc",
    "sbp_debug_attn_fwd_bf16", "sbp_debug_attn_bwd_bf16", "sbp_lmhead_ce_forward_stream",
    "sbp_dpo_workspace_size", "sbp_dpo_token_weights", "sbp_lmhead_ce_workspace_size_host",
    "sbp_lmhead_ce_backward_stream_host", "sbp_decoder_layer_backward_stream_reverse",
    "sbp_debug_gemm_stall_bf16", "sbp_embedding_scaled_forward",
    "sbp_embedding_scaled_backward_workspace_size", "sbp_embedding_scaled_backward",
    "sbp_rope_table", "sbp_qk_norm_rope_forward", "sbp_qk_norm_rope_backward_workspace_size",
    "sbp_qk_norm_rope_backward", "sbp_grad_norm_workspace_size", "sbp_grad_sqsum",
    "sbp_grad_clip", "sbp_grad_clip_norm", "sbp_decoder_layer_qk_norm_workspace_size",
    "sbp_decoder_layer_qk_norm_forward_stream", "sbp_decoder_layer_qk_norm_backward_stream",
]

WEIGHT_FIELDS = ("ln1_g", "wq", "wk", "wv", "bq", "bk", "bv", "wo", "ln2_g", "w_gate", "w_up",
                 "w_down")
# gains of the per-head norms of queries and keys, which a layer may have besides (sbp_step.h)
QK_NORM_FIELDS = ("q_norm_g", "k_norm_g")


class SbpError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code


class Profile(C.Structure):
    _fields_ = [("launches", C.c_longlong * 4), ("ms", C.c_double * 4),
                ("busy_ms", C.c_double * 4)]


class LayerCfg(C.Structure):
    _fields_ = [("batch", C.c_int64), ("seq_len", C.c_int64), ("d_model", C.c_int64),
                ("n_heads", C.c_int64), ("n_kv_heads", C.c_int64), ("head_dim", C.c_int64),
                ("ffn", C.c_int64), ("rms_eps", C.c_float), ("rope_theta", C.c_double),
                ("dtype", C.c_int), ("num_chunks", C.c_int)]


class LayerWeights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in WEIGHT_FIELDS]


class LayerGrads(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in WEIGHT_FIELDS]


class QkGains(C.Structure):
    _fields_ = [("q_g", C.c_void_p), ("k_g", C.c_void_p)]


class QkCfg(C.Structure):
    _fields_ = [("rows", C.c_int64), ("n_heads", C.c_int64), ("n_kv_heads", C.c_int64),
                ("head_dim", C.c_int64), ("seq_len", C.c_int64), ("table_len", C.c_int64),
                ("eps", C.c_float), ("dtype", C.c_int)]


_lib = None


def load(path: Optional[str] = None):
    """Open libsbp.so (built by build.py).  Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libsbp.so not found at {p}; run "
                           "`python -m memory_efficient_exact_chunk_b200.build`")
    lib = C.CDLL(p)
    vp, i64, sz = C.c_void_p, C.c_int64, C.c_size_t
    lib.sbp_last_error.restype = C.c_char_p
    lib.sbp_version.restype = C.c_char_p
    lib.sbp_chunk_bounds.argtypes = [i64, C.c_int, C.POINTER(C.c_int64)]
    lib.sbp_get_device_status.argtypes = [vp, vp]
    lib.sbp_lmhead_ce_workspace_size.restype = sz
    lib.sbp_lmhead_ce_workspace_size.argtypes = [i64, i64, i64, C.c_int, C.c_int]
    lib.sbp_lmhead_ce_backward_stream.argtypes = [i64, i64, i64, C.c_int, C.c_int] + [vp] * 7 + \
        [vp, sz, vp]
    lib.sbp_lmhead_ce_workspace_size_host.restype = sz
    lib.sbp_lmhead_ce_workspace_size_host.argtypes = [i64, i64, i64, C.c_int, C.c_int]
    lib.sbp_lmhead_ce_backward_stream_host.argtypes = [i64, i64, i64, C.c_int, C.c_int] + \
        [vp] * 7 + [vp, sz, vp]
    lib.sbp_lmhead_ce_forward_stream.argtypes = [i64, i64, i64, C.c_int, C.c_int] + [vp] * 6 + \
        [vp, sz, vp]
    lib.sbp_dpo_workspace_size.restype = sz
    lib.sbp_dpo_workspace_size.argtypes = [i64]
    lib.sbp_dpo_token_weights.argtypes = [i64, i64, vp, vp, vp, C.c_float, vp, vp, vp, vp, sz, vp]
    lib.sbp_decoder_layer_workspace_size.restype = sz
    lib.sbp_decoder_layer_workspace_size.argtypes = [C.POINTER(LayerCfg)]
    lib.sbp_decoder_layer_backward_stream.argtypes = [C.POINTER(LayerCfg),
                                                      C.POINTER(LayerWeights), vp, vp, vp,
                                                      C.POINTER(LayerGrads), vp, sz, vp]
    lib.sbp_decoder_layer_backward_stream_reverse.argtypes = \
        lib.sbp_decoder_layer_backward_stream.argtypes
    lib.sbp_decoder_layer_forward_stream.argtypes = [C.POINTER(LayerCfg),
                                                     C.POINTER(LayerWeights), vp, vp, vp, sz, vp]
    lib.sbp_rmsnorm_forward.argtypes = [i64, i64, C.c_int, C.c_float, vp, vp, vp, vp, vp]
    lib.sbp_rmsnorm_backward_workspace_size.restype = sz
    lib.sbp_rmsnorm_backward_workspace_size.argtypes = [i64, i64]
    lib.sbp_rmsnorm_backward.argtypes = [i64, i64, C.c_int, vp, vp, vp, vp, vp, C.c_int, vp, vp,
                                         sz, vp]
    lib.sbp_embedding_forward.argtypes = [i64, i64, i64, C.c_int, vp, vp, vp, vp]
    lib.sbp_embedding_backward_workspace_size.restype = sz
    lib.sbp_embedding_backward_workspace_size.argtypes = [i64, i64]
    lib.sbp_embedding_backward.argtypes = [i64, i64, i64, vp, vp, vp, vp, sz, vp]
    lib.sbp_embedding_scaled_forward.argtypes = [i64, i64, i64, C.c_int, C.c_float, vp, vp, vp, vp]
    lib.sbp_embedding_scaled_backward_workspace_size.restype = sz
    lib.sbp_embedding_scaled_backward_workspace_size.argtypes = [i64, i64, i64]
    lib.sbp_embedding_scaled_backward.argtypes = [i64, i64, i64, C.c_float, vp, vp, vp, C.c_int,
                                                  vp, sz, vp]
    lib.sbp_rope_table.argtypes = [i64, i64, C.c_double, vp, vp, vp]
    lib.sbp_qk_norm_rope_forward.argtypes = [C.POINTER(QkCfg), vp, i64, vp, i64] + [vp] * 5 + \
        [vp, i64, vp, i64, vp]
    lib.sbp_qk_norm_rope_backward_workspace_size.restype = sz
    lib.sbp_qk_norm_rope_backward_workspace_size.argtypes = [C.POINTER(QkCfg)]
    lib.sbp_qk_norm_rope_backward.argtypes = [C.POINTER(QkCfg), vp, i64, vp, i64] + [vp] * 5 + \
        [vp, i64] * 4 + [vp, vp, vp, sz, vp]
    lib.sbp_decoder_layer_qk_norm_workspace_size.restype = sz
    lib.sbp_decoder_layer_qk_norm_workspace_size.argtypes = [C.POINTER(LayerCfg)]
    lib.sbp_decoder_layer_qk_norm_forward_stream.argtypes = [
        C.POINTER(LayerCfg), C.POINTER(LayerWeights), C.POINTER(QkGains), vp, vp, vp, sz, vp]
    lib.sbp_decoder_layer_qk_norm_backward_stream.argtypes = [
        C.POINTER(LayerCfg), C.POINTER(LayerWeights), C.POINTER(QkGains), vp, vp, vp,
        C.POINTER(LayerGrads), vp, vp, C.c_int, vp, sz, vp]
    lib.sbp_grad_norm_workspace_size.restype = sz
    lib.sbp_grad_norm_workspace_size.argtypes = [i64]
    lib.sbp_grad_sqsum.argtypes = [i64, vp, vp, vp, vp, sz, vp]
    lib.sbp_grad_clip.argtypes = [i64, vp, vp, vp, vp, C.c_float, vp, vp]
    lib.sbp_grad_clip_norm.argtypes = [i64, vp, vp, vp, C.c_float, vp, vp, sz, vp]
    lib.sbp_debug_gemm_bf16.argtypes = [i64, i64, i64, vp, C.c_int, i64, vp, C.c_int, i64, vp, i64,
                                         C.c_int, C.c_int, i64, vp, vp]
    lib.sbp_lmhead_ce_backward_noalloc.argtypes = [i64, i64, i64, C.c_int, C.c_int] + [vp] * 7 + \
        [vp]
    lib.sbp_debug_gemm_stall_bf16.argtypes = [i64, i64, i64, vp, vp, vp, i64, vp, vp]
    lib.sbp_debug_attn_fwd_bf16.argtypes = [i64] * 7 + [vp] * 5 + [C.c_int, vp, vp]
    lib.sbp_debug_attn_bwd_bf16.argtypes = [i64] * 7 + [vp] * 9 + [C.c_int, vp, vp]
    lib.sbp_launch_count.restype = C.c_longlong
    lib.sbp_profile_end.argtypes = [C.POINTER(Profile)]
    _lib = lib
    return lib


def _check(code: int):
    if code != 0:
        raise SbpError(code, load().sbp_last_error().decode())


def chunk_bounds(seq_len: int, num_chunks: int):
    arr = (C.c_int64 * (num_chunks + 1))()
    _check(load().sbp_chunk_bounds(seq_len, num_chunks, arr))
    return [(arr[i], arr[i + 1]) for i in range(num_chunks)]


# ----------------------------------------------------------------------------- torch helpers
_TORCH = None


def _torch():
    """torch, imported at the first use (the calls below are short: a global is cheaper than the
    import statement)."""
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def _dtype_code(t):
    torch = _torch()
    if t.dtype is torch.bfloat16:
        return SBP_BF16
    if t.dtype is torch.float32:
        return SBP_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def allocating(stream):
    """Where torch allocates for `stream` (None: the current stream).  Memory taken from another
    stream's pool may still be in use by that stream's queued work."""
    return contextlib.nullcontext() if stream is None else _torch().cuda.stream(stream)


def workspace(nbytes: int, device="cuda", stream=None):
    """A 256-byte aligned device buffer of at least nbytes (torch allocations are aligned) for
    calls on `stream`."""
    torch = _torch()
    with allocating(stream):
        t = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    if stream is not None and t.is_cuda:      # it may be passed to calls on the current one too
        t.record_stream(torch.cuda.current_stream(t.device))
    return t


def device_status(ws, stream=None):
    _check(load().sbp_get_device_status(_ptr(ws), _stream(stream)))


# ----------------------------------------------------------------------------- LM head
def lmhead_ce_workspace_size(n_tokens, hidden, vocab, num_chunks, dtype_code):
    return load().sbp_lmhead_ce_workspace_size(n_tokens, hidden, vocab, num_chunks, dtype_code)


def lmhead_ce_backward(hidden_states, weight, targets, loss_weights, num_chunks, loss_out,
                       d_hidden, d_weight, ws=None, stream=None):
    """loss_out[0] = sum_t w_t CE_t; d_hidden overwritten; d_weight += (all fp32)."""
    N, d = hidden_states.shape
    V = weight.shape[0]
    dt = _dtype_code(hidden_states)
    need = lmhead_ce_workspace_size(N, d, V, num_chunks, dt)
    if ws is None:
        ws = workspace(need, hidden_states.device, stream)
    _check(load().sbp_lmhead_ce_backward_stream(
        N, d, V, num_chunks, dt, _ptr(hidden_states), _ptr(weight), _ptr(targets),
        _ptr(loss_weights), _ptr(loss_out), _ptr(d_hidden), _ptr(d_weight), _ptr(ws),
        ws.numel(), _stream(stream)))
    return ws


def lmhead_ce_backward_host(hidden_states_host, weight, targets_host, loss_weights_host,
                            num_chunks, loss_out, d_hidden, d_weight, ws=None, stream=None):
    """sbp_lmhead_ce_backward_stream_host: hidden states, targets and loss weights in (pinned)
    host memory, staged chunk by chunk by the library; everything else on the device."""
    N, d = hidden_states_host.shape
    V = weight.shape[0]
    dt = _dtype_code(hidden_states_host)
    if ws is None:
        ws = workspace(int(load().sbp_lmhead_ce_workspace_size_host(N, d, V, num_chunks, dt)),
                       weight.device, stream)
    _check(load().sbp_lmhead_ce_backward_stream_host(
        N, d, V, num_chunks, dt, _ptr(hidden_states_host), _ptr(weight), _ptr(targets_host),
        _ptr(loss_weights_host), _ptr(loss_out), _ptr(d_hidden), _ptr(d_weight), _ptr(ws),
        ws.numel(), _stream(stream)))
    return ws


def lmhead_ce_workspace_size_host(N, d, V, D, dt) -> int:
    return int(load().sbp_lmhead_ce_workspace_size_host(N, d, V, D, dt))


def lmhead_ce_forward(hidden_states, weight, targets, loss_weights, num_chunks, token_ce,
                      loss_out=None, ws=None, stream=None):
    """token_ce[t] = CE_t where loss_weights[t] != 0, else 0 (include/sbp_dpo.h); loss_out[0]
    (optional) = sum_t w_t CE_t."""
    N, d = hidden_states.shape
    V = weight.shape[0]
    dt = _dtype_code(hidden_states)
    need = lmhead_ce_workspace_size(N, d, V, num_chunks, dt)
    if ws is None:
        ws = workspace(need, hidden_states.device, stream)
    _check(load().sbp_lmhead_ce_forward_stream(
        N, d, V, num_chunks, dt, _ptr(hidden_states), _ptr(weight), _ptr(targets),
        _ptr(loss_weights), _ptr(token_ce), _ptr(loss_out) if loss_out is not None else None,
        _ptr(ws), ws.numel(), _stream(stream)))
    return ws


def dpo_workspace_size(n_pairs: int) -> int:
    return int(load().sbp_dpo_workspace_size(n_pairs))


def dpo_token_weights(n_pairs, seq_len, token_ce, response_mask, ref_logp, beta, loss_out,
                      weights, seq_logp=None, ws=None, stream=None):
    """DPO loss into loss_out[0] and per-token loss weights (include/sbp_dpo.h)."""
    if ws is None:
        ws = workspace(dpo_workspace_size(n_pairs), token_ce.device, stream)
    _check(load().sbp_dpo_token_weights(
        n_pairs, seq_len, _ptr(token_ce), _ptr(response_mask), _ptr(ref_logp), float(beta),
        _ptr(loss_out), _ptr(seq_logp) if seq_logp is not None else None, _ptr(weights),
        _ptr(ws), ws.numel(), _stream(stream)))
    return ws


def lmhead_ce_backward_noalloc(hidden_states, weight, targets, loss_weights, num_chunks, loss_out,
                               d_hidden, d_weight, stream=None):
    """As lmhead_ce_backward, with the library's own fixed scratch instead of a workspace
    (include/sbp_noalloc.h): nothing is allocated, sizes above the scratch are rejected."""
    N, d = hidden_states.shape
    V = weight.shape[0]
    _check(load().sbp_lmhead_ce_backward_noalloc(
        N, d, V, num_chunks, _dtype_code(hidden_states), _ptr(hidden_states), _ptr(weight),
        _ptr(targets), _ptr(loss_weights), _ptr(loss_out), _ptr(d_hidden), _ptr(d_weight),
        _stream(stream)))


# ----------------------------------------------------------------------------- decoder layer
def layer_cfg(batch, seq_len, d_model, n_heads, n_kv_heads, head_dim, ffn, rms_eps, rope_theta,
              dtype_code, num_chunks) -> LayerCfg:
    return LayerCfg(batch, seq_len, d_model, n_heads, n_kv_heads, head_dim, ffn, rms_eps,
                    rope_theta, dtype_code, num_chunks)


def _struct(cls, tensors: Dict[str, object]):
    return cls(**{n: (tensors[n].data_ptr() if tensors.get(n) is not None else None)
                  for n in WEIGHT_FIELDS})


def has_qk_norm(weights) -> bool:
    """Whether a layer's weights name the gains of query/key norms (both or none)."""
    n = sum(weights.get(f) is not None for f in QK_NORM_FIELDS)
    if n == 1:
        raise ValueError("q_norm_g and k_norm_g must be both set or both absent")
    return n == 2


def layer_workspace_size(cfg: LayerCfg, qk_norm: bool = False) -> int:
    lib = load()
    if qk_norm:
        return lib.sbp_decoder_layer_qk_norm_workspace_size(C.byref(cfg))
    return lib.sbp_decoder_layer_workspace_size(C.byref(cfg))


def _layer_ws(cfg, qk_norm, ws, device, stream):
    need = layer_workspace_size(cfg, qk_norm)
    if need == 0:
        raise SbpError(1, "invalid layer configuration")
    return workspace(need, device, stream) if ws is None else ws


def _qk_gains(cfg, weights, device):
    import torch
    dtype = torch.bfloat16 if cfg.dtype == SBP_BF16 else torch.float32
    for f in QK_NORM_FIELDS:
        _is(weights[f], f, dtype, (cfg.head_dim,))
        if weights[f].device != device:
            raise ValueError(f"{f}: must be on {device}")
    return QkGains(*[weights[f].data_ptr() for f in QK_NORM_FIELDS])


def _layer_backward(reverse, cfg, weights, x, dy, dx, grads, ws, stream):
    lib = load()
    qk_norm = has_qk_norm(weights)
    ws = _layer_ws(cfg, qk_norm, ws, x.device, stream)
    w = _struct(LayerWeights, weights)
    g = _struct(LayerGrads, grads)
    if qk_norm:
        import torch
        gains = _qk_gains(cfg, weights, x.device)
        for f in QK_NORM_FIELDS:
            if grads.get(f) is None:
                raise ValueError(f"grads: {f} is missing")
            _is(grads[f], f"grads[{f!r}]", torch.float32, (cfg.head_dim,))
        _check(lib.sbp_decoder_layer_qk_norm_backward_stream(
            C.byref(cfg), C.byref(w), C.byref(gains), _ptr(x), _ptr(dy), _ptr(dx), C.byref(g),
            *[_ptr(grads[f]) for f in QK_NORM_FIELDS], int(reverse), _ptr(ws), ws.numel(),
            _stream(stream)))
        return ws
    fn = (lib.sbp_decoder_layer_backward_stream_reverse if reverse
          else lib.sbp_decoder_layer_backward_stream)
    _check(fn(C.byref(cfg), C.byref(w), _ptr(x), _ptr(dy), _ptr(dx), C.byref(g), _ptr(ws),
              ws.numel(), _stream(stream)))
    return ws


def decoder_layer_backward(cfg: LayerCfg, weights, x, dy, dx, grads, ws=None, stream=None):
    """The streamed backward of a layer.  Weights with q_norm_g and k_norm_g [head_dim] add the
    per-head norms of queries and keys (include/sbp_step.h); grads then has both too."""
    return _layer_backward(False, cfg, weights, x, dy, dx, grads, ws, stream)


def decoder_layer_backward_reverse(cfg: LayerCfg, weights, x, dy, dx, grads, ws=None,
                                   stream=None):
    """The layer backward with the chunks visited from last to first."""
    return _layer_backward(True, cfg, weights, x, dy, dx, grads, ws, stream)


def decoder_layer_forward(cfg: LayerCfg, weights, x, y, ws=None, stream=None):
    lib = load()
    qk_norm = has_qk_norm(weights)
    ws = _layer_ws(cfg, qk_norm, ws, x.device, stream)
    w = _struct(LayerWeights, weights)
    if qk_norm:
        gains = _qk_gains(cfg, weights, x.device)
        _check(lib.sbp_decoder_layer_qk_norm_forward_stream(
            C.byref(cfg), C.byref(w), C.byref(gains), _ptr(x), _ptr(y), _ptr(ws), ws.numel(),
            _stream(stream)))
    else:
        _check(lib.sbp_decoder_layer_forward_stream(C.byref(cfg), C.byref(w), _ptr(x), _ptr(y),
                                                    _ptr(ws), ws.numel(), _stream(stream)))
    return ws


# ----------------------------------------------------------------------------- support
def rmsnorm_forward(x2d, g, eps, y2d, rstd=None, stream=None):
    rows, cols = x2d.shape
    _check(load().sbp_rmsnorm_forward(rows, cols, _dtype_code(x2d), eps, _ptr(x2d), _ptr(g),
                                      _ptr(y2d), _ptr(rstd), _stream(stream)))


def rmsnorm_backward(x2d, g, rstd, dy2d, dx2d, dg, accumulate=False, ws=None, stream=None):
    rows, cols = x2d.shape
    need = load().sbp_rmsnorm_backward_workspace_size(rows, cols)
    if ws is None or ws.numel() < need:
        ws = workspace(need, x2d.device, stream)
    _check(load().sbp_rmsnorm_backward(rows, cols, _dtype_code(x2d), _ptr(x2d), _ptr(g),
                                       _ptr(rstd), _ptr(dy2d), _ptr(dx2d), int(accumulate),
                                       _ptr(dg), _ptr(ws), ws.numel(), _stream(stream)))
    return ws


def embedding_forward(ids, table, y, stream=None):
    rows = ids.numel()
    V, cols = table.shape
    _check(load().sbp_embedding_forward(rows, cols, V, _dtype_code(table), _ptr(ids),
                                        _ptr(table), _ptr(y), _stream(stream)))


def embedding_backward(ids, dy2d, d_table, ws=None, stream=None):
    rows = ids.numel()
    V, cols = d_table.shape
    need = load().sbp_embedding_backward_workspace_size(rows, V)
    if ws is None or ws.numel() < need:
        ws = workspace(need, dy2d.device, stream)
    _check(load().sbp_embedding_backward(rows, cols, V, _ptr(ids), _ptr(dy2d), _ptr(d_table),
                                         _ptr(ws), ws.numel(), _stream(stream)))
    return ws


# ----------------------------------------------------------------------------- step operators
# These calls are short, so their checks are kept cheap: shapes are compared as they are (a
# torch.Size is a tuple), pointers go to ctypes as integers.
def _on_device(stream, *tensors):
    """The index of the one CUDA device of `tensors` (None entries are left out) and the raw
    stream.  The library launches on the current device: tensors and stream have to be its."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("tensors must be on one CUDA device")
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    # the device and the current stream's handle as torch keeps them: torch.cuda's own calls make
    # a Stream object (3 us)
    own = _torch()._C
    if dev != own._cuda_getDevice() or (stream is not None and stream.device.index != dev):
        raise ValueError(f"tensors on cuda:{dev}: the current device and the stream must be its")
    return dev, own._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _is(t, name, dtype, shape):
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def _with_ws(ws, dev, stream, need, call):
    """call(address, bytes) with ws, or with a new workspace of need() bytes where ws is None or
    too small for the library; the workspace used.  (Sizes that the library refuses need 0 bytes;
    the call itself then says why.)"""
    if ws is not None:
        if not ws.is_contiguous() or ws.get_device() != dev:
            raise ValueError(f"the workspace must be a contiguous buffer on cuda:{dev}")
        code = call(ws.data_ptr(), ws.nbytes)
        if code == 0:
            return ws
        if code != 3:                    # SBP_ERR_WORKSPACE, before anything is queued
            _check(code)
    ws = workspace(need(), f"cuda:{dev}", stream)
    _check(call(ws.data_ptr(), ws.nbytes))
    return ws


def _addr(t):
    return None if t is None else t.data_ptr()


def embedding_scaled_forward(ids, table, scale, y, stream=None):
    """y[r] = scale * table[ids[r]]; ids int32, any shape; ids outside [0, vocab) give zero rows
    (include/sbp_step.h)."""
    shape = table.shape
    V, cols = shape
    rows = ids.numel()
    dtype, dt = table.dtype, _dtype_code(table)
    _is(ids, "ids", _torch().int32, ids.shape)
    _is(table, "table", dtype, shape)
    _is(y, "y", dtype, (rows, cols) if y.dim() == 2 else (*ids.shape, cols))
    _, st = _on_device(stream, ids, table, y)
    code = load().sbp_embedding_scaled_forward(rows, cols, V, dt, scale, ids.data_ptr(),
                                               table.data_ptr(), y.data_ptr(), st)
    if code:
        _check(code)


def embedding_scaled_backward_workspace_size(rows, cols, vocab) -> int:
    return int(load().sbp_embedding_scaled_backward_workspace_size(rows, cols, vocab))


def embedding_scaled_backward(ids, dy, scale, d_table, accumulate=True, ws=None, stream=None):
    """d_table (+)= scale * the sum of dy's rows of each id, by sorted tokens; without
    `accumulate` the whole table is written.  Returns the workspace, to be passed again."""
    torch = _torch()
    shape = d_table.shape
    V, cols = shape
    rows = ids.numel()
    _is(ids, "ids", torch.int32, ids.shape)
    _is(d_table, "d_table", torch.float32, shape)
    _is(dy, "dy", torch.float32, (rows, cols) if dy.dim() == 2 else (*ids.shape, cols))
    dev, st = _on_device(stream, ids, dy, d_table)
    fn = load().sbp_embedding_scaled_backward
    return _with_ws(ws, dev, stream,
                    lambda: embedding_scaled_backward_workspace_size(rows, cols, V),
                    lambda p, n: fn(rows, cols, V, scale, ids.data_ptr(), dy.data_ptr(),
                                    d_table.data_ptr(), 1 if accumulate else 0, p, n, st))


def rope_table(n_positions, head_dim, theta, device="cuda", stream=None):
    """(cos, sin) tables [n_positions, head_dim // 2] fp32 of the decoder layer's RoPE."""
    torch = _torch()
    if n_positions < 1 or head_dim < 2:
        raise ValueError("rope_table: need positive sizes")
    with allocating(stream):
        cos = torch.empty(n_positions, head_dim // 2, dtype=torch.float32, device=device)
        sin = torch.empty_like(cos)
    _, st = _on_device(stream, cos)
    _check(load().sbp_rope_table(n_positions, head_dim, theta, cos.data_ptr(), sin.data_ptr(),
                                 st))
    return cos, sin


def _heads(t, name, dtype, shape):
    """Row stride of a [rows, heads, head_dim] tensor whose rows may lie apart."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    rows, n, hd = shape
    sr, sh, s1 = t.stride()
    if s1 != 1 or (n > 1 and sh != hd):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    if rows == 1:
        return n * hd
    if sr < n * hd:
        raise ValueError(f"{name}: the rows overlap")
    return sr


def _qk_call(q, k, q_g, k_g, cos, sin, eps, positions, seq_len):
    """Checks of what both directions share; the leading arguments of both calls."""
    torch = _torch()
    dtype, dt, shape = q.dtype, _dtype_code(q), q.shape
    rows, H, hd = shape
    gain, table = (hd,), (cos.shape[0], hd // 2)
    ldq = _heads(q, "q", dtype, shape)
    _is(q_g, "q_g", dtype, gain)
    _is(cos, "cos", torch.float32, table)
    _is(sin, "sin", torch.float32, table)
    pos = None
    if positions is not None:
        _is(positions, "positions", torch.int32, (rows,))
        pos = positions.data_ptr()
    seq = rows if seq_len is None else seq_len
    if k is None:
        cfg = QkCfg(rows, H, 0, hd, seq, table[0], eps, dt)
        return (C.byref(cfg), q.data_ptr(), ldq, None, 0, q_g.data_ptr(), None, pos,
                cos.data_ptr(), sin.data_ptr())
    Hkv = k.shape[1]
    ldk = _heads(k, "k", dtype, (rows, Hkv, hd))
    _is(k_g, "k_g", dtype, gain)
    cfg = QkCfg(rows, H, Hkv, hd, seq, table[0], eps, dt)
    return (C.byref(cfg), q.data_ptr(), ldq, k.data_ptr(), ldk, q_g.data_ptr(), k_g.data_ptr(), pos,
            cos.data_ptr(), sin.data_ptr())


def qk_norm_rope_forward(q, k, q_g, k_g, cos, sin, eps, q_out, k_out, positions=None,
                         seq_len=None, stream=None):
    """Per-head RMS norm with RoPE of q [rows, heads, head_dim] and k [rows, kv_heads, head_dim]
    (rows may be strided, k may be None) into q_out and k_out, which may be q and k
    (include/sbp_step.h).  The position of row r is positions[r], or r % seq_len (default: r)."""
    args = _qk_call(q, k, q_g, k_g, cos, sin, eps, positions, seq_len)
    ldqo, ldko = _heads(q_out, "q_out", q.dtype, q.shape), 0
    if k is None:
        k_g = k_out = None
    else:
        ldko = _heads(k_out, "k_out", q.dtype, k.shape)
    _, st = _on_device(stream, q, k, q_g, k_g, cos, sin, positions, q_out, k_out)
    code = load().sbp_qk_norm_rope_forward(*args, q_out.data_ptr(), ldqo, _addr(k_out), ldko, st)
    if code:
        _check(code)


def qk_norm_rope_backward(q, k, q_g, k_g, cos, sin, eps, dq_out, dk_out, dq, dk, dq_g, dk_g,
                          positions=None, seq_len=None, ws=None, stream=None):
    """Backward of qk_norm_rope_forward from its inputs: dq, dk overwritten (they may be dq_out,
    dk_out), dq_g, dk_g accumulated (one vector may be both, of a gain that is shared); all
    gradients fp32.  Returns the workspace."""
    f32 = _torch().float32
    args = _qk_call(q, k, q_g, k_g, cos, sin, eps, positions, seq_len)
    gain = (q.shape[2],)
    lddqo, lddq = _heads(dq_out, "dq_out", f32, q.shape), _heads(dq, "dq", f32, q.shape)
    _is(dq_g, "dq_g", f32, gain)
    lddko = lddk = 0
    if k is None:
        k_g = dk_out = dk = dk_g = None
    else:
        lddko, lddk = _heads(dk_out, "dk_out", f32, k.shape), _heads(dk, "dk", f32, k.shape)
        _is(dk_g, "dk_g", f32, gain)
    dev, st = _on_device(stream, q, k, q_g, k_g, cos, sin, positions, dq_out, dk_out, dq, dk,
                         dq_g, dk_g)
    lib = load()
    return _with_ws(ws, dev, stream, lambda: lib.sbp_qk_norm_rope_backward_workspace_size(args[0]),
                    lambda p, n: lib.sbp_qk_norm_rope_backward(
                        *args, dq_out.data_ptr(), lddqo, _addr(dk_out), lddko, dq.data_ptr(),
                        lddq, _addr(dk), lddk, dq_g.data_ptr(), _addr(dk_g), p, n, st))


class GradList:
    """The gradients of a model in the form the norm and the clipping take: checked once, their
    pointers and sizes in host arrays.  No two may share memory (the gradient of a tied weight
    belongs into the list once).

    The list stands for the memory that its tensors have when it is made, and keeps that memory:
    where a tensor gets other memory (`t.data = ...`, `t.set_(...)`) a new list has to be made, and
    a storage in the list must not be resized.  Calls with the old list work on the memory that it
    kept, and raise ValueError once they see the change: each call looks at LOOK tensors in turn,
    all of them where there are no more (looking at one costs 0.07 us, at 300 more than some calls
    take)."""

    LOOK = 8

    def __init__(self, tensors):
        self.tensors = list(tensors)
        if not self.tensors:
            raise ValueError("no gradients")
        f32, n = _torch().float32, len(self.tensors)
        self.device = self.tensors[0].get_device()
        for i, t in enumerate(self.tensors):
            _is(t, f"gradient {i}", f32, t.shape)
            if self.device < 0 or t.get_device() != self.device:
                raise ValueError(f"gradient {i}: all gradients must be on one CUDA device")
        self.sizes = [t.numel() for t in self.tensors]
        ptrs = [t.data_ptr() for t in self.tensors]
        self.memory = [t.untyped_storage() for t in self.tensors]
        k = self.LOOK
        self.parts = itertools.cycle([(self.tensors[i:i + k], ptrs[i:i + k])
                                      for i in range(0, n, k)])
        self.ptrs = (C.c_void_p * n)(*ptrs)
        self.numel = (C.c_int64 * n)(*self.sizes)
        # (start, end, index) of the non-empty ones by address
        self.spans = sorted((p, p + 4 * m, i) for i, (p, m) in enumerate(zip(ptrs, self.sizes))
                            if m)
        for (_, end, i), (start, _, j) in zip(self.spans, self.spans[1:]):
            if start < end:
                raise ValueError(f"gradients {i} and {j} share memory")

    def __len__(self):
        return len(self.tensors)

    def look(self):
        """Raises where one of the next LOOK tensors has other memory than the list."""
        tensors, addresses = next(self.parts)
        if list(map(_TORCH.Tensor.data_ptr, tensors)) != addresses:
            raise ValueError("a gradient has other memory than when its GradList was made: make "
                             "a new list")

    def takes(self, out) -> bool:
        """Whether the results may go to `out`: tensors of the same sizes, each either the
        gradient itself or apart from every gradient."""
        if out.sizes != self.sizes or out.device != self.device:
            return False
        a, b = self.spans, out.spans
        if not a or a[-1][1] <= b[0][0] or b[-1][1] <= a[0][0]:
            return True
        i = 0
        for start, end, k in b:
            while i < len(a) and a[i][1] <= start:
                i += 1
            if i < len(a) and a[i][0] < end and a[i] != (start, end, k):
                return False
        return True


def _grad_args(grads, out, stream, *scalars):
    if isinstance(grads, GradList):
        grads.look()
    else:
        grads = GradList(grads)
    into = None
    if out is not None and out is not grads:
        if isinstance(out, GradList):
            out.look()
        else:
            out = GradList(out)
        if not grads.takes(out):
            raise ValueError("out must have the gradients' sizes and device, and share memory "
                             "with no other gradient than its own")
        into = out.ptrs
    dev, st = _on_device(stream, grads.tensors[0], *scalars)
    return grads, into, dev, st


def grad_norm_workspace_size(n_tensors) -> int:
    return int(load().sbp_grad_norm_workspace_size(n_tensors))


def grad_sqsum(grads, sqsum, ws=None, stream=None):
    """sqsum[0] (float64) = the sum of the squares of all gradients (a GradList, or a list of
    fp32 tensors).  Returns the workspace."""
    _is(sqsum, "sqsum", _torch().float64, (1,))
    grads, _, dev, st = _grad_args(grads, None, stream, sqsum)
    n, fn = len(grads), load().sbp_grad_sqsum
    return _with_ws(ws, dev, stream, lambda: grad_norm_workspace_size(n),
                    lambda p, b: fn(n, grads.ptrs, grads.numel, sqsum.data_ptr(), p, b, st))


def grad_clip(grads, sqsum, max_norm, norm_out=None, out=None, stream=None):
    """out (default: in place) = grads * min(1, max_norm / (sqrt(sqsum) + 1e-6))."""
    torch = _torch()
    _is(sqsum, "sqsum", torch.float64, (1,))
    if norm_out is not None:
        _is(norm_out, "norm_out", torch.float32, (1,))
    grads, into, _, st = _grad_args(grads, out, stream, sqsum, norm_out)
    _check(load().sbp_grad_clip(len(grads), grads.ptrs, into, grads.numel, sqsum.data_ptr(),
                                max_norm, _addr(norm_out), st))


def grad_clip_norm(grads, max_norm, norm_out, out=None, ws=None, stream=None):
    """norm_out[0] = the global norm of all gradients, which are clipped to max_norm (in place,
    or into `out`).  Returns the workspace."""
    _is(norm_out, "norm_out", _torch().float32, (1,))
    grads, into, dev, st = _grad_args(grads, out, stream, norm_out)
    n, fn = len(grads), load().sbp_grad_clip_norm
    return _with_ws(ws, dev, stream, lambda: grad_norm_workspace_size(n),
                    lambda p, b: fn(n, grads.ptrs, into, grads.numel, max_norm,
                                    norm_out.data_ptr(), p, b, st))


# ----------------------------------------------------------------------------- test hooks
def debug_gemm_bf16(A, a_trans, B, b_trans, C, accumulate=False, path=0, kblk=0, ws=None,
                    stream=None):
    """C (+)= op(A) op(B) with bf16 A/B and fp32 C (see include/sbp_debug.h)."""
    M = A.shape[1] if a_trans else A.shape[0]
    K = A.shape[0] if a_trans else A.shape[1]
    N = B.shape[0] if b_trans else B.shape[1]
    if ws is None:
        ws = workspace(256, C.device)
        ws.zero_()
    _check(load().sbp_debug_gemm_bf16(M, N, K, _ptr(A), int(a_trans), A.stride(0), _ptr(B),
                                      int(b_trans), B.stride(0), _ptr(C), C.stride(0),
                                      int(accumulate), int(path), int(kblk), _ptr(ws),
                                      _stream(stream)))
    return ws


def debug_gemm_stall_bf16(A, B, C, wait_limit_ns, ws=None, stream=None):
    """The single-CTA GEMM of C = A B^T with no operand copies issued, so that its bounded
    waits run out after wait_limit_ns (include/sbp_debug.h); returns the workspace whose
    status word the kernel raises."""
    M, K = A.shape
    N = B.shape[0]
    if ws is None:
        ws = workspace(256, C.device)
        ws.zero_()
    _check(load().sbp_debug_gemm_stall_bf16(M, N, K, _ptr(A), _ptr(B), _ptr(C),
                                            int(wait_limit_ns), _ptr(ws), _stream(stream)))
    return ws


# ----------------------------------------------------------------------------- profiling
def launch_count() -> int:
    return int(load().sbp_launch_count())


def profile_begin():
    _check(load().sbp_profile_begin())


def profile_end() -> dict:
    p = Profile()
    _check(load().sbp_profile_end(C.byref(p)))
    names = ("gemm_tc", "gemm_simt", "attn_fwd", "attn_bwd")
    return {n: {"launches": p.launches[i], "ms": p.ms[i], "busy_ms": p.busy_ms[i]}
            for i, n in enumerate(names)}


def debug_attn_fwd_workspace_bytes(B, Tc, H, hd):
    """Workspace of sbp_debug_attn_fwd_bf16: the status word, then the key-range split's
    partial O (fp32), its maxima and sums, and two flags per query-tile pair."""
    pairs = ((Tc + 127) // 128 + 1) // 2
    return 256 + 4 * B * Tc * H * (hd + 2) + 8 * B * H * pairs


def debug_attn_fwd_bf16(q, Kp, Vp, o, lse, s, path=0, ws=None, stream=None):
    """Attention forward of a chunk (include/sbp_debug.h); q/o [B*Tc, H, hd], Kp/Vp
    [B, T, Hkv, hd] bf16, lse [B*Tc, H] fp32."""
    B, T, Hkv, hd = Kp.shape
    R, H, _ = q.shape
    Tc = R // B
    need = debug_attn_fwd_workspace_bytes(B, Tc, H, hd)
    if ws is None:
        ws = workspace(need, q.device)
        ws.zero_()
    elif ws.numel() * ws.element_size() < need:
        raise ValueError(f"attention forward workspace needs {need} bytes")
    _check(load().sbp_debug_attn_fwd_bf16(B, T, Tc, s, H, Hkv, hd, _ptr(q), _ptr(Kp), _ptr(Vp),
                                          _ptr(o), _ptr(lse), int(path), _ptr(ws),
                                          _stream(stream)))
    return ws


def debug_attn_bwd_bf16(q, Kp, Vp, o, dO, lse, dq, dKp, dVp, s, path=0, stream=None):
    """Attention backward of a chunk (include/sbp_debug.h)."""
    B, T, Hkv, hd = Kp.shape
    R, H, _ = q.shape
    Tc = R // B
    tcp = (Tc + 127) // 128 * 128
    ws = workspace(256 + max(4 * R * H, 8 * H * B * tcp), q.device)
    ws.zero_()
    _check(load().sbp_debug_attn_bwd_bf16(B, T, Tc, s, H, Hkv, hd, _ptr(q), _ptr(Kp), _ptr(Vp),
                                          _ptr(o), _ptr(dO), _ptr(lse), _ptr(dq), _ptr(dKp),
                                          _ptr(dVp), int(path), _ptr(ws), _stream(stream)))
    return ws

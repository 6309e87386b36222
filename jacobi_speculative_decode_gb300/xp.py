"""Thin ctypes binding of libxp.so (the C ABI in include/xp.h), same names as the C calls.

Argument marshalling only: tensors become raw pointers, ``None`` becomes NULL,
the stream defaults to torch's current stream.  Every step of the pass runs in
the library's CUDA kernels; there is no Python or CPU fallback -- a missing
library or device raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libxp.so")

XP_BF16, XP_F32, XP_Q8, XP_Q4 = 0, 1, 2, 3
XP_PASSES_AUTO, XP_PASSES_PERSISTENT, XP_PASSES_PER_STAGE = 0, 1, 2
STATUS = {0: "XP_OK", 1: "XP_EINVAL", 2: "XP_ECAPACITY", 3: "XP_ENOTPREPARED", 4: "XP_ECUDA",
          5: "XP_EBADTOKEN", 6: "XP_ETIMEOUT", 7: "XP_EUNSUPPORTED", 8: "XP_ERANGE",
          9: "XP_EBADPAGE", 10: "XP_ENOPAGES", 11: "XP_ESHARED", 12: "XP_ELENGTH", 13: "XP_EEMPTY"}
XP_OK, XP_EINVAL, XP_ECAPACITY, XP_ENOTPREPARED, XP_ECUDA, XP_EBADTOKEN, XP_ETIMEOUT, \
    XP_EUNSUPPORTED, XP_ERANGE, XP_EBADPAGE, XP_ENOPAGES, XP_ESHARED, XP_ELENGTH, \
    XP_EEMPTY = range(14)


class XPError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)} ({status_str(code)})")
        self.code = code


class xp_weights(ctypes.Structure):
    _fields_ = [("V", ctypes.c_int), ("hidden", ctypes.c_int), ("r", ctypes.c_int),
                ("H", ctypes.c_int), ("B", ctypes.c_int), ("max_N", ctypes.c_int),
                ("dtype", ctypes.c_int),
                ("w1", ctypes.c_void_p), ("down_h", ctypes.c_void_p), ("down_g", ctypes.c_void_p),
                ("in_proj", ctypes.c_void_p), ("mix_L", ctypes.c_void_p),
                ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p),
                ("w_down", ctypes.c_void_p), ("w2", ctypes.c_void_p)]


class xp_cache_desc(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_int), ("page_size", ctypes.c_int), ("layers", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("max_seqs", ctypes.c_int),
                ("dtype", ctypes.c_int),
                ("stride_layer", ctypes.c_int64), ("stride_page", ctypes.c_int64),
                ("stride_token", ctypes.c_int64), ("stride_head", ctypes.c_int64),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p)]


class xp_attn(ctypes.Structure):
    _fields_ = [("layer", ctypes.c_int), ("N", ctypes.c_int), ("T", ctypes.c_int),
                ("heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int),
                ("prefix_len", ctypes.c_int), ("max_len", ctypes.c_int),
                ("scale", ctypes.c_float),
                ("q_stride_n", ctypes.c_int64), ("q_stride_t", ctypes.c_int64),
                ("q_stride_h", ctypes.c_int64), ("o_stride_n", ctypes.c_int64),
                ("o_stride_t", ctypes.c_int64), ("o_stride_h", ctypes.c_int64)]


_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_S = ctypes.c_size_t
_SIGS = {
    "xp_head_prep_bytes": (_S, [ctypes.POINTER(xp_weights)]),
    "xp_workspace_bytes": (_S, [ctypes.POINTER(xp_weights), _I, _I]),
    "xp_workspace_init": (_I, [_P, _S, _P]),
    "xp_head_create": (_I, [ctypes.POINTER(xp_weights), _P, _S, _P, ctypes.POINTER(_P)]),
    "xp_head_refill": (_I, [_P, ctypes.POINTER(xp_weights), _P]),
    "xp_head_destroy": (None, [_P]),
    "xp_fold_mix": (_I, [_P, _P, _I, _I, _I, _P]),
    "xp_hidden_cache": (_I, [_P, _P, _I, _P, _P, _S, _P]),
    "xp_latent_pass": (_I, [_P, _P, _P, _P, _I, _P, _P]),
    "xp_readout_argmax": (_I, [_P, _P, _P, _I64, _I64, _I, _P, _P, _P, _S, _P]),
    "xp_readout_argmax_noalloc": (_I, [_P, _P, _P, _I64, _I64, _I, _P, _P, _P]),
    "xp_refine_logits": (_I, [_P, _P, _P, _I64, _I64, _I, _P, _I64, _P]),
    "xp_selftest_wait_timeout": (_I, [_P, _P]),
    "xp_init_argmax": (_I, [_P, _P, _I64, _I64, _P, _I, _P, _P, _P, _S, _P]),
    "xp_topc_gather": (_I, [_P, _P, _I64, _I64, _I, _I, _P, _P, _P, _P, _P]),
    "xp_topc_readout_argmax": (_I, [_P, _P, _P, _P, _P, _I, _I, _P, _P, _P]),
    "xp_jacobi_refine": (_I, [_P, _P, _I64, _I64, _P, _P, _P, _I, _I, _I, _P, _P, _S, _P]),
    "xp_jacobi_passes": (_I, [_P, _P, _I64, _I64, _P, _P, _I, _I, _P, _P, _S, _P]),
    "xp_set_pass_mode": (_I, [_P, _I]),
    "xp_passes_persistent": (_I, [_P, _P, _I64, _I64, _I]),
    "xp_set_readout_pairs": (_I, [_P, _I]),
    "xp_readout_pairs": (_I, [_P, _I]),
    "xp_get_error": (_I, [_P, _P]),
    "xp_readout_kernel_name": (ctypes.c_char_p, [_P]),
    "xp_profile_timeline": (_I, [_P, _P, _S, _I, ctypes.POINTER(_S)]),
    "xp_status_str": (ctypes.c_char_p, [_I]),
    "xp_verify_workspace_bytes": (_S, [_P, _I]),
    "xp_verify_drafts": (_I, [_P, _P, _I64, _I64, _P, _I64, _P, _P, _I, _I, _I, _I, _P, _P, _P, _I64, _P, _P,
                              _P, _P, _S, _P]),
    "xp_logprobs_workspace_bytes": (_S, [_P, _I, _I]),
    "xp_token_logprobs": (_I, [_P, _P, _I64, _I64, _P, _I, _I, _I, _I, _P, _I, _P, _P, _P, _P, _P, _P, _S,
                               _P]),
    "xp_quant_head_bytes": (_S, [_I, _I, _I]),
    "xp_cache_read": (_I, [_P, _I, _P, _I64, _I, _P, _P, _I, _I, _P, _P, _I64, _I64, _I64, _I, _I, _I, _P]),
    "xp_cache_prep_bytes": (_S, [ctypes.POINTER(xp_cache_desc)]),
    "xp_cache_create": (_I, [ctypes.POINTER(xp_cache_desc), _P, _S, _P, ctypes.POINTER(_P)]),
    "xp_cache_destroy": (None, [_P]),
    "xp_cache_get_error": (_I, [_P, _P]),
    "xp_cache_append": (_I, [_P, _I, _P, _P, _I64, _I64, _I64, _I, _I, _I, _P, _I64, _P, _I, _I, _P]),
    "xp_cache_append_columns": (_I, [_P, _I, _P, _P, _I64, _I64, _I64, _I, _I, _I, _P, _I64, _I, _P, _I, _I,
                                     _P]),
    "xp_cache_copy": (_I, [_P, _P, _P, _I, _P]),
    "xp_cache_resize": (_I, [_P, _P, _I64, _P, _P, _P, _I, _I, _I, _P, _I64, _P, _P, _P]),
    "xp_cache_fork": (_I, [_P, _P, _I64, _P, _I, _P, _P, _I, _I, _P, _I, _P, _I64, _P, _P, _P]),
    "xp_cache_compact": (_I, [_P, _P, _I64, _P, _I, _I, _P, _I, _P, _I64, _P, _P, _P, _P]),
    "xp_attention_workspace_bytes": (_S, [_P, ctypes.POINTER(xp_attn)]),
    "xp_prefix_attention": (_I, [_P, ctypes.POINTER(xp_attn), _P, _P, _I, _P, _I64, _I, _P, _P, _P,
                                 _P, _S, _P]),
}

_lib = None
torch = None   # once something has needed it


def _need_torch():
    global torch
    import torch as module
    torch = module


def lib() -> ctypes.CDLL:
    """Load libxp.so once (raises if it was never built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "jacobi_speculative_decode_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def exported_symbols():
    return list(_SIGS)


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream, device=None):
    """The handle of a stream, or of the current one (on `device`, where the caller has looked it up)."""
    if stream is None:
        import torch
        if device is None:
            if not torch.cuda.is_initialized() and not torch.cuda.is_available():
                raise RuntimeError("no CUDA device: libxp has no CPU path")
            device = torch.cuda.current_device()
        # without a Stream object around it where torch gives it so (not a public call)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return raw(device) if raw else torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _nbytes(x):
    """Size in bytes of a buffer given as a tensor (0 for None)."""
    if x is None:
        return 0
    return x.numel() * x.element_size()


def _check(name, code):
    if code != XP_OK:
        raise XPError(name, code)


def status_str(code: int) -> str:
    return lib().xp_status_str(code).decode()


# ------------------------------------------------------------------ sizing ---

def make_weights(V, hidden, r, H, B, max_N, dtype, w1=None, down_h=None, down_g=None,
                 in_proj=None, mix_L=None, w_gate=None, w_up=None, w_down=None, w2=None):
    return xp_weights(V, hidden, r, H, B, max_N, dtype, _ptr(w1), _ptr(down_h), _ptr(down_g),
                      _ptr(in_proj), _ptr(mix_L), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                      _ptr(w2))


def xp_head_prep_bytes(w: xp_weights) -> int:
    return lib().xp_head_prep_bytes(ctypes.byref(w))


def xp_workspace_bytes(w: xp_weights, N: int, topc: int = 0) -> int:
    return lib().xp_workspace_bytes(ctypes.byref(w), N, topc)


# ------------------------------------------------------------------- calls ---

def xp_workspace_init(ws, stream=None):
    _check("xp_workspace_init", lib().xp_workspace_init(_ptr(ws), ws.numel() * ws.element_size(),
                                                        _stream(stream)))


def xp_head_create(w: xp_weights, prep, stream=None):
    out = ctypes.c_void_p()
    _check("xp_head_create", lib().xp_head_create(ctypes.byref(w), _ptr(prep),
                                                  prep.numel() * prep.element_size(),
                                                  _stream(stream), ctypes.byref(out)))
    return out.value


def xp_head_refill(head, w: xp_weights, stream=None):
    _check("xp_head_refill", lib().xp_head_refill(head, ctypes.byref(w), _stream(stream)))


def xp_head_destroy(head):
    lib().xp_head_destroy(head)


def xp_fold_mix(raw, mix, r, B, dtype, stream=None):
    _check("xp_fold_mix", lib().xp_fold_mix(_ptr(raw), _ptr(mix), r, B, dtype, _stream(stream)))


def xp_hidden_cache(head, h_full, N, xh, ws, stream=None):
    _check("xp_hidden_cache", lib().xp_hidden_cache(head, _ptr(h_full), N, _ptr(xh), _ptr(ws),
                                                    _nbytes(ws), _stream(stream)))


def xp_latent_pass(head, blk, am1, xh, N, lat, stream=None):
    _check("xp_latent_pass", lib().xp_latent_pass(head, _ptr(blk), _ptr(am1), _ptr(xh), N,
                                                  _ptr(lat), _stream(stream)))


def xp_readout_argmax(head, lat, base, stride_n, stride_b, N, blk, win_val, ws, stream=None):
    _check("xp_readout_argmax", lib().xp_readout_argmax(
        head, _ptr(lat), _ptr(base), stride_n, stride_b, N, _ptr(blk), _ptr(win_val), _ptr(ws),
        _nbytes(ws), _stream(stream)))


def xp_readout_argmax_noalloc(head, lat, base, stride_n, stride_b, N, blk, win_val, stream=None):
    """xp_readout_argmax without a workspace, for callers that cannot allocate device memory."""
    _check("xp_readout_argmax_noalloc", lib().xp_readout_argmax_noalloc(
        head, _ptr(lat), _ptr(base), stride_n, stride_b, N, _ptr(blk), _ptr(win_val),
        _stream(stream)))


def xp_selftest_wait_timeout(head, stream=None):
    """Launch one wait that can only end by its time limit (sets XP_ETIMEOUT)."""
    _check("xp_selftest_wait_timeout", lib().xp_selftest_wait_timeout(head, _stream(stream)))


def xp_refine_logits(head, lat, base, stride_n, stride_b, N, out, ld_out, stream=None):
    """Draft rows' fp32 logits base + lat.w2 (the bias alone when base is None)."""
    _check("xp_refine_logits", lib().xp_refine_logits(
        head, _ptr(lat), _ptr(base), stride_n, stride_b, N, _ptr(out), ld_out, _stream(stream)))


def xp_init_argmax(head, base, stride_n, stride_b, anchor, N, blk, win_val, ws, stream=None):
    _check("xp_init_argmax", lib().xp_init_argmax(
        head, _ptr(base), stride_n, stride_b, _ptr(anchor), N, _ptr(blk), _ptr(win_val),
        _ptr(ws), _nbytes(ws), _stream(stream)))


def xp_topc_gather(head, base, stride_n, stride_b, N, C, cand, base_c, w2c, blk, stream=None):
    _check("xp_topc_gather", lib().xp_topc_gather(
        head, _ptr(base), stride_n, stride_b, N, C, _ptr(cand), _ptr(base_c), _ptr(w2c),
        _ptr(blk), _stream(stream)))


def xp_topc_readout_argmax(head, lat, base_c, cand, w2c, N, C, blk, win_val, stream=None):
    _check("xp_topc_readout_argmax", lib().xp_topc_readout_argmax(
        head, _ptr(lat), _ptr(base_c), _ptr(cand), _ptr(w2c), N, C, _ptr(blk), _ptr(win_val),
        _stream(stream)))


def xp_jacobi_refine(head, base, stride_n, stride_b, h_full, anchor, am1, N, K, topc, blk, ws,
                     stream=None):
    _check("xp_jacobi_refine", lib().xp_jacobi_refine(
        head, _ptr(base), stride_n, stride_b, _ptr(h_full), _ptr(anchor), _ptr(am1), N, K, topc,
        _ptr(blk), _ptr(ws), _nbytes(ws), _stream(stream)))


def xp_jacobi_passes(head, base, stride_n, stride_b, xh, am1, N, K, blk, ws, stream=None):
    """K passes on an initialised blk (refined in place), given the hidden cache xh."""
    _check("xp_jacobi_passes", lib().xp_jacobi_passes(
        head, _ptr(base), stride_n, stride_b, _ptr(xh), _ptr(am1), N, K, _ptr(blk), _ptr(ws),
        _nbytes(ws), _stream(stream)))


def xp_set_pass_mode(head, mode: int):
    _check("xp_set_pass_mode", lib().xp_set_pass_mode(head, mode))


def xp_passes_persistent(head, base, stride_n, stride_b, N) -> bool:
    return bool(lib().xp_passes_persistent(head, _ptr(base), stride_n, stride_b, N))


def xp_set_readout_pairs(head, on: bool):
    _check("xp_set_readout_pairs", lib().xp_set_readout_pairs(head, int(on)))


def xp_readout_pairs(head, N) -> bool:
    return bool(lib().xp_readout_pairs(head, N))


def xp_get_error(head, stream=None) -> int:
    """Synchronise the stream, read and clear the device error word; returns the status code."""
    return lib().xp_get_error(head, _stream(stream))


def xp_profile_timeline(head, buf, K: int) -> int:
    """Record the persistent refine's per-CTA phase stamps into buf (None: stop); returns
    the bytes K passes need."""
    needed = ctypes.c_size_t()
    _check("xp_profile_timeline", lib().xp_profile_timeline(head, _ptr(buf), _nbytes(buf), K,
                                                            ctypes.byref(needed)))
    return needed.value


def xp_readout_kernel_name(head) -> str:
    return lib().xp_readout_kernel_name(head).decode()


# ------------------------------------- verification, cache and attention calls ---
#
# These calls take their sizes and strides from the tensors; a tensor that the C call could
# not read as it is (not on the current device, another type, a strided last dimension, too few
# elements) is refused with ValueError (whose text is made only then: a call's checks are part of
# its latency).

def _want(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _here(names, *tensors):
    """All of them on the current device (None passes), which is returned."""
    if torch is None:
        _need_torch()
    device = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            name = next(n for n, x in zip(names.split(), tensors) if x is t)
            raise ValueError(f"{name}: not on the current CUDA device")
    return device


def _code(name, t):
    """The library's type code of a tensor's dtype."""
    if torch is None:
        _need_torch()
    dtype = t.dtype
    if dtype == torch.bfloat16:
        return XP_BF16
    if dtype != torch.float32:
        raise ValueError(f"{name}: bf16 or fp32")
    return XP_F32


def _ints(name, t, n):
    """A contiguous int32 vector of at least n elements on the GPU (None passes): its pointer."""
    if torch is None:
        _need_torch()
    if t is None:
        return None
    if t.dtype == torch.int32 and t.is_cuda and t.is_contiguous() and t.numel() >= n:
        return t.data_ptr()
    raise ValueError(f"{name}: a contiguous int32 CUDA tensor of at least {n} elements")


def _table(name, t, rows=None):
    """An int32 page table [rows, width], unit stride over the columns: its rows' stride."""
    return _columns(name, t, rows)[0]


def _columns(name, t, rows=None):
    """The same: its rows' stride and its columns."""
    if torch is None:
        _need_torch()
    shape = t.shape
    if t.dtype == torch.int32 and len(shape) == 2:
        (have, width), (ld, step) = shape, t.stride()
        if width > 0 and (step == 1 or width == 1) and (rows is None or have >= rows):
            return (ld if have > 1 else width), width
    raise ValueError(f"{name}: an int32 tensor [rows, width], unit stride over the columns")


def _flat(name, t, dtype, n):
    """A contiguous tensor of a type and at least n elements (None passes): its pointer."""
    if t is None:
        return None
    if not (t.dtype == dtype and t.is_contiguous() and t.numel() >= n):
        raise ValueError(f"{name}: contiguous {dtype} of at least {n} elements")
    return t.data_ptr()


def _rows(k, v):
    """K and V rows of the same strides: their sizes and strides."""
    shape, strides = k.shape, k.stride()
    _want(len(shape) == 4 and strides[3] == 1 and shape == v.shape and strides == v.stride() and k.dtype == v.dtype,
          "k, v: [N, T, kv_heads, head_dim] of the same strides")
    return *shape, *strides[:3]


def xp_verify_workspace_bytes(head, N: int) -> int:
    return lib().xp_verify_workspace_bytes(head, N)


def xp_verify_drafts(head, target, draft, blk, n_draft, temperature, u, noise, tokens, counts, prob,
                     ws, stream=None):
    """Accept drafted slots and draw one token a block.  target [N, B, V]; draft
    [N*(B-1), >= V] fp32 logits, or None for greedy (one-hot) drafts; blk [N, B]; u [N, B-1];
    noise [N, >= V]; out: tokens [N, B], counts [N], prob [N, B-1] (or None)."""
    import torch
    N, B, V = target.shape
    f32, i64, i32 = torch.float32, torch.int64, torch.int32
    device = _here("target draft blk n_draft temperature u noise tokens counts prob ws", target, draft, blk,
                   n_draft, temperature, u, noise, tokens, counts, prob, ws)
    sn, sb, sv = target.stride()
    _want(sv == 1, "target: [N, B, V] with unit stride over V")
    _want(draft is None or (draft.dtype == f32 and draft.dim() == 2 and draft.stride(1) == 1
                            and draft.shape[0] >= N * (B - 1) and draft.shape[1] >= V),
          "draft: fp32 [N*(B-1), >= V] with unit stride over V")
    _want(noise.dtype == f32 and noise.dim() == 2 and noise.stride(1) == 1 and noise.shape[0] >= N
          and noise.shape[1] >= V, "noise: fp32 [N, >= V] with unit stride over V")
    for name, t, dt, count in (("blk", blk, i64, N * B), ("n_draft", n_draft, i32, N),
                               ("temperature", temperature, f32, N), ("u", u, f32, N * (B - 1)),
                               ("tokens", tokens, i64, N * B), ("counts", counts, i32, N),
                               ("prob", prob, f32, N * (B - 1))):
        if t is not None and not (t.dtype == dt and t.is_contiguous() and t.numel() >= count):
            raise ValueError(f"{name}: contiguous {dt} of at least {count} elements")
    _check("xp_verify_drafts", lib().xp_verify_drafts(
        head, _ptr(target), sn, sb, _ptr(draft),
        draft.stride(0) if draft is not None else 0, _ptr(blk), _ptr(n_draft), N, B, V,
        _code("target", target), _ptr(temperature), _ptr(u), _ptr(noise), noise.stride(0) if N > 1 else noise.shape[1], _ptr(tokens),
        _ptr(counts), _ptr(prob), _ptr(ws), _nbytes(ws), _stream(stream, device)))


def xp_logprobs_workspace_bytes(head, rows: int, top: int) -> int:
    return lib().xp_logprobs_workspace_bytes(head, rows, top)


def xp_token_logprobs(head, logits, tokens, temperature, logprob, entropy, rank, top_ids, top_logprobs, ws,
                      stream=None):
    """Log probabilities of tokens [N, B] (-1: none) under logits [N, B, V] at temperature [N] (None: 1).
    Out, each may be None: logprob, entropy [N, B], rank [N, B] int32, top_ids int64 and top_logprobs
    [N, B, top], top up to 32."""
    device = _here("logits tokens temperature logprob entropy rank top_ids top_logprobs ws", logits, tokens,
                   temperature, logprob, entropy, rank, top_ids, top_logprobs, ws)
    N, B, V = logits.shape
    sn, sb, sv = logits.stride()
    _want(sv == 1, "logits: [N, B, V] with unit stride over V")
    top = 0
    some = top_ids if top_ids is not None else top_logprobs
    if some is not None:
        top = some.shape[-1]
        for t in (top_ids, top_logprobs):
            _want(t is None or t.shape == (N, B, top), "top_ids, top_logprobs: [N, B, top]")
    f32, i64 = torch.float32, torch.int64
    _check("xp_token_logprobs", lib().xp_token_logprobs(
        head, logits.data_ptr(), sn, sb, _flat("tokens", tokens, i64, N * B), N, B, V, _code("logits", logits),
        _flat("temperature", temperature, f32, N), top, _flat("logprob", logprob, f32, N * B),
        _flat("entropy", entropy, f32, N * B), _flat("rank", rank, torch.int32, N * B),
        _flat("top_ids", top_ids, i64, N * B * top), _flat("top_logprobs", top_logprobs, f32, N * B * top),
        _ptr(ws), _nbytes(ws), _stream(stream, device)))


def make_cache_desc(k, v, max_seqs: int = 4096) -> xp_cache_desc:
    """Descriptor of K and V pools seen as [layers, pages, page_size, kv_heads, head_dim] (views
    with the heads outside the tokens too)."""
    _here("k v", k, v)
    _want(k.dim() == 5 and k.shape == v.shape and k.stride() == v.stride() and k.dtype == v.dtype
          and k.stride(4) == 1,
          "k, v: bf16 or fp32 tensors [layers, pages, page_size, kv_heads, head_dim] of the "
          "same strides, unit stride over head_dim")
    layers, pages, ps, heads, dim = k.shape
    return xp_cache_desc(pages, ps, layers, heads, dim, max_seqs, _code("k", k), k.stride(0),
                         k.stride(1), k.stride(2), k.stride(3), _ptr(k), _ptr(v))


def xp_quant_head_bytes(page_size: int, head_dim: int, bits: int) -> int:
    """Bytes of one head of a page of a cache of 8 or 4 bits (0: sizes it cannot have)."""
    return lib().xp_quant_head_bytes(page_size, head_dim, _bits(bits))


def _bits(bits: int) -> int:
    _want(bits in (4, 8), "bits: 8 or 4")
    return XP_Q8 if bits == 8 else XP_Q4


def make_quant_cache_desc(k, v, page_size: int, head_dim: int, bits: int, max_seqs: int = 4096) -> xp_cache_desc:
    """Descriptor of K and V pools of 8 or 4 bits: uint8 [layers, pages, kv_heads, xp_quant_head_bytes]."""
    import torch
    _here("k v", k, v)
    size = xp_quant_head_bytes(page_size, head_dim, bits)
    _want(size > 0, "page_size: positive; head_dim: a multiple of 16 up to 256")
    _want(k.dim() == 4 and k.shape == v.shape and k.stride() == v.stride()
          and k.dtype == v.dtype == torch.uint8 and k.shape[3] == size and k.stride(3) == 1
          and (k.shape[2] == 1 or k.stride(2) == size),
          f"k, v: uint8 tensors [layers, pages, kv_heads, {size}] of the same strides, a page's heads dense")
    layers, pages, heads, _ = k.shape
    return xp_cache_desc(pages, page_size, layers, heads, head_dim, max_seqs, _bits(bits), k.stride(0),
                         k.stride(1), head_dim * bits // 8, size, _ptr(k), _ptr(v))


def xp_cache_prep_bytes(d: xp_cache_desc) -> int:
    return lib().xp_cache_prep_bytes(ctypes.byref(d))


def xp_cache_create(d: xp_cache_desc, prep, stream=None):
    out = ctypes.c_void_p()
    device = _here("prep", prep)
    _check("xp_cache_create", lib().xp_cache_create(ctypes.byref(d), _ptr(prep), _nbytes(prep),
                                                    _stream(stream, device), ctypes.byref(out)))
    return out.value


def xp_cache_destroy(cache):
    lib().xp_cache_destroy(cache)


def xp_cache_get_error(cache, stream=None) -> int:
    """Synchronise the stream, read and clear the cache's error word; returns the status code."""
    return lib().xp_cache_get_error(cache, _stream(stream))


def xp_cache_append(cache, layer, k, v, table, lens, stream=None):
    """Write the K and V rows [N, T, kv_heads, head_dim] of the newest tokens (lens counts them).
    Only the table's own columns are read, those of a wider tensor that it is a part of are not."""
    device = _here("k v table lens", k, v, table, lens)
    N, T, heads, dim, sn, st, sh = _rows(k, v)
    ld, width = _columns("table", table, N)
    _check("xp_cache_append", lib().xp_cache_append_columns(
        cache, layer, k.data_ptr(), v.data_ptr(), sn, st, sh, heads, dim, _code("k", k), table.data_ptr(), ld,
        width, _ints("lens", lens, N), N, T, _stream(stream, device)))


def xp_cache_read(cache, layer, table, lens, first, k, v, stream=None):
    """Read back T positions of every row into k, v [N, T, kv_heads, head_dim] (bf16 or fp32, whatever the
    cache's type), from position first[n] on (None: 0); zeros where a position is not in [0, lens[n])."""
    device = _here("table lens first k v", table, lens, first, k, v)
    N, T, heads, dim, sn, st, sh = _rows(k, v)
    ld, width = _columns("table", table, N)
    _check("xp_cache_read", lib().xp_cache_read(
        cache, layer, table.data_ptr(), ld, width, _ints("lens", lens, N), _ints("first", first, N), N, T, k.data_ptr(), v.data_ptr(),
        sn, st, sh, heads, dim, _code("k", k), _stream(stream, device)))


def xp_cache_copy(cache, src, dst, stream=None):
    """Copy whole pages src[i] -> dst[i] in every layer."""
    device = _here("src dst", src, dst)
    _ints("src", src, 0)
    _ints("dst", dst, src.numel())
    _check("xp_cache_copy", lib().xp_cache_copy(cache, _ptr(src), _ptr(dst), src.numel(),
                                                _stream(stream, device)))


def xp_cache_resize(cache, table, lens, new_lens, refs, table_out, lens_out, refs_out, stream=None):
    """Lengths lens -> new_lens: give back or take pages (outputs may be the inputs)."""
    N, width = table.shape
    device = _here("table lens new_lens refs table_out lens_out refs_out", table, lens, new_lens, refs, table_out,
                   lens_out, refs_out)
    ld, ld_out = _table("table", table), _table("table_out", table_out, N)
    _want(table_out.shape[1] >= width, "table_out: as wide as table")
    for name, t in (("lens", lens), ("new_lens", new_lens), ("lens_out", lens_out)):
        _ints(name, t, N)
    _ints("refs", refs, 1)
    _ints("refs_out", refs_out, refs.numel())
    _check("xp_cache_resize", lib().xp_cache_resize(
        cache, _ptr(table), ld, _ptr(lens), _ptr(new_lens), _ptr(refs), refs.numel(), N, width,
        _ptr(table_out), ld_out, _ptr(lens_out), _ptr(refs_out), _stream(stream, device)))


def xp_cache_fork(cache, table, lens, parent, cut, refs, child_table, child_lens, refs_out,
                  stream=None):
    """Children parent[i] continued at min(lens[parent[i]], cut[i]) (cut may be None)."""
    rows, width = table.shape
    M = parent.numel()
    device = _here("table lens parent cut refs child_table child_lens refs_out", table, lens, parent, cut, refs,
                   child_table, child_lens, refs_out)
    ld, ld_child = _table("table", table), _table("child_table", child_table, M)
    _want(child_table.shape[1] >= width, "child_table: as wide as table")
    for name, t, n in (("lens", lens, rows), ("parent", parent, M), ("cut", cut, M),
                       ("child_lens", child_lens, M), ("refs", refs, 1)):
        _ints(name, t, n)
    _ints("refs_out", refs_out, refs.numel())
    _check("xp_cache_fork", lib().xp_cache_fork(
        cache, _ptr(table), ld, _ptr(lens), rows, _ptr(parent), _ptr(cut), M, width, _ptr(refs),
        refs.numel(), _ptr(child_table), ld_child, _ptr(child_lens), _ptr(refs_out), _stream(stream, device)))


def xp_cache_compact(cache, table, lens, refs, table_out, refs_out, map=None, live=None,
                     stream=None):
    """Pack the pages in use to the pool's front; map[page] is each page's new id."""
    N, width = table.shape
    device = _here("table lens refs table_out refs_out map live", table, lens, refs, table_out, refs_out, map,
                   live)
    ld, ld_out = _table("table", table), _table("table_out", table_out, N)
    _want(table_out.shape[1] >= width, "table_out: as wide as table")
    _ints("lens", lens, N)
    _ints("refs", refs, 1)
    _ints("refs_out", refs_out, refs.numel())
    _ints("map", map, refs.numel())
    _ints("live", live, 1)
    _check("xp_cache_compact", lib().xp_cache_compact(
        cache, _ptr(table), ld, _ptr(lens), N, width, _ptr(refs), refs.numel(), _ptr(table_out),
        ld_out, _ptr(refs_out), _ptr(map), _ptr(live), _stream(stream, device)))


def make_attn(q, out, layer: int, prefix_len: int, max_len: int, scale: float) -> xp_attn:
    """Sizes and strides of one attention call: q, out [N, T, heads, head_dim]."""
    _want(q.dim() == 4 and q.shape == out.shape and q.dtype == out.dtype and q.stride(3) == 1
          and out.stride(3) == 1, "q, out: [N, T, heads, head_dim] of one type, unit stride last")
    N, T, heads, dim = q.shape
    a = xp_attn(layer, N, T, heads, dim, _code("q", q), prefix_len, max_len, scale, *q.stride()[:3], *out.stride()[:3])
    a.q_like = (q.shape, q.stride(), q.dtype)
    a.out_like = (out.shape, out.stride(), out.dtype)
    return a


def xp_attention_workspace_bytes(cache, attn: xp_attn) -> int:
    return lib().xp_attention_workspace_bytes(cache, ctypes.byref(attn))


def xp_prefix_attention(cache, attn, q, prefix_table, table, lens, out, lse, ws, stream=None):
    """Attention of attn.N sequences of attn.T new tokens over a shared prefix and their tails
    (attn from make_attn for tensors of these shapes and strides)."""
    _want((q.shape, q.stride(), q.dtype) == attn.q_like
          and (out.shape, out.stride(), out.dtype) == attn.out_like,
          "q, out: the shapes, strides and type that make_attn was given")
    device = _here("q prefix_table table lens out lse ws", q, prefix_table, table, lens, out, lse, ws)
    N, columns, ld, width = attn.N, None, 0, 0
    if table is not None:
        columns, (ld, width) = table.data_ptr(), _columns("table", table, N)
    _want(lse is None or (lse.is_contiguous() and lse.dtype == torch.float32
                          and lse.numel() >= N * attn.T * attn.heads),
          "lse: contiguous fp32 [N, T, heads]")
    _check("xp_prefix_attention", lib().xp_prefix_attention(
        cache, ctypes.byref(attn), q.data_ptr(), _ints("prefix_table", prefix_table, 0),
        0 if prefix_table is None else prefix_table.numel(), columns, ld, width, _ints("lens", lens, N),
        out.data_ptr(), None if lse is None else lse.data_ptr(), _ptr(ws), _nbytes(ws), _stream(stream, device)))


# ------------------------------------------------------ torch conveniences ---

def torch_dtype(dtype: str):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]


def to_device(a: np.ndarray, dtype: str, device="cuda"):
    """Storage array from the generator (bf16 as uint16 bits) -> device tensor, bit for bit."""
    import torch
    if a.dtype == np.uint16:
        t = torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16)
    else:
        t = torch.from_numpy(np.ascontiguousarray(a))
    return t.to(device)


def to_host_storage(t) -> np.ndarray:
    """Device tensor -> numpy storage form (bf16 as uint16 bits)."""
    import torch
    t = t.detach().cpu().contiguous()
    if t.dtype == torch.bfloat16:
        return t.view(torch.int16).numpy().view(np.uint16)
    return t.numpy()


class Head:
    """Owns a head's prepared device memory (a torch buffer) and its handle."""

    def __init__(self, shape: dict, weights: dict, dtype: str, max_N: int, stream=None):
        import torch
        self.dtype = dtype
        self.code = XP_BF16 if dtype == "bf16" else XP_F32
        self.shape = dict(shape, max_N=max_N)
        self.V, self.hidden, self.r, self.H, self.B = (shape[k] for k in ("V", "hidden", "r", "H", "B"))
        self.max_N = max_N
        w = make_weights(self.V, self.hidden, self.r, self.H, self.B, max_N, self.code, **weights)
        self.prep = torch.empty(xp_head_prep_bytes(w), dtype=torch.uint8, device="cuda")
        self.handle = xp_head_create(w, self.prep, stream)

    def weights_struct(self, **weights) -> xp_weights:
        return make_weights(self.V, self.hidden, self.r, self.H, self.B, self.max_N, self.code,
                            **weights)

    def workspace(self, N: int, topc: int = 0):
        import torch
        w = self.weights_struct()
        return torch.zeros(xp_workspace_bytes(w, N, topc), dtype=torch.uint8, device="cuda")

    def logprobs_workspace(self, rows: int, top: int):
        import torch
        return torch.zeros(xp_logprobs_workspace_bytes(self.handle, rows, top), dtype=torch.uint8,
                           device="cuda")

    def verify_workspace(self, N: int):
        import torch
        return torch.zeros(xp_verify_workspace_bytes(self.handle, N), dtype=torch.uint8,
                           device="cuda")

    def close(self):
        if self.handle:
            xp_head_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Cache:
    """A paged cache over the caller's K and V pools, seen as [layers, pages, page_size, kv_heads,
    head_dim] (kept alive here), with its prepared scratch and handle."""

    def __init__(self, k, v, max_seqs: int = 4096, stream=None):
        self.handle = None
        self._create(k, v, make_cache_desc(k, v, max_seqs), stream)

    def _create(self, k, v, desc, stream):
        import torch
        self.k, self.v = k, v
        self.prep = torch.empty(max(256, xp_cache_prep_bytes(desc)), dtype=torch.uint8,
                                device=k.device)
        self.handle = xp_cache_create(desc, self.prep, stream)

    def attention_workspace(self, attn: xp_attn):
        import torch
        return torch.empty(xp_attention_workspace_bytes(self.handle, attn), dtype=torch.uint8,
                           device=self.k.device)

    def close(self):
        if self.handle:
            xp_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class QuantCache(Cache):
    """A paged cache held in 8 or 4 bits over the caller's K and V pools, uint8 [layers, pages, kv_heads,
    xp_quant_head_bytes] (`pool` makes one).  Every call on caches takes it."""

    def __init__(self, k, v, page_size: int, head_dim: int, bits: int, max_seqs: int = 4096, stream=None):
        self.handle = None
        self._create(k, v, make_quant_cache_desc(k, v, page_size, head_dim, bits, max_seqs), stream)

    @staticmethod
    def pool(layers: int, pages: int, page_size: int, kv_heads: int, head_dim: int, bits: int):
        import torch
        size = xp_quant_head_bytes(page_size, head_dim, bits)
        _want(size > 0, "page_size: positive; head_dim: a multiple of 16 up to 256")
        return torch.empty(layers, pages, kv_heads, size, dtype=torch.uint8, device="cuda")


def head_from_inputs(inp: dict, wl, max_N: int | None = None, stream=None):
    """Device head from generator output: raw mixer folded on the GPU by xp_fold_mix.

    Returns (Head, dict of the device weight tensors used).
    """
    import torch
    d = wl.dtype
    t = {k: to_device(inp[k], d) for k in ("w1", "down_h", "down_g", "in_proj", "raw_mix",
                                            "w_gate", "w_up", "w_down", "w2")}
    code = XP_BF16 if d == "bf16" else XP_F32
    mix = torch.empty_like(t["raw_mix"])
    xp_fold_mix(t["raw_mix"], mix, wl.r, wl.B, code, stream)
    t["mix_L"] = mix
    shape = dict(V=wl.V, hidden=wl.hidden, r=wl.r, H=wl.H, B=wl.B)
    weights = {k: t[k] for k in ("w1", "down_h", "down_g", "in_proj", "mix_L", "w_gate", "w_up",
                                 "w_down", "w2")}
    head = Head(shape, weights, d, max_N or wl.N, stream)
    return head, t

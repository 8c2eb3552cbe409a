"""Thin ctypes binding over ``libbgattn.so`` (the C ABI in include/bg_attn.h).

Argument marshalling only: every function passes device pointers, sizes and
the current CUDA stream straight to the library; all of the work runs in the
library's CUDA kernels.  There is no CPU fallback: if the library is missing
or fails to load, every call raises.

The functions carry the C names.  Tensor arguments are torch CUDA tensors
(torch is used for device memory and streams only); ``raw`` exposes the
ctypes functions themselves for callers that manage pointers directly.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Optional

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbgattn.so")

BG_OK, BG_ERR_INVALID_ARG, BG_ERR_UNSUPPORTED, BG_ERR_DEVICE_DATA, BG_ERR_CUDA = 0, 1, 2, 3, 4
BG_DEVSTAT_CU_SEQLENS = 0x01
BG_DEVSTAT_SEQ_TOO_LONG = 0x02
BG_DEVSTAT_PARENT = 0x04
BG_DEVSTAT_CU_PROMPT = 0x08
BG_DEVSTAT_EMPTY_ROW = 0x10
BG_DEVSTAT_PLAN = 0x20
BG_DEVSTAT_GROUP = 0x40
BG_DEVSTAT_TOKEN = 0x80
BG_DEVSTAT_TIMEOUT = 0x100
BG_DEVSTAT_BIAS = 0x200
BG_DEVSTAT_MASK = 0x400
BG_DEVSTAT_PENALTY = 0x800
BG_MAX_SUFFIX = 16
BG_MAX_SEQLEN = 65536
BG_NOALLOC_SCRATCH_BYTES = 1 << 20
BG_MAX_BEAM = 512
BG_MAX_VOCAB = 1 << 22
BG_MAX_TOP = 32
BG_DTYPE_F32, BG_DTYPE_BF16 = 0, 1
BG_MAX_AXES = 4
BG_MAX_HEADS = 65536
BG_MAX_BIAS = 8191
BG_MAX_TREE = 1024

# Every symbol include/bg_attn.h declares, with its ctypes signature.
_P, _I32, _F32, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
_SHARED_PLAN = [_P, _I32, _I32, _I32, _P, _I32, _I32, _P, _I32, _I32, _I32, _I32, _P, _SZ, _P, _P]
_SHARED_RUN = [_P, _P, _P, _P, _I32, _I32, _I32, _P, _P, _P, _I32, _I32, _P, _I32, _I32, _I32, _I32, _F32, _F32, _P, _P,
               _P, _SZ, _P, _P]
_I64 = ctypes.c_int64
_TREE_RUN = [_P, _P, _P, _P, _P, _I32, _I32, _I32, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _F32, _F32, _P, _P, _P, _SZ, _P,
             _P]
SIGNATURES = {
    "bg_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "bg_packed_prefill_workspace_size": ([_I32] * 6, _SZ),
    "bg_packed_prefill_attn": ([_P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _F32, _P, _P, _P, _SZ, _P, _P],
                               ctypes.c_int),
    "bg_packed_prefill_plan": ([_P, _I32, _I32, _I32, _P, _SZ, _P, _P], ctypes.c_int),
    "bg_packed_prefill_attn_planned": ([_P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _F32, _P, _P, _P, _SZ, _P,
                                        _P], ctypes.c_int),
    "bg_packed_prefill_attn_fp8": ([_P, _F32, _P, _F32, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _F32, _P, _P, _P,
                                    _SZ, _P, _P], ctypes.c_int),
    "bg_packed_prefill_attn_noalloc": ([_P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _F32, _P, _P, _P, _P],
                                       ctypes.c_int),
    "bg_packed_last_token_attn": ([_P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _F32, _P, _P, _P, _P],
                                  ctypes.c_int),
    "bg_beam_decode_attn": ([_P, _P, _P, _P, _I32, _I32, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _F32, _P,
                             _P, _P], ctypes.c_int),
    "bg_beam_suffix_reorder": ([_P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _P, _P],
                               ctypes.c_int),
    "bg_beam_decode_step": ([_P, _P, _P, _P, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _I32, _I32, _I32, _I32, _I32,
                             _I32, _I32, _F32, _P, _P, _P], ctypes.c_int),
    "bg_beam_select_workspace_size": ([_I32] * 3, _SZ),
    "bg_shared_attn_workspace_size": ([_I32] * 8, _SZ),
    "bg_shared_prefill_plan": (_SHARED_PLAN, ctypes.c_int),
    "bg_shared_last_token_plan": (_SHARED_PLAN, ctypes.c_int),
    "bg_shared_prefill_attn": (_SHARED_RUN, ctypes.c_int),
    "bg_shared_prefill_attn_planned": (_SHARED_RUN, ctypes.c_int),
    "bg_shared_last_token_attn": (_SHARED_RUN, ctypes.c_int),
    "bg_shared_last_token_attn_planned": (_SHARED_RUN, ctypes.c_int),
    "bg_tree_attn_workspace_size": ([_I32] * 7, _SZ),
    "bg_tree_plan": ([_P, _P, _I32, _I32, _I32, _P, _I32, _I32, _I32, _I32, _I32, _P, _SZ, _P, _P], ctypes.c_int),
    "bg_tree_attn": (_TREE_RUN, ctypes.c_int),
    "bg_tree_attn_planned": (_TREE_RUN, ctypes.c_int),
    "bg_packed_qk_norm_rope": ([_P, _I64, _P, _I64, _P, _I64, _I32, _I32, _I32, _I32, _P, _P, _F32, _F32, _P, _I32, _P, _P,
                                _I32, _I32, _F32, _P, _P, _P, _P], ctypes.c_int),
    "bg_beam_qk_norm_rope": ([_P, _I64, _P, _I64, _P, _I64, _I32, _I32, _I32, _I32, _I32, _P, _P, _F32, _F32, _P, _I32, _P,
                              _I32, _P, _I32, _I32, _F32, _P, _P, _P, _I32, _I32, _P], ctypes.c_int),
    "bg_adjust_logits": ([_P, _I32, _I64, _I32, _I32, _I32, _P, _P, _I32, _P, _P, _I32, _P, _P, _P, _P, _P, _P, _I32, _P,
                          _I64, _I32, _P, _P, _I32, _I64, _P, _P], ctypes.c_int),
    "bg_token_logprobs": ([_P, _I32, ctypes.c_int64, _I32, _I32, _P, _I32, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "bg_selftest_wait_timeout": ([_P, _P, _P], ctypes.c_int),
    "bg_selftest_logprobs_timeout": ([_P, _I32, _I32, _P, _I32, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "bg_beam_select": ([_P, _P, _I32, _I32, _I32, _P, _P, _P, _P, _SZ, _P], ctypes.c_int),
}


class BgError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")


_lib = None


def load(path: Optional[str] = None):
    """Load the library (once).  Raises if it is not built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with attention_packed_varlen_causal_gb300.build.build() "
                           "(there is no fallback implementation)")
    lib = ctypes.CDLL(p)
    for name, (args, res) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    if path is None:
        _lib = lib
    return lib


class _Raw:
    def __getattr__(self, name):
        return getattr(load(), name)


raw = _Raw()


def status_string(status: int) -> str:
    return load().bg_status_string(int(status)).decode()


def _ptr(t) -> Optional[int]:
    return None if t is None else int(t.data_ptr())


def _stream(stream) -> Optional[int]:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _check(fn: str, status: int):
    if status != BG_OK:
        raise BgError(fn, status)


def bg_packed_prefill_workspace_size(num_seqs: int, total_tokens: int, max_seqlen: int, Hq: int, Hkv: int,
                                     head_dim: int) -> int:
    return int(load().bg_packed_prefill_workspace_size(num_seqs, total_tokens, max_seqlen, Hq, Hkv, head_dim))


def bg_packed_prefill_attn(q, k, v, cu_seqlens, max_seqlen: int, out, *, lse=None, scale: Optional[float] = None,
                           workspace=None, dev_status=None, stream=None):
    """q [T,Hq,d], k/v [T,Hkv,d] bf16 CUDA tensors; cu_seqlens int32 [B+1] CUDA;
    out bf16 [T,Hq,d] (written); lse fp32 [T,Hq] or None; workspace a uint8
    CUDA tensor of at least bg_packed_prefill_workspace_size bytes."""
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    B = cu_seqlens.numel() - 1
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    need = bg_packed_prefill_workspace_size(B, T, max_seqlen, Hq, Hkv, d)
    if workspace is None:
        raise ValueError(f"workspace of {need} bytes required (the library never allocates)")
    st = load().bg_packed_prefill_attn(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), B, T, int(max_seqlen), Hq, Hkv, d,
                                       float(scale), _ptr(out), _ptr(lse), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _ptr(dev_status),
                                       _stream(stream))
    _check("bg_packed_prefill_attn", st)
    return out


def bg_packed_prefill_plan(cu_seqlens, total_tokens: int, max_seqlen: int, *, workspace=None, dev_status=None,
                           stream=None):
    """The work list of a packing (cu_seqlens int32 [B+1] CUDA) into workspace, for
    bg_packed_prefill_attn_planned calls with the same packing."""
    B = cu_seqlens.numel() - 1
    if workspace is None:
        raise ValueError("workspace required (the library never allocates)")
    st = load().bg_packed_prefill_plan(_ptr(cu_seqlens), B, int(total_tokens), int(max_seqlen), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(), _ptr(dev_status),
                                       _stream(stream))
    _check("bg_packed_prefill_plan", st)


def bg_packed_prefill_attn_planned(q, k, v, cu_seqlens, max_seqlen: int, out, *, lse=None,
                                   scale: Optional[float] = None, workspace=None, dev_status=None, stream=None):
    """bg_packed_prefill_attn with the work list a bg_packed_prefill_plan call left in
    workspace (same cu_seqlens, max_seqlen and total tokens)."""
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    B = cu_seqlens.numel() - 1
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if workspace is None:
        raise ValueError("workspace required (the library never allocates)")
    st = load().bg_packed_prefill_attn_planned(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), B, T, int(max_seqlen), Hq,
                                               Hkv, d, float(scale), _ptr(out), _ptr(lse), _ptr(workspace),
                                               workspace.numel() * workspace.element_size(), _ptr(dev_status),
                                               _stream(stream))
    _check("bg_packed_prefill_attn_planned", st)
    return out


def bg_packed_prefill_attn_fp8(q_codes, q_scale: float, k_codes, k_scale: float, v, cu_seqlens, max_seqlen: int, out,
                               *, lse=None, scale: Optional[float] = None, workspace=None, dev_status=None,
                               stream=None):
    """q_codes uint8 [T,Hq,d] and k_codes uint8 [T,Hkv,d] E4M3 codes (torch.uint8 or
    torch.float8_e4m3fn CUDA tensors) with their per-tensor scales; v bf16 [T,Hkv,d];
    cu_seqlens int32 [B+1]; out bf16 [T,Hq,d] (written); lse fp32 [T,Hq] or None; workspace
    as for bg_packed_prefill_attn.  ``scale`` is the softmax scale of the dequantised
    values (default 1/sqrt(d))."""
    T, Hq, d = q_codes.shape
    Hkv = k_codes.shape[1]
    B = cu_seqlens.numel() - 1
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    need = bg_packed_prefill_workspace_size(B, T, max_seqlen, Hq, Hkv, d)
    if workspace is None:
        raise ValueError(f"workspace of {need} bytes required (the library never allocates)")
    st = load().bg_packed_prefill_attn_fp8(_ptr(q_codes), float(q_scale), _ptr(k_codes), float(k_scale), _ptr(v),
                                           _ptr(cu_seqlens), B, T, int(max_seqlen), Hq, Hkv, d, float(scale), _ptr(out),
                                           _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                           _ptr(dev_status), _stream(stream))
    _check("bg_packed_prefill_attn_fp8", st)
    return out


def bg_packed_prefill_attn_noalloc(q, k, v, cu_seqlens, max_seqlen: int, out, *, lse=None,
                                   scale: Optional[float] = None, dev_status=None, stream=None):
    """As bg_packed_prefill_attn, for callers that cannot allocate: the work
    list lives in the library's own fixed device array (no workspace
    argument).  Calls on one device share that array, so calls that can
    overlap on the GPU must be serialised; the first call on a device should
    precede any stream capture."""
    T, Hq, d = q.shape
    Hkv = k.shape[1]
    B = cu_seqlens.numel() - 1
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    st = load().bg_packed_prefill_attn_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), B, T, int(max_seqlen), Hq,
                                               Hkv, d, float(scale), _ptr(out), _ptr(lse), _ptr(dev_status),
                                               _stream(stream))
    _check("bg_packed_prefill_attn_noalloc", st)
    return out


def bg_packed_last_token_attn(q, k, v, cu_seqlens, max_seqlen: int, out, *, lse=None,
                              scale: Optional[float] = None, dev_status=None, stream=None):
    """q [B,Hq,d] (each sequence's last valid row); k, v [T,Hkv,d]; cu_seqlens
    int32 [B+1]; out [B,Hq,d] (written); lse fp32 [B,Hq] or None."""
    B, Hq, d = q.shape
    T, Hkv = k.shape[0], k.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    st = load().bg_packed_last_token_attn(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), B, T, int(max_seqlen), Hq,
                                          Hkv, d, float(scale), _ptr(out), _ptr(lse), _ptr(dev_status),
                                          _stream(stream))
    _check("bg_packed_last_token_attn", st)
    return out


def bg_beam_decode_attn(q, prompt_k, prompt_v, cu_prompt, max_prompt_len: int, suffix_k, suffix_v, suffix_len: int,
                        out, *, scale: Optional[float] = None, dev_status=None, stream=None):
    """q [R,W,Hq,d]; prompt_k/v [sumP,Hkv,d]; cu_prompt int32 [R+1];
    suffix_k/v [R,W,S_max,Hkv,d]; out [R,W,Hq,d] (written)."""
    R, W, Hq, d = q.shape
    Hkv = prompt_k.shape[1]
    S_max = suffix_k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    st = load().bg_beam_decode_attn(_ptr(q), _ptr(prompt_k), _ptr(prompt_v), _ptr(cu_prompt), prompt_k.shape[0],
                                    int(max_prompt_len), _ptr(suffix_k), _ptr(suffix_v), int(suffix_len), S_max, R, W,
                                    Hq, Hkv, d, float(scale), _ptr(out), _ptr(dev_status), _stream(stream))
    _check("bg_beam_decode_attn", st)
    return out


def bg_beam_suffix_reorder(src_k, src_v, dst_k, dst_v, parent_idx, n_tokens: int, *, new_k=None, new_v=None,
                           dev_status=None, stream=None):
    """src/dst [R,W,S_max,Hkv,d] bf16; parent_idx int32 [R,W]; new_k/new_v
    [R,W,Hkv,d] or None.  dst[r,b,:n] = src[r,parent[r,b],:n], dst[r,b,n] = new[r,b]."""
    R, W, S_max, Hkv, d = src_k.shape
    st = load().bg_beam_suffix_reorder(_ptr(src_k), _ptr(src_v), _ptr(dst_k), _ptr(dst_v), _ptr(parent_idx),
                                       _ptr(new_k), _ptr(new_v), R, W, S_max, int(n_tokens), Hkv, d,
                                       _ptr(dev_status), _stream(stream))
    _check("bg_beam_suffix_reorder", st)
    return dst_k, dst_v


def bg_beam_decode_step(q, prompt_k, prompt_v, cu_prompt, max_prompt_len: int, src_suffix_k, src_suffix_v,
                        parent_idx, new_k, new_v, dst_suffix_k, dst_suffix_v, suffix_len: int, out, *,
                        scale: Optional[float] = None, dev_status=None, stream=None):
    """One decode step in one call: dst[r,b,:t-1] = src[r,parent[r,b],:t-1], dst[r,b,t-1] = new[r,b],
    then out = decode attention over [prompt ; dst[:, :, :t]] (t = suffix_len >= 1).
    src/dst [R,W,S_max,Hkv,d] bf16 (src may be None when t == 1); parent_idx int32 [R,W];
    new_k/new_v [R,W,Hkv,d]; out [R,W,Hq,d] (written)."""
    R, W, Hq, d = q.shape
    Hkv = prompt_k.shape[1]
    S_max = dst_suffix_k.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    st = load().bg_beam_decode_step(_ptr(q), _ptr(prompt_k), _ptr(prompt_v), _ptr(cu_prompt), prompt_k.shape[0],
                                    int(max_prompt_len), _ptr(src_suffix_k), _ptr(src_suffix_v), _ptr(parent_idx),
                                    _ptr(new_k), _ptr(new_v), _ptr(dst_suffix_k), _ptr(dst_suffix_v),
                                    int(suffix_len), S_max, R, W, Hq, Hkv, d, float(scale), _ptr(out),
                                    _ptr(dev_status), _stream(stream))
    _check("bg_beam_decode_step", st)
    return out


def bg_selftest_wait_timeout(dev_status, waited_ns, *, stream=None):
    """Makes one bounded pipeline wait run out on the device: dev_status (int32) receives
    BG_DEVSTAT_TIMEOUT, waited_ns (int64) the nanoseconds waited."""
    st = load().bg_selftest_wait_timeout(_ptr(dev_status), _ptr(waited_ns), _stream(stream))
    _check("bg_selftest_wait_timeout", st)


def bg_beam_select_workspace_size(R: int, W: int, V: int) -> int:
    return int(load().bg_beam_select_workspace_size(R, W, V))


def bg_beam_select(logits, cum, token_out, parent_out, score_out, *, workspace=None, stream=None):
    """logits fp32 [R,W,V]; cum fp32 [R,W]; token_out/parent_out int32 [R,W] and
    score_out fp32 [R,W] (written); workspace a uint8 CUDA tensor of at least
    bg_beam_select_workspace_size bytes."""
    R, W, V = logits.shape
    need = bg_beam_select_workspace_size(R, W, V)
    if workspace is None:
        raise ValueError(f"workspace of {need} bytes required (the library never allocates)")
    st = load().bg_beam_select(_ptr(logits), _ptr(cum), R, W, V, _ptr(token_out), _ptr(parent_out), _ptr(score_out),
                               _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check("bg_beam_select", st)
    return token_out, parent_out, score_out


def _expect(fn: str, device, checks):
    """Each of ``checks`` is (name, tensor or None, dtype, shape): contiguous, on ``device``."""
    for name, t, dtype, shape in checks:
        if t is not None and not (t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous()):
            raise ValueError(f"{fn}: {name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, "
                             f"got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _alike(dtype, index: int, tensors) -> bool:
    """Whether all of ``tensors`` (or None) are contiguous, of ``dtype`` and on device ``index``.  The checks of
    the shared-prefix and log-probability calls begin with it, as it takes a third of ``_expect``'s time
    (their smallest problems run for 7 to 20 us); ``_expect`` finds the message if one fails."""
    for t in tensors:
        if t is not None and (t.dtype is not dtype or t.get_device() != index or not t.is_contiguous()):
            return False
    return True


def _fits(*sizes) -> bool:
    """Whether all sizes are int32; ctypes would pass the low 32 bits of larger ones."""
    for n in sizes:
        if not -0x80000000 <= n <= 0x7fffffff:
            return False
    return True


def _raw_stream(index: int) -> int:
    """The current stream of device ``index``: torch's own shortcut, which makes no object, where there is one."""
    import torch
    short = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return short(index) if short is not None else torch.cuda.current_stream(index).cuda_stream


def _launch(fn: str, index: int, stream, *args):
    """Calls the library's ``fn`` with device ``index`` current, on ``stream`` or that device's current one."""
    import torch
    if index < 0:
        raise ValueError(f"{fn}: CUDA tensors expected")
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            return _launch(fn, index, stream, *args)
    st = _raw_stream(index) if stream is None else stream.cuda_stream
    _check(fn, getattr(load(), fn)(*args, st))


def bg_shared_attn_workspace_size(num_groups: int, num_seqs: int, total_tokens: int, max_seqlen: int,
                                  max_prefix_len: int, Hq: int, Hkv: int, head_dim: int) -> int:
    if not _fits(num_groups, num_seqs, total_tokens, max_seqlen, max_prefix_len, Hq, Hkv, head_dim):
        return 0
    return int(load().bg_shared_attn_workspace_size(num_groups, num_seqs, total_tokens, max_seqlen, max_prefix_len, Hq,
                                                    Hkv, head_dim))


def _workspace(fn: str, workspace, sizes, index: int):
    """Pointer and bytes of the workspace; ``sizes`` are bg_shared_attn_workspace_size's arguments, for the message."""
    if workspace is None:
        raise ValueError(f"{fn}: workspace of {bg_shared_attn_workspace_size(*sizes)} bytes required (the library never "
                         "allocates)")
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"{fn}: workspace must be contiguous on the other tensors' device, got {workspace.device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _shared_run(fn: str, last: bool, q, k, v, cu_seqlens, max_seqlen, prefix_k, prefix_v, cu_prefix, max_prefix_len,
                cu_group, out, lse, scale, softcap, workspace, dev_status, stream):
    import torch
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    rows, Hq, d = q.shape
    kv = k.shape
    T, Hkv = kv[0], kv[1]
    S, R = cu_seqlens.numel() - 1, cu_group.numel() - 1
    if (prefix_k is None) != (prefix_v is None):
        raise ValueError(f"{fn}: prefix_k and prefix_v come together")
    P = 0 if prefix_k is None else prefix_k.shape[0]
    index = q.get_device()
    if not (_alike(bf16, index, (q, k, v, prefix_k, prefix_v, out)) and
            _alike(i32, index, (cu_seqlens, cu_prefix, cu_group, dev_status)) and
            (lse is None or (_alike(f32, index, (lse,)) and lse.shape == (rows, Hq))) and
            rows == (S if last else T) and out.shape == q.shape and kv == (T, Hkv, d) and v.shape == kv and
            (prefix_k is None or prefix_k.shape == prefix_v.shape == (P, Hkv, d)) and
            cu_seqlens.dim() == cu_prefix.dim() == cu_group.dim() == 1 and cu_prefix.numel() == R + 1):
        _expect(fn, q.device, (
            ("q", q, bf16, (S if last else T, Hq, d)), ("k", k, bf16, (T, Hkv, d)), ("v", v, bf16, (T, Hkv, d)),
            ("cu_seqlens", cu_seqlens, i32, (S + 1,)), ("prefix_k", prefix_k, bf16, (P, Hkv, d)),
            ("prefix_v", prefix_v, bf16, (P, Hkv, d)), ("cu_prefix", cu_prefix, i32, (R + 1,)),
            ("cu_group", cu_group, i32, (R + 1,)), ("out", out, bf16, (rows, Hq, d)), ("lse", lse, f32, (rows, Hq)),
            ("dev_status", dev_status, i32, dev_status.shape if dev_status is not None else ())))
    max_seqlen, max_prefix_len = int(max_seqlen), int(max_prefix_len)
    if not _fits(S, T, P, max_seqlen, max_prefix_len):
        raise BgError(fn, BG_ERR_UNSUPPORTED)
    ws, ws_bytes = _workspace(fn, workspace, (R, S, T, max_seqlen, max_prefix_len, Hq, Hkv, d), index)
    _launch(fn, index, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_seqlens.data_ptr(), S, T, max_seqlen,
            _ptr(prefix_k), _ptr(prefix_v), cu_prefix.data_ptr(), P, max_prefix_len, cu_group.data_ptr(), R, Hq, Hkv, d,
            1.0 / math.sqrt(d) if scale is None else float(scale), float(softcap), out.data_ptr(), _ptr(lse), ws,
            ws_bytes, _ptr(dev_status))
    return out


def bg_shared_prefill_attn(q, k, v, cu_seqlens, max_seqlen: int, prefix_k, prefix_v, cu_prefix, max_prefix_len: int,
                           cu_group, out, *, lse=None, scale: Optional[float] = None, softcap: float = 0.0,
                           workspace=None, dev_status=None, stream=None):
    """Causal attention of the samples' tokens over their request's prefix and their own sample.
    q [T,Hq,d], k/v [T,Hkv,d] bf16, packed by cu_seqlens int32 [S+1]; prefix_k/prefix_v [P,Hkv,d] (or
    None) packed by cu_prefix int32 [R+1]; samples cu_group[r] .. cu_group[r+1]-1 belong to request r
    (int32 [R+1]); out [T,Hq,d] (written); lse fp32 [T,Hq] or None; scores capped by softcap * tanh(x /
    softcap) if softcap > 0 (then the prefixes' own rows too come from this call, each prefix as the one
    sample of a request without one: bg_packed_prefill_attn does not cap); workspace a uint8 CUDA tensor of bg_shared_attn_workspace_size bytes."""
    return _shared_run("bg_shared_prefill_attn", False, q, k, v, cu_seqlens, max_seqlen, prefix_k, prefix_v, cu_prefix,
                       max_prefix_len, cu_group, out, lse, scale, softcap, workspace, dev_status, stream)


def bg_shared_last_token_attn(q, k, v, cu_seqlens, max_seqlen: int, prefix_k, prefix_v, cu_prefix, max_prefix_len: int,
                              cu_group, out, *, lse=None, scale: Optional[float] = None, softcap: float = 0.0,
                              workspace=None, dev_status=None, stream=None):
    """As bg_shared_prefill_attn with one query per sample, over the prefix and the whole sample:
    q and out [S,Hq,d], lse fp32 [S,Hq] or None."""
    return _shared_run("bg_shared_last_token_attn", True, q, k, v, cu_seqlens, max_seqlen, prefix_k, prefix_v,
                       cu_prefix, max_prefix_len, cu_group, out, lse, scale, softcap, workspace, dev_status, stream)


def bg_shared_prefill_attn_planned(q, k, v, cu_seqlens, max_seqlen: int, prefix_k, prefix_v, cu_prefix,
                                   max_prefix_len: int, cu_group, out, *, lse=None, scale: Optional[float] = None,
                                   softcap: float = 0.0, workspace=None, dev_status=None, stream=None):
    """bg_shared_prefill_attn with the work list that bg_shared_prefill_plan left in workspace."""
    return _shared_run("bg_shared_prefill_attn_planned", False, q, k, v, cu_seqlens, max_seqlen, prefix_k, prefix_v,
                       cu_prefix, max_prefix_len, cu_group, out, lse, scale, softcap, workspace, dev_status, stream)


def bg_shared_last_token_attn_planned(q, k, v, cu_seqlens, max_seqlen: int, prefix_k, prefix_v, cu_prefix,
                                      max_prefix_len: int, cu_group, out, *, lse=None, scale: Optional[float] = None,
                                      softcap: float = 0.0, workspace=None, dev_status=None, stream=None):
    """bg_shared_last_token_attn with the work list that bg_shared_last_token_plan left in workspace."""
    return _shared_run("bg_shared_last_token_attn_planned", True, q, k, v, cu_seqlens, max_seqlen, prefix_k, prefix_v,
                       cu_prefix, max_prefix_len, cu_group, out, lse, scale, softcap, workspace, dev_status, stream)


def _shared_plan(fn: str, cu_seqlens, total_tokens, max_seqlen, cu_prefix, total_prefix, max_prefix_len, cu_group, Hq,
                 Hkv, head_dim, workspace, dev_status, stream):
    import torch
    i32 = torch.int32
    S, R = cu_seqlens.numel() - 1, cu_group.numel() - 1
    index = cu_seqlens.get_device()
    _expect(fn, cu_seqlens.device, (
        ("cu_seqlens", cu_seqlens, i32, (S + 1,)), ("cu_prefix", cu_prefix, i32, (R + 1,)),
        ("cu_group", cu_group, i32, (R + 1,)),
        ("dev_status", dev_status, i32, dev_status.shape if dev_status is not None else ())))
    T, P, max_seqlen, max_prefix_len = int(total_tokens), int(total_prefix), int(max_seqlen), int(max_prefix_len)
    if not _fits(S, T, P, max_seqlen, max_prefix_len, Hq, Hkv, head_dim):
        raise BgError(fn, BG_ERR_UNSUPPORTED)
    ws, ws_bytes = _workspace(fn, workspace, (R, S, T, max_seqlen, max_prefix_len, Hq, Hkv, head_dim), index)
    _launch(fn, index, stream, cu_seqlens.data_ptr(), S, T, max_seqlen, cu_prefix.data_ptr(), P, max_prefix_len,
            cu_group.data_ptr(), R, Hq, Hkv, head_dim, ws, ws_bytes, _ptr(dev_status))


def bg_shared_prefill_plan(cu_seqlens, total_tokens: int, max_seqlen: int, cu_prefix, total_prefix: int,
                           max_prefix_len: int, cu_group, Hq: int, Hkv: int, head_dim: int, *, workspace=None,
                           dev_status=None, stream=None):
    """The work list of a packing into workspace, for bg_shared_prefill_attn_planned calls with it."""
    _shared_plan("bg_shared_prefill_plan", cu_seqlens, total_tokens, max_seqlen, cu_prefix, total_prefix,
                 max_prefix_len, cu_group, Hq, Hkv, head_dim, workspace, dev_status, stream)


def bg_shared_last_token_plan(cu_seqlens, total_tokens: int, max_seqlen: int, cu_prefix, total_prefix: int,
                              max_prefix_len: int, cu_group, Hq: int, Hkv: int, head_dim: int, *, workspace=None,
                              dev_status=None, stream=None):
    """The work list of a packing into workspace, for bg_shared_last_token_attn_planned calls with it."""
    _shared_plan("bg_shared_last_token_plan", cu_seqlens, total_tokens, max_seqlen, cu_prefix, total_prefix,
                 max_prefix_len, cu_group, Hq, Hkv, head_dim, workspace, dev_status, stream)


def bg_token_logprobs(logits, tokens=None, *, logprob=None, entropy=None, top_token=None, top_logprob=None,
                      dev_status=None, stream=None):
    """logits fp32 or bf16 [N,V] (rows may be strided, columns not); tokens int32 [N] or None;
    written: logprob fp32 [N] (with tokens), entropy fp32 [N] or None, top_token int32 [N,K] and
    top_logprob fp32 [N,K] or both None."""
    import torch
    fn = "bg_token_logprobs"
    N, V = logits.shape
    dtype = {torch.float32: BG_DTYPE_F32, torch.bfloat16: BG_DTYPE_BF16}.get(logits.dtype)
    if dtype is None or (V > 1 and N > 0 and logits.stride(1) != 1):
        raise ValueError(f"{fn}: logits must be float32 or bfloat16 with contiguous rows, got {logits.dtype} with "
                         f"strides {logits.stride()}")
    if not _fits(N, V):
        raise BgError(fn, BG_ERR_UNSUPPORTED)
    index = logits.get_device()
    K = 0 if top_token is None else top_token.shape[-1]
    f32, i32 = torch.float32, torch.int32
    if not (_alike(i32, index, (tokens, top_token, dev_status)) and _alike(f32, index, (logprob, entropy, top_logprob)) and
            (tokens is None or tokens.shape == (N,)) and (logprob is None or logprob.shape == (N,)) and
            (entropy is None or entropy.shape == (N,)) and (top_token is None or top_token.shape == (N, K)) and
            (top_logprob is None or top_logprob.shape == (N, K))):
        _expect(fn, logits.device, (
            ("tokens", tokens, i32, (N,)), ("logprob", logprob, f32, (N,)), ("entropy", entropy, f32, (N,)),
            ("top_token", top_token, i32, (N, K)), ("top_logprob", top_logprob, f32, (N, K)),
            ("dev_status", dev_status, i32, dev_status.shape if dev_status is not None else ())))
    _launch(fn, index, stream, logits.data_ptr(), dtype, logits.stride(0) if N > 1 else max(V, 1), N, V, _ptr(tokens), K,
            _ptr(logprob), _ptr(entropy), _ptr(top_token), _ptr(top_logprob), _ptr(dev_status))
    return logprob, entropy, top_token, top_logprob


def bg_selftest_logprobs_timeout(logits, tokens, stalled_row: int, *, logprob, entropy, top_token, top_logprob, dev_status,
                                 stream=None):
    """bg_token_logprobs of fp32 logits [N,V] with K = 1 whose rows from stalled_row on are never loaded: the waits
    run out after a second, those rows get NaN and -1, and dev_status (int32 [1]) BG_DEVSTAT_TIMEOUT."""
    import torch
    fn = "bg_selftest_logprobs_timeout"
    N, V = logits.shape
    f32, i32 = torch.float32, torch.int32
    _expect(fn, logits.device, (
        ("logits", logits, f32, (N, V)), ("tokens", tokens, i32, (N,)), ("logprob", logprob, f32, (N,)),
        ("entropy", entropy, f32, (N,)), ("top_token", top_token, i32, (N, 1)), ("top_logprob", top_logprob, f32, (N, 1)),
        ("dev_status", dev_status, i32, (1,))))
    if not _fits(N, V, stalled_row):
        raise BgError(fn, BG_ERR_UNSUPPORTED)
    _launch(fn, logits.get_device(), stream, logits.data_ptr(), N, V, tokens.data_ptr(), stalled_row, logprob.data_ptr(),
            entropy.data_ptr(), top_token.data_ptr(), top_logprob.data_ptr(), dev_status.data_ptr())


def bg_tree_attn_workspace_size(num_requests: int, total_nodes: int, max_nodes: int, max_prefix_len: int, Hq: int, Hkv: int,
                                head_dim: int) -> int:
    if not _fits(num_requests, total_nodes, max_nodes, max_prefix_len, Hq, Hkv, head_dim):
        return 0
    return int(load().bg_tree_attn_workspace_size(num_requests, total_nodes, max_nodes, max_prefix_len, Hq, Hkv, head_dim))


def _tree_workspace(fn: str, workspace, sizes, index: int):
    if workspace is None:
        raise ValueError(f"{fn}: workspace of {bg_tree_attn_workspace_size(*sizes)} bytes required (the library never "
                         "allocates)")
    if workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"{fn}: workspace must be contiguous on the other tensors' device, got {workspace.device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _tree_run(fn: str, q, k, v, parent, cu_nodes, max_nodes, prefix_k, prefix_v, cu_prefix, max_prefix_len, out, lse, scale,
              softcap, workspace, dev_status, stream):
    import torch
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    T, Hq, d = q.shape
    kv = k.shape
    Hkv = kv[1]
    R = cu_nodes.numel() - 1
    if (prefix_k is None) != (prefix_v is None):
        raise ValueError(f"{fn}: prefix_k and prefix_v come together")
    P = 0 if prefix_k is None else prefix_k.shape[0]
    index = q.get_device()
    if not (_alike(bf16, index, (q, k, v, prefix_k, prefix_v, out)) and
            _alike(i32, index, (parent, cu_nodes, cu_prefix, dev_status)) and
            (lse is None or (_alike(f32, index, (lse,)) and lse.shape == (T, Hq))) and
            out.shape == q.shape and kv == (T, Hkv, d) and v.shape == kv and parent.shape == (T,) and
            (prefix_k is None or prefix_k.shape == prefix_v.shape == (P, Hkv, d)) and
            cu_nodes.dim() == cu_prefix.dim() == 1 and cu_prefix.numel() == R + 1):
        _expect(fn, q.device, (
            ("q", q, bf16, (T, Hq, d)), ("k", k, bf16, (T, Hkv, d)), ("v", v, bf16, (T, Hkv, d)),
            ("parent", parent, i32, (T,)), ("cu_nodes", cu_nodes, i32, (R + 1,)),
            ("prefix_k", prefix_k, bf16, (P, Hkv, d)), ("prefix_v", prefix_v, bf16, (P, Hkv, d)),
            ("cu_prefix", cu_prefix, i32, (R + 1,)), ("out", out, bf16, (T, Hq, d)), ("lse", lse, f32, (T, Hq)),
            ("dev_status", dev_status, i32, dev_status.shape if dev_status is not None else ())))
    max_nodes, max_prefix_len = int(max_nodes), int(max_prefix_len)
    if not _fits(R, T, P, max_nodes, max_prefix_len):
        raise BgError(fn, BG_ERR_UNSUPPORTED)
    ws, ws_bytes = _tree_workspace(fn, workspace, (R, T, max_nodes, max_prefix_len, Hq, Hkv, d), index)
    _launch(fn, index, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), parent.data_ptr(), cu_nodes.data_ptr(), R, T,
            max_nodes, _ptr(prefix_k), _ptr(prefix_v), cu_prefix.data_ptr(), P, max_prefix_len, Hq, Hkv, d,
            1.0 / math.sqrt(d) if scale is None else float(scale), float(softcap), out.data_ptr(), _ptr(lse), ws,
            ws_bytes, _ptr(dev_status))
    return out


def bg_tree_attn(q, k, v, parent, cu_nodes, max_nodes: int, prefix_k, prefix_v, cu_prefix, max_prefix_len: int, out, *,
                 lse=None, scale: Optional[float] = None, softcap: float = 0.0, workspace=None, dev_status=None,
                 stream=None):
    """Attention of the nodes of drafted trees over their request's prefix, their ancestors and themselves.
    q [T,Hq,d], k/v [T,Hkv,d] bf16, request r at rows cu_nodes[r] .. cu_nodes[r+1]-1 (int32 [R+1]); parent
    int32 [T]: a lower node of the same request, counted from its first, or -1; prefix_k/prefix_v [P,Hkv,d]
    (or None) packed by cu_prefix int32 [R+1]; out [T,Hq,d] (written); lse fp32 [T,Hq] or None; workspace a
    uint8 CUDA tensor of bg_tree_attn_workspace_size bytes."""
    return _tree_run("bg_tree_attn", q, k, v, parent, cu_nodes, max_nodes, prefix_k, prefix_v, cu_prefix, max_prefix_len,
                     out, lse, scale, softcap, workspace, dev_status, stream)


def bg_tree_attn_planned(q, k, v, parent, cu_nodes, max_nodes: int, prefix_k, prefix_v, cu_prefix, max_prefix_len: int, out,
                         *, lse=None, scale: Optional[float] = None, softcap: float = 0.0, workspace=None,
                         dev_status=None, stream=None):
    """bg_tree_attn with the work list and the masks that bg_tree_plan left in workspace."""
    return _tree_run("bg_tree_attn_planned", q, k, v, parent, cu_nodes, max_nodes, prefix_k, prefix_v, cu_prefix,
                     max_prefix_len, out, lse, scale, softcap, workspace, dev_status, stream)


def bg_tree_plan(parent, cu_nodes, max_nodes: int, cu_prefix, total_prefix: int, max_prefix_len: int, Hq: int, Hkv: int,
                 head_dim: int, *, workspace=None, dev_status=None, stream=None):
    """The work list and masks of the trees (parent int32 [T], cu_nodes int32 [R+1]) into workspace, for
    bg_tree_attn_planned calls with them."""
    import torch
    fn, i32 = "bg_tree_plan", torch.int32
    T, R = parent.numel(), cu_nodes.numel() - 1
    index = parent.get_device()
    _expect(fn, parent.device, (
        ("parent", parent, i32, (T,)), ("cu_nodes", cu_nodes, i32, (R + 1,)), ("cu_prefix", cu_prefix, i32, (R + 1,)),
        ("dev_status", dev_status, i32, dev_status.shape if dev_status is not None else ())))
    P, max_nodes, max_prefix_len = int(total_prefix), int(max_nodes), int(max_prefix_len)
    if not _fits(R, T, P, max_nodes, max_prefix_len, Hq, Hkv, head_dim):
        raise BgError(fn, BG_ERR_UNSUPPORTED)
    ws, ws_bytes = _tree_workspace(fn, workspace, (R, T, max_nodes, max_prefix_len, Hq, Hkv, head_dim), index)
    _launch(fn, index, stream, parent.data_ptr(), cu_nodes.data_ptr(), R, T, max_nodes, cu_prefix.data_ptr(), P,
            max_prefix_len, Hq, Hkv, head_dim, ws, ws_bytes, _ptr(dev_status))


def _rows_of_heads(fn: str, name: str, t, lead, index: int):
    """Row stride of ``t``, whose last two dimensions (heads, d) are side by side and whose ``lead`` leading ones step
    through rows at one distance (a view into the fused projection's output, for instance)."""
    import torch
    shape, st = t.shape, t.stride()
    ok = t.dtype is torch.bfloat16 and t.get_device() == index and st[-1] == 1 and (shape[-2] == 1 or st[-2] == shape[-1])
    row = st[lead - 1]
    if lead == 2 and shape[0] > 1:
        if shape[1] == 1:
            row = st[0]
        else:
            ok = ok and st[0] == shape[1] * row
    rows = shape[0] if lead == 1 else shape[0] * shape[1]
    if not ok:
        raise ValueError(f"{fn}: {name} must be bfloat16 rows of heads side by side at one distance, on the other tensors' "
                         f"device, got {t.dtype} {tuple(shape)} with strides {st} on {t.device}")
    return row if rows > 1 else (shape[-2] * shape[-1] + 7) // 8 * 8


@functools.lru_cache(maxsize=64)
def _axes(axis_of):
    return (_I32 * len(axis_of))(*axis_of)


def _qk_norm_rope(fn: str, q, k, v, positions, place_shape, outs, lead, q_weight, k_weight, inv_freq):
    """Checks of both forms, with the messages; returns the row strides of q, k and v."""
    import torch
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    index = q.get_device()
    d = q.shape[-1]
    if k.shape[:lead] != q.shape[:lead] or k.shape[-1] != d or (v is not None and v.shape != k.shape):
        raise ValueError(f"{fn}: q, k and v must have the same rows and head_dim, got {tuple(q.shape)}, {tuple(k.shape)}, "
                         f"{None if v is None else tuple(v.shape)}")
    lead_axes = tuple(positions.shape[:1]) if positions.dim() > len(place_shape) else ()
    _expect(fn, q.device, [("positions", positions, i32, lead_axes + place_shape),
                           ("inv_freq", inv_freq, f32, (inv_freq.numel(),)), ("q_weight", q_weight, bf16, (d,)),
                           ("k_weight", k_weight, bf16, (d,))] + [(n, t, bf16, s) for n, t, s in outs])
    return tuple(0 if t is None else _rows_of_heads(fn, n, t, lead, index) for n, t in (("q", q), ("k", k), ("v", v)))


def _rope_common(fn: str, d: int, index: int, positions, places: int, q_weight, k_weight, inv_freq, axis_of):
    """Quick checks of what both forms share, (whether they pass, axes, axis_of as an array, rotated dimensions)."""
    import torch
    f32 = torch.float32
    ps, n = positions.shape, inv_freq.shape[0]
    ok = (0 < len(ps) <= 2 and ps[-1] == places and positions.dtype is torch.int32 and positions.get_device() == index and
          positions.is_contiguous() and inv_freq.dtype is f32 and inv_freq.get_device() == index and inv_freq.is_contiguous() and
          inv_freq.dim() == 1 and (q_weight is None or q_weight.shape == (d,)) and (k_weight is None or k_weight.shape == (d,)))
    if axis_of is not None:
        if len(axis_of) != n:
            raise ValueError(f"{fn}: axis_of must have an axis for each of the {n} frequencies, got {len(axis_of)}")
        axis_of = _axes(tuple(axis_of))
    return ok, ps[0] if len(ps) == 2 else 1, axis_of, 2 * n


def bg_packed_qk_norm_rope(q, k, v, positions, q_out, k_out, v_out=None, *, inv_freq, q_weight=None, k_weight=None,
                           eps: float = 1e-6, weight_offset: float = 0.0, axis_of=None, interleaved: bool = False,
                           rope_scale: float = 1.0, stream=None):
    """Norm of every head of q [T,Hq,d] and k [T,Hkv,d] (bf16; rows may be strided, as views into a fused projection
    are) with q_weight/k_weight bf16 [d] (None: no norm), then the rotation of the first 2 * len(inv_freq) dimensions
    by positions int32 [T] or [axes,T] times inv_freq fp32; axis_of: the axis of each frequency (a list).
    q_out [T,Hq,d], k_out and v_out [T,Hkv,d] contiguous (written); v [T,Hkv,d] is copied to v_out, or both are None."""
    import torch
    fn = "bg_packed_qk_norm_rope"
    qs, ks = q.shape, k.shape
    T, Hq, d = qs
    Hkv = ks[1]
    index = q.get_device()
    ok, axes, axis_of, rot = _rope_common(fn, d, index, positions, T, q_weight, k_weight, inv_freq, axis_of)
    bf16 = torch.bfloat16
    a, b = q.stride(), k.stride()
    c = b if v is None else v.stride()
    # as the calls usually are: rows of heads, d apart, of more than one token
    if not (ok and T > 1 and a[2] == b[2] == c[2] == 1 and a[1] == b[1] == c[1] == d and ks == (T, Hkv, d) and
            q.dtype is bf16 and k.dtype is bf16 and k.get_device() == index and
            (v is None or (v.shape == ks and v.dtype is bf16 and v.get_device() == index)) and
            _alike(bf16, index, (q_out, k_out, v_out, q_weight, k_weight)) and q_out.shape == qs and k_out.shape == ks and
            (v_out is None or v_out.shape == ks)):
        a, b, c = ((n,) for n in _qk_norm_rope(fn, q, k, v, positions, (T,), (
            ("q_out", q_out, (T, Hq, d)), ("k_out", k_out, (T, Hkv, d)), ("v_out", v_out, (T, Hkv, d))), 1, q_weight,
            k_weight, inv_freq))
    if T > 0x7fffffff or Hq > 0x7fffffff or Hkv > 0x7fffffff:
        raise BgError(fn, BG_ERR_UNSUPPORTED)
    _launch(fn, index, stream, q.data_ptr(), a[0], k.data_ptr(), b[0], _ptr(v), c[0], T, Hq, Hkv, d, _ptr(q_weight),
            _ptr(k_weight), float(eps), float(weight_offset), positions.data_ptr(), axes, axis_of, inv_freq.data_ptr(), rot,
            int(interleaved), float(rope_scale), q_out.data_ptr(), k_out.data_ptr(), _ptr(v_out))
    return q_out, k_out, v_out


def bg_beam_qk_norm_rope(q, k, v, base_pos, step: int, q_out, suffix_k, suffix_v, slot: int, *, inv_freq, q_weight=None,
                         k_weight=None, eps: float = 1e-6, weight_offset: float = 0.0, axis_of=None,
                         interleaved: bool = False, rope_scale: float = 1.0, stream=None):
    """bg_packed_qk_norm_rope for the new token of every beam: q [R,W,Hq,d], k/v [R,W,Hkv,d] bf16 (strided rows as
    there), all beams of request r at base_pos int32 [R] or [axes,R] plus step; q_out [R,W,Hq,d] and slot ``slot`` of
    suffix_k/suffix_v [R,W,S_max,Hkv,d] are written."""
    import torch
    fn = "bg_beam_qk_norm_rope"
    qs, ks, ss = q.shape, k.shape, suffix_k.shape
    R, W, Hq, d = qs
    Hkv, S_max = ks[2], ss[2]
    index = q.get_device()
    ok, axes, axis_of, rot = _rope_common(fn, d, index, base_pos, R, q_weight, k_weight, inv_freq, axis_of)
    bf16 = torch.bfloat16
    a, b, c = q.stride(), k.stride(), v.stride()
    # as the calls usually are: rows of heads, d apart, at one distance, of more than one beam
    if not (ok and W > 1 and a[3] == b[3] == c[3] == 1 and a[2] == b[2] == c[2] == d and
            (R == 1 or (a[0] == W * a[1] and b[0] == W * b[1] and c[0] == W * c[1])) and ks == (R, W, Hkv, d) and v.shape == ks and
            q.dtype is bf16 and k.dtype is bf16 and v.dtype is bf16 and k.get_device() == index == v.get_device() and
            _alike(bf16, index, (q_out, suffix_k, suffix_v, q_weight, k_weight)) and q_out.shape == qs and
            ss == (R, W, S_max, Hkv, d) and suffix_v.shape == ss):
        suffix = (R, W, S_max, Hkv, d)
        a, b, c = ((0, n) for n in _qk_norm_rope(fn, q, k, v, base_pos, (R,), (
            ("q_out", q_out, (R, W, Hq, d)), ("suffix_k", suffix_k, suffix), ("suffix_v", suffix_v, suffix)), 2, q_weight,
            k_weight, inv_freq))
    if not _fits(R, W, Hq, Hkv, S_max, step, slot):
        raise BgError(fn, BG_ERR_UNSUPPORTED)
    _launch(fn, index, stream, q.data_ptr(), a[1], k.data_ptr(), b[1], v.data_ptr(), c[1], R, W, Hq, Hkv, d,
            _ptr(q_weight), _ptr(k_weight), float(eps), float(weight_offset), base_pos.data_ptr(), axes, axis_of, int(step),
            inv_freq.data_ptr(), rot, int(interleaved), float(rope_scale), q_out.data_ptr(), suffix_k.data_ptr(),
            suffix_v.data_ptr(), S_max, int(slot))
    return q_out, suffix_k, suffix_v


def bg_adjust_logits(logits, out, *, rows_per_group: int = 1, prompt_tokens=None, cu_prompt=None, own_tokens=None,
                     own_lens=None, repetition=None, frequency=None, presence=None, bias_tokens=None, bias_values=None,
                     cu_bias=None, mask=None, mask_index=None, dev_status=None, stream=None):
    """Penalties, biases and masks on logits fp32 or bf16 [N,V] into out [N,V] (rows may be strided; out may be logits).
    Groups of rows_per_group rows share prompt_tokens int32 (packed by cu_prompt int32 [G+1]), repetition/frequency/
    presence fp32 [G] and bias_tokens int32, bias_values fp32 (packed by cu_bias int32 [G+1]); own_tokens int32 [N,S],
    of which row i has own_lens[i] (int32 [N] or None: S); mask int32 or uint32 [M,words], bit v % 32 of word v // 32 set
    where v is allowed, mask_index int32 [N] (-1: no mask) or None: row i has mask i."""
    import torch
    fn = "bg_adjust_logits"
    N, V = logits.shape
    kinds = {torch.float32: BG_DTYPE_F32, torch.bfloat16: BG_DTYPE_BF16}
    index = logits.get_device()
    for name, t in (("logits", logits), ("out", out)):
        if t.dtype not in kinds or t.shape != (N, V) or (V > 1 and N > 0 and t.stride(1) != 1) or t.get_device() != index:
            raise ValueError(f"{fn}: {name} must be float32 or bfloat16 with contiguous rows of shape {(N, V)} on "
                             f"{logits.device}, got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")
    rows_per_group = int(rows_per_group)
    if rows_per_group < 1 or N % rows_per_group:
        raise ValueError(f"{fn}: {N} rows are no whole groups of {rows_per_group}")
    G = N // rows_per_group
    f32, i32 = torch.float32, torch.int32
    if (prompt_tokens is None) != (cu_prompt is None) or (bias_tokens is None) != (cu_bias is None) or \
            (bias_tokens is None) != (bias_values is None):
        raise ValueError(f"{fn}: prompt_tokens and cu_prompt, and bias_tokens, bias_values and cu_bias, come together")
    P = 0 if prompt_tokens is None else prompt_tokens.numel()
    B = 0 if bias_tokens is None else bias_tokens.numel()
    S = 0 if own_tokens is None else own_tokens.shape[-1]
    M, words = (0, 0) if mask is None else (mask.shape[0], mask.shape[-1])
    if mask is not None and mask.dtype is getattr(torch, "uint32", None):
        mask = mask.view(i32)
    if not (_alike(i32, index, (prompt_tokens, cu_prompt, own_tokens, own_lens, bias_tokens, cu_bias, mask, mask_index,
                                dev_status)) and
            _alike(f32, index, (repetition, frequency, presence, bias_values)) and
            (prompt_tokens is None or (prompt_tokens.dim() == 1 and cu_prompt.shape == (G + 1,))) and
            (own_tokens is None or own_tokens.shape == (N, S)) and (own_lens is None or own_lens.shape == (N,)) and
            (repetition is None or repetition.shape == (G,)) and (frequency is None or frequency.shape == (G,)) and
            (presence is None or presence.shape == (G,)) and
            (bias_tokens is None or (bias_tokens.shape == bias_values.shape == (B,) and cu_bias.shape == (G + 1,))) and
            (mask is None or mask.dim() == 2) and (mask_index is None or mask_index.shape == (N,))):
        _expect(fn, logits.device, (
            ("prompt_tokens", prompt_tokens, i32, (P,)), ("cu_prompt", cu_prompt, i32, (G + 1,)),
            ("own_tokens", own_tokens, i32, (N, S)), ("own_lens", own_lens, i32, (N,)), ("repetition", repetition, f32, (G,)),
            ("frequency", frequency, f32, (G,)), ("presence", presence, f32, (G,)), ("bias_tokens", bias_tokens, i32, (B,)),
            ("bias_values", bias_values, f32, (B,)), ("cu_bias", cu_bias, i32, (G + 1,)), ("mask", mask, i32, (M, words)),
            ("mask_index", mask_index, i32, (N,)),
            ("dev_status", dev_status, i32, dev_status.shape if dev_status is not None else ())))
    if not _fits(N, V, P, B, S, M):
        raise BgError(fn, BG_ERR_UNSUPPORTED)
    _launch(fn, index, stream, logits.data_ptr(), kinds[logits.dtype], logits.stride(0) if N > 1 else V, G, rows_per_group, V,
            _ptr(prompt_tokens), _ptr(cu_prompt), P, _ptr(own_tokens), _ptr(own_lens), S, _ptr(repetition),
            _ptr(frequency), _ptr(presence), _ptr(bias_tokens), _ptr(bias_values), _ptr(cu_bias), B, _ptr(mask), words, M,
            _ptr(mask_index), out.data_ptr(), kinds[out.dtype], out.stride(0) if N > 1 else V, _ptr(dev_status))
    return out

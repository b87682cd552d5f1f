"""Python binding of libattn_b200.so (argument marshalling only).

Every function here has the name of the C entry point it calls (declared in
include/attn_b200.h).  It takes torch tensors, allocates the outputs with torch
when they are not given, passes raw device pointers, sizes and the current
CUDA stream, and raises ``AttnError`` on a non-OK status.  All arithmetic
happens in the CUDA kernels; there is no fallback: if the library is missing
or the device is not a B200, the call raises.
"""
from __future__ import annotations

import ctypes
import math
from pathlib import Path

import torch

_LIB_PATH = Path(__file__).resolve().parent / "libattn_b200.so"
_lib = None

MASK_NONE, MASK_CAUSAL, MASK_PATCH = 0, 1, 2
BF16, FP8_E4M3 = 0, 1


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, status_string(status), status))


def library_path() -> Path:
    return _LIB_PATH


def lib():
    """Loads the CUDA library (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not _LIB_PATH.exists():
            raise RuntimeError("libattn_b200.so is not built; run "
                               "`python -m attention_paged_kv_gqa_b200.build`")
        L = ctypes.CDLL(str(_LIB_PATH))
        P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.attn_check_device.argtypes = [I]
        L.attn_check_device.restype = I
        L.attn_status_string.argtypes = [I]
        L.attn_status_string.restype = ctypes.c_char_p
        L.attn_device_error.argtypes = [ctypes.POINTER(I), P]
        L.attn_device_error.restype = I
        L.attn_selftest_wait_expiry.argtypes = [ctypes.c_longlong, P]
        L.attn_selftest_wait_expiry.restype = I
        L.attn_fwd_dense.argtypes = [P, P, P, P, P, I, I, I, I, I, I, P, P, P, F, I, I, F, I,
                                     P, P, P, P]
        L.attn_fwd_dense.restype = I
        L.attn_fwd_varlen_paged.argtypes = [P, P, P, P, I, I, I, P, P, P, I, I, I, I, I, I, I,
                                            F, I, P, I, F, I, P, P, P, P, P, P, Z, P]
        L.attn_fwd_varlen_paged.restype = I
        L.attn_fwd_varlen_paged_only_qv.argtypes = [P, P, P, I, I, I, P, P, P, I, I, I, I, I, I, I,
                                                    F, I, P, I, F, I, P, P, P, P, P]
        L.attn_fwd_varlen_paged_only_qv.restype = I
        L.attn_decode_paged_only_qv.argtypes = [P, P, P, I, I, I, P, I, I, I, I, F, I, F, I, I, P, P,
                                                P, Z, P]
        L.attn_decode_paged_only_qv.restype = I
        L.attn_fwd_patch.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, I, P, P, P, P, P, P]
        L.attn_fwd_patch.restype = I
        L.attn_decode_workspace_size.argtypes = [I, I, I, I, I, I, I]
        L.attn_decode_workspace_size.restype = Z
        L.attn_decode_paged.argtypes = [P, P, P, P, I, I, I, P, I, I, I, I, F, I, F, I, I, P, P,
                                        P, P, P, P, Z, P]
        L.attn_decode_paged.restype = I
        L.attn_fwd_varlen_paged_qv.argtypes = [P, P, P, P, P, I, I, I, P, P, P, I, I, I, I, I, I,
                                               I, F, I, P, I, F, I, P, P, P]
        L.attn_fwd_varlen_paged_qv.restype = I
        L.attn_decode_paged_qv.argtypes = [P, P, P, P, P, I, I, I, P, I, I, I, I, F, I, F, I, I,
                                           P, P, P, Z, P]
        L.attn_decode_paged_qv.restype = I
        L.attn_decode_paged_noalloc.argtypes = [P, P, P, P, I, I, I, P, I, I, I, I, F, I, P, P, P]
        L.attn_decode_paged_noalloc.restype = I
        L.attn_kv_append_paged.argtypes = [P, P, P, P, P, I, I, I, P, P, P, I, I, I, I, I, P]
        L.attn_kv_append_paged.restype = I
        L.attn_decode_paged_append.argtypes = [P, P, P, P, P, P, I, I, I, P, P, I, I, I, I, F, I, F,
                                               I, I, P, P, P, Z, P]
        L.attn_decode_paged_append.restype = I
        L.attn_bwd_workspace_size.argtypes = [I, I]
        L.attn_bwd_workspace_size.restype = Z
        L.attn_bwd_varlen.argtypes = [P, P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, F,
                                      I, I, P, Z, P]
        L.attn_bwd_varlen.restype = I
        L.attn_rope.argtypes = [P] * 8 + [I, I, I, I, P, I, I, P, I, P, I, I, P]
        L.attn_rope.restype = I
        append = [P] * 7 + [P, P]                       # q .. v_cache
        pages = [P, I, I, I]                            # block_table .. block_size
        rope = [P, I, I, P, I, P, I]                    # cos_sin .. interleaved
        L.attn_kv_append_rope_paged.argtypes = append + pages + [P, P, P, I, I, I, I, I] + rope + [I, P, P, P, P]
        L.attn_kv_append_rope_paged.restype = I
        L.attn_kv_append_paged_q4.argtypes = append + [P, P] + pages + [P, P, P, I, I, I, I, I, I] + rope + [P]
        L.attn_kv_append_paged_q4.restype = I
        L.attn_kv_gather_paged_q4.argtypes = [P] * 4 + pages + [P, P, I, I, I, I, I, P, P, P]
        L.attn_kv_gather_paged_q4.restype = I
        L.attn_decode_q4_workspace_size.argtypes = [I] * 4
        L.attn_decode_q4_workspace_size.restype = Z
        L.attn_decode_paged_q4.argtypes = [P] * 5 + pages + [P, I, I, I, I, I, F, I, F, P, P, P, Z, P]
        L.attn_decode_paged_q4.restype = I
        L.attn_fwd_q4_workspace_size.argtypes = [I] * 6
        L.attn_fwd_q4_workspace_size.restype = Z
        L.attn_fwd_varlen_paged_q4.argtypes = [P] * 5 + pages + [P, P] + [I] * 8 + [F, I, I, F, P, P, P, Z, P]
        L.attn_fwd_varlen_paged_q4.restype = I
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().attn_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != 0:
        raise AttnError(status, where)


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float8_e4m3fn:
        return FP8_E4M3
    raise TypeError("q/k/v must be bfloat16 or float8_e4m3fn, got %s" % t.dtype)


def _scale(scale):
    return 0.0 if scale is None else float(scale)


def _strides3(t: torch.Tensor):
    if t.stride(-1) != 1:
        raise ValueError("head_dim must be the contiguous dimension")
    return (ctypes.c_int64 * 3)(t.stride(0), t.stride(1), t.stride(2))


def attn_check_device(device: int = 0) -> int:
    return lib().attn_check_device(int(device))


def attn_device_error(stream=None) -> int:
    code = ctypes.c_int(0)
    st = lib().attn_device_error(ctypes.byref(code), _stream(stream))
    if st not in (0, 7, 9):
        _check(st, "attn_device_error")
    return code.value


def attn_selftest_wait_expiry(limit_ns: int, stream=None):
    """Launches the bounded-wait test kernel (a wait nothing satisfies, limited to limit_ns)."""
    _check(lib().attn_selftest_wait_expiry(int(limit_ns), _stream(stream)),
           "attn_selftest_wait_expiry")


def attn_fwd_dense(q, k, v, *, causal=False, scale=None, window_left=-1, softcap=0.0,
                   descale_q=None, descale_k=None, descale_v=None, out=None, lse=None,
                   return_lse=True, stream=None):
    """q [B, Lq, Hq, D], k/v [B, Lk, Hkv, D] -> (o [B, Lq, Hq, D] bf16, lse [B, Hq, Lq] fp32).

    window_left >= 0 (causal only): row i keeps keys i' - window_left .. i';
    softcap > 0: each logit s becomes softcap * tanh(s / softcap).
    """
    B, Lq, Hq, D = q.shape
    Lk, Hkv = k.shape[1], k.shape[2]
    if out is None:
        out = torch.empty((B, Lq, Hq, D), dtype=torch.bfloat16, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq, Lq), dtype=torch.float32, device=q.device)
    st = lib().attn_fwd_dense(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Lq, Lk, Hq, Hkv,
                              D, _strides3(q), _strides3(k), _strides3(v), _scale(scale),
                              MASK_CAUSAL if causal else MASK_NONE, int(window_left),
                              float(softcap), _dtype_code(q),
                              _ptr(descale_q), _ptr(descale_k), _ptr(descale_v), _stream(stream))
    _check(st, "attn_fwd_dense")
    return out, lse


def attn_fwd_varlen_paged(q, k_cache, v_cache, *, cu_seqlens_q, max_seqlen_q, block_table=None,
                          cu_seqlens_k=None, seqused_k=None, mask=MASK_NONE, scale=None,
                          patch_kv_range=None, window_left=-1, softcap=0.0, descale_q=None,
                          descale_k=None, descale_v=None, out=None, lse=None, return_lse=True,
                          stream=None):
    """q [total_q, Hq, D]; paged k/v [num_blocks, 16, Hkv, D] (or packed [total_k, Hkv, D]).

    Returns (o [total_q, Hq, D] bf16, lse [Hq, total_q] fp32).
    """
    total_q, Hq, D = q.shape
    B = cu_seqlens_q.numel() - 1
    if block_table is not None:
        num_blocks, block_size, Hkv = k_cache.shape[0], k_cache.shape[1], k_cache.shape[2]
        mbps, total_k = block_table.shape[1], 0
    else:
        num_blocks, block_size, mbps = 0, 0, 0
        total_k, Hkv = k_cache.shape[0], k_cache.shape[1]
    if out is None:
        out = torch.empty((total_q, Hq, D), dtype=torch.bfloat16, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((Hq, total_q), dtype=torch.float32, device=q.device)
    st = lib().attn_fwd_varlen_paged(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), mbps, num_blocks, block_size,
        _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), _ptr(seqused_k), B, total_q, total_k,
        int(max_seqlen_q), Hq, Hkv, D, _scale(scale), int(mask), _ptr(patch_kv_range),
        int(window_left), float(softcap), _dtype_code(q), _ptr(descale_q), _ptr(descale_k), _ptr(descale_v), _ptr(out), _ptr(lse),
        None, 0, _stream(stream))
    _check(st, "attn_fwd_varlen_paged")
    return out, lse


def attn_fwd_varlen_paged_only_qv(qv, v_cache, *, cu_seqlens_q, max_seqlen_q, block_table=None,
                                  cu_seqlens_k=None, seqused_k=None, mask=MASK_NONE, scale=None,
                                  patch_kv_range=None, window_left=-1, softcap=0.0,
                                  descale_qv=None, descale_v=None, out=None, lse=None,
                                  return_lse=True, stream=None):
    """The only_qv score (scale * qv . v): qv [total_q, Hq, D]; v paged or packed as in
    attn_fwd_varlen_paged.  Returns (o [total_q, Hq, D] bf16, lse [Hq, total_q] fp32)."""
    total_q, Hq, D = qv.shape
    B = cu_seqlens_q.numel() - 1
    if block_table is not None:
        num_blocks, block_size, Hkv = v_cache.shape[0], v_cache.shape[1], v_cache.shape[2]
        mbps, total_k = block_table.shape[1], 0
    else:
        num_blocks, block_size, mbps = 0, 0, 0
        total_k, Hkv = v_cache.shape[0], v_cache.shape[1]
    if out is None:
        out = torch.empty((total_q, Hq, D), dtype=torch.bfloat16, device=qv.device)
    if lse is None and return_lse:
        lse = torch.empty((Hq, total_q), dtype=torch.float32, device=qv.device)
    st = lib().attn_fwd_varlen_paged_only_qv(
        _ptr(qv), _ptr(v_cache), _ptr(block_table), mbps, num_blocks, block_size,
        _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), _ptr(seqused_k), B, total_q, total_k,
        int(max_seqlen_q), Hq, Hkv, D, _scale(scale), int(mask), _ptr(patch_kv_range),
        int(window_left), float(softcap), _dtype_code(qv), _ptr(descale_qv), _ptr(descale_v),
        _ptr(out), _ptr(lse), _stream(stream))
    _check(st, "attn_fwd_varlen_paged_only_qv")
    return out, lse


def attn_fwd_varlen_paged_qv(q, qv, k_cache, v_cache, *, cu_seqlens_q, max_seqlen_q,
                             block_table=None, cu_seqlens_k=None, seqused_k=None, mask=MASK_NONE,
                             scale=None, patch_kv_range=None, window_left=-1, softcap=0.0,
                             out=None, lse=None, return_lse=True, stream=None):
    """The forward with the Qv score term, scale * (q.k + qv.v): q, qv [total_q, Hq, D] bf16;
    K/V paged or packed as in attn_fwd_varlen_paged.
    Returns (o [total_q, Hq, D] bf16, lse [Hq, total_q] fp32)."""
    total_q, Hq, D = q.shape
    B = cu_seqlens_q.numel() - 1
    if block_table is not None:
        num_blocks, block_size, Hkv = k_cache.shape[0], k_cache.shape[1], k_cache.shape[2]
        mbps, total_k = block_table.shape[1], 0
    else:
        num_blocks, block_size, mbps = 0, 0, 0
        total_k, Hkv = k_cache.shape[0], k_cache.shape[1]
    if out is None:
        out = torch.empty((total_q, Hq, D), dtype=torch.bfloat16, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((Hq, total_q), dtype=torch.float32, device=q.device)
    st = lib().attn_fwd_varlen_paged_qv(
        _ptr(q), _ptr(qv), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), mbps, num_blocks,
        block_size, _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), _ptr(seqused_k), B, total_q, total_k,
        int(max_seqlen_q), Hq, Hkv, D, _scale(scale), int(mask), _ptr(patch_kv_range),
        int(window_left), float(softcap), _dtype_code(q), _ptr(out), _ptr(lse), _stream(stream))
    _check(st, "attn_fwd_varlen_paged_qv")
    return out, lse


def attn_fwd_patch(q, k, v, *, cu_seqlens_q, cu_seqlens_k, patch_kv_range, max_seqlen_q,
                   max_interval, scale=None, descale_q=None, descale_k=None, descale_v=None,
                   out=None, lse=None, return_lse=True, stream=None):
    """Patch cross-attention with intervals of at most max_interval keys (see the header):
    q [total_q, Hq, D], packed k/v [total_k, Hkv, D] -> (o, lse [Hq, total_q])."""
    total_q, Hq, D = q.shape
    total_k, Hkv = k.shape[0], k.shape[1]
    B = cu_seqlens_q.numel() - 1
    if out is None:
        out = torch.empty((total_q, Hq, D), dtype=torch.bfloat16, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((Hq, total_q), dtype=torch.float32, device=q.device)
    st = lib().attn_fwd_patch(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
                              _ptr(patch_kv_range), B, total_q, total_k, int(max_seqlen_q), Hq, Hkv, D,
                              _scale(scale), int(max_interval), _dtype_code(q), _ptr(descale_q),
                              _ptr(descale_k), _ptr(descale_v), _ptr(out), _ptr(lse), _stream(stream))
    _check(st, "attn_fwd_patch")
    return out, lse


def attn_decode_workspace_size(B, num_heads_q, num_heads_kv, head_dim, max_blocks_per_seq,
                               block_size=16, num_splits=0) -> int:
    return int(lib().attn_decode_workspace_size(B, num_heads_q, num_heads_kv, head_dim,
                                                max_blocks_per_seq, block_size, num_splits))


def attn_decode_paged(q, k_cache, v_cache, block_table, seqused_k, *, scale=None, num_splits=0,
                      window_left=-1, softcap=0.0, descale_q=None, descale_k=None,
                      descale_v=None, out=None, lse=None, workspace=None, return_lse=True,
                      stream=None):
    """q [B, Hq, D] against a paged cache -> (o [B, Hq, D] bf16, lse [B, Hq] fp32).

    The query is the newest cached token; window_left >= 0 keeps the keys
    L-1-window_left .. L-1; softcap > 0 caps the logits as in the prefill calls.
    With q and the cache in float8_e4m3fn, descale_q/k/v ([Hkv] fp32 each) are
    required (head_dim 128, automatic split).
    """
    B, Hq, D = q.shape
    num_blocks, block_size, Hkv = k_cache.shape[0], k_cache.shape[1], k_cache.shape[2]
    mbps = block_table.shape[1]
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    ws_bytes = attn_decode_workspace_size(B, Hq, Hkv, D, mbps, block_size, num_splits)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=q.device)
    st = lib().attn_decode_paged(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), mbps,
                                 num_blocks, block_size, _ptr(seqused_k), B, Hq, Hkv, D,
                                 _scale(scale), int(window_left), float(softcap), int(num_splits),
                                 _dtype_code(q), _ptr(descale_q), _ptr(descale_k), _ptr(descale_v),
                                 _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
                                 _stream(stream))
    _check(st, "attn_decode_paged")
    return out, lse


def attn_decode_paged_qv(q, qv, k_cache, v_cache, block_table, seqused_k, *, scale=None,
                         num_splits=0, window_left=-1, softcap=0.0, out=None, lse=None,
                         workspace=None, return_lse=True, stream=None):
    """Paged decode whose logit adds the Qv term: scale * (q.k + qv.v).

    q, qv [B, Hq, D] bf16 -> (o [B, Hq, D] bf16, lse [B, Hq] fp32); arguments as
    attn_decode_paged.
    """
    B, Hq, D = q.shape
    num_blocks, block_size, Hkv = k_cache.shape[0], k_cache.shape[1], k_cache.shape[2]
    mbps = block_table.shape[1]
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    ws_bytes = attn_decode_workspace_size(B, Hq, Hkv, D, mbps, block_size, num_splits)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=q.device)
    st = lib().attn_decode_paged_qv(_ptr(q), _ptr(qv), _ptr(k_cache), _ptr(v_cache),
                                    _ptr(block_table), mbps, num_blocks, block_size,
                                    _ptr(seqused_k), B, Hq, Hkv, D, _scale(scale),
                                    int(window_left), float(softcap), int(num_splits),
                                    _dtype_code(q), _ptr(out), _ptr(lse), _ptr(workspace),
                                    workspace.numel(), _stream(stream))
    _check(st, "attn_decode_paged_qv")
    return out, lse


def attn_decode_paged_only_qv(qv, v_cache, block_table, seqused_k, *, scale=None, num_splits=0,
                              window_left=-1, softcap=0.0, out=None, lse=None, workspace=None,
                              return_lse=True, stream=None):
    """Paged decode with the only_qv score: qv [B, Hq, D] -> (o [B, Hq, D] bf16, lse [B, Hq])."""
    B, Hq, D = qv.shape
    num_blocks, block_size, Hkv = v_cache.shape[0], v_cache.shape[1], v_cache.shape[2]
    mbps = block_table.shape[1]
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=qv.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=qv.device)
    ws_bytes = attn_decode_workspace_size(B, Hq, Hkv, D, mbps, block_size, num_splits)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=qv.device)
    st = lib().attn_decode_paged_only_qv(_ptr(qv), _ptr(v_cache), _ptr(block_table), mbps,
                                         num_blocks, block_size, _ptr(seqused_k), B, Hq, Hkv, D,
                                         _scale(scale), int(window_left), float(softcap),
                                         int(num_splits), _dtype_code(qv), _ptr(out), _ptr(lse),
                                         _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "attn_decode_paged_only_qv")
    return out, lse


def attn_decode_paged_noalloc(q, k_cache, v_cache, block_table, seqused_k, *, scale=None,
                              out=None, lse=None, return_lse=True, stream=None):
    """attn_decode_paged whose split-KV scratch is the library's fixed device array.

    For callers that must not allocate device memory while they run: the C
    call allocates nothing (the outputs are allocated here only when not given).
    """
    B, Hq, D = q.shape
    num_blocks, block_size, Hkv = k_cache.shape[0], k_cache.shape[1], k_cache.shape[2]
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    st = lib().attn_decode_paged_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                         block_table.shape[1], num_blocks, block_size,
                                         _ptr(seqused_k), B, Hq, Hkv, D, _scale(scale),
                                         _dtype_code(q), _ptr(out), _ptr(lse), _stream(stream))
    _check(st, "attn_decode_paged_noalloc")
    return out, lse


def attn_kv_append_paged(k_new, v_new, k_cache, v_cache, block_table, seqused_k, *,
                         cu_seqlens_new=None, seqused_k_out=None, stream=None):
    """Writes new tokens' K/V ([total_new, Hkv, D]) into the paged cache in place.

    Sequence b's i-th new token goes to position seqused_k[b] + i.  Returns
    seqused_k_out (lengths after), allocated here when not given.
    cu_seqlens_new None means one new token per sequence.
    """
    total_new, Hkv, D = k_new.shape
    B = seqused_k.numel()
    num_blocks, block_size = k_cache.shape[0], k_cache.shape[1]
    if seqused_k_out is None:
        seqused_k_out = torch.empty_like(seqused_k)
    st = lib().attn_kv_append_paged(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                    _ptr(block_table), block_table.shape[1], num_blocks,
                                    block_size, _ptr(cu_seqlens_new), _ptr(seqused_k),
                                    _ptr(seqused_k_out), B, total_new, Hkv, D, _dtype_code(k_new),
                                    _stream(stream))
    _check(st, "attn_kv_append_paged")
    return seqused_k_out


def attn_decode_paged_append(q, k_new, v_new, k_cache, v_cache, block_table, seqused_k, *,
                             seqused_k_out=None, scale=None, num_splits=0, window_left=-1,
                             softcap=0.0, out=None, lse=None, workspace=None, return_lse=True,
                             stream=None):
    """Appends one token per sequence (k_new/v_new [B, Hkv, D]) to the paged cache, then
    decodes q [B, Hq, D] over the updated cache.  Returns (o, lse, seqused_k_out)."""
    B, Hq, D = q.shape
    num_blocks, block_size, Hkv = k_cache.shape[0], k_cache.shape[1], k_cache.shape[2]
    mbps = block_table.shape[1]
    if seqused_k_out is None:
        seqused_k_out = torch.empty_like(seqused_k)
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.bfloat16, device=q.device)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    ws_bytes = attn_decode_workspace_size(B, Hq, Hkv, D, mbps, block_size, num_splits)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=q.device)
    st = lib().attn_decode_paged_append(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), mbps,
        num_blocks, block_size, _ptr(seqused_k), _ptr(seqused_k_out), B, Hq, Hkv, D, _scale(scale),
        int(window_left), float(softcap), int(num_splits), _dtype_code(q), _ptr(out), _ptr(lse),
        _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "attn_decode_paged_append")
    return out, lse, seqused_k_out


def attn_bwd_varlen(q, k, v, o, dout, lse, *, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                    max_seqlen_k, mask=MASK_NONE, scale=None, window_left=-1, dq=None, dk=None,
                    dv=None, workspace=None, stream=None):
    """Gradients of the varlen forward: (dq [total_q, Hq, D], dk, dv [total_k, Hkv, D]).

    q, o, dout [total_q, Hq, D] bf16; k, v [total_k, Hkv, D] bf16; lse [Hq, total_q]
    fp32 from the forward.
    """
    total_q, Hq, D = q.shape
    total_k, Hkv = k.shape[0], k.shape[1]
    B = cu_seqlens_q.numel() - 1
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    ws_bytes = int(lib().attn_bwd_workspace_size(Hq, total_q))
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), dtype=torch.uint8, device=q.device)
    st = lib().attn_bwd_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq),
                               _ptr(dk), _ptr(dv), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), B,
                               total_q, total_k, int(max_seqlen_q), int(max_seqlen_k), Hq, Hkv, D,
                               _scale(scale), int(mask), int(window_left), _ptr(workspace),
                               workspace.numel(), _stream(stream))
    _check(st, "attn_bwd_varlen")
    return dq, dk, dv


def attn_bwd_dense(q, k, v, o, dout, lse, *, causal=False, scale=None, window_left=-1,
                   stream=None):
    """Dense [B, L, H, D] convenience over attn_bwd_varlen (lse [B, Hq, Lq] from
    attn_fwd_dense).  Returns (dq, dk, dv) in the dense layouts."""
    B, Lq, Hq, D = q.shape
    Lk, Hkv = k.shape[1], k.shape[2]
    dev = q.device
    cq = torch.arange(B + 1, dtype=torch.int32, device=dev) * Lq
    ck = torch.arange(B + 1, dtype=torch.int32, device=dev) * Lk
    lse_v = lse.permute(1, 0, 2).reshape(Hq, B * Lq).contiguous()
    dq, dk, dv = attn_bwd_varlen(q.reshape(B * Lq, Hq, D), k.reshape(B * Lk, Hkv, D),
                                 v.reshape(B * Lk, Hkv, D), o.reshape(B * Lq, Hq, D),
                                 dout.reshape(B * Lq, Hq, D), lse_v, cu_seqlens_q=cq,
                                 cu_seqlens_k=ck, max_seqlen_q=Lq, max_seqlen_k=Lk,
                                 mask=MASK_CAUSAL if causal else MASK_NONE, scale=scale,
                                 window_left=window_left, stream=stream)
    return dq.reshape(B, Lq, Hq, D), dk.reshape(B, Lk, Hkv, D), dv.reshape(B, Lk, Hkv, D)


# ---------------------------------------------------------------- rotary positions, 4-bit cache
# These calls check their tensors (type, shape, layout, device) before the pointers
# leave for C, and run on the tensors' device whichever device is current.  A decode
# step's kernels take a few microseconds, so the checks' passing path is kept short:
# one comparison each, with the message worked out only for a tensor that fails.

_BF16, _F32, _I32, _I16, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.int16, torch.uint8
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _need(ok, where, what):
    if not ok:
        raise ValueError("%s: %s" % (where, what))


def _refuse(t, dtype, shape, dev, where, name):
    """Why t is not a contiguous tensor of this type and shape on this device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s: %s must be a tensor" % (where, name))
    if t.dtype != dtype:
        raise TypeError("%s: %s must be %s, got %s" % (where, name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s: %s must have shape %s, got %s" % (where, name, tuple(shape), tuple(t.shape)))
    if t.device != dev:
        raise ValueError("%s: %s is on %s, not on %s" % (where, name, t.device, dev))
    raise ValueError("%s: %s must be contiguous" % (where, name))


def _tensor(t, dtype, shape, dev, where, name):
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev
            and t.is_contiguous()):
        _refuse(t, dtype, shape, dev, where, name)


def _dims(t, n, where, name):
    """The shape of a tensor of n dimensions."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s: %s must be a tensor" % (where, name))
    s = t.shape
    if len(s) != n:
        raise ValueError("%s: %s must have %s dimensions, got shape %s" %
                         (where, name, ("no", "one", "two", "three", "four")[n], tuple(s)))
    return s


def _cuda(t, where, name):
    """The shape and device of the [rows, heads, head_dim] tensor that leads a call."""
    s = _dims(t, 3, where, name)
    if not t.is_cuda:
        raise ValueError("%s: %s must be a CUDA tensor" % (where, name))
    return s, t.device


_Strides = ctypes.c_int64 * 2
_strides = {}              # (token, head) strides -> the array that C takes


def _pair(row, head):
    a = _strides.get((row, head))
    if a is None:
        if len(_strides) > 512:
            _strides.clear()
        a = _strides[row, head] = _Strides(row, head)
    return a


def _new_heads(t, shape):
    """A new contiguous bf16 [rows, heads, head_dim] tensor beside t, and its strides."""
    return torch.empty_like(t, memory_format=torch.contiguous_format), _pair(shape[1] * shape[2], shape[2])


def _heads(t, shape, dev, where, name):
    """The (token, head) strides of a bf16 view with contiguous heads."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _BF16 or t.shape != shape or t.device != dev:
        _refuse(t, _BF16, shape, dev, where, name)
    row, head, one = t.stride()
    if one != 1 or (row | head) & 7 or t.data_ptr() & 15:
        raise ValueError("%s: %s needs a contiguous head_dim, strides that are multiples of 8 and a "
                         "16-byte aligned start" % (where, name))
    return _pair(row, head)


def _call(fn, dev, *args):
    """fn(*args, the current stream of dev) with dev current."""
    i = dev.index
    raw = _raw_stream(i) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream
    if _current_device() != i:
        with torch.cuda.device(dev):
            return fn(*args, raw)
    return fn(*args, raw)


def _on(stream, call, *args, **kw):
    """call(*args, **kw) with `stream` current.  What it allocates is that stream's memory (another
    stream's may still be in use there), and is not handed out again before the stream that was
    current is done with it."""
    dev = next((a.device for a in args if isinstance(a, torch.Tensor)), stream.device)
    _need(stream.device == dev, call.__name__, "the stream is of %s, the tensors are on %s" % (stream.device, dev))
    here = torch.cuda.current_stream(dev)
    with torch.cuda.stream(stream):
        out = call(*args, **kw)
    if here != stream:
        for t in out:
            if t is not None:
                t.record_stream(here)
    return out


def _at(t):
    return None if t is None else t.data_ptr()


def _rope_args(cos_sin, positions, pair_axis, total, dev, where, optional):
    """(cos_sin, max_position, rot_dim, positions, n_axes, pair_axis) as the C calls take them."""
    if cos_sin is None:
        _need(optional, where, "cos_sin is required")
        _need(positions is None and pair_axis is None, where, "positions and pair_axis need cos_sin")
        return None, 0, 0, None, 1, None
    rows, rot = _dims(cos_sin, 2, where, "cos_sin")
    _tensor(cos_sin, _F32, (rows, rot), dev, where, "cos_sin")
    axes = 1
    if positions is None:
        _need(optional, where, "positions is required")
    elif isinstance(positions, torch.Tensor) and positions.dim() == 1:
        _tensor(positions, _I32, (total,), dev, where, "positions")
    else:
        axes = _dims(positions, 2, where, "positions")[0]
        _tensor(positions, _I32, (axes, total), dev, where, "positions")
    if pair_axis is not None:
        _tensor(pair_axis, _I32, (rot // 2,), dev, where, "pair_axis")
    elif axes != 1:
        _need(False, where, "several axes need pair_axis")
    return cos_sin.data_ptr(), rows, rot, _at(positions), axes, _at(pair_axis)


def attn_rope(q, k=None, *, cos_sin, positions, pair_axis=None, interleaved=False, inverse=False,
              out_q=None, out_k=None, stream=None):
    """Rotates q [total, Hq, D] and k [total, Hkv, D] (bf16, strided views allowed) by their
    positions -> (q_out, k_out); k None gives (q_out, None).

    cos_sin: fp32 [max_position, rot_dim], cosines then sines; positions: int32 [total], or
    [n_axes, total] with pair_axis int32 [rot_dim / 2] naming each pair's axis.  interleaved
    pairs columns (2 i, 2 i + 1) in place of (i, i + rot_dim / 2).  inverse turns the other
    way: the gradient of the forward rotation.  out_q / out_k may be q / k themselves.
    """
    if stream is not None:
        return _on(stream, attn_rope, q, k, cos_sin=cos_sin, positions=positions, pair_axis=pair_axis,
                   interleaved=interleaved, inverse=inverse, out_q=out_q, out_k=out_k)
    where = "attn_rope"
    (total, Hq, D), dev = _cuda(q, where, "q")
    sq = _heads(q, (total, Hq, D), dev, where, "q")
    rope = _rope_args(cos_sin, positions, pair_axis, total, dev, where, False)
    if out_q is None:
        out_q, so = _new_heads(q, (total, Hq, D))
    else:
        so = _heads(out_q, (total, Hq, D), dev, where, "out_q")
    Hkv, sk, sko = 0, None, None
    if k is not None:
        Hkv = _dims(k, 3, where, "k")[1]
        sk = _heads(k, (total, Hkv, D), dev, where, "k")
        if out_k is None:
            out_k, sko = _new_heads(k, (total, Hkv, D))
        else:
            sko = _heads(out_k, (total, Hkv, D), dev, where, "out_k")
    else:
        _need(out_k is None, where, "out_k without k")
    if total == 0:
        return out_q, out_k
    st = _call(lib().attn_rope, dev, q.data_ptr(), out_q.data_ptr(), _at(k), _at(out_k), sq, so, sk, sko, total,
               Hq, Hkv, D, *rope, 1 if interleaved else 0, 1 if inverse else 0)
    _check(st, where)
    return out_q, out_k


def _append_args(q, k_new, v_new, block_table, seqused_k, cu_seqlens_new, seqused_k_out, out_q, q_dtype, where):
    (total, Hkv, D), dev = _cuda(k_new, where, "k_new")
    sk = _heads(k_new, (total, Hkv, D), dev, where, "k_new")
    sv = _heads(v_new, (total, Hkv, D), dev, where, "v_new")
    Hq, sq = 0, None
    if q is not None:
        Hq = _dims(q, 3, where, "q")[1]
        sq = _heads(q, (total, Hq, D), dev, where, "q")
        if out_q is None:
            out_q = torch.empty_like(q, dtype=q_dtype, memory_format=torch.contiguous_format)
        else:
            _tensor(out_q, q_dtype, (total, Hq, D), dev, where, "out_q")
            _need(out_q.data_ptr() % 16 == 0, where, "out_q must be 16-byte aligned")
    else:
        _need(out_q is None, where, "out_q without q")
    B = _dims(seqused_k, 1, where, "seqused_k")[0]
    _tensor(seqused_k, _I32, (B,), dev, where, "seqused_k")
    mbps = _dims(block_table, 2, where, "block_table")[1]
    _tensor(block_table, _I32, (B, mbps), dev, where, "block_table")
    if cu_seqlens_new is not None:
        _tensor(cu_seqlens_new, _I32, (B + 1,), dev, where, "cu_seqlens_new")
    else:
        _need(total == B, where, "without cu_seqlens_new there is one new token per sequence")
    if seqused_k_out is None:
        seqused_k_out = torch.empty_like(seqused_k)
    else:
        _tensor(seqused_k_out, _I32, (B,), dev, where, "seqused_k_out")
    return dev, total, Hq, Hkv, D, B, mbps, sq, sk, sv, out_q, seqused_k_out


def attn_kv_append_rope_paged(q, k_new, v_new, k_cache, v_cache, block_table, seqused_k, *, cos_sin=None,
                              positions=None, pair_axis=None, interleaved=False, cu_seqlens_new=None,
                              descale_q=None, descale_k=None, descale_v=None, out_q=None,
                              seqused_k_out=None, stream=None):
    """attn_kv_append_paged with the rotation of q and k (and for an e4m3 cache the
    quantisation) on the way -> (q_out [total_new, Hq, D] of the cache's type, the new lengths).

    q may be None (q_out is then None).  positions None: each token's position in the cache.
    """
    if stream is not None:
        return _on(stream, attn_kv_append_rope_paged, q, k_new, v_new, k_cache, v_cache, block_table, seqused_k,
                   cos_sin=cos_sin, positions=positions, pair_axis=pair_axis, interleaved=interleaved,
                   cu_seqlens_new=cu_seqlens_new, descale_q=descale_q, descale_k=descale_k,
                   descale_v=descale_v, out_q=out_q, seqused_k_out=seqused_k_out)
    where = "attn_kv_append_rope_paged"
    n, bs, _, _ = _dims(k_cache, 4, where, "k_cache")
    fp8 = k_cache.dtype is torch.float8_e4m3fn
    kind = torch.float8_e4m3fn if fp8 else _BF16
    dev, total, Hq, Hkv, D, B, mbps, sq, sk, sv, out_q, used = _append_args(
        q, k_new, v_new, block_table, seqused_k, cu_seqlens_new, seqused_k_out, out_q, kind, where)
    _tensor(k_cache, kind, (n, bs, Hkv, D), dev, where, "k_cache")
    _tensor(v_cache, kind, (n, bs, Hkv, D), dev, where, "v_cache")
    if fp8:
        for name, d in (("descale_k", descale_k), ("descale_v", descale_v), ("descale_q", descale_q)):
            if q is None and name == "descale_q":
                descale_q = None
                continue
            _need(isinstance(d, torch.Tensor) and d.numel() == 1, where, name + " must be a one-element tensor")
            _tensor(d, _F32, d.shape, dev, where, name)
    else:
        descale_q = descale_k = descale_v = None
    rope = _rope_args(cos_sin, positions, pair_axis, total, dev, where, True)
    if total == 0:
        return out_q, used.copy_(seqused_k)      # (an empty tensor has no address to pass)
    st = _call(lib().attn_kv_append_rope_paged, dev, _at(q), _at(out_q), k_new.data_ptr(), v_new.data_ptr(), sq, sk,
               sv, k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), mbps, n, bs, _at(cu_seqlens_new),
               seqused_k.data_ptr(), used.data_ptr(), B, total, Hq, Hkv, D, *rope, 1 if interleaved else 0,
               FP8_E4M3 if fp8 else BF16, _at(descale_q), _at(descale_k), _at(descale_v))
    _check(st, where)
    return out_q, used


def _q4_cache(k_cache, v_cache, k_meta, v_meta, dev, where):
    """Checks a 4-bit cache -> (num_blocks, block_size, Hkv, D, group_size)."""
    s = _dims(k_cache, 4, where, "k_cache")
    n, h, bs, half = s
    _tensor(k_cache, _U8, s, dev, where, "k_cache")
    _tensor(v_cache, _U8, s, dev, where, "v_cache")
    G = _dims(k_meta, 4, where, "k_meta")[3]
    _tensor(k_meta, _I16, (n, h, bs, G), dev, where, "k_meta")
    _tensor(v_meta, _I16, (n, h, bs, G), dev, where, "v_meta")
    if G < 1 or 2 * half % G:
        _need(False, where, "head_dim must be a multiple of the metas per token")
    return n, bs, h, 2 * half, 2 * half // G


def attn_kv_append_paged_q4(q, k_new, v_new, k_cache, v_cache, k_meta, v_meta, block_table, seqused_k, *,
                            cos_sin=None, positions=None, pair_axis=None, interleaved=False,
                            cu_seqlens_new=None, out_q=None, seqused_k_out=None, stream=None):
    """Appends new tokens to a 4-bit cache, rotating q and k on the way (cos_sin None: no
    rotation) -> (q_out [total_new, Hq, D] bf16 or None, the new lengths).

    k_cache / v_cache: uint8 [num_blocks, Hkv, 16, D / 2]; k_meta / v_meta: int16
    [num_blocks, Hkv, 16, D / group_size], group_size 32, 64 or 128 (the format is described
    in the header).
    """
    if stream is not None:
        return _on(stream, attn_kv_append_paged_q4, q, k_new, v_new, k_cache, v_cache, k_meta, v_meta, block_table,
                   seqused_k, cos_sin=cos_sin, positions=positions, pair_axis=pair_axis, interleaved=interleaved,
                   cu_seqlens_new=cu_seqlens_new, out_q=out_q, seqused_k_out=seqused_k_out)
    where = "attn_kv_append_paged_q4"
    dev, total, Hq, Hkv, D, B, mbps, sq, sk, sv, out_q, used = _append_args(
        q, k_new, v_new, block_table, seqused_k, cu_seqlens_new, seqused_k_out, out_q, _BF16, where)
    n, bs, h, Dc, gs = _q4_cache(k_cache, v_cache, k_meta, v_meta, dev, where)
    if h != Hkv or Dc != D:
        _need(False, where, "k_new and the cache have different heads")
    rope = _rope_args(cos_sin, positions, pair_axis, total, dev, where, True)
    if total == 0:
        return out_q, used.copy_(seqused_k)      # (an empty tensor has no address to pass)
    st = _call(lib().attn_kv_append_paged_q4, dev, _at(q), _at(out_q), k_new.data_ptr(), v_new.data_ptr(), sq, sk,
               sv, k_cache.data_ptr(), v_cache.data_ptr(), k_meta.data_ptr(), v_meta.data_ptr(), block_table.data_ptr(),
               mbps, n, bs, _at(cu_seqlens_new), seqused_k.data_ptr(), used.data_ptr(), B, total, Hq, Hkv, D, gs, *rope,
               1 if interleaved else 0)
    _check(st, where)
    return out_q, used


def attn_kv_gather_paged_q4(k_cache, v_cache, k_meta, v_meta, block_table, cu_seqlens, total, *, starts=None,
                            out_k=None, out_v=None, stream=None):
    """Reads tokens of a 4-bit cache back -> packed (k, v) [total, Hkv, D] bf16, exactly.

    Sequence b's tokens starts[b] .. (None: 0 ..) go to rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1.
    """
    if stream is not None:
        return _on(stream, attn_kv_gather_paged_q4, k_cache, v_cache, k_meta, v_meta, block_table, cu_seqlens, total,
                   starts=starts, out_k=out_k, out_v=out_v)
    where = "attn_kv_gather_paged_q4"
    B = _dims(cu_seqlens, 1, where, "cu_seqlens")[0] - 1
    _need(B >= 0 and cu_seqlens.is_cuda, where, "cu_seqlens must be a CUDA tensor of B + 1 entries")
    dev = cu_seqlens.device
    _tensor(cu_seqlens, _I32, (B + 1,), dev, where, "cu_seqlens")
    n, bs, Hkv, D, gs = _q4_cache(k_cache, v_cache, k_meta, v_meta, dev, where)
    mbps = _dims(block_table, 2, where, "block_table")[1]
    _tensor(block_table, _I32, (B, mbps), dev, where, "block_table")
    if starts is not None:
        _tensor(starts, _I32, (B,), dev, where, "starts")
    total = int(total)
    shape = (total, Hkv, D)
    if out_k is None:
        out_k = torch.empty(shape, dtype=_BF16, device=dev)
    else:
        _tensor(out_k, _BF16, shape, dev, where, "out_k")
    if out_v is None:
        out_v = torch.empty_like(out_k)
    else:
        _tensor(out_v, _BF16, shape, dev, where, "out_v")
    if total == 0:
        return out_k, out_v
    st = _call(lib().attn_kv_gather_paged_q4, dev, k_cache.data_ptr(), v_cache.data_ptr(), k_meta.data_ptr(),
               v_meta.data_ptr(), block_table.data_ptr(), mbps, n, bs, cu_seqlens.data_ptr(), _at(starts), B, total, Hkv,
               D, gs, out_k.data_ptr(), out_v.data_ptr())
    _check(st, where)
    return out_k, out_v


def attn_decode_q4_workspace_size(B, num_heads_q, num_heads_kv, head_dim) -> int:
    return lib().attn_decode_q4_workspace_size(B, num_heads_q, num_heads_kv, head_dim)


def attn_fwd_q4_workspace_size(B, max_seqlen_q, num_heads_q, num_heads_kv, head_dim, total_k) -> int:
    return lib().attn_fwd_q4_workspace_size(B, max_seqlen_q, num_heads_q, num_heads_kv, head_dim, total_k)


def _outputs(q, out, lse, lse_shape, return_lse, dev, where):
    _tensor(q, _BF16, q.shape, dev, where, "q")
    if out is None:
        out = torch.empty_like(q)
    else:
        _tensor(out, _BF16, q.shape, dev, where, "out")
    if lse is not None:
        _tensor(lse, _F32, lse_shape, dev, where, "lse")
    elif return_lse:
        lse = q.new_empty(lse_shape, dtype=_F32)
    return out, lse


def _space(workspace, need, q, dev, where):
    if workspace is None:
        return q.new_empty((max(need, 16),), dtype=_U8)
    _tensor(workspace, _U8, _dims(workspace, 1, where, "workspace"), dev, where, "workspace")
    return workspace


def attn_decode_paged_q4(q, k_cache, v_cache, k_meta, v_meta, block_table, seqused_k, *, scale=None,
                         window_left=-1, softcap=0.0, out=None, lse=None, workspace=None,
                         return_lse=True, stream=None):
    """attn_decode_paged over a 4-bit cache: q [B, Hq, D] bf16 -> (o [B, Hq, D] bf16, lse [B, Hq] fp32)."""
    if stream is not None:
        return _on(stream, attn_decode_paged_q4, q, k_cache, v_cache, k_meta, v_meta, block_table, seqused_k,
                   scale=scale, window_left=window_left, softcap=softcap, out=out, lse=lse,
                   workspace=workspace, return_lse=return_lse)
    where = "attn_decode_paged_q4"
    (B, Hq, D), dev = _cuda(q, where, "q")
    n, bs, Hkv, Dc, gs = _q4_cache(k_cache, v_cache, k_meta, v_meta, dev, where)
    if Dc != D:
        _need(False, where, "q and the cache have different head_dims")
    mbps = _dims(block_table, 2, where, "block_table")[1]
    _tensor(block_table, _I32, (B, mbps), dev, where, "block_table")
    _tensor(seqused_k, _I32, (B,), dev, where, "seqused_k")
    out, lse = _outputs(q, out, lse, (B, Hq), return_lse, dev, where)
    if B == 0:
        return out, lse
    L = lib()
    workspace = _space(workspace, L.attn_decode_q4_workspace_size(B, Hq, Hkv, D), q, dev, where)
    st = _call(L.attn_decode_paged_q4, dev, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
               k_meta.data_ptr(), v_meta.data_ptr(), block_table.data_ptr(), mbps, n, bs, seqused_k.data_ptr(), B, Hq, Hkv,
               D, gs, _scale(scale), int(window_left), float(softcap), out.data_ptr(), _at(lse), workspace.data_ptr(),
               workspace.numel())
    _check(st, where)
    return out, lse


def attn_fwd_varlen_paged_q4(q, k_cache, v_cache, k_meta, v_meta, *, block_table, cu_seqlens_q, max_seqlen_q,
                             seqused_k, total_k, mask=MASK_NONE, scale=None, window_left=-1, softcap=0.0,
                             out=None, lse=None, workspace=None, return_lse=True, stream=None):
    """attn_fwd_varlen_paged over a 4-bit cache: packed q [total_q, Hq, D] bf16, the newest of
    each sequence's seqused_k tokens -> (o [total_q, Hq, D] bf16, lse [Hq, total_q] fp32).

    total_k: at least the sum of seqused_k (rows of the workspace); mask NONE or CAUSAL.
    """
    if stream is not None:
        return _on(stream, attn_fwd_varlen_paged_q4, q, k_cache, v_cache, k_meta, v_meta,
                   block_table=block_table, cu_seqlens_q=cu_seqlens_q, max_seqlen_q=max_seqlen_q,
                   seqused_k=seqused_k, total_k=total_k, mask=mask, scale=scale, window_left=window_left,
                   softcap=softcap, out=out, lse=lse, workspace=workspace, return_lse=return_lse)
    where = "attn_fwd_varlen_paged_q4"
    (total_q, Hq, D), dev = _cuda(q, where, "q")
    B = _dims(seqused_k, 1, where, "seqused_k")[0]
    _tensor(seqused_k, _I32, (B,), dev, where, "seqused_k")
    _tensor(cu_seqlens_q, _I32, (B + 1,), dev, where, "cu_seqlens_q")
    n, bs, Hkv, Dc, gs = _q4_cache(k_cache, v_cache, k_meta, v_meta, dev, where)
    if Dc != D:
        _need(False, where, "q and the cache have different head_dims")
    mbps = _dims(block_table, 2, where, "block_table")[1]
    _tensor(block_table, _I32, (B, mbps), dev, where, "block_table")
    out, lse = _outputs(q, out, lse, (Hq, total_q), return_lse, dev, where)
    if total_q == 0:
        return out, lse
    L, most, total_k = lib(), int(max_seqlen_q), int(total_k)
    workspace = _space(workspace, L.attn_fwd_q4_workspace_size(B, most, Hq, Hkv, D, total_k), q, dev, where)
    st = _call(L.attn_fwd_varlen_paged_q4, dev, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
               k_meta.data_ptr(), v_meta.data_ptr(), block_table.data_ptr(), mbps, n, bs, cu_seqlens_q.data_ptr(),
               seqused_k.data_ptr(), B, total_q, total_k, most, Hq, Hkv, D, gs, _scale(scale), int(mask),
               int(window_left), float(softcap), out.data_ptr(), _at(lse), workspace.data_ptr(), workspace.numel())
    _check(st, where)
    return out, lse

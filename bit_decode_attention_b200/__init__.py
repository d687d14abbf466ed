"""bit_decode_attention_b200 -- NVFP4 KV cache with fused NVFP4 -> FP8 decode
attention for NVIDIA B200 (sm_100a).

Thin Python binding over the C ABI of libnvfp4kv.so (include/nvfp4kv.h).
The functions below carry the C names and only marshal arguments: torch
tensors supply device memory and the current CUDA stream, every step of the
computation runs in the library's kernels.  There is no CPU path.

Formats and flow follow "NVIDIA解説: NVFP4 KV Cacheで長コンテキストLLM推論を最適化"
(sections "E2M1 + 2レベルスケーリング" and "量子化・逆量子化フロー").
"""
from __future__ import annotations

import contextlib
import ctypes
import dataclasses
from typing import Optional

import torch

from . import _native
from ._native import (NVFP4_ERR_CAPACITY, NVFP4_ERR_INVALID_ARG, NVFP4_ERR_NONFINITE,  # noqa: F401
                      NVFP4_ERR_TIMEOUT, NVFP4_ERR_UNSUPPORTED, NVFP4_ERR_WORKSPACE, NVFP4_OK,
                      NativeError)

__all__ = [
    "KVPlane", "nvfp4_cache_bytes", "nvfp4_calib_tensor_scale", "nvfp4_kv_quantize_append",
    "nvfp4_kv_quantize_append_kv",
    "nvfp4_kv_dequant_fp8", "nvfp4_decode_attention_workspace", "nvfp4_decode_attention",
    "nvfp4_version", "NativeError", "nvfp4_decode_attention_noalloc",
    "mxfp4_cache_bytes", "mxfp4_kv_quantize_append",
    "PagedKVPlane", "nvfp4_kv_quantize_append_paged", "nvfp4_decode_attention_paged",
    "nvfp4_prefill_attention", "nvfp4_decode_attention_append", "nvfp4_set_wait_limit",
    "nvfp4_qk_norm_rope_append", "nvfp4_qk_norm_rope_append_paged", "nvfp4_tree_attention_workspace",
    "nvfp4_tree_attention", "nvfp4_tree_attention_paged", "nvfp4_verify_drafts",
    "KVPlaneList", "nvfp4_kv_commit_path", "nvfp4_kv_commit_path_paged",
]


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    # the handle of torch.cuda.current_stream(), without building a Stream object
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return _native.NVFP4_IN_BF16
    if t.dtype == torch.float32:
        return _native.NVFP4_IN_F32
    raise TypeError("inputs must be bfloat16 or float32, got %s" % t.dtype)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


@dataclasses.dataclass
class KVPlane:
    """One NVFP4 cache plane (K or V) in device memory.

    codes  uint8 [B][H_kv][S_max][D/2]  (element 2j low nibble of byte j)
    scales uint8 [B][H_kv][S_max][D/16] (one E4M3 byte per 16 elements)
    """
    codes: torch.Tensor
    scales: torch.Tensor

    @classmethod
    def allocate(cls, B: int, H_kv: int, S_max: int, D: int, device="cuda") -> "KVPlane":
        codes = torch.zeros(B, H_kv, S_max, D // 2, dtype=torch.uint8, device=device)
        scales = torch.zeros(B, H_kv, S_max, D // 16, dtype=torch.uint8, device=device)
        return cls(codes, scales)

    @classmethod
    def allocate_mxfp4(cls, B: int, H_kv: int, S_max: int, D: int, device="cuda") -> "KVPlane":
        """An MXFP4 plane: the same codes, scales uint8 [B][H_kv][S_max][D/32] (E8M0)."""
        codes = torch.zeros(B, H_kv, S_max, D // 2, dtype=torch.uint8, device=device)
        scales = torch.zeros(B, H_kv, S_max, D // 32, dtype=torch.uint8, device=device)
        return cls(codes, scales)

    @property
    def shape(self):
        B, H, S, Dh = self.codes.shape
        return B, H, S, 2 * Dh

    def struct(self) -> _native.KVPlaneStruct:
        B, H, S, D = self.shape
        return _native.KVPlaneStruct(self.codes.data_ptr(), self.scales.data_ptr(), B, H, S, D)


@dataclasses.dataclass
class PagedKVPlane:
    """One paged NVFP4 cache plane: a page pool and the block table.

    codes       uint8 [num_pages][H_kv][page_tokens][D/2]
    scales      uint8 [num_pages][H_kv][page_tokens][D/16]
    block_table int32 [B][max_pages]; token t of sequence b lives in page
                block_table[b][t // page_tokens], slot t % page_tokens
    K and V planes of one cache share the block table.
    """
    codes: torch.Tensor
    scales: torch.Tensor
    block_table: torch.Tensor

    @classmethod
    def allocate(cls, num_pages: int, H_kv: int, page_tokens: int, D: int, block_table: torch.Tensor,
                 device="cuda") -> "PagedKVPlane":
        codes = torch.zeros(num_pages, H_kv, page_tokens, D // 2, dtype=torch.uint8, device=device)
        scales = torch.zeros(num_pages, H_kv, page_tokens, D // 16, dtype=torch.uint8, device=device)
        return cls(codes, scales, block_table)

    def struct(self) -> _native.PagedPlaneStruct:
        P, H, T, Dh = self.codes.shape
        B, M = self.block_table.shape
        return _native.PagedPlaneStruct(self.codes.data_ptr(), self.scales.data_ptr(),
                                        self.block_table.data_ptr(), P, H, T, 2 * Dh, B, M)


def nvfp4_version() -> str:
    return _native.lib().nvfp4_version().decode()


def nvfp4_set_wait_limit(polls: int) -> None:
    """Testing hook: pipeline-wait give-up limit of the tensor-core attention
    kernel (sleeping polls; 0 = give up unless already complete; < 0 = default)."""
    _native.lib().nvfp4_set_wait_limit(int(polls))


def nvfp4_cache_bytes(B: int, H_kv: int, S_max: int, D: int) -> int:
    return int(_native.lib().nvfp4_cache_bytes(B, H_kv, S_max, D))


def nvfp4_calib_tensor_scale(x: torch.Tensor, s_tensor: Optional[torch.Tensor] = None,
                             status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Per-tensor scale fl32(amax / 2688) as a 1-element device float tensor."""
    _need_cuda(x)
    if s_tensor is None:
        s_tensor = torch.empty(1, dtype=torch.float32, device=x.device)
    st = _native.lib().nvfp4_calib_tensor_scale(_ptr(x), _dtype_code(x), x.numel(), _ptr(s_tensor),
                                                _ptr(status), _stream(stream))
    _native.check("nvfp4_calib_tensor_scale", st)
    return s_tensor


def nvfp4_kv_quantize_append(x_new: torch.Tensor, start_pos: torch.Tensor, s_tensor: torch.Tensor,
                             plane: KVPlane, new_lens: Optional[torch.Tensor] = None,
                             status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Quantize x_new [B][n_new][H_kv][D] and write it at slots start_pos[b]... of `plane`."""
    _need_cuda(x_new, start_pos, s_tensor, new_lens, status)
    n_new = x_new.shape[1]
    pl = plane.struct()
    st = _native.lib().nvfp4_kv_quantize_append(_ptr(x_new), _dtype_code(x_new), n_new,
                                                _ptr(start_pos), _ptr(new_lens), _ptr(s_tensor),
                                                ctypes.byref(pl), _ptr(status), _stream(stream))
    _native.check("nvfp4_kv_quantize_append", st)


def nvfp4_kv_quantize_append_paged(x_new: torch.Tensor, start_pos: torch.Tensor, s_tensor: torch.Tensor,
                                   plane: PagedKVPlane, new_lens: Optional[torch.Tensor] = None,
                                   status: Optional[torch.Tensor] = None, stream=None) -> None:
    """nvfp4_kv_quantize_append into a paged plane (slots found through its block table)."""
    _need_cuda(x_new, start_pos, s_tensor, new_lens, status, plane.block_table)
    pl = plane.struct()
    st = _native.lib().nvfp4_kv_quantize_append_paged(_ptr(x_new), _dtype_code(x_new), x_new.shape[1],
                                                      _ptr(start_pos), _ptr(new_lens), _ptr(s_tensor),
                                                      ctypes.byref(pl), _ptr(status), _stream(stream))
    _native.check("nvfp4_kv_quantize_append_paged", st)


def nvfp4_kv_quantize_append_kv(x_k: torch.Tensor, x_v: torch.Tensor, start_pos: torch.Tensor,
                                s_tensor_k: torch.Tensor, s_tensor_v: torch.Tensor, k: KVPlane, v: KVPlane,
                                new_lens: Optional[torch.Tensor] = None,
                                status: Optional[torch.Tensor] = None, stream=None) -> None:
    """nvfp4_kv_quantize_append for K into `k` and V into `v` in one launch."""
    _need_cuda(x_k, x_v, start_pos, s_tensor_k, s_tensor_v, new_lens, status)
    if x_k.shape != x_v.shape or x_k.dtype != x_v.dtype:
        raise ValueError("x_k and x_v must have the same shape and dtype")
    n_new = x_k.shape[1]
    pk, pv = k.struct(), v.struct()
    st = _native.lib().nvfp4_kv_quantize_append_kv(_ptr(x_k), _ptr(x_v), _dtype_code(x_k), n_new,
                                                   _ptr(start_pos), _ptr(new_lens), _ptr(s_tensor_k),
                                                   _ptr(s_tensor_v), ctypes.byref(pk), ctypes.byref(pv),
                                                   _ptr(status), _stream(stream))
    _native.check("nvfp4_kv_quantize_append_kv", st)


def mxfp4_cache_bytes(B: int, H_kv: int, S_max: int, D: int) -> int:
    return int(_native.lib().mxfp4_cache_bytes(B, H_kv, S_max, D))


def mxfp4_kv_quantize_append(x_new: torch.Tensor, start_pos: torch.Tensor, plane: KVPlane,
                             new_lens: Optional[torch.Tensor] = None,
                             status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Quantize x_new [B][n_new][H_kv][D] to MXFP4 (32-element blocks, E8M0
    scales) and write it at slots start_pos[b]... of an MXFP4 `plane`."""
    _need_cuda(x_new, start_pos, new_lens, status)
    B, H, S, D = plane.shape
    if plane.scales.shape[-1] != D // 32:
        raise ValueError("an MXFP4 plane holds D/32 scale bytes per token (KVPlane.allocate_mxfp4)")
    pl = plane.struct()
    st = _native.lib().mxfp4_kv_quantize_append(_ptr(x_new), _dtype_code(x_new), x_new.shape[1],
                                                _ptr(start_pos), _ptr(new_lens), ctypes.byref(pl),
                                                _ptr(status), _stream(stream))
    _native.check("mxfp4_kv_quantize_append", st)


def nvfp4_kv_dequant_fp8(plane: KVPlane, s_tensor: torch.Tensor, seq_lens: torch.Tensor,
                         out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """E4M3 bytes [B][H_kv][S_max][D] for the first seq_lens[b] slots."""
    _need_cuda(s_tensor, seq_lens, out, status)
    B, H, S, D = plane.shape
    if out is None:
        out = torch.zeros(B, H, S, D, dtype=torch.uint8, device=plane.codes.device)
    pl = plane.struct()
    st = _native.lib().nvfp4_kv_dequant_fp8(ctypes.byref(pl), _ptr(s_tensor), _ptr(seq_lens),
                                            _ptr(out), _ptr(status), _stream(stream))
    _native.check("nvfp4_kv_dequant_fp8", st)
    return out


def nvfp4_decode_attention_workspace(B: int, H_q: int, H_kv: int, D: int) -> int:
    return int(_native.lib().nvfp4_decode_attention_workspace(B, H_q, H_kv, D))


def new_workspace(B: int, H_q: int, H_kv: int, D: int, device="cuda") -> torch.Tensor:
    """Zero-filled workspace for nvfp4_decode_attention (reusable across calls)."""
    n = nvfp4_decode_attention_workspace(B, H_q, H_kv, D)
    if n == 0:
        raise ValueError("unsupported attention shape")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def nvfp4_prefill_attention(q: torch.Tensor, k: KVPlane, v: KVPlane, s_tensor_k: torch.Tensor,
                            s_tensor_v: torch.Tensor, start_pos: torch.Tensor, softmax_scale: float = 0.0,
                            out: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """Causal attention of a prompt chunk over the NVFP4 cache (the chunk's K/V
    already appended at start_pos); q [B][C][H_q][128] -> fp32 [B][C][H_q][128]."""
    _need_cuda(q, s_tensor_k, s_tensor_v, start_pos, out, status)
    B, C, H_q, D = q.shape
    if out is None:
        out = torch.empty(B, C, H_q, D, dtype=torch.float32, device=q.device)
    kp, vp = k.struct(), v.struct()
    st = _native.lib().nvfp4_prefill_attention(
        _ptr(q), _dtype_code(q), C, H_q, ctypes.byref(kp), ctypes.byref(vp), _ptr(s_tensor_k),
        _ptr(s_tensor_v), _ptr(start_pos), ctypes.c_float(softmax_scale), _ptr(out), _ptr(status),
        _stream(stream))
    _native.check("nvfp4_prefill_attention", st)
    return out


def nvfp4_decode_attention(q: torch.Tensor, k: KVPlane, v: KVPlane, s_tensor_k: torch.Tensor,
                           s_tensor_v: torch.Tensor, seq_lens: torch.Tensor,
                           softmax_scale: float = 0.0, out: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None,
                           status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """softmax(q K^T * scale) V over the NVFP4 cache; q [B][H_q][D] -> fp32 [B][H_q][D]."""
    _need_cuda(q, s_tensor_k, s_tensor_v, seq_lens, out, workspace, status)
    B, H_q, D = q.shape
    Bk, H_kv, S, Dk = k.shape
    if out is None:
        out = torch.empty(B, H_q, D, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = new_workspace(B, H_q, H_kv, D, device=q.device)
    kp, vp = k.struct(), v.struct()
    st = _native.lib().nvfp4_decode_attention(
        _ptr(q), _dtype_code(q), H_q, ctypes.byref(kp), ctypes.byref(vp), _ptr(s_tensor_k),
        _ptr(s_tensor_v), _ptr(seq_lens), ctypes.c_float(softmax_scale), _ptr(out),
        _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream))
    _native.check("nvfp4_decode_attention", st)
    return out


def nvfp4_decode_attention_append(q: torch.Tensor, x_k_new: torch.Tensor, x_v_new: torch.Tensor,
                                  start_pos: torch.Tensor, k: KVPlane, v: KVPlane, s_tensor_k: torch.Tensor,
                                  s_tensor_v: torch.Tensor, softmax_scale: float = 0.0,
                                  out: Optional[torch.Tensor] = None, new_lens: Optional[torch.Tensor] = None,
                                  workspace: Optional[torch.Tensor] = None,
                                  status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Append one token per sequence (x_k_new / x_v_new [B][1][H_kv][D]) at slot
    start_pos[b], then attend over start_pos[b] + 1 tokens; fp32 [B][H_q][D]."""
    _need_cuda(q, x_k_new, x_v_new, start_pos, s_tensor_k, s_tensor_v, out, new_lens, workspace, status)
    if x_k_new.shape != x_v_new.shape or x_k_new.dtype != x_v_new.dtype:
        raise ValueError("x_k_new and x_v_new must have the same shape and dtype")
    B, H_q, D = q.shape
    Bk, H_kv, S, Dk = k.shape
    if tuple(x_k_new.shape) != (Bk, 1, H_kv, Dk):
        raise ValueError("x_k_new must be [B][1][H_kv][D]")
    if out is None:
        out = torch.empty(B, H_q, D, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = new_workspace(B, H_q, H_kv, D, device=q.device)
    kp, vp = k.struct(), v.struct()
    st = _native.lib().nvfp4_decode_attention_append(
        _ptr(q), _dtype_code(q), H_q, _ptr(x_k_new), _ptr(x_v_new), _dtype_code(x_k_new), _ptr(start_pos),
        _ptr(new_lens), ctypes.byref(kp), ctypes.byref(vp), _ptr(s_tensor_k), _ptr(s_tensor_v),
        ctypes.c_float(softmax_scale), _ptr(out), _ptr(workspace), workspace.numel(), _ptr(status),
        _stream(stream))
    _native.check("nvfp4_decode_attention_append", st)
    return out


def nvfp4_decode_attention_paged(q: torch.Tensor, k: PagedKVPlane, v: PagedKVPlane,
                                 s_tensor_k: torch.Tensor, s_tensor_v: torch.Tensor,
                                 seq_lens: torch.Tensor, softmax_scale: float = 0.0,
                                 out: Optional[torch.Tensor] = None,
                                 workspace: Optional[torch.Tensor] = None,
                                 status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """nvfp4_decode_attention over paged K/V planes that share one block table."""
    _need_cuda(q, s_tensor_k, s_tensor_v, seq_lens, out, workspace, status, k.block_table)
    B, H_q, D = q.shape
    H_kv = k.codes.shape[1]
    if out is None:
        out = torch.empty(B, H_q, D, dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = new_workspace(B, H_q, H_kv, D, device=q.device)
    kp, vp = k.struct(), v.struct()
    st = _native.lib().nvfp4_decode_attention_paged(
        _ptr(q), _dtype_code(q), H_q, ctypes.byref(kp), ctypes.byref(vp), _ptr(s_tensor_k),
        _ptr(s_tensor_v), _ptr(seq_lens), ctypes.c_float(softmax_scale), _ptr(out),
        _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream))
    _native.check("nvfp4_decode_attention_paged", st)
    return out


def nvfp4_decode_attention_noalloc(q: torch.Tensor, k: KVPlane, v: KVPlane, s_tensor_k: torch.Tensor,
                                   s_tensor_v: torch.Tensor, seq_lens: torch.Tensor,
                                   softmax_scale: float = 0.0, out: Optional[torch.Tensor] = None,
                                   status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """nvfp4_decode_attention without a workspace, for callers that may not
    allocate device memory: scratch is the library's built-in device buffer
    (shared by all calls on a device; calls must not overlap on the GPU)."""
    _need_cuda(q, s_tensor_k, s_tensor_v, seq_lens, out, status)
    B, H_q, D = q.shape
    if out is None:
        out = torch.empty(B, H_q, D, dtype=torch.float32, device=q.device)
    kp, vp = k.struct(), v.struct()
    st = _native.lib().nvfp4_decode_attention_noalloc(
        _ptr(q), _dtype_code(q), H_q, ctypes.byref(kp), ctypes.byref(vp), _ptr(s_tensor_k),
        _ptr(s_tensor_v), _ptr(seq_lens), ctypes.c_float(softmax_scale), _ptr(out), _ptr(status),
        _stream(stream))
    _native.check("nvfp4_decode_attention_noalloc", st)
    return out


# ---------------------------------------------------------------------------
# a step of tree-drafted decoding
# ---------------------------------------------------------------------------
def _target(stream):
    """(current device, stream handle) of a call."""
    cur = torch.cuda.current_device()
    return cur, stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(cur)


def _need_kind(k, v, kind):
    if type(k) is not kind or type(v) is not kind:
        raise TypeError("k and v must be %s" % kind.__name__)


def _allocating(stream):
    """Tensors that a call makes for itself are made on its stream: filled there before
    its kernels, and not given to another stream's work while they run."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _like_rows(x: torch.Tensor, dtype, stream) -> torch.Tensor:
    """A dense output like x, zeros: rows behind a sequence's count, and rows of a sequence
    or token that the kernel refuses, are not written."""
    with _allocating(stream):
        return torch.zeros(x.shape, dtype=dtype, device=x.device)


def _qk_norm_rope_append(func, kind, x_q, x_k, x_v, start_pos, s_tensor_k, s_tensor_v, k, v, w_q, w_k, eps, rope_table,
                         interleaved, positions, n_valid, q_out, new_lens, status, stream):
    _need_kind(k, v, kind)
    if q_out is None:
        q_out = _like_rows(x_q, x_q.dtype, stream)
    st = _native.binding().qk_norm_rope_append(
        *_target(stream), kind is PagedKVPlane, x_q, x_k, x_v, start_pos, s_tensor_k, s_tensor_v, k, v, w_q, w_k, eps,
        rope_table, interleaved, positions, n_valid, q_out, new_lens, status)
    if st:
        _native.check(func, st)
    return q_out


def nvfp4_qk_norm_rope_append(x_q: torch.Tensor, x_k: torch.Tensor, x_v: torch.Tensor, start_pos: torch.Tensor,
                              s_tensor_k: torch.Tensor, s_tensor_v: torch.Tensor, k: KVPlane, v: KVPlane,
                              w_q: Optional[torch.Tensor] = None, w_k: Optional[torch.Tensor] = None,
                              eps: float = 1e-6, rope_table: Optional[torch.Tensor] = None,
                              interleaved: bool = False, positions: Optional[torch.Tensor] = None,
                              n_valid: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                              new_lens: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                              stream=None) -> torch.Tensor:
    """RMS norm of each query and key head (eps < 0: none), rotation by the rows
    of rope_table [P][R] (R/2 cosines, R/2 sines; None: none), K and V quantized
    into the cache at slots start_pos[b] + i; returns the queries [B][n][H_q][D].
    x_q, x_k, x_v [B][n][heads][D] may be slices of one packed projection.  Rows
    that are not computed (padding, refused ones) are zero where q_out is None."""
    return _qk_norm_rope_append("nvfp4_qk_norm_rope_append", KVPlane, x_q, x_k, x_v, start_pos, s_tensor_k, s_tensor_v,
                                k, v, w_q, w_k, eps, rope_table, interleaved, positions, n_valid, q_out, new_lens,
                                status, stream)


def nvfp4_qk_norm_rope_append_paged(x_q: torch.Tensor, x_k: torch.Tensor, x_v: torch.Tensor, start_pos: torch.Tensor,
                                    s_tensor_k: torch.Tensor, s_tensor_v: torch.Tensor, k: PagedKVPlane,
                                    v: PagedKVPlane, w_q: Optional[torch.Tensor] = None,
                                    w_k: Optional[torch.Tensor] = None, eps: float = 1e-6,
                                    rope_table: Optional[torch.Tensor] = None, interleaved: bool = False,
                                    positions: Optional[torch.Tensor] = None, n_valid: Optional[torch.Tensor] = None,
                                    q_out: Optional[torch.Tensor] = None, new_lens: Optional[torch.Tensor] = None,
                                    status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """nvfp4_qk_norm_rope_append into paged planes that share one block table."""
    return _qk_norm_rope_append("nvfp4_qk_norm_rope_append_paged", PagedKVPlane, x_q, x_k, x_v, start_pos, s_tensor_k,
                                s_tensor_v, k, v, w_q, w_k, eps, rope_table, interleaved, positions, n_valid, q_out,
                                new_lens, status, stream)


def nvfp4_tree_attention_workspace(B: int, N: int, H_q: int, H_kv: int, D: int) -> int:
    return int(_native.lib().nvfp4_tree_attention_workspace(B, N, H_q, H_kv, D))


def _tree_attention(func, kind, q, k, v, s_tensor_k, s_tensor_v, start_pos, tree_mask, n_nodes, softmax_scale, out,
                    out_dtype, workspace, status, stream):
    _need_kind(k, v, kind)
    if out is None:
        out = _like_rows(q, out_dtype, stream)
    if workspace is None:
        B, N, H_q, D = q.shape
        size = nvfp4_tree_attention_workspace(B, N, H_q, k.codes.shape[1], D)
        if size == 0:
            raise ValueError("unsupported attention shape")
        with _allocating(stream):
            workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
    st = _native.binding().tree_attention(
        *_target(stream), kind is PagedKVPlane, q, k, v, s_tensor_k, s_tensor_v, start_pos, tree_mask, n_nodes,
        softmax_scale, out, workspace, status)
    if st:
        _native.check(func, st)
    return out


def nvfp4_tree_attention(q: torch.Tensor, k: KVPlane, v: KVPlane, s_tensor_k: torch.Tensor, s_tensor_v: torch.Tensor,
                         start_pos: torch.Tensor, tree_mask: Optional[torch.Tensor] = None,
                         n_nodes: Optional[torch.Tensor] = None, softmax_scale: float = 0.0,
                         out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.float32,
                         workspace: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """Attention of a tree's N nodes (K/V appended at start_pos[b] + i) over the
    cache; q [B][N][H_q][D] bf16 -> [B][N][H_q][D] of out_dtype.  tree_mask int32
    [N][ceil(N/32)] or [B][N][ceil(N/32)]: bit j of row i lets node i see node j
    (None: a chain, j <= i).  Rows that are not computed (padding, refused
    sequences) are zero where out is None."""
    return _tree_attention("nvfp4_tree_attention", KVPlane, q, k, v, s_tensor_k, s_tensor_v, start_pos, tree_mask,
                           n_nodes, softmax_scale, out, out_dtype, workspace, status, stream)


def nvfp4_tree_attention_paged(q: torch.Tensor, k: PagedKVPlane, v: PagedKVPlane, s_tensor_k: torch.Tensor,
                               s_tensor_v: torch.Tensor, start_pos: torch.Tensor,
                               tree_mask: Optional[torch.Tensor] = None, n_nodes: Optional[torch.Tensor] = None,
                               softmax_scale: float = 0.0, out: Optional[torch.Tensor] = None,
                               out_dtype: torch.dtype = torch.float32, workspace: Optional[torch.Tensor] = None,
                               status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """nvfp4_tree_attention over paged planes that share one block table."""
    return _tree_attention("nvfp4_tree_attention_paged", PagedKVPlane, q, k, v, s_tensor_k, s_tensor_v, start_pos,
                           tree_mask, n_nodes, softmax_scale, out, out_dtype, workspace, status, stream)


def nvfp4_verify_drafts(target_probs: torch.Tensor, draft_probs: Optional[torch.Tensor], tokens: torch.Tensor,
                        parents: torch.Tensor, u_accept: torch.Tensor, u_sample: torch.Tensor,
                        n_nodes: Optional[torch.Tensor] = None, path: Optional[torch.Tensor] = None,
                        n_accepted: Optional[torch.Tensor] = None, next_token: Optional[torch.Tensor] = None,
                        status: Optional[torch.Tensor] = None, stream=None):
    """Walk the drafted tree from node 0 by the given random numbers; returns
    (path int32 [B][N], -1 behind its end; n_accepted int32 [B]; next_token
    int32 [B]).  target_probs, draft_probs [B][N][V] (row i follows node i;
    draft_probs None: the drafts were chosen, not drawn), tokens int32 [B][N],
    parents int32 [N] or [B][N], u_accept [B][N] and u_sample [B] in [0, 1)."""
    if path is None or n_accepted is None or next_token is None:
        B, N, _ = target_probs.shape
        dev = target_probs.device
        with _allocating(stream):
            path = torch.full((B, N), -1, dtype=torch.int32, device=dev) if path is None else path
            n_accepted = torch.zeros(B, dtype=torch.int32, device=dev) if n_accepted is None else n_accepted
            next_token = torch.full((B,), -1, dtype=torch.int32, device=dev) if next_token is None else next_token
    st = _native.binding().verify_drafts(*_target(stream), target_probs, draft_probs, tokens, parents, u_accept, u_sample,
                                         n_nodes, path, n_accepted, next_token, status)
    if st:
        _native.check("nvfp4_verify_drafts", st)
    return path, n_accepted, next_token


class KVPlaneList:
    """The planes of a cache (all layers' K and V: KVPlane, or PagedKVPlane that
    share one block table), checked and laid out once for nvfp4_kv_commit_path.
    Holds the planes, and the tensors they had when the list was made, which stay
    the ones that are moved: a plane whose tensors are replaced needs a new list."""

    def __init__(self, planes):
        self.planes = tuple(planes)
        if not self.planes:
            raise ValueError("a plane list needs at least one plane")
        self.kind = type(self.planes[0])
        if self.kind not in (KVPlane, PagedKVPlane):
            raise TypeError("planes must be KVPlane or PagedKVPlane")
        for p in self.planes:
            _need_kind(self.planes[0], p, self.kind)
        self.device = self.planes[0].codes.get_device()
        if self.device < 0:
            raise ValueError("planes must be CUDA tensors")
        data, self.B = _native.binding().planes(self.device, self.kind is PagedKVPlane, self.planes)
        self._structs = ctypes.create_string_buffer(data, len(data))
        self.address = ctypes.addressof(self._structs)
        self._count = len(self.planes)
        # what the structs point at, whatever becomes of the planes' attributes
        self._tensors = [tuple(vars(p).values()) for p in self.planes]

    def __len__(self):
        return self._count


def _commit_path(func, kind, planes, start_pos, path, n_accepted, new_lens, status, stream):
    if not isinstance(planes, KVPlaneList):
        planes = KVPlaneList(planes)
    if planes.kind is not kind:
        raise TypeError("planes must be %s" % kind.__name__)
    cur, handle = _target(stream)
    if planes.device != cur:
        raise ValueError("planes must be on the current CUDA device (%d), got %d" % (cur, planes.device))
    st = _native.binding().commit_path(cur, handle, kind is PagedKVPlane, planes.address, len(planes), planes.B,
                                       start_pos, path, n_accepted, new_lens, status)
    if st:
        _native.check(func, st)


def nvfp4_kv_commit_path(planes, start_pos: torch.Tensor, path: torch.Tensor, n_accepted: torch.Tensor,
                         new_lens: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                         stream=None) -> None:
    """Keep the accepted path's cache slots: slot start_pos[b] + path[b][j] moves
    to start_pos[b] + j for j < n_accepted[b], in every plane given (all layers'
    K and V as a KVPlaneList or a sequence of KVPlane, none of them twice; one launch
    for 64 planes)."""
    _commit_path("nvfp4_kv_commit_path", KVPlane, planes, start_pos, path, n_accepted, new_lens, status, stream)


def nvfp4_kv_commit_path_paged(planes, start_pos: torch.Tensor, path: torch.Tensor, n_accepted: torch.Tensor,
                               new_lens: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                               stream=None) -> None:
    """nvfp4_kv_commit_path in paged planes that share one block table."""
    _commit_path("nvfp4_kv_commit_path_paged", PagedKVPlane, planes, start_pos, path, n_accepted, new_lens, status,
                 stream)

"""GB300-native weight-absorbed MLA decode.

Python binding of ``libmla.so``, the C-ABI library declared in ``include/mla.h``.
The functions here only marshal arguments: every step of the path (schedule,
W_UK absorption, paged decode, LSE combine, W_UV un-absorption) runs in the
library's sm_103a kernels.  PyTorch supplies device memory and streams.
There is no fallback: if the library is not built, calls raise.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

__all__ = [
    "MLAError", "lib", "library_path", "num_sm_parts", "metadata_size", "decode_metadata",
    "decode_workspace_size", "decode", "decode_sparse", "decode_fp8", "decode_sparse_fp8", "absorb_q", "unabsorb_o",
    "absorb_plan_max_batch", "absorb_q_plan",
    "bmm_fp8_workspace_size", "absorb_q_fp8", "absorb_q_fp8_plan", "unabsorb_o_fp8", "extend_workspace_size", "extend_chunked",
    "rope_axes", "cache_append", "cache_append_fp8", "attn_weights", "attn_weights_fp8", "evict", "evict_fp8",
    "get_device_status",
    "schedule_params", "debug_withhold_first_load", "DecodeStep", "EXPORTED_SYMBOLS",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libmla.so")

MLA_OK = 0
STATUS_NAMES = {0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED", 3: "MLA_ERR_WORKSPACE",
                4: "MLA_ERR_CUDA", 5: "MLA_ERR_TIMEOUT", 6: "MLA_ERR_DEVICE_BOUNDS"}

_c_int, _c_size, _c_float, _c_ll, _p = ctypes.c_int, ctypes.c_size_t, ctypes.c_float, ctypes.c_int64, ctypes.c_void_p
_SIGNATURES = {
    "mla_status_string": (ctypes.c_char_p, [_c_int]),
    "mla_num_sm_parts": (_c_int, [_c_int, _c_int, _c_int]),
    "mla_metadata_size": (_c_size, [_c_int, _c_int]),
    "mla_decode_metadata": (_c_int, [_p, _c_int, _c_int, _c_int, _c_int, _c_int, _p, _p]),
    "mla_schedule_params": (None, [ctypes.POINTER(_c_int), ctypes.POINTER(_c_int), ctypes.POINTER(_c_int)]),
    "mla_decode_workspace_size": (_c_size, [_c_int, _c_int, _c_int, _c_int]),
    "mla_decode": (_c_int, [_p, _p, _c_ll, _p, _c_int, _p, _c_int, _c_int, _c_int, _c_float, _c_int,
                            _p, _c_int, _p, _c_size, _p, _p, _p]),
    "mla_decode_sparse": (_c_int, [_p, _p, _c_ll, _p, _c_int, _p, _p, _c_ll, _p, _c_int, _c_int, _c_int, _c_float,
                                   _c_int, _p, _c_int, _p, _c_size, _p, _p, _p]),
    "mla_decode_fp8": (_c_int, [_p, _p, _c_float, _c_ll, _p, _c_int, _p, _c_int, _c_int, _c_int, _c_float, _c_int,
                                _p, _c_int, _p, _c_size, _p, _p, _p]),
    "mla_decode_sparse_fp8": (_c_int, [_p, _p, _c_float, _c_ll, _p, _c_int, _p, _p, _c_ll, _p, _c_int, _c_int, _c_int,
                                       _c_float, _c_int, _p, _c_int, _p, _c_size, _p, _p, _p]),
    "mla_absorb_q": (_c_int, [_p, _c_ll, _p, _c_ll, _p, _p, _c_int, _c_int, _p]),
    "mla_absorb_q_rope": (_c_int, [_p, _c_ll, _p, _c_ll, _p, _c_float, _p, _p, _c_int, _c_int, _p]),
    "mla_absorb_plan_max_batch": (_c_int, []),
    "mla_absorb_q_plan": (_c_int, [_p, _c_ll, _p, _c_ll, _p, _c_float, _p, _p, _c_int, _c_int, _p, _c_int, _c_int, _p,
                                   _p]),
    "mla_unabsorb_o": (_c_int, [_p, _p, _p, _c_int, _c_int, _p]),
    "mla_bmm_fp8_workspace_size": (_c_size, []),
    "mla_absorb_q_fp8": (_c_int, [_p, _c_ll, _p, _c_ll, _p, _c_float, _p, _c_float, _p, _c_int, _c_int, _p, _c_size, _p]),
    "mla_absorb_q_fp8_plan": (_c_int, [_p, _c_ll, _p, _c_ll, _p, _c_float, _p, _c_float, _p, _c_int, _c_int, _p,
                                       _c_size, _p, _c_int, _c_int, _p, _p]),
    "mla_unabsorb_o_fp8": (_c_int, [_p, _p, _c_float, _p, _c_int, _c_int, _p, _c_size, _p]),
    "mla_extend_workspace_size": (_c_size, [_c_int, _c_int, _c_int]),
    "mla_extend_chunked": (_c_int, [_p, _p, _p, _p, _p, _c_ll, _p, _c_int, _c_int, _c_int, _c_float, _c_int, _p, _c_size,
                                    _p, _p, _p]),
    "mla_decode_noalloc": (_c_int, [_p, _p, _c_ll, _p, _c_int, _p, _c_int, _c_int, _c_int, _c_float, _c_int,
                                    _c_int, _p, _p, _p]),
    "mla_rope_axes": (_c_int, [_p, _c_ll, _c_ll, _p, _c_ll, _c_ll, _p, _c_ll, _p, _c_int, _c_int, _c_float, _c_int,
                               _c_int, _c_int, _p]),
    "mla_cache_append": (_c_int, [_p, _c_ll, _p, _c_ll, _p, _c_ll, _p, _c_int, _p, _p, _c_int, _c_int, _p, _c_ll, _p,
                                  _c_int, _c_int, _c_float, _p]),
    "mla_cache_append_fp8": (_c_int, [_p, _c_ll, _p, _c_ll, _p, _c_float, _c_ll, _p, _c_int, _p, _p, _c_int, _c_int, _p,
                                      _c_ll, _p, _c_int, _c_int, _c_float, _p]),
    "mla_attn_weights": (_c_int, [_p, _p, _p, _c_ll, _p, _c_int, _p, _c_int, _c_int, _c_int, _c_float, _c_int, _p, _c_ll,
                                  _p]),
    "mla_attn_weights_fp8": (_c_int, [_p, _p, _p, _c_float, _c_ll, _p, _c_int, _p, _c_int, _c_int, _c_int, _c_float,
                                      _c_int, _p, _c_ll, _p]),
    "mla_evict": (_c_int, [_p, _c_ll, _p, _c_int, _p, _c_int, _p, _c_ll, _p, _c_ll, _c_int, _c_int, _c_int, _p, _p, _p,
                           _p, _c_ll, _p]),
    "mla_evict_fp8": (_c_int, [_p, _c_ll, _p, _c_int, _p, _c_int, _p, _c_ll, _p, _c_ll, _c_int, _c_int, _c_int, _p, _p,
                               _p, _p, _c_ll, _p]),
    "mla_get_device_status": (_c_int, [_p]),
    "mla_debug_withhold_first_load": (None, [_c_int]),
}
EXPORTED_SYMBOLS = tuple(_SIGNATURES)

_lib = None


class MLAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)}")


def lib() -> ctypes.CDLL:
    """Load libmla.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise RuntimeError(f"{library_path} is missing: build it with "
                               "`python -m mla_absorbed_decode_gb300.build_lib`")
        handle = ctypes.CDLL(library_path)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _check(status: int, what: str):
    if status != MLA_OK:
        raise MLAError(status, what)


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _ptr(t: torch.Tensor) -> int:
    return t.data_ptr()


def num_sm_parts(s_q: int, H: int, device: int | None = None) -> int:
    dev = torch.cuda.current_device() if device is None else device
    n = lib().mla_num_sm_parts(dev, s_q, H)
    if n <= 0:
        raise MLAError(-n if n < 0 else 4, "mla_num_sm_parts")
    return n


def metadata_size(B: int, parts: int) -> int:
    return lib().mla_metadata_size(B, parts)


def schedule_params() -> tuple[int, int, int]:
    """(set-up cost per segment, parts that saturate HBM, cost of an extra segment), in pages."""
    f, h, c = _c_int(), _c_int(), _c_int()
    lib().mla_schedule_params(ctypes.byref(f), ctypes.byref(h), ctypes.byref(c))
    return f.value, h.value, c.value


def decode_metadata(seqlens: torch.Tensor, s_q: int, H: int, causal: bool, parts: int,
                    out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Split-KV tile schedule for these sequence lengths (int32 tensor on the device)."""
    B = seqlens.numel()
    n_ints = metadata_size(B, parts) // 4
    if out is None:
        out = torch.empty(n_ints, dtype=torch.int32, device=seqlens.device)
    _check(lib().mla_decode_metadata(_ptr(seqlens), B, s_q, H, int(causal), parts, _ptr(out), _stream(stream)),
           "mla_decode_metadata")
    return out


def decode_workspace_size(B: int, s_q: int, H: int, parts: int) -> int:
    return lib().mla_decode_workspace_size(B, s_q, H, parts)


def decode(q, kv_cache, block_table, seqlens, softmax_scale: float, causal: bool, metadata, parts: int,
           workspace=None, out=None, lse=None, stream=None):
    """Absorbed MLA decode: returns (out [B,s_q,H,512] bf16, lse [B,s_q,H] fp32)."""
    B, s_q, H, _ = q.shape
    dev = q.device
    if out is None:
        out = torch.empty((B, s_q, H, 512), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, s_q, H), dtype=torch.float32, device=dev)
    need = decode_workspace_size(B, s_q, H, parts)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _check(lib().mla_decode(_ptr(q), _ptr(kv_cache), kv_cache.shape[0], _ptr(block_table), block_table.shape[1],
                            _ptr(seqlens), B, s_q, H, float(softmax_scale), int(causal), _ptr(metadata), parts,
                            _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out), _ptr(lse),
                            _stream(stream)), "mla_decode")
    return out, lse


def decode_sparse(q, kv_cache, block_table, seqlens, indices, topk_lens, softmax_scale: float, causal: bool, metadata,
                  parts: int, workspace=None, out=None, lse=None, stream=None):
    """Sparse (top-k) absorbed decode over indices[b, :topk_lens[b]] (int32 token positions);
    metadata from decode_metadata(topk_lens, ...).  Returns (out [B,s_q,H,512] bf16, lse [B,s_q,H] fp32)."""
    B, s_q, H, _ = q.shape
    dev = q.device
    if out is None:
        out = torch.empty((B, s_q, H, 512), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, s_q, H), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(decode_workspace_size(B, s_q, H, parts), dtype=torch.uint8, device=dev)
    _check(lib().mla_decode_sparse(_ptr(q), _ptr(kv_cache), kv_cache.shape[0], _ptr(block_table), block_table.shape[1],
                                   _ptr(seqlens), _ptr(indices), indices.stride(0), _ptr(topk_lens), B, s_q, H,
                                   float(softmax_scale), int(causal), _ptr(metadata), parts, _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _ptr(out), _ptr(lse),
                                   _stream(stream)), "mla_decode_sparse")
    return out, lse


def decode_fp8(q, kv_cache, kv_scale: float, block_table, seqlens, softmax_scale: float, causal: bool, metadata,
               parts: int, workspace=None, out=None, lse=None, stream=None):
    """Absorbed MLA decode over an FP8 cache: kv_cache [num_blocks,64,576] uint8 E4M3 codes (or a
    float8_e4m3fn tensor), cached value = code value * kv_scale.  Returns (out, lse) as decode."""
    B, s_q, H, _ = q.shape
    dev = q.device
    if kv_cache.element_size() != 1:
        raise TypeError("decode_fp8: kv_cache must hold one byte per value (E4M3 codes)")
    if out is None:
        out = torch.empty((B, s_q, H, 512), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, s_q, H), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(decode_workspace_size(B, s_q, H, parts), dtype=torch.uint8, device=dev)
    _check(lib().mla_decode_fp8(_ptr(q), _ptr(kv_cache), float(kv_scale), kv_cache.shape[0], _ptr(block_table),
                                block_table.shape[1], _ptr(seqlens), B, s_q, H, float(softmax_scale), int(causal),
                                _ptr(metadata), parts, _ptr(workspace), workspace.numel() * workspace.element_size(),
                                _ptr(out), _ptr(lse), _stream(stream)), "mla_decode_fp8")
    return out, lse


def decode_sparse_fp8(q, kv_cache, kv_scale: float, block_table, seqlens, indices, topk_lens, softmax_scale: float,
                      causal: bool, metadata, parts: int, workspace=None, out=None, lse=None, stream=None):
    """decode_sparse over an FP8 cache (E4M3 codes scaled by kv_scale, as in decode_fp8)."""
    B, s_q, H, _ = q.shape
    dev = q.device
    if kv_cache.element_size() != 1:
        raise TypeError("decode_sparse_fp8: kv_cache must hold one byte per value (E4M3 codes)")
    if out is None:
        out = torch.empty((B, s_q, H, 512), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, s_q, H), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(decode_workspace_size(B, s_q, H, parts), dtype=torch.uint8, device=dev)
    _check(lib().mla_decode_sparse_fp8(_ptr(q), _ptr(kv_cache), float(kv_scale), kv_cache.shape[0], _ptr(block_table),
                                       block_table.shape[1], _ptr(seqlens), _ptr(indices), indices.stride(0),
                                       _ptr(topk_lens), B, s_q, H, float(softmax_scale), int(causal), _ptr(metadata),
                                       parts, _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out),
                                       _ptr(lse), _stream(stream)), "mla_decode_sparse_fp8")
    return out, lse


def absorb_q(q_nope: torch.Tensor, w_uk: torch.Tensor, q: torch.Tensor, q_pe: torch.Tensor | None = None,
             stream=None, positions: torch.Tensor | None = None, rope_theta: float = 10000.0) -> torch.Tensor:
    """q[n, h, 0:512] = q_nope[n, h, :] @ w_uk[h] and q[n, h, 512:576] = q_pe[n, h, :], RoPE-rotated
    by positions[n] (int32 [N]) when positions is given; q is [N, H, 576] (or [B, s_q, H, 576])."""
    N, H, _ = q_nope.shape
    pe_ptr, pe_stride = (0, 0) if q_pe is None else (_ptr(q_pe), q_pe.stride(0))
    if positions is None:
        _check(lib().mla_absorb_q(_ptr(q_nope), q_nope.stride(0), pe_ptr or None, pe_stride, _ptr(w_uk), _ptr(q), N,
                                  H, _stream(stream)), "mla_absorb_q")
    else:
        _check(lib().mla_absorb_q_rope(_ptr(q_nope), q_nope.stride(0), pe_ptr or None, pe_stride, _ptr(positions),
                                       float(rope_theta), _ptr(w_uk), _ptr(q), N, H, _stream(stream)),
               "mla_absorb_q_rope")
    return q


def absorb_plan_max_batch() -> int:
    return lib().mla_absorb_plan_max_batch()


def absorb_q_plan(q_nope: torch.Tensor, w_uk: torch.Tensor, q: torch.Tensor, seqlens: torch.Tensor, num_parts: int,
                  metadata: torch.Tensor, q_pe: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                  rope_theta: float = 10000.0, stream=None) -> torch.Tensor:
    """absorb_q and decode_metadata(seqlens, ..., num_parts, out=metadata) in one launch
    (B = len(seqlens), s_q = N / B); returns q."""
    N, H, _ = q_nope.shape
    pe_ptr, pe_stride = (0, 0) if q_pe is None else (_ptr(q_pe), q_pe.stride(0))
    _check(lib().mla_absorb_q_plan(_ptr(q_nope), q_nope.stride(0), pe_ptr or None, pe_stride,
                                   _ptr(positions) if positions is not None else None, float(rope_theta), _ptr(w_uk),
                                   _ptr(q), N, H, _ptr(seqlens), seqlens.numel(), int(num_parts), _ptr(metadata),
                                   _stream(stream)), "mla_absorb_q_plan")
    return q


def unabsorb_o(o_lat: torch.Tensor, w_uv: torch.Tensor, o: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """o[n, h, :] = o_lat[n, h, :] @ w_uv[h]; o_lat is [N, H, 512] -> o [N, H, 128]."""
    N, H = o_lat.shape[0], o_lat.shape[1]
    if o is None:
        o = torch.empty((N, H, 128), dtype=torch.bfloat16, device=o_lat.device)
    _check(lib().mla_unabsorb_o(_ptr(o_lat), _ptr(w_uv), _ptr(o), N, H, _stream(stream)), "mla_unabsorb_o")
    return o


def bmm_fp8_workspace_size() -> int:
    return lib().mla_bmm_fp8_workspace_size()


def _fp8_workspace(dev, workspace):
    if workspace is None:
        workspace = torch.empty(bmm_fp8_workspace_size(), dtype=torch.uint8, device=dev)
    return workspace


def absorb_q_fp8(q_nope: torch.Tensor, w_uk_t: torch.Tensor, w_uk_scale: float, q: torch.Tensor,
                 q_pe: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                 rope_theta: float = 10000.0, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q[n, h, 0:512] = bmm_fp8(input_to_float8(q_nope), W_UK)[n, h] with w_uk_t [H, 512, 128] E4M3
    codes (uint8 or float8_e4m3fn) and scale w_uk_scale; q[n, h, 512:576] = q_pe[n, h], RoPE-rotated
    by positions[n] when positions is given."""
    N, H, _ = q_nope.shape
    if w_uk_t.element_size() != 1:
        raise TypeError("absorb_q_fp8: w_uk_t must hold one E4M3 code per value")
    ws = _fp8_workspace(q_nope.device, workspace)
    pe_ptr, pe_stride = (0, 0) if q_pe is None else (_ptr(q_pe), q_pe.stride(0))
    _check(lib().mla_absorb_q_fp8(_ptr(q_nope), q_nope.stride(0), pe_ptr or None, pe_stride,
                                  None if positions is None else _ptr(positions), float(rope_theta), _ptr(w_uk_t),
                                  float(w_uk_scale), _ptr(q), N, H, _ptr(ws), ws.numel() * ws.element_size(),
                                  _stream(stream)), "mla_absorb_q_fp8")
    return q


def absorb_q_fp8_plan(q_nope: torch.Tensor, w_uk_t: torch.Tensor, w_uk_scale: float, q: torch.Tensor,
                      seqlens: torch.Tensor, num_parts: int, metadata: torch.Tensor, q_pe: torch.Tensor | None = None,
                      positions: torch.Tensor | None = None, rope_theta: float = 10000.0,
                      workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """absorb_q_fp8 and decode_metadata(seqlens, ..., num_parts, out=metadata) in one pass
    (B = len(seqlens), s_q = N / B); returns q."""
    N, H, _ = q_nope.shape
    if w_uk_t.element_size() != 1:
        raise TypeError("absorb_q_fp8_plan: w_uk_t must hold one E4M3 code per value")
    ws = _fp8_workspace(q_nope.device, workspace)
    pe_ptr, pe_stride = (0, 0) if q_pe is None else (_ptr(q_pe), q_pe.stride(0))
    _check(lib().mla_absorb_q_fp8_plan(_ptr(q_nope), q_nope.stride(0), pe_ptr or None, pe_stride,
                                       None if positions is None else _ptr(positions), float(rope_theta),
                                       _ptr(w_uk_t), float(w_uk_scale), _ptr(q), N, H, _ptr(ws),
                                       ws.numel() * ws.element_size(), _ptr(seqlens), seqlens.numel(),
                                       int(num_parts), _ptr(metadata), _stream(stream)), "mla_absorb_q_fp8_plan")
    return q


def unabsorb_o_fp8(o_lat: torch.Tensor, w_uv_t: torch.Tensor, w_uv_scale: float, o: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """o[n, h, :] = bmm_fp8(input_to_float8(o_lat), W_UV)[n, h] with w_uv_t [H, 128, 512] E4M3 codes
    and scale w_uv_scale; o_lat is [N, H, 512] -> o [N, H, 128] bf16."""
    N, H = o_lat.shape[0], o_lat.shape[1]
    if w_uv_t.element_size() != 1:
        raise TypeError("unabsorb_o_fp8: w_uv_t must hold one E4M3 code per value")
    if o is None:
        o = torch.empty((N, H, 128), dtype=torch.bfloat16, device=o_lat.device)
    ws = _fp8_workspace(o_lat.device, workspace)
    _check(lib().mla_unabsorb_o_fp8(_ptr(o_lat), _ptr(w_uv_t), float(w_uv_scale), _ptr(o), N, H, _ptr(ws),
                                    ws.numel() * ws.element_size(), _stream(stream)), "mla_unabsorb_o_fp8")
    return o


def extend_workspace_size(T: int, H: int, chunk_tokens: int) -> int:
    return lib().mla_extend_workspace_size(T, H, chunk_tokens)


def extend_chunked(q_nope: torch.Tensor, q_pe: torch.Tensor, w_uk: torch.Tensor, w_uv: torch.Tensor,
                   kv_cache: torch.Tensor, block_row: torch.Tensor, seqlen: int, softmax_scale: float,
                   chunk_tokens: int = 2048, workspace: torch.Tensor | None = None, out: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None, stream=None):
    """Chunked extend on the expanded path (MHA_CHUNKED_KV): the T new tokens (the last T of the
    request's seqlen cached tokens, causal) attend to the cache expanded chunk by chunk, merged by
    LSE.  q_nope [T,H,128], q_pe [T,H,64] (RoPE applied), w_uk [H,128,512], w_uv [H,512,128],
    block_row int32 [>= ceil(seqlen/64)].  Returns (out [T,H,128] bf16, lse [T,H] fp32)."""
    T, H, _ = q_nope.shape
    dev = q_nope.device
    if out is None:
        out = torch.empty((T, H, 128), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(extend_workspace_size(T, H, chunk_tokens), dtype=torch.uint8, device=dev)
    _check(lib().mla_extend_chunked(_ptr(q_nope), _ptr(q_pe), _ptr(w_uk), _ptr(w_uv), _ptr(kv_cache),
                                    kv_cache.shape[0], _ptr(block_row), int(seqlen), T, H, float(softmax_scale),
                                    int(chunk_tokens), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _ptr(out), _ptr(lse), _stream(stream)), "mla_extend_chunked")
    return out, lse


# The latent-cache calls.  The kernels read raw addresses, so a tensor of another type, shape or device must
# not reach them; the checks are plain conditions (a decode step makes these calls for every layer).
_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _bad(name: str, what: str, wanted: str, t: torch.Tensor, dtype=None) -> Exception:
    kind = TypeError if dtype is not None and t.dtype is not dtype else ValueError
    return kind(f"{name}: {what} must be {wanted} on one GPU with the call's other tensors; got {t.dtype} "
                f"{list(t.shape)} with strides {list(t.stride())} on {t.device}")


def _paged(name: str, kv_cache: torch.Tensor, block_table: torch.Tensor, seqlens: torch.Tensor, fp8: bool):
    """Checks a call's cache, table and lengths; returns (device index, B, num_blocks, max_blocks)."""
    dev = kv_cache.get_device()
    shape = kv_cache.shape
    if fp8 and kv_cache.element_size() != 1:
        raise TypeError(f"{name}: kv_cache must hold one byte per value (E4M3 codes)")
    if (dev < 0 or not (fp8 or kv_cache.dtype is _BF16) or len(shape) != 3 or shape[1] != 64 or shape[2] != 576
            or not kv_cache.is_contiguous()):
        raise _bad(name, "kv_cache", "a contiguous [num_blocks, 64, 576]", kv_cache, None if fp8 else _BF16)
    if seqlens.dtype is not _I32 or seqlens.get_device() != dev or seqlens.dim() != 1 or not seqlens.is_contiguous():
        raise _bad(name, "seqlens", "a contiguous int32 [B]", seqlens, _I32)
    B = seqlens.numel()
    table = block_table.shape
    if (block_table.dtype is not _I32 or block_table.get_device() != dev or len(table) != 2 or table[0] != B
            or not block_table.is_contiguous()):
        raise _bad(name, "block_table", "a contiguous int32 [B, max_blocks]", block_table, _I32)
    return dev, B, shape[0], table[1]


def _rows(name: str, what: str, t: torch.Tensor, dtype: torch.dtype, dev: int, B: int, max_blocks: int) -> int:
    """Checks a [B, slots] tensor whose rows may be strided; returns the elements between rows, of which a request may
    use as many as there are columns."""
    shape, strides = t.shape, t.stride()
    if (t.dtype is not dtype or t.get_device() != dev or len(shape) != 2 or shape[0] != B or shape[1] < 1
            or (shape[1] > 1 and strides[1] != 1)):
        raise _bad(name, what, f"{dtype} [B, slots] with contiguous rows", t, dtype)
    slots = shape[1]
    stride = strides[0] if B > 1 else slots
    if stride != slots and (stride < slots or slots < 64 * max_blocks):
        raise ValueError(f"{name}: {what}: rows that are a part of wider ones must have a slot for every entry of block_table")
    return stride


def _launch(dev: int, fn: str, args, stream):
    """Calls the library with the tensors' device current (it launches on the current device) and that device's current
    stream unless one is given."""
    raw = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        status = getattr(_lib or lib(), fn)(*args, raw)
    else:
        with torch.cuda.device(dev):
            status = getattr(_lib or lib(), fn)(*args, raw)
    if status != MLA_OK:
        raise MLAError(status, fn)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """An output of a call on `stream`, from that stream's memory."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


@functools.lru_cache(maxsize=64)   # a model has one
def _sections(sections: tuple):
    """Host array of a rotation's sections."""
    if not 1 <= len(sections) <= 4 or min(sections) < 0 or sum(sections) != 32:
        raise ValueError("sections must be 1 to 4 counts of pairs that sum to 32")
    return (_c_int * len(sections))(*sections), len(sections)


def _axes(name: str, positions: torch.Tensor, sections, N: int, dev: int):
    """Checks positions ([N], or [axes, N]) and sections; returns (pointer, stride, host sections, axes)."""
    host, axes = _sections(sections if type(sections) is tuple else tuple(sections))
    shape, strides = positions.shape, positions.stride()
    if (positions.dtype is not _I32 or positions.get_device() != dev or not 1 <= len(shape) <= 2 or shape[-1] != N
            or (shape[0] if len(shape) == 2 else 1) != axes or (N > 1 and strides[-1] != 1)):
        raise _bad(name, "positions", f"int32 [{axes} axes, N] (or [N] for one axis) with contiguous rows", positions, _I32)
    return positions.data_ptr(), strides[0] if axes > 1 else N, host, axes


def rope_axes(x: torch.Tensor, positions: torch.Tensor, sections=(32,), out: torch.Tensor | None = None,
              rope_theta: float = 10000.0, interleaved: bool = False, inverse: bool = False, stream=None) -> torch.Tensor:
    """RoPE with several position axes: x [N, H, 64] bf16 (any strides that keep the last dim
    contiguous), positions int32 [axes, N], sections = how many of the 32 adjacent pairs each axis
    turns, one section after the other or (interleaved) dealt out in turn.  out may be x or a view such
    as q[..., 512:] of the decode query.  inverse turns back: the gradient of x from that of out."""
    dev = x.get_device()
    shape, xs = x.shape, x.stride()
    if dev < 0 or x.dtype is not _BF16 or len(shape) != 3 or shape[2] != 64 or xs[2] != 1:
        raise _bad("rope_axes", "x", "a bfloat16 [N, H, 64] with contiguous rows", x, _BF16)
    N, H, _ = shape
    if out is None:
        out = _empty((N, H, 64), _BF16, x.device, stream)
    os_ = out.stride()
    if out.dtype is not _BF16 or out.get_device() != dev or out.shape != shape or os_[2] != 1:
        raise _bad("rope_axes", "out", "a bfloat16 of x's shape with contiguous rows", out, _BF16)
    if N == 0 or H == 0:
        return out
    pos, pos_stride, host, axes = _axes("rope_axes", positions, sections, N, dev)
    many, heads = N > 1, H > 1   # the stride of a dim of one element says nothing
    _launch(dev, "mla_rope_axes", (
        x.data_ptr(), xs[0] if many else 0, xs[1] if heads else 0, out.data_ptr(), os_[0] if many else 0,
        os_[1] if heads else 0, pos, pos_stride, host, axes, interleaved, rope_theta, inverse, N, H), stream)
    return out


def _append(name, c, k_pe, kv_cache, kv_scale, block_table, seqlens, new_offsets, positions, sections, rope_theta,
            interleaved, stream):
    dev, B, num_blocks, max_blocks = _paged(name, kv_cache, block_table, seqlens, kv_scale is not None)
    shape, cs, ps = c.shape, c.stride(), k_pe.stride()
    if c.dtype is not _BF16 or c.get_device() != dev or len(shape) != 2 or shape[1] != 512 or cs[1] != 1:
        raise _bad(name, "c", "a bfloat16 [N, 512] with contiguous rows", c, _BF16)
    N = shape[0]
    if k_pe.dtype is not _BF16 or k_pe.get_device() != dev or k_pe.shape != (N, 64) or ps[1] != 1:
        raise _bad(name, "k_pe", f"a bfloat16 [{N}, 64] with contiguous rows", k_pe, _BF16)
    off = None
    if new_offsets is not None:
        if (new_offsets.dtype is not _I32 or new_offsets.get_device() != dev or new_offsets.shape != (B + 1,)
                or not new_offsets.is_contiguous()):
            raise _bad(name, "new_offsets", "a contiguous int32 [B + 1]", new_offsets, _I32)
        off = new_offsets.data_ptr()
    if N == 0 or B == 0:
        return kv_cache
    rot = (None, 0, None, 0) if positions is None else _axes(name, positions, sections, N, dev)
    pool = (kv_cache.data_ptr(),) if kv_scale is None else (kv_cache.data_ptr(), kv_scale)
    _launch(dev, "mla_" + name, (
        c.data_ptr(), cs[0] if N > 1 else 512, k_pe.data_ptr(), ps[0] if N > 1 else 64, *pool, num_blocks,
        block_table.data_ptr(), max_blocks, seqlens.data_ptr(), off, N, B, *rot, interleaved, rope_theta), stream)
    return kv_cache


def cache_append(c, k_pe, kv_cache, block_table, seqlens, new_offsets=None, positions=None, sections=(32,),
                 rope_theta: float = 10000.0, interleaved: bool = False, stream=None) -> torch.Tensor:
    """A step's new rows [c, k_pe] (bf16 [N, 512] and [N, 64], rows may be strided) into the paged cache:
    request b's rows are its last tokens, seqlens counts them already.  Rows are dealt to the requests
    by new_offsets (int32 [B + 1]) or evenly.  With positions ([axes, N] or [N] int32) k_pe is turned
    on the way, as in rope_axes.  Returns kv_cache."""
    return _append("cache_append", c, k_pe, kv_cache, None, block_table, seqlens, new_offsets, positions, sections,
                   rope_theta, interleaved, stream)


def cache_append_fp8(c, k_pe, kv_cache, kv_scale: float, block_table, seqlens, new_offsets=None, positions=None,
                     sections=(32,), rope_theta: float = 10000.0, interleaved: bool = False,
                     stream=None) -> torch.Tensor:
    """cache_append into an FP8 cache: E4M3 codes of value / kv_scale (round to nearest even, saturating)."""
    return _append("cache_append_fp8", c, k_pe, kv_cache, kv_scale, block_table, seqlens, new_offsets, positions,
                   sections, rope_theta, interleaved, stream)


def _weights(name, q, lse, kv_cache, kv_scale, block_table, seqlens, softmax_scale, causal, weights, stream):
    dev, B, num_blocks, max_blocks = _paged(name, kv_cache, block_table, seqlens, kv_scale is not None)
    shape = q.shape
    if (q.dtype is not _BF16 or q.get_device() != dev or len(shape) != 4 or shape[0] != B or shape[3] != 576
            or not q.is_contiguous()):
        raise _bad(name, "q", "a contiguous bfloat16 [B, s_q, H, 576]", q, _BF16)
    if lse.dtype is not _F32 or lse.get_device() != dev or lse.shape != shape[:3] or not lse.is_contiguous():
        raise _bad(name, "lse", "a contiguous float32 [B, s_q, H]", lse, _F32)
    stride = _rows(name, "weights", weights, _F32, dev, B, max_blocks)
    if q.numel() == 0:
        return weights
    pool = (kv_cache.data_ptr(),) if kv_scale is None else (kv_cache.data_ptr(), kv_scale)
    _launch(dev, "mla_" + name, (
        q.data_ptr(), lse.data_ptr(), *pool, num_blocks, block_table.data_ptr(), max_blocks, seqlens.data_ptr(), B,
        shape[1], shape[2], softmax_scale, causal, weights.data_ptr(), stride), stream)
    return weights


def attn_weights(q, lse, kv_cache, block_table, seqlens, softmax_scale: float, causal: bool, weights,
                 stream=None) -> torch.Tensor:
    """weights[b, t] += the attention weight that the step's heads and query positions gave cached token
    t (fp32 [B, slots], slots >= every length; q and lse as of decode).  Returns weights."""
    return _weights("attn_weights", q, lse, kv_cache, None, block_table, seqlens, softmax_scale, causal, weights, stream)


def attn_weights_fp8(q, lse, kv_cache, kv_scale: float, block_table, seqlens, softmax_scale: float, causal: bool,
                     weights, stream=None) -> torch.Tensor:
    """attn_weights over an FP8 cache (E4M3 codes scaled by kv_scale, as in decode_fp8)."""
    return _weights("attn_weights_fp8", q, lse, kv_cache, kv_scale, block_table, seqlens, softmax_scale, causal, weights,
                    stream)


def _evict(name, fp8, kv_cache, block_table, seqlens, weights, budget, sink, recent, arrival, width, new_seqlens, kept,
           weights_out, arrival_out, stream):
    dev, B, num_blocks, max_blocks = _paged(name, kv_cache, block_table, seqlens, fp8)
    w_stride = _rows(name, "weights", weights, _F32, dev, B, max_blocks)
    a_ptr, a_stride = None, 0
    if arrival is not None:
        a_stride = _rows(name, "arrival", arrival, _I32, dev, B, max_blocks)
        a_ptr = arrival.data_ptr()
    if width is None:
        width = weights.shape[1]

    def given(what, t, dtype, shape):
        if t is None:
            return _empty(shape, dtype, weights.device, stream)
        if t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
            raise _bad(name, what, f"a contiguous {dtype} {list(shape)}", t, dtype)
        return t

    wide = (B, width)
    outs = (given("new_seqlens", new_seqlens, _I32, (B,)), given("kept", kept, _I32, wide),
            given("weights_out", weights_out, _F32, wide), given("arrival_out", arrival_out, _I32, wide))
    if B == 0:
        return outs
    _launch(dev, "mla_" + name, (
        kv_cache.data_ptr(), num_blocks, block_table.data_ptr(), max_blocks, seqlens.data_ptr(), B, weights.data_ptr(),
        w_stride, a_ptr, a_stride, budget, sink, recent, outs[0].data_ptr(), outs[1].data_ptr(), outs[2].data_ptr(),
        outs[3].data_ptr(), width), stream)
    return outs


def evict(kv_cache, block_table, seqlens, weights, budget: int, sink: int = 0, recent: int = 0, arrival=None,
          width: int | None = None, new_seqlens=None, kept=None, weights_out=None, arrival_out=None, stream=None):
    """Of every request's cached tokens the min(length, budget) of largest accumulated weight stay, its
    first `sink` and newest `recent` ones (by arrival number; the slot without `arrival`) before all
    others, ties to the lower slot; kv_cache is changed in place: slots that fall free below the new
    length take the staying tokens from beyond it.  Returns (new_seqlens [B] int32 (may be seqlens),
    kept [B, width] int32: the old slot of the token in each slot, weights_out, arrival_out [B, width]:
    what belongs to the slots from now on, later tokens' included).  width: slots a request from now
    on (default: as weights has)."""
    return _evict("evict", False, kv_cache, block_table, seqlens, weights, budget, sink, recent, arrival, width,
                  new_seqlens, kept, weights_out, arrival_out, stream)


def evict_fp8(kv_cache, block_table, seqlens, weights, budget: int, sink: int = 0, recent: int = 0, arrival=None,
              width: int | None = None, new_seqlens=None, kept=None, weights_out=None, arrival_out=None, stream=None):
    """evict over an FP8 cache (one byte a value)."""
    return _evict("evict_fp8", True, kv_cache, block_table, seqlens, weights, budget, sink, recent, arrival, width,
                  new_seqlens, kept, weights_out, arrival_out, stream)


def get_device_status(stream=None) -> int:
    """Synchronize the stream; return and clear the kernels' device status word."""
    return lib().mla_get_device_status(_stream(stream))


def debug_withhold_first_load(enable: bool = True):
    lib().mla_debug_withhold_first_load(int(enable))


class DecodeStep:
    """One decode step of an MLA layer for a fixed batch shape: W_UK absorption,
    absorbed decode over the paged latent cache, LSE combine, W_UV un-absorption.

    Buffers (q, out, lse, o, metadata, workspace) are allocated once here, with
    torch, and reused; `run` launches only library kernels.  With kv_scale given, the
    cache passed to `run` / `capture` is an FP8 (E4M3) cache with that per-tensor scale.
    """

    def __init__(self, B: int, s_q: int, H: int, seqlens: torch.Tensor, causal: bool, softmax_scale: float,
                 parts: int | None = None, device="cuda", kv_scale: float | None = None):
        self.B, self.s_q, self.H = B, s_q, H
        self.causal, self.scale = causal, softmax_scale
        self.kv_scale = kv_scale
        self.parts = parts if parts is not None else num_sm_parts(s_q, H)
        dev = torch.device(device)
        self.q = torch.empty((B, s_q, H, 576), dtype=torch.bfloat16, device=dev)
        self.out = torch.empty((B, s_q, H, 512), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((B, s_q, H), dtype=torch.float32, device=dev)
        self.o = torch.empty((B * s_q, H, 128), dtype=torch.bfloat16, device=dev)
        self.workspace = torch.empty(decode_workspace_size(B, s_q, H, self.parts), dtype=torch.uint8, device=dev)
        self.seqlens = seqlens
        self.metadata = decode_metadata(seqlens, s_q, H, causal, self.parts)
        self._plan_stream = torch.cuda.Stream(device=dev)

    def plan(self, stream=None):
        """Recompute the split schedule (after seqlens changed)."""
        decode_metadata(self.seqlens, self.s_q, self.H, self.causal, self.parts, out=self.metadata, stream=stream)

    def plan_beside(self, work):
        """plan() on a side stream while `work()` (stream work that does not read the
        metadata, such as the W_UK absorption) runs on the current stream; the current
        stream then waits for both.  The schedule sees everything issued before the call."""
        cur = torch.cuda.current_stream(self.q.device)
        self._plan_stream.wait_stream(cur)
        with torch.cuda.stream(self._plan_stream):
            self.plan()
        work()
        cur.wait_stream(self._plan_stream)

    def absorb(self, q_nope, q_pe, w_uk, positions=None, rope_theta: float = 10000.0, stream=None, sections=None,
               interleaved: bool = False):
        """The W_UK absorption and the rest of the decode query: q_pe as it is, rotated by positions
        (int32 [B*s_q]) inside the absorption, or, with sections, by positions [axes, B*s_q] (rope_axes)."""
        self._check_axes(positions, sections)
        absorb_q(q_nope, w_uk, self.q, q_pe=None if sections is not None else q_pe, stream=stream,
                 positions=None if sections is not None else positions, rope_theta=rope_theta)
        self._rotate(q_pe, positions, rope_theta, sections, interleaved, stream)

    @staticmethod
    def _check_axes(positions, sections):
        if sections is not None and positions is None:
            raise ValueError("sections need positions [axes, B*s_q]")

    def _rotate(self, q_pe, positions, rope_theta, sections, interleaved, stream=None):
        if sections is not None:
            rope_axes(q_pe, positions, sections, out=self.q.view(self.B * self.s_q, self.H, 576)[..., 512:],
                      rope_theta=rope_theta, interleaved=interleaved, stream=stream)

    def absorb_and_plan(self, q_nope, q_pe, w_uk, positions=None, rope_theta: float = 10000.0, stream=None,
                        sections=None, interleaved: bool = False):
        """absorb() with plan() in the absorption's launch (B <= absorb_plan_max_batch(); else the
        two calls, the schedule on a side stream beside the absorption)."""
        self._check_axes(positions, sections)
        if sections is not None:
            self.absorb_and_plan(q_nope, None, w_uk, stream=stream)
            self._rotate(q_pe, positions, rope_theta, sections, interleaved, stream)
            return
        if self.B <= absorb_plan_max_batch():
            absorb_q_plan(q_nope, w_uk, self.q, self.seqlens, self.parts, self.metadata, q_pe=q_pe,
                          positions=positions, rope_theta=rope_theta, stream=stream)
        else:
            self.plan_beside(lambda: absorb_q(q_nope, w_uk, self.q, q_pe=q_pe, stream=stream, positions=positions,
                                              rope_theta=rope_theta))

    def _decode(self, kv_cache, block_table, stream=None):
        if self.kv_scale is None:
            decode(self.q, kv_cache, block_table, self.seqlens, self.scale, self.causal, self.metadata, self.parts,
                   workspace=self.workspace, out=self.out, lse=self.lse, stream=stream)
        else:
            decode_fp8(self.q, kv_cache, self.kv_scale, block_table, self.seqlens, self.scale, self.causal,
                       self.metadata, self.parts, workspace=self.workspace, out=self.out, lse=self.lse, stream=stream)

    def append(self, c, k_pe, kv_cache, block_table, positions=None, rope_theta: float = 10000.0, sections=(32,),
               interleaved: bool = False, stream=None):
        """The step's new rows (c [B*s_q,512], k_pe [B*s_q,64]) into the cache as each request's last s_q
        tokens (seqlens counts them), before `run`; k_pe rotated by positions where they are given.  In a batch
        padded with empty requests cache_append, whose new_offsets give those no row, is the call to make."""
        rot = dict(positions=positions, sections=sections, rope_theta=rope_theta, interleaved=interleaved, stream=stream)
        if self.kv_scale is None:
            cache_append(c, k_pe, kv_cache, block_table, self.seqlens, **rot)
        else:
            cache_append_fp8(c, k_pe, kv_cache, self.kv_scale, block_table, self.seqlens, **rot)

    def accumulate_weights(self, kv_cache, block_table, weights, stream=None):
        """Adds the attention weight of the step that `run` / `replay` has just done to weights [B, slots]."""
        if self.kv_scale is None:
            attn_weights(self.q, self.lse, kv_cache, block_table, self.seqlens, self.scale, self.causal, weights,
                         stream=stream)
        else:
            attn_weights_fp8(self.q, self.lse, kv_cache, self.kv_scale, block_table, self.seqlens, self.scale,
                             self.causal, weights, stream=stream)

    def evict(self, kv_cache, block_table, weights, budget: int, sink: int = 0, recent: int = 0, arrival=None,
              width: int | None = None, kept=None, weights_out=None, arrival_out=None, stream=None):
        """Evicts down to `budget` tokens a request (see evict()); seqlens is changed in place and the schedule
        recomputed.  Returns (kept, weights_out, arrival_out)."""
        call = evict if self.kv_scale is None else evict_fp8
        outs = call(kv_cache, block_table, self.seqlens, weights, budget, sink=sink, recent=recent, arrival=arrival,
                    width=width, new_seqlens=self.seqlens, kept=kept, weights_out=weights_out, arrival_out=arrival_out,
                    stream=stream)
        self.plan(stream=stream)
        return outs[1:]

    def run(self, q_nope, q_pe, w_uk, w_uv, kv_cache, block_table, stream=None, positions=None,
            rope_theta: float = 10000.0, sections=None, interleaved: bool = False):
        """q_nope [B*s_q,H,128], q_pe [B*s_q,H,64] -> o [B*s_q,H,128] (bf16); with positions
        (int32 [B*s_q]) q_pe is RoPE-rotated inside the absorption, with sections too by
        positions [axes, B*s_q] (rope_axes)."""
        self.absorb(q_nope, q_pe, w_uk, positions, rope_theta, stream, sections, interleaved)
        self._decode(kv_cache, block_table, stream=stream)
        unabsorb_o(self.out.view(self.B * self.s_q, self.H, 512), w_uv, o=self.o, stream=stream)
        return self.o

    def capture(self, q_nope, q_pe, w_uk, w_uv, kv_cache, block_table, plan=True, before=None, after=None,
                positions=None, rope_theta: float = 10000.0, sections=None, interleaved: bool = False):
        """Record the step (plan() if `plan`, then run()) into a CUDA graph; `replay()` relaunches it
        with one host call.  `before` / `after` are optional callables whose stream work (for example
        copies of the step's inputs from pinned host buffers, or of its result back) is recorded in
        the same graph.  The graph holds the addresses of every buffer: refill them in place between
        replays.  The step runs once, uncaptured, first (one-time library set-up happens there)."""
        rot = dict(positions=positions, rope_theta=rope_theta, sections=sections, interleaved=interleaved)

        def body():
            if before is not None:
                before()
            if plan:   # the schedule in the absorption's launch
                self.absorb_and_plan(q_nope, q_pe, w_uk, **rot)
            else:
                self.absorb(q_nope, q_pe, w_uk, **rot)
            self._decode(kv_cache, block_table)
            unabsorb_o(self.out.view(self.B * self.s_q, self.H, 512), w_uv, o=self.o)
            if after is not None:
                after()
        side = torch.cuda.Stream(device=self.q.device)
        side.wait_stream(torch.cuda.current_stream(self.q.device))
        with torch.cuda.stream(side):
            body()
        torch.cuda.current_stream(self.q.device).wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            body()
        self._graph = graph
        return graph

    def replay(self):
        """Relaunch the captured step on the current stream (see `capture`); returns o."""
        if getattr(self, "_graph", None) is None:
            raise RuntimeError("DecodeStep.replay() before capture()")
        self._graph.replay()
        return self.o

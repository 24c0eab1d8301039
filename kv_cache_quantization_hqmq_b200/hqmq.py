"""Thin Python binding of libhqmq (include/hqmq.h).

Argument marshalling only: every step of the HQMQ path runs in the CUDA
kernels of libhqmq.so.  torch provides device memory and streams.  There is no
fallback: if the library is missing or fails to load, importing this module
raises.

Entry points keep the C names.  Tensors are passed where the C ABI takes
device pointers; shapes and dtypes are read from them; `stream` defaults to
torch's current stream.  Non-zero return codes raise HQMQError.

A serving flow, per (layer, role) cache x [B, H, T, 128] (bf16):

    hqmq_make_codebook(seed, S, n_groups, 0, cb)          # once per model
    hqmq_make_search_table(cb_call, S, H, table)          # once per model (S <= 48)
    hqmq_encode_med3(x, 3.0, HQMQ_GRAN_CHUNK, cb_call, S, table, words, radius, rmed,
                     thr, out_idx, out_val, slab_off, cap, ws, tile_off=tile_off)
    # optional 2b bits per chunk: hqmq_quantize_radius(radius, thr, x.shape, S, rwords)
    # decode step, every (layer, role) at once, against the prefill's thr:
    hqmq_append_batch(x_new, thr_all, HQMQ_GRAN_CHUNK, cb_all, S, words_new, radius_new,
                      oi_new, ov_new, so_new, cap_new, tile_off=to_new)
    # attention of the new queries straight from the codes:
    k = kv_codes(words_k, radius_k, cb_k, out_idx_k, out_val_k, tile_off_k, cap, 0)
    v = kv_codes(words_v, radius_v, cb_v, out_idx_v, out_val_v, tile_off_v, cap, 0)
    hqmq_attention_decode(q, k, v, S, H, T, o, alloc_attention_ws(B, H), seq_len=lens)
    # or the dense cache: hqmq_decode(words, radius, cb_call, S, out_idx, out_val,
    #                                  slab_off, cap, 0, y, tile_off=tile_off)

The same over pages, for caches that grow and share prefixes (once per layer):

    words, radius, flags, val = alloc_kv_pages(n_pages, H, 64, S, out_cap=128)
    kp = kv_pages(words, radius, cb_k, flags, val, thr_k, table_k)     # vp likewise
    ws = alloc_attention_paged_ws(B, Hq, kp, max_pages, prefix_len)
    # every step: queries and keys normed and rotated, K and V quantised into the pages
    hqmq_qk_norm_rope(q, k, q, k, pos, rope_inv_freq(128, 500000.0), q_weight, k_weight)
    hqmq_paged_write(k_new, v_new, kp, vp, block_table, cu_tokens, pos0)
    hqmq_attention_paged(q_new, kp, vp, block_table, seq_len, o, ws,
                         prefix_table=prefix_table, prefix_len=prefix_len)
    # or the dense tokens: hqmq_paged_read(kp, block_table, seq_len, y)
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libhqmq.so")

HQMQ_OK, HQMQ_ERR_ARG, HQMQ_ERR_ALIGN, HQMQ_ERR_CUDA, HQMQ_ERR_WORKSPACE = 0, 1, 2, 3, 4
HQMQ_BF16, HQMQ_F32 = 0, 1
HQMQ_GRAN_CHUNK, HQMQ_GRAN_ELEMENT = 0, 1
FLAG_OUTLIER_OVERFLOW, FLAG_SATURATED, FLAG_NONFINITE, FLAG_BAD_INDEX = 1, 2, 4, 8
FLAG_MED3_FALLBACK = 16
FLAG_BAD_PAGE, FLAG_TIMEOUT = 32, 64


class HQMQError(RuntimeError):
    def __init__(self, fn, rc):
        super().__init__("%s failed: %s (%d)" % (fn, _lib.hqmq_error_string(rc).decode(), rc))
        self.rc = rc


if not os.path.exists(LIB_PATH):
    raise ImportError("libhqmq.so is not built (%s); run "
                      "`python -m kv_cache_quantization_hqmq_b200.build`" % LIB_PATH)

_lib = ctypes.CDLL(LIB_PATH)
_P, _I, _U32, _U64, _F = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_float
_I64 = ctypes.c_int64
_SIGS = {
    "hqmq_version": (ctypes.c_char_p, []),
    "hqmq_error_string": (ctypes.c_char_p, [_I]),
    "hqmq_index_bits": (_U32, [_U32]),
    "hqmq_index_words": (_U64, [_I, _I, _I, _I, _U32]),
    "hqmq_make_codebook": (_I, [_U64, _U32, _U32, _U32, _P, _P]),
    "hqmq_outlier_workspace_size": (_U64, [_I, _I, _I, _I, _I]),
    "hqmq_outlier_extract": (_I, [_P, _I, _I, _I, _I, _I, _F, _I, _P, _P, _P, _P, _P, _P, _U64,
                                  _P, _U64, _P, _P]),
    "hqmq_list_tiles": (_U64, [_I, _I, _I, _I]),
    "hqmq_encode": (_I, [_P, _I, _I, _I, _I, _I, _P, _U32, _P, _I, _P, _P, _P, _P]),
    "hqmq_decode": (_I, [_P, _P, _P, _U32, _P, _P, _P, _P, _U64, _I, _I, _I, _I, _I, _P, _I, _P,
                         _P]),
    "hqmq_outlier_extract_noalloc": (_I, [_P, _I, _I, _I, _I, _I, _F, _I, _P, _P, _P, _P, _P,
                                          _U64, _P, _P]),
    "hqmq_encode_med3_workspace_size": (_U64, [_I, _I, _I, _I, _I]),
    "hqmq_encode_med3": (_I, [_P, _I, _I, _I, _I, _I, _F, _I, _P, _U32, _P, _P, _P, _P, _P, _P,
                              _P, _P, _P, _U64, _P, _U64, _P, _P]),
    "hqmq_search_table_bytes": (_U64, [_U32]),
    "hqmq_make_search_table": (_I, [_P, _U32, _U32, _P, _P]),
    "hqmq_encode_lut": (_I, [_P, _I, _I, _I, _I, _I, _P, _U32, _P, _P, _I, _P, _P, _P, _P]),
    "hqmq_quantize_radius": (_I, [_P, _P, _I, _I, _I, _I, _U32, _P, _P]),
    "hqmq_append_batch": (_I, [_P, _I, _I, _I, _I, _I, _I, _P, _I, _P, _U32, _P, _P, _P, _P, _P,
                               _P, _U64, _P, _P]),
    "hqmq_outlier_extract_given_thr_workspace_size": (_U64, [_I, _I, _I, _I]),
    "hqmq_outlier_extract_given_thr": (_I, [_P, _I, _I, _I, _I, _I, _P, _I, _P, _P, _P, _P, _U64,
                                            _P, _U64, _P, _P]),
    "hqmq_decode_qradius": (_I, [_P, _P, _P, _P, _U32, _P, _P, _P, _U64, _I, _I, _I, _I, _I, _P,
                                 _I, _P, _P]),
    "hqmq_joint_block": (None, [_U32, _P, _P]),
    "hqmq_joint_words": (_U64, [_I, _I, _I, _I, _U32]),
    "hqmq_pack_joint": (_I, [_P, _P, _U32, _I, _I, _I, _I, _P, _P, _P]),
    "hqmq_list_flags": (_I, [_P, _P, _U64, _I, _I, _I, _I, _P, _P]),
    "hqmq_decode_joint": (_I, [_P, _P, _P, _U32, _P, _P, _P, _U64, _I, _I, _I, _I, _P, _I, _P]),
    "hqmq_attention_workspace_size": (_U64, [_I, _I]),
    "hqmq_attention_decode": (_I, [_P, _P, _P, _P, _U32, _I, _I, _I, _I, _I, _F, _P, _I, _P,
                                   _U64, _P, _P]),
    "hqmq_qk_norm_rope": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _I, _F, _P, _P, _I, _I, _P]),
    "hqmq_paged_write": (_I, [_P, _P, _P, _P, _I, _I64, _I64, _I64, _I64, _I, _I, _P, _P, _P, _I,
                              _P, _P]),
    "hqmq_paged_read": (_I, [_P, _I, _P, _P, _I, _I, _P, _I, _P, _P]),
    "hqmq_attention_paged_workspace_size": (_U64, [_I, _I, _I, _I, _I]),
    "hqmq_attention_paged": (_I, [_P, _P, _P, _I, _I, _P, _P, _I, _P, _I, _F, _P, _I, _P, _P, _U64,
                                  _P, _P]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def lib():
    return _lib


def _check(name, rc):
    if rc != HQMQ_OK:
        raise HQMQError(name, rc)


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return HQMQ_BF16
    if t.dtype == torch.float32:
        return HQMQ_F32
    raise TypeError("HQMQ tensors are bf16 or fp32, got %s" % t.dtype)


def _shape4(x):
    if x.dim() != 4:
        raise ValueError("expected a [B, H, T, D] tensor, got shape %s" % (tuple(x.shape),))
    if not x.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return tuple(int(v) for v in x.shape)


# ---------------------------------------------------------------- queries
def hqmq_version():
    return _lib.hqmq_version().decode()


def hqmq_index_bits(S):
    return int(_lib.hqmq_index_bits(S))


def hqmq_index_words(B, H, T, D, S):
    return int(_lib.hqmq_index_words(B, H, T, D, S))


def hqmq_outlier_workspace_size(B, H, T, D, gran=HQMQ_GRAN_CHUNK):
    return int(_lib.hqmq_outlier_workspace_size(B, H, T, D, gran))


def hqmq_encode_med3_workspace_size(B, H, T, D, gran=HQMQ_GRAN_CHUNK):
    return int(_lib.hqmq_encode_med3_workspace_size(B, H, T, D, gran))


# ---------------------------------------------------------------- calls
def hqmq_make_codebook(seed, S, n_groups, group0, codebook, stream=None):
    """codebook: fp32 device tensor of n_groups * S * 4 elements."""
    assert codebook.dtype == torch.float32 and codebook.numel() == n_groups * S * 4
    _check("hqmq_make_codebook", _lib.hqmq_make_codebook(seed, S, n_groups, group0,
                                                         _ptr(codebook), _stream(stream)))
    return codebook


def hqmq_outlier_extract(x, C, gran, rmed, thr, out_idx, out_val, slab_off, cap, ws,
                         status=None, stream=None, tile_off=None):
    """tile_off: optional uint32 [hqmq_list_tiles(B, H, T, D) + 1] output."""
    B, H, T, D = _shape4(x)
    _check("hqmq_outlier_extract", _lib.hqmq_outlier_extract(
        _ptr(x), _dtype_code(x), B, H, T, D, float(C), gran, _ptr(rmed), _ptr(thr),
        _ptr(out_idx), _ptr(out_val), _ptr(slab_off), _ptr(tile_off), int(cap), _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(status), _stream(stream)))


def hqmq_list_tiles(B, H, T, D):
    return int(_lib.hqmq_list_tiles(B, H, T, D))


def hqmq_outlier_extract_noalloc(x, C, gran, rmed, thr, out_idx, out_val, slab_off, cap,
                                 status=None, stream=None):
    """Med3x with the library's fixed 1 MiB device scratch instead of a
    caller workspace, for callers that cannot allocate device memory.  Calls
    on one device share that scratch: do not let two of them overlap."""
    B, H, T, D = _shape4(x)
    _check("hqmq_outlier_extract_noalloc", _lib.hqmq_outlier_extract_noalloc(
        _ptr(x), _dtype_code(x), B, H, T, D, float(C), gran, _ptr(rmed), _ptr(thr),
        _ptr(out_idx), _ptr(out_val), _ptr(slab_off), int(cap), _ptr(status), _stream(stream)))


def hqmq_encode(x, codebook, S, thr, gran, idx_words, radius, status=None, stream=None):
    B, H, T, D = _shape4(x)
    _check("hqmq_encode", _lib.hqmq_encode(
        _ptr(x), _dtype_code(x), B, H, T, D, _ptr(codebook), S, _ptr(thr), gran,
        _ptr(idx_words), _ptr(radius), _ptr(status), _stream(stream)))


def hqmq_search_table_bytes(S):
    return int(_lib.hqmq_search_table_bytes(S))


def hqmq_make_search_table(codebook, S, n_groups, table, stream=None):
    """table: uint8 device tensor of n_groups * hqmq_search_table_bytes(S) bytes."""
    assert table.numel() * table.element_size() >= n_groups * hqmq_search_table_bytes(S)
    _check("hqmq_make_search_table", _lib.hqmq_make_search_table(
        _ptr(codebook), S, n_groups, _ptr(table), _stream(stream)))
    return table


def hqmq_encode_lut(x, codebook, S, table, thr, gran, idx_words, radius, status=None,
                    stream=None):
    B, H, T, D = _shape4(x)
    _check("hqmq_encode_lut", _lib.hqmq_encode_lut(
        _ptr(x), _dtype_code(x), B, H, T, D, _ptr(codebook), S, _ptr(table), _ptr(thr), gran,
        _ptr(idx_words), _ptr(radius), _ptr(status), _stream(stream)))


def hqmq_encode_med3(x, C, gran, codebook, S, table, idx_words, radius, rmed, thr, out_idx,
                     out_val, slab_off, cap, ws, status=None, stream=None, tile_off=None):
    """Med3x + encode (table may be None: S-codeword loop); tile_off: optional
    uint32 [hqmq_list_tiles(B, H, T, D) + 1] output."""
    B, H, T, D = _shape4(x)
    _check("hqmq_encode_med3", _lib.hqmq_encode_med3(
        _ptr(x), _dtype_code(x), B, H, T, D, float(C), gran, _ptr(codebook), S, _ptr(table),
        _ptr(idx_words), _ptr(radius), _ptr(rmed), _ptr(thr), _ptr(out_idx), _ptr(out_val),
        _ptr(slab_off), _ptr(tile_off), int(cap), _ptr(ws), ws.numel() * ws.element_size(),
        _ptr(status), _stream(stream)))


def hqmq_decode(idx_words, radius, codebook, S, out_idx, out_val, slab_off, cap, gran, y,
                status=None, stream=None, tile_off=None):
    """tile_off: the list's tile offsets (applied in the main pass), or None."""
    B, H, T, D = _shape4(y)
    _check("hqmq_decode", _lib.hqmq_decode(
        _ptr(idx_words), _ptr(radius), _ptr(codebook), S, _ptr(out_idx), _ptr(out_val),
        _ptr(slab_off), _ptr(tile_off), int(cap), gran, B, H, T, D, _ptr(y), _dtype_code(y),
        _ptr(status), _stream(stream)))


def hqmq_outlier_extract_given_thr_workspace_size(B, H, T, D):
    return int(_lib.hqmq_outlier_extract_given_thr_workspace_size(B, H, T, D))


def hqmq_outlier_extract_given_thr(x, thr, gran, out_idx, out_val, slab_off, cap, ws,
                                   status=None, stream=None, tile_off=None):
    """Med3x list of x under a given threshold thr [H] (no median of its own):
    the streaming form for decode-phase tokens."""
    B, H, T, D = _shape4(x)
    _check("hqmq_outlier_extract_given_thr", _lib.hqmq_outlier_extract_given_thr(
        _ptr(x), _dtype_code(x), B, H, T, D, _ptr(thr), gran, _ptr(out_idx), _ptr(out_val),
        _ptr(slab_off), _ptr(tile_off), int(cap), _ptr(ws), ws.numel() * ws.element_size(),
        _ptr(status), _stream(stream)))


def hqmq_append_batch(x, thr, gran, codebook, S, idx_words, radius, out_idx, out_val, slab_off,
                      cap, tile_off=None, status=None, stream=None):
    """n_calls small calls in one launch; x: [n_calls, B, H, T, D]; every other
    array holds the calls' arrays back to back (see include/hqmq.h)."""
    if x.dim() != 5 or not x.is_contiguous():
        raise ValueError("x must be a contiguous [n_calls, B, H, T, D] tensor")
    C, B, H, T, D = (int(v) for v in x.shape)
    _check("hqmq_append_batch", _lib.hqmq_append_batch(
        _ptr(x), _dtype_code(x), C, B, H, T, D, _ptr(thr), gran, _ptr(codebook), S,
        _ptr(idx_words), _ptr(radius), _ptr(out_idx), _ptr(out_val), _ptr(slab_off),
        _ptr(tile_off), int(cap), _ptr(status), _stream(stream)))


def hqmq_quantize_radius(radius, thr, shape, S, rcode_words, stream=None):
    """Radius codes (b bits per chunk, uniform on [0, thr_h], 24 S levels) of a
    call's fp16 radii; shape = (B, H, T, D)."""
    B, H, T, D = shape
    _check("hqmq_quantize_radius", _lib.hqmq_quantize_radius(
        _ptr(radius), _ptr(thr), B, H, T, D, S, _ptr(rcode_words), _stream(stream)))
    return rcode_words


def hqmq_decode_qradius(idx_words, rcode_words, thr, codebook, S, out_idx, out_val, tile_off,
                        cap, gran, y, status=None, stream=None):
    """hqmq_decode with the radii taken from their codes; a list needs tile_off."""
    B, H, T, D = _shape4(y)
    _check("hqmq_decode_qradius", _lib.hqmq_decode_qradius(
        _ptr(idx_words), _ptr(rcode_words), _ptr(thr), _ptr(codebook), S, _ptr(out_idx),
        _ptr(out_val), _ptr(tile_off), int(cap), gran, B, H, T, D, _ptr(y), _dtype_code(y),
        _ptr(status), _stream(stream)))


def hqmq_joint_block(S):
    """(chunks per block, bits per block) of the joint (index, level) code."""
    n, w = ctypes.c_uint32(0), ctypes.c_uint32(0)
    _lib.hqmq_joint_block(S, ctypes.byref(n), ctypes.byref(w))
    return n.value, w.value


def hqmq_joint_words(B, H, T, D, S):
    return int(_lib.hqmq_joint_words(B, H, T, D, S))


def alloc_joint(B, H, T, D, S, device="cuda"):
    n = hqmq_joint_words(B, H, T, D, S)
    if n == 0:
        raise ValueError("bad shape/S for the joint code")
    return torch.empty(n, dtype=torch.int32, device=device)


def hqmq_pack_joint(idx_words, rcode_words, S, shape, joint, status=None, stream=None):
    """The joint code of a call (shape = (B, H, T, D)) from its index and
    radius-code words."""
    B, H, T, D = shape
    _check("hqmq_pack_joint", _lib.hqmq_pack_joint(
        _ptr(idx_words), _ptr(rcode_words), S, B, H, T, D, _ptr(joint), _ptr(status),
        _stream(stream)))
    return joint


def hqmq_list_flags(out_idx, slab_off, cap, shape, flags, stream=None):
    """The 1-bit outlier flags (uint32 [B*H*T*D/128]) of a chunk-mode list."""
    B, H, T, D = shape
    _check("hqmq_list_flags", _lib.hqmq_list_flags(
        _ptr(out_idx), _ptr(slab_off), int(cap), B, H, T, D, _ptr(flags), _stream(stream)))
    return flags


def hqmq_decode_joint(joint, thr, codebook, S, flags, out_val, tile_off, cap, y, stream=None):
    """Decode from the joint code; flags (with the list's values and tile
    offsets) restore the chunk-mode outliers, or None."""
    B, H, T, D = _shape4(y)
    _check("hqmq_decode_joint", _lib.hqmq_decode_joint(
        _ptr(joint), _ptr(thr), _ptr(codebook), S, _ptr(flags), _ptr(out_val), _ptr(tile_off),
        int(cap), B, H, T, D, _ptr(y), _dtype_code(y), _stream(stream)))


class KVCodes(ctypes.Structure):
    """hqmq_kv_codes: one coded K or V cache (device pointers)."""
    _fields_ = [("idx_words", _P), ("radius", _P), ("codebook", _P), ("out_idx", _P),
                ("out_val", _P), ("tile_off", _P), ("cap", _U64), ("gran", _I),
                ("rcode_words", _P), ("thr", _P)]


def kv_codes(idx_words, radius, codebook, out_idx=None, out_val=None, tile_off=None, cap=0,
             gran=HQMQ_GRAN_CHUNK, rcode_words=None, thr=None):
    """The hqmq_kv_codes record of one coded cache (the tensors must outlive
    the calls that use it).  rcode_words + thr: the quantized-radius format
    (radius may then be None)."""
    c = KVCodes(_ptr(idx_words), _ptr(radius), _ptr(codebook), _ptr(out_idx), _ptr(out_val),
                _ptr(tile_off), int(cap) if out_idx is not None else 0, int(gran),
                _ptr(rcode_words), _ptr(thr))
    c._keep = (idx_words, radius, codebook, out_idx, out_val, tile_off, rcode_words, thr)
    return c


def hqmq_attention_workspace_size(B, Hk):
    return int(_lib.hqmq_attention_workspace_size(B, Hk))


def hqmq_attention_decode(q, k, v, S, Hk, T, o, ws, scale=None, seq_len=None, status=None,
                          stream=None):
    """o[b, h] = softmax(scale q[b, h] K^T) V over the first seq_len[b] tokens
    of the coded caches k, v (KVCodes from kv_codes; [B, Hk, T, 128]).
    q: bf16 [B, Hq, 128]; o: bf16 or fp32 [B, Hq, 128]; seq_len: int32 [B]
    or None; scale defaults to 1/sqrt(128)."""
    if q.dim() != 3 or q.dtype != torch.bfloat16 or not q.is_contiguous():
        raise ValueError("q must be a contiguous bf16 [B, Hq, D] tensor")
    B, Hq, D = (int(v_) for v_ in q.shape)
    if scale is None:
        scale = D ** -0.5
    _check("hqmq_attention_decode", _lib.hqmq_attention_decode(
        _ptr(q), _ptr(seq_len), ctypes.byref(k), ctypes.byref(v), S, B, Hq, Hk, T, D,
        float(scale), _ptr(o), _dtype_code(o), _ptr(ws), ws.numel() * ws.element_size(),
        _ptr(status), _stream(stream)))
    return o


def alloc_attention_ws(B, Hk, device="cuda"):
    return torch.empty(hqmq_attention_workspace_size(B, Hk), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------- paged cache
_BF16, _F32, _I32, _F64 = torch.bfloat16, torch.float32, torch.int32, torch.float64
_DTYPE_CODE = {torch.bfloat16: HQMQ_BF16, torch.float32: HQMQ_F32}


# torch.cuda.current_device without its check that CUDA is up: tensors on a device are there already, and
# without any the answer does not match theirs
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
# the current stream's handle without a Stream object (None: a torch that has no such shortcut)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_INT_MAX = 0x7FFFFFFF                                     # ctypes cuts larger numbers off


def _here(*tensors):
    """The current CUDA device, on which all of the tensors have to be (the calls launch there)."""
    dev = _current_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:       # (-1 for a CPU tensor)
            raise ValueError("tensors must be on the current CUDA device %d, got one on %s "
                             "(call under torch.cuda.device)" % (dev, t.device))
    return dev


def _on(stream, dev):
    """The stream's handle; None: torch's current stream of the device."""
    if stream is None:
        return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream
    return _stream(stream)


def _code(t):
    c = _DTYPE_CODE.get(t.dtype)
    return _dtype_code(t) if c is None else c


def _addr(t):
    return None if t is None else t.data_ptr()


def _ints(name, t, shape):
    if t is None or t.dtype is not _I32 or t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor of shape %s, got %s"
                         % (name, tuple(shape), t if t is None else (t.dtype, tuple(t.shape))))


def _table(t, n_seqs=None, name="block_table"):
    s = () if t is None else t.shape
    if len(s) != 2 or (n_seqs is not None and s[0] != n_seqs) or t.dtype is not _I32 or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 [n_seqs, max_pages], got %s"
                         % (name, t if t is None else (t.dtype, tuple(s))))
    return s[1]


class KVPages(ctypes.Structure):
    """hqmq_kv_pages: a paged coded K or V cache (device pointers)."""
    _fields_ = [("idx_words", _P), ("radius", _P), ("flags", _P), ("out_val", _P),
                ("codebook", _P), ("thr", _P), ("table", _P), ("S", _U32), ("n_pages", _I),
                ("page_size", _I), ("heads", _I), ("out_cap", _I)]


def alloc_kv_pages(n_pages, heads, page_size, S, out_cap=0, device="cuda"):
    """(idx_words, radius, flags, out_val) of an empty pool: int32 [n_pages, heads, page_size, b],
    fp16 bits as int16 [..., 32], int32 [n_pages, heads, page_size] and int16 [n_pages, heads,
    out_cap, 4]; the last two None if out_cap is 0 (no outliers)."""
    words = torch.zeros(n_pages, heads, page_size, hqmq_index_bits(S), dtype=torch.int32, device=device)
    radius = torch.zeros(n_pages, heads, page_size, 32, dtype=torch.int16, device=device)
    if not out_cap:
        return words, radius, None, None
    flags = torch.zeros(n_pages, heads, page_size, dtype=torch.int32, device=device)
    out_val = torch.zeros(n_pages, heads, out_cap, 4, dtype=torch.int16, device=device)
    return words, radius, flags, out_val


def kv_pages(idx_words, radius, codebook, flags=None, out_val=None, thr=None, table=None):
    """The hqmq_kv_pages record of one paged cache (the tensors must outlive the
    calls that use it), shapes as alloc_kv_pages gives them; codebook: fp32
    [heads, S, 4]; thr: fp32 [heads] (to write with flags); table: the search
    tables of the heads' codebooks or None."""
    if codebook.dim() != 3 or codebook.shape[2] != 4:
        raise ValueError("codebook must be fp32 [heads, S, 4]")
    heads, S = int(codebook.shape[0]), int(codebook.shape[1])
    b = hqmq_index_bits(S)
    if idx_words.dim() != 4 or idx_words.shape[1] != heads or idx_words.shape[3] != b:
        raise ValueError("idx_words must be [n_pages, %d, page_size, %d], got %s"
                         % (heads, b, tuple(idx_words.shape)))
    n_pages, _, P, _ = (int(v) for v in idx_words.shape)
    if (flags is None) != (out_val is None):
        raise ValueError("flags and out_val come together")
    cap = int(out_val.shape[2]) if out_val is not None and out_val.dim() == 4 else 0
    want = (("idx_words", idx_words, (n_pages, heads, P, b), 4),
            ("radius", radius, (n_pages, heads, P, 32), 2),
            ("flags", flags, (n_pages, heads, P), 4),
            ("out_val", out_val, (n_pages, heads, cap, 4), 2),
            ("codebook", codebook, (heads, S, 4), 4), ("thr", thr, (heads,), 4))
    for name, t, shape, size in want:
        if t is None and name in ("flags", "out_val", "thr"):
            continue
        if tuple(t.shape) != shape or t.element_size() != size or not t.is_contiguous():
            raise ValueError("%s must be contiguous %s of %d-byte elements, got %s %s"
                             % (name, shape, size, t.dtype, tuple(t.shape)))
    if codebook.dtype != torch.float32 or (thr is not None and thr.dtype != torch.float32):
        raise ValueError("codebook and thr are fp32")
    if table is not None and (not hqmq_search_table_bytes(S) or not table.is_contiguous() or
                              table.numel() * table.element_size() < heads * hqmq_search_table_bytes(S)):
        raise ValueError("table must hold the search tables of %d heads" % heads)
    _here(idx_words, radius, flags, out_val, codebook, thr, table)
    c = KVPages(_ptr(idx_words), _ptr(radius), _ptr(flags), _ptr(out_val), _ptr(codebook), _ptr(thr),
                _ptr(table), S, n_pages, P, heads, cap)
    c._keep = (idx_words, radius, flags, out_val, codebook, thr, table)
    c._ref = ctypes.byref(c)
    return c


class _HeadView(ctypes.Structure):
    """hqmq_head_view."""
    _fields_ = [("data", _P), ("stride_b", _I64), ("stride_t", _I64), ("stride_h", _I64), ("heads", _I)]


_pack_view = struct.Struct("=4qi4x").pack                # its bytes
assert ctypes.sizeof(_HeadView) == 40 == len(_pack_view(0, 0, 0, 0, 0))


def _head_view(x, heads, D):
    sb, st, sh, sd = x.stride()
    if sd != 1 and D > 1:
        raise ValueError("the last dimension must be contiguous")
    return _pack_view(x.data_ptr(), sb, st, sh, heads)


def rope_inv_freq(R, base=10000.0, device="cuda"):
    """fp64 [R / 2] of base^(-2 i / R), the d_inv_freq of hqmq_qk_norm_rope."""
    return base ** -(torch.arange(0, R, 2, dtype=torch.float64, device=device) / R)


def hqmq_qk_norm_rope(q, k, q_out, k_out, pos, inv_freq, q_weight=None, k_weight=None, eps=1e-6,
                      interleaved=False, stream=None):
    """RMS norm (where a weight is given) of every head vector of q [B, T, Hq, D] and
    k [B, T, Hk, D] and the rotation of its first 2 len(inv_freq) elements by
    pos [B, T] (int32) * inv_freq (fp64, or None), into q_out and k_out: the same
    shapes, strides of their own (q_out may be q).  q or k may be None."""
    x = q if q is not None else k
    if x is None or x.dim() != 4:
        raise ValueError("q and k are [B, T, heads, D]")
    shape, dt = x.shape, x.dtype
    B, T, _, D = shape
    views, w, w_dt = [], None, HQMQ_BF16
    for t, t_out, wt in ((q, q_out, q_weight), (k, k_out, k_weight)):
        if t is None:
            if t_out is not None or wt is not None:
                raise ValueError("an output or weight without its input")
            views += (None, None)
            continue
        s = shape if t is x else t.shape
        if t_out is None or len(s) != 4 or t_out.shape != s or t.dtype is not dt or t_out.dtype is not dt or \
                (t is not x and (s[0] != B or s[1] != T or s[3] != D)):
            raise ValueError("q, k and their outputs must agree in B, T, D and dtype")
        if wt is not None:
            if wt.dim() != 1 or wt.shape[0] != D or not wt.is_contiguous():
                raise ValueError("weights are contiguous [D]")
            if w is not None and wt.dtype is not w.dtype:
                raise ValueError("the weights must have one dtype")
            w, w_dt = wt, _code(wt)
        v = _head_view(t, s[2], D)
        views += (v, v if t_out is t else _head_view(t_out, s[2], D))
    R = 0
    if inv_freq is not None:
        if inv_freq.dtype is not _F64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be a contiguous fp64 vector")
        R = 2 * inv_freq.shape[0]
        _ints("pos", pos, (B, T))
    dev = _here(q, k, q_out, k_out, pos, inv_freq, q_weight, k_weight)
    rc = _lib.hqmq_qk_norm_rope(
        *views, _code(x), B, T, D, _addr(q_weight), _addr(k_weight), w_dt, eps, _addr(pos), _addr(inv_freq), R, 1 if interleaved else 0, _on(stream, dev))
    if rc:
        _check("hqmq_qk_norm_rope", rc)


def hqmq_paged_write(xk, xv, k, v, block_table, cu_tokens, pos0, status=None, stream=None):
    """Quantises new tokens xk, xv ([n_tokens, heads, 128], bf16 or fp32, any token
    and head strides) into the pages k, v (KVPages): sequence b's are rows
    cu_tokens[b] .. cu_tokens[b+1]-1 and go to positions pos0[b], pos0[b]+1, ...
    block_table: int32 [n_seqs, max_pages]; cu_tokens: int32 [n_seqs + 1]; pos0:
    int32 [n_seqs].  xv and v may be None."""
    s, ks, vs, v_ref, v_keep = xk.shape, xk.stride(), (0, 0, 1), None, None
    if v is not None:
        if xv is None or xv.shape != s or xv.dtype is not xk.dtype:
            raise ValueError("xk and xv must agree in shape and dtype (and xv be there where v is)")
        vs, v_ref, v_keep = xv.stride(), v._ref, v._keep[0]
    if len(s) != 3 or s[1] != k.heads or s[2] != 128 or ks[2] != 1 or vs[2] != 1 or s[0] > _INT_MAX:
        raise ValueError("new tokens are [n_tokens < 2^31, %d, 128] with a contiguous last dimension, got "
                         "%s" % (k.heads, tuple(s)))
    max_pages = _table(block_table)
    n_seqs = block_table.shape[0]
    _ints("pos0", pos0, (n_seqs,))
    _ints("cu_tokens", cu_tokens, (n_seqs + 1,))
    dev = _here(xk, xv, k._keep[0], v_keep, block_table, cu_tokens, pos0, status)
    rc = _lib.hqmq_paged_write(
        k._ref, v_ref, xk.data_ptr(), _addr(xv), _code(xk), ks[0], ks[1], vs[0], vs[1], s[0], n_seqs,
        cu_tokens.data_ptr(), pos0.data_ptr(), block_table.data_ptr(), max_pages, _addr(status), _on(stream, dev))
    if rc:
        _check("hqmq_paged_write", rc)


def hqmq_paged_read(c, block_table, seq_len, y, status=None, stream=None):
    """y[b, h, t] (contiguous [n_seqs, heads, T, 128], bf16 or fp32) = the token at
    position t < seq_len[b] of sequence b; the other rows are left as they are."""
    B, H, T, D = _shape4(y)
    if H != c.heads or D != 128:
        raise ValueError("y must be [n_seqs, %d, T, 128]" % c.heads)
    _ints("seq_len", seq_len, (B,))
    max_pages = _table(block_table, B)
    dev = _here(c._keep[0], block_table, seq_len, y, status)
    rc = _lib.hqmq_paged_read(c._ref, B, seq_len.data_ptr(), block_table.data_ptr(), max_pages, T, y.data_ptr(),
                              _code(y), _addr(status), _on(stream, dev))
    if rc:
        _check("hqmq_paged_read", rc)
    return y


def hqmq_attention_paged_workspace_size(B, Hq, Hk, max_tokens, prefix_len=0):
    if max(B, Hq, Hk, max_tokens, prefix_len) > _INT_MAX:
        return 0
    return int(_lib.hqmq_attention_paged_workspace_size(B, Hq, Hk, max_tokens, prefix_len))


def alloc_attention_paged_ws(B, Hq, k, max_pages, prefix_len=0, device="cuda"):
    """Workspace of hqmq_attention_paged over pages like k (KVPages)."""
    n = hqmq_attention_paged_workspace_size(B, Hq, k.heads, max_pages * k.page_size, prefix_len)
    if n == 0:
        raise ValueError("sizes that hqmq_attention_paged does not take")
    return torch.empty(n, dtype=torch.uint8, device=device)


def hqmq_attention_paged(q, k, v, block_table, seq_len, o, ws, prefix_table=None, prefix_len=0,
                         scale=None, lse=None, status=None, stream=None):
    """o[b, h] = softmax(scale q[b, h] K^T) V over the prefix's prefix_len tokens
    (prefix_table: int32 pages, shared by the batch and processed once for it)
    and the seq_len[b] tokens of sequence b's row of block_table (None: the
    prefix alone).  q: bf16 [B, Hq, 128]; o: bf16 or fp32 [B, Hq, 128]; lse:
    fp32 [B, Hq] or None; scale defaults to 1/sqrt(128)."""
    if q.dim() != 3 or q.dtype is not _BF16 or not q.is_contiguous():
        raise ValueError("q must be a contiguous bf16 [B, Hq, 128] tensor")
    B, Hq, D = q.shape
    if D != 128 or o.shape != q.shape or not o.is_contiguous():
        raise ValueError("q and o are contiguous [B, Hq, 128]")
    max_pages = 0
    if block_table is not None:
        max_pages = _table(block_table, B)
        _ints("seq_len", seq_len, (B,))
    if prefix_len > 0:
        need = (prefix_len + k.page_size - 1) // k.page_size
        if prefix_len > _INT_MAX:
            raise ValueError("prefix_len must be below 2^31, got %d" % prefix_len)
        if prefix_table is None or prefix_table.dim() != 1 or prefix_table.shape[0] < need:
            raise ValueError("prefix_table must hold the prefix's %d pages" % need)
        _ints("prefix_table", prefix_table, prefix_table.shape)
    if lse is not None and (lse.dtype is not _F32 or lse.shape != (B, Hq) or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous fp32 [B, Hq] tensor")
    dev = _here(q, k._keep[0], v._keep[0], block_table, seq_len, o, ws, prefix_table, lse, status)
    rc = _lib.hqmq_attention_paged(
        q.data_ptr(), k._ref, v._ref, B, Hq, _addr(seq_len), _addr(block_table), max_pages, _addr(prefix_table),
        prefix_len, D ** -0.5 if scale is None else scale, o.data_ptr(), _code(o), _addr(lse), ws.data_ptr(),
        ws.numel() * ws.element_size(), _addr(status), _on(stream, dev))
    if rc:
        _check("hqmq_attention_paged", rc)
    return o


# ---------------------------------------------------------------- buffers
def new_status(device="cuda"):
    """A zeroed device hqmq_status (4 x 64-bit words)."""
    return torch.zeros(4, dtype=torch.int64, device=device)


def read_status(status):
    v = status.cpu().numpy().view("uint64")
    return {"flags": int(v[0] & 0xFFFFFFFF), "n_outliers": int(v[1]),
            "n_saturated": int(v[2]), "n_nonfinite": int(v[3])}


def alloc_codes(B, H, T, D, S, device="cuda"):
    """(idx_words uint32 as int32, radius fp16 bits as int16) for one call."""
    nw = hqmq_index_words(B, H, T, D, S)
    if nw == 0:
        raise ValueError("bad shape/S")
    words = torch.empty(nw, dtype=torch.int32, device=device)
    radius = torch.empty(B * H * T * D // 4, dtype=torch.int16, device=device)
    return words, radius


def alloc_tile_off(B, H, T, D, device="cuda"):
    """uint32 (as int32) [hqmq_list_tiles + 1]: a call's list tile offsets."""
    n = hqmq_list_tiles(B, H, T, D)
    if n == 0:
        raise ValueError("bad shape")
    return torch.empty(n + 1, dtype=torch.int32, device=device)


def alloc_outliers(B, H, T, D, cap, gran=HQMQ_GRAN_CHUNK, device="cuda"):
    """(rmed, thr, out_idx, out_val, slab_off, ws) for one call's Med3x step."""
    rmed = torch.empty(H, dtype=torch.float32, device=device)
    thr = torch.empty(H, dtype=torch.float32, device=device)
    out_idx = torch.empty(max(cap, 1), dtype=torch.int32, device=device)
    out_val = torch.empty(max(cap, 1) * (4 if gran == HQMQ_GRAN_CHUNK else 1), dtype=torch.int16,
                          device=device)
    slab_off = torch.empty(B * H + 1, dtype=torch.int32, device=device)
    ws = torch.empty(hqmq_outlier_workspace_size(B, H, T, D, gran), dtype=torch.uint8,
                     device=device)
    return rmed, thr, out_idx, out_val, slab_off, ws

"""ctypes binding over libkvc.so (C ABI in include/kvc.h).

Argument marshalling only: every step of the coder runs in the library's
HIP kernels.  torch supplies device memory and the current HIP stream.
Importing this module loads the library and raises ImportError if it has not
been built (``python -m entropy_coding_amd.build``); there is no fallback.
"""

from __future__ import annotations

import ctypes
import math
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# KVC_LIBRARY names another build of the same library (the CPU tests load
# the sanitizer build this way); by default the in-tree libkvc.so.
LIB_PATH = os.environ.get("KVC_LIBRARY") or os.path.join(_HERE, "libkvc.so")

KVC_OK, KVC_ERR_INVALID, KVC_ERR_CAPACITY, KVC_ERR_CORRUPT, KVC_ERR_MISMATCH, KVC_ERR_DEVICE = 0, -1, -2, -3, -4, -5
KVC_BF16, KVC_E4M3, KVC_F32 = 0, 1, 2
HEADER_BYTES = 128
DECODE_WORKSPACE_BYTES = 917504
NOALLOC_SCRATCH_BYTES = 917504
ESTIMATE_WORKSPACE_BYTES = 256
ENCODE_STAGES = 2     # side-information checksum + per-call tables, coding kernel (with the stream's layout)
DECODE_STAGES = 2     # side-information checksum + escape bucket table, decoding kernel

EXPORTS = [
    "kvc_version", "kvc_status_string", "kvc_phi_tables", "kvc_narrow_table", "kvc_encode_sizes", "kvc_encode", "kvc_encode_result",
    "kvc_stream_info", "kvc_decode", "kvc_decode_async", "kvc_decode_result", "kvc_decode_noalloc",
    "kvc_decode_paged", "kvc_reload",
    "kvc_calibrate_sigma", "kvc_calibrate_sigma_blocks", "kvc_calibrate_sigma_rate", "kvc_calibrate_split",
    "kvc_build_marginal", "kvc_estimate_bits", "kvc_cdf_table",
    "kvc_build_block_table", "kvc_block_table_result", "kvc_paged_append",
    "kvc_paged_attention_sizes", "kvc_paged_attention", "kvc_paged_attention_result",
    "kvc_paged_qkv", "kvc_verify_drafts_sizes", "kvc_verify_drafts", "kvc_verify_drafts_result",
    "kvc_paged_compact", "kvc_paged_compact_result", "kvc_fork_pages", "kvc_release_pages", "kvc_shared_pages_result",
]

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -m entropy_coding_amd.build`")
_lib = ctypes.CDLL(LIB_PATH)


class kvc_params(ctypes.Structure):
    _fields_ = [
        ("kv_dtype", ctypes.c_int32), ("mu_dtype", ctypes.c_int32),
        ("w_narrow_bp", ctypes.c_uint32), ("w_wide_bp", ctypes.c_uint32),
        ("chunk_tokens", ctypes.c_uint32), ("sigma_block_tokens", ctypes.c_uint32),
        ("narrow_dof", ctypes.c_uint32), ("channel_split", ctypes.c_uint32),
        ("planes", ctypes.c_int64), ("tokens", ctypes.c_int64), ("channels", ctypes.c_int64),
    ]


class kvc_paged_kv(ctypes.Structure):
    _fields_ = [
        ("d_pools", ctypes.c_void_p), ("d_block_table", ctypes.c_void_p),
        ("n_pools", ctypes.c_int64), ("pool_bytes", ctypes.c_uint64),
        ("batch", ctypes.c_int64), ("heads", ctypes.c_int64), ("max_pages", ctypes.c_int64),
        ("num_pages", ctypes.c_int64), ("page_tokens", ctypes.c_uint32), ("reserved", ctypes.c_uint32),
    ]


class kvc_encode_info(ctypes.Structure):
    _fields_ = [("stage_ms", ctypes.c_float * ENCODE_STAGES)]


class kvc_decode_info(ctypes.Structure):
    _fields_ = [("stage_ms", ctypes.c_float * 2), ("reserved", ctypes.c_uint32),
                ("fallback_symbols", ctypes.c_uint64)]


class kvc_block_table(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64), ("max_pages", ctypes.c_int64), ("num_pages", ctypes.c_int64),
        ("free_capacity", ctypes.c_int64), ("max_rows", ctypes.c_int64),
        ("page_tokens", ctypes.c_uint32), ("trim", ctypes.c_uint32),
        ("d_cached_lens", ctypes.c_void_p), ("d_new_lens", ctypes.c_void_p), ("d_held_in", ctypes.c_void_p),
        ("d_held_out", ctypes.c_void_p), ("d_block_table", ctypes.c_void_p), ("d_free_pages", ctypes.c_void_p),
        ("d_free_in", ctypes.c_void_p), ("d_free_out", ctypes.c_void_p), ("d_row_starts", ctypes.c_void_p),
        ("d_slots", ctypes.c_void_p), ("d_positions", ctypes.c_void_p),
    ]


class kvc_attention(ctypes.Structure):
    _fields_ = [
        ("d_q", ctypes.c_void_p), ("q_row_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
        ("d_out", ctypes.c_void_p), ("out_row_stride", ctypes.c_int64), ("d_lse", ctypes.c_void_p),
        ("d_row_starts", ctypes.c_void_p), ("d_context_lens", ctypes.c_void_p), ("d_tree_mask", ctypes.c_void_p),
        ("mask_words", ctypes.c_int64), ("rows", ctypes.c_int64), ("rows_per_sequence", ctypes.c_int64),
        ("max_tokens", ctypes.c_int64), ("q_heads", ctypes.c_int64), ("channels", ctypes.c_int64),
        ("kv_dtype", ctypes.c_int32), ("softmax_scale", ctypes.c_float), ("k_scale", ctypes.c_float),
        ("v_scale", ctypes.c_float),
    ]


class kvc_qkv(ctypes.Structure):
    _fields_ = [
        ("d_q", ctypes.c_void_p), ("q_row_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
        ("d_k", ctypes.c_void_p), ("k_row_stride", ctypes.c_int64), ("k_head_stride", ctypes.c_int64),
        ("d_v", ctypes.c_void_p), ("v_row_stride", ctypes.c_int64), ("v_head_stride", ctypes.c_int64),
        ("d_q_out", ctypes.c_void_p), ("q_out_row_stride", ctypes.c_int64),
        ("d_q_norm", ctypes.c_void_p), ("d_k_norm", ctypes.c_void_p), ("d_frequencies", ctypes.c_void_p),
        ("d_positions", ctypes.c_void_p), ("d_slots", ctypes.c_void_p),
        ("rows", ctypes.c_int64), ("q_heads", ctypes.c_int64), ("channels", ctypes.c_int64), ("rotary", ctypes.c_int64),
        ("kv_dtype", ctypes.c_int32), ("norm_dtype", ctypes.c_int32), ("neighbours", ctypes.c_uint32),
        ("eps", ctypes.c_float), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
    ]


class kvc_drafts(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int64), ("rows", ctypes.c_int64), ("vocab", ctypes.c_int64),
        ("d_row_starts", ctypes.c_void_p), ("d_tokens", ctypes.c_void_p), ("d_parents", ctypes.c_void_p),
        ("d_target", ctypes.c_void_p), ("target_row_stride", ctypes.c_int64), ("d_draft", ctypes.c_void_p),
        ("draft_row_stride", ctypes.c_int64), ("d_accept", ctypes.c_void_p), ("d_sample", ctypes.c_void_p),
        ("d_kept", ctypes.c_void_p), ("d_kept_lens", ctypes.c_void_p), ("d_out_tokens", ctypes.c_void_p),
    ]


class kvc_shared_pages(ctypes.Structure):
    _fields_ = [
        ("free_capacity", ctypes.c_int64), ("d_block_table", ctypes.c_void_p), ("d_held_in", ctypes.c_void_p),
        ("d_held_out", ctypes.c_void_p), ("d_free_pages", ctypes.c_void_p), ("d_free_in", ctypes.c_void_p),
        ("d_free_out", ctypes.c_void_p), ("d_extra", ctypes.c_void_p),
    ]


_P = ctypes.c_void_p
_U64 = ctypes.c_uint64
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_U32 = ctypes.c_uint32


def _sig(name, res, args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = args
    return f


_lib_version = _sig("kvc_version", ctypes.c_int, [])
_lib_status_string = _sig("kvc_status_string", ctypes.c_char_p, [ctypes.c_int])
_lib_phi_tables = _sig("kvc_phi_tables", ctypes.c_int, [_P, _P])
_lib_narrow_table = _sig("kvc_narrow_table", ctypes.c_int, [_U32, _P])
_lib_encode_sizes = _sig("kvc_encode_sizes", ctypes.c_int, [ctypes.POINTER(kvc_params), ctypes.POINTER(_U64), ctypes.POINTER(_U64)])
_lib_encode = _sig("kvc_encode", ctypes.c_int,
                   [ctypes.POINTER(kvc_params), _P, _P, _P, _P, _P, _U64, ctypes.POINTER(_U64), _P, _P, _U64, _P, _P])
_lib_encode_result = _sig("kvc_encode_result", ctypes.c_int, [_P, _P, ctypes.POINTER(_U64), _P])
_lib_stream_info = _sig("kvc_stream_info", ctypes.c_int, [_P, _U64, ctypes.POINTER(kvc_params), ctypes.POINTER(_U64)])
_DECODE_ARGS = [_P, _P, _U64, _P, _U64, _P, _U64, _P, _U64, _P, _U64, _P, _U64, _P]
_lib_decode = _sig("kvc_decode", ctypes.c_int, _DECODE_ARGS + [_P])
_lib_decode_async = _sig("kvc_decode_async", ctypes.c_int, _DECODE_ARGS)
_lib_decode_result = _sig("kvc_decode_result", ctypes.c_int, [_P, _P, _P])
_lib_reload = _sig("kvc_reload", ctypes.c_int,
                   [_I64, _P, _P, _P, _U64, _P, _U64, _P, _U64, _P, _U64, _P, _U64, _P, _U64, _P, _P,
                    ctypes.POINTER(_I64)])
_lib_decode_noalloc = _sig("kvc_decode_noalloc", ctypes.c_int, [_P, _P, _U64, _P, _U64, _P, _U64, _P, _U64, _P, _U64, _P])
_lib_decode_paged = _sig("kvc_decode_paged", ctypes.c_int,
                         [_P, _P, _U64, _P, _U64, _P, _U64, _P, _U64, ctypes.POINTER(kvc_paged_kv), _P, _U64, _P, _P])
_lib_calibrate = _sig("kvc_calibrate_sigma", ctypes.c_int,
                      [_P, _P, _I32, _I32, _I64, _I64, _I64, _I64, ctypes.c_float, _P, _P, _U64, _P])
_lib_calibrate_blocks = _sig("kvc_calibrate_sigma_blocks", ctypes.c_int,
                             [_P, _P, _I32, _I32, _I64, _I64, _I64, _I64, _I64, ctypes.c_float, _P, _P, _U64, _P])
_lib_calibrate_rate = _sig("kvc_calibrate_sigma_rate", ctypes.c_int,
                           [_P, _P, _I32, _I32, _I64, _I64, _I64, _I64, _I64, ctypes.c_float, _U32, _U32, _U32, _P,
                            _P, _P, _U64, _P])
_lib_calibrate_split = _sig("kvc_calibrate_split", ctypes.c_int,
                            [_P, _P, _I32, _I32, _I64, _I64, _I64, _I64, _I64, _P, _U32, _U32, _U32, _P, _P, _P, _U64,
                             _P])
_lib_marginal = _sig("kvc_build_marginal", ctypes.c_int, [_P, _I32, _U64, _U32, _U32, _P, _P])
_lib_estimate = _sig("kvc_estimate_bits", ctypes.c_int, [ctypes.POINTER(kvc_params), _P, _P, _P, _P, _P, _P, _U64, _P])
_lib_cdf_table = _sig("kvc_cdf_table", ctypes.c_int, [_I32, _I32, _U32, _U32, _U32, _P, _P, _I64, _P, _P, _P])

_F32 = ctypes.c_float
_lib_block_table = _sig("kvc_build_block_table", ctypes.c_int,
                        [ctypes.POINTER(kvc_block_table), _P, _U64, _P, ctypes.POINTER(_I64)])
_lib_block_table_result = _sig("kvc_block_table_result", ctypes.c_int, [_P, _P, ctypes.POINTER(_I64)])
_lib_append = _sig("kvc_paged_append", ctypes.c_int,
                   [ctypes.POINTER(kvc_paged_kv), _I64, _I32, _I64, _P, _P, _I32, _I64, _I64, _I64, _P, _F32, _F32, _P])
_lib_attention_sizes = _sig("kvc_paged_attention_sizes", ctypes.c_int,
                            [ctypes.POINTER(kvc_paged_kv), ctypes.POINTER(kvc_attention), ctypes.POINTER(_U64)])
_lib_attention = _sig("kvc_paged_attention", ctypes.c_int,
                      [ctypes.POINTER(kvc_paged_kv), _I64, ctypes.POINTER(kvc_attention), _P, _U64, _P])
_lib_attention_result = _sig("kvc_paged_attention_result", ctypes.c_int, [_P, _P])
_lib_qkv = _sig("kvc_paged_qkv", ctypes.c_int, [ctypes.POINTER(kvc_paged_kv), _I64, ctypes.POINTER(kvc_qkv), _P])
_lib_verify_sizes = _sig("kvc_verify_drafts_sizes", ctypes.c_int, [ctypes.POINTER(kvc_drafts), ctypes.POINTER(_U64)])
_lib_verify = _sig("kvc_verify_drafts", ctypes.c_int, [ctypes.POINTER(kvc_drafts), _P, _U64, _P])
_lib_verify_result = _sig("kvc_verify_drafts_result", ctypes.c_int, [_P, _P])
_lib_compact = _sig("kvc_paged_compact", ctypes.c_int,
                    [ctypes.POINTER(kvc_paged_kv), _I32, _I64, _I64, _P, _P, _P, _P, _P, _U64, _P])
_lib_compact_result = _sig("kvc_paged_compact_result", ctypes.c_int, [_P, _P])
_SHARED_ARGS = [ctypes.POINTER(kvc_paged_kv), _I32, _I64, ctypes.POINTER(kvc_shared_pages), _I64]
_lib_fork = _sig("kvc_fork_pages", ctypes.c_int, _SHARED_ARGS + [_P, _P, _P, _P, _U64, _P])
_lib_release = _sig("kvc_release_pages", ctypes.c_int, _SHARED_ARGS + [_P, _P, _U64, _P])
_lib_shared_result = _sig("kvc_shared_pages_result", ctypes.c_int, [_P, _P])


class KvcError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {kvc_status_string(status)} ({status})")


def _check(st: int, where: str):
    if st != KVC_OK:
        raise KvcError(st, where)


def _stream(stream=None) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _host_header(header) -> np.ndarray:
    """A host copy of a stream header (bytes, numpy or a device tensor holding
    at least the header) as a contiguous 128-byte array."""
    if isinstance(header, torch.Tensor):
        header = header[:HEADER_BYTES].cpu().numpy()
    h = np.frombuffer(bytes(header[:HEADER_BYTES]), dtype=np.uint8).copy()
    if h.size != HEADER_BYTES:
        raise KvcError(KVC_ERR_CORRUPT, "stream header")
    return h


def _kv_dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16 or t.dtype == torch.int16:
        return KVC_BF16
    if t.dtype == torch.float8_e4m3fn or t.dtype == torch.uint8:
        return KVC_E4M3
    raise TypeError(f"KV must be bf16 (or int16 patterns) or e4m3 (or uint8 patterns), got {t.dtype}")


def _mu_dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16 or t.dtype == torch.int16:
        return KVC_BF16
    if t.dtype == torch.float32:
        return KVC_F32
    raise TypeError(f"mu must be bf16 or float32, got {t.dtype}")


def _need(t: torch.Tensor, name: str):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous device tensor")


def kvc_version() -> int:
    return _lib_version()


def kvc_status_string(status: int) -> str:
    return _lib_status_string(status).decode()


def kvc_phi_tables():
    """(narrow, wide) base tables of the library, computed on the host."""
    a = np.zeros(12289, dtype=np.uint32)
    b = np.zeros(12289, dtype=np.uint32)
    _check(_lib_phi_tables(a.ctypes.data, b.ctypes.data), "kvc_phi_tables")
    return a, b


def kvc_narrow_table(narrow_dof: int = 0):
    """The narrow part's base table (Phi, or Student's t with narrow_dof
    degrees of freedom), computed on the host."""
    a = np.zeros(12289, dtype=np.uint32)
    _check(_lib_narrow_table(narrow_dof, a.ctypes.data), "kvc_narrow_table")
    return a


def make_params(kv_dtype, mu_dtype, planes, tokens, channels, weights=(9500, 300), chunk_tokens=0,
                sigma_block_tokens=0, narrow_dof=0, channel_split=0) -> kvc_params:
    return kvc_params(kv_dtype, mu_dtype, weights[0], weights[1], chunk_tokens, sigma_block_tokens,
                      narrow_dof, channel_split, planes, tokens, channels)


def side_info(sigma: torch.Tensor, channel_split: torch.Tensor) -> torch.Tensor:
    """The side buffer of a stream with per-channel weights: sigma's words,
    then the narrow weights [G, D] (basis points) as uint32 words, in one
    float32 device tensor (pass it wherever sigma goes)."""
    w = channel_split.to(torch.int32).contiguous()
    return torch.cat([sigma.reshape(-1).to(torch.float32), w.view(torch.float32).reshape(-1)])


def sigma_shape(planes: int, tokens: int, channels: int, sigma_block_tokens: int = 0):
    """Shape of sigma: [G, D], or [G, ceil(T / B), D] with sigma blocks."""
    if sigma_block_tokens == 0:
        return (planes, channels)
    return (planes, -(-tokens // sigma_block_tokens), channels)


def kvc_encode_sizes(p: kvc_params):
    a, b = _U64(), _U64()
    _check(_lib_encode_sizes(ctypes.byref(p), ctypes.byref(a), ctypes.byref(b)), "kvc_encode_sizes")
    return a.value, b.value


class Encoder:
    """Holds the output and workspace buffers of one shape so that repeated
    calls allocate nothing."""

    def __init__(self, p: kvc_params, device="cuda", out_capacity: int | None = None):
        self.p = p
        max_stream, ws = kvc_encode_sizes(p)
        self.capacity = max_stream if out_capacity is None else out_capacity
        self.out = torch.empty(self.capacity, dtype=torch.uint8, device=device)
        self.workspace = torch.empty(ws, dtype=torch.uint8, device=device)
        self.header = np.zeros(HEADER_BYTES, dtype=np.uint8)     # host copy of the last stream's header

    def _check_inputs(self, kv, mu, sigma):
        p = self.p
        n = p.planes * p.tokens * p.channels
        if kv.numel() != n or mu.numel() != n or _kv_dtype(kv) != p.kv_dtype or _mu_dtype(mu) != p.mu_dtype:
            raise ValueError("kv / mu do not match the encoder's parameters")
        words = math.prod(sigma_shape(p.planes, p.tokens, p.channels, p.sigma_block_tokens))
        if p.channel_split:
            words += p.planes * p.channels                  # the narrow weights follow sigma
        if sigma.numel() != words:
            raise ValueError("sigma does not match the encoder's parameters")

    def __call__(self, kv, mu, sigma, prefix=None, stream=None, info: dict | None = None) -> torch.Tensor:
        self._check_inputs(kv, mu, sigma)
        n = _U64(0)
        inf = kvc_encode_info() if info is not None else None
        st = _lib_encode(ctypes.byref(self.p), _ptr(kv), _ptr(mu), _ptr(sigma), _ptr(prefix),
                         _ptr(self.out), self.capacity, ctypes.byref(n), self.header.ctypes.data,
                         _ptr(self.workspace), self.workspace.numel(), _stream(stream),
                         ctypes.byref(inf) if inf is not None else None)
        _check(st, "kvc_encode")
        if inf is not None:
            info["stage_ms"] = list(inf.stage_ms)
        return self.out[: n.value]

    def enqueue(self, kv, mu, sigma, prefix=None, stream=None):
        """Queue an encode without waiting for it; result() gives the stream."""
        self._check_inputs(kv, mu, sigma)
        st = _lib_encode(ctypes.byref(self.p), _ptr(kv), _ptr(mu), _ptr(sigma), _ptr(prefix),
                         _ptr(self.out), self.capacity, None, None, _ptr(self.workspace), self.workspace.numel(),
                         _stream(stream), None)
        _check(st, "kvc_encode")

    def result(self, stream=None) -> torch.Tensor:
        n = _U64(0)
        _check(_lib_encode_result(_ptr(self.workspace), _stream(stream), ctypes.byref(n), self.header.ctypes.data),
               "kvc_encode_result")
        return self.out[: n.value]


def kvc_encode(kv: torch.Tensor, mu: torch.Tensor, sigma: torch.Tensor, prefix: torch.Tensor | None = None,
               weights=(9500, 300), chunk_tokens: int = 0, stream=None,
               sigma_block_tokens: int = 0, narrow_dof: int = 0,
               channel_split: torch.Tensor | None = None) -> torch.Tensor:
    """Encode KV [G, T, D] under the mixture around mu with sigma [G, D] (or
    [G, ceil(T / B), D] with sigma_block_tokens = B) and, when channel_split
    [G, D] is given, each channel's own narrow weight (decode then takes
    side_info(sigma, channel_split) as its sigma); returns the stream as a
    uint8 device tensor."""
    for t, nm in ((kv, "kv"), (mu, "mu"), (sigma, "sigma")):
        _need(t, nm)
    if prefix is not None:
        _need(prefix, "prefix")
    g, t, d = kv.shape
    if tuple(mu.shape) != (g, t, d) or tuple(sigma.shape) != sigma_shape(g, t, d, sigma_block_tokens) \
            or sigma.dtype != torch.float32:
        raise ValueError("shapes: kv and mu [G, T, D], sigma [G, D] (or [G, ceil(T / B), D]) float32")
    split = 0
    if channel_split is not None:
        if tuple(channel_split.shape) != (g, d):
            raise ValueError("channel_split is [G, D]")
        sigma = side_info(sigma, channel_split)
        split = 1
    p = make_params(_kv_dtype(kv), _mu_dtype(mu), g, t, d, weights, chunk_tokens, sigma_block_tokens, narrow_dof,
                    split)
    return Encoder(p, kv.device)(kv, mu, sigma, prefix, stream).clone()


def kvc_stream_info(header: bytes | np.ndarray):
    h = np.frombuffer(bytes(header[:HEADER_BYTES]), dtype=np.uint8).copy()
    p = kvc_params()
    total = _U64()
    _check(_lib_stream_info(h.ctypes.data, h.size, ctypes.byref(p), ctypes.byref(total)), "kvc_stream_info")
    return p, total.value


def _decode_args(header, stream_bytes, mu, sigma, prefix, kv_out, workspace, stream):
    h = _host_header(stream_bytes if header is None else header)
    args = [h.ctypes.data, _ptr(stream_bytes), stream_bytes.numel(), _ptr(mu), _nbytes(mu), _ptr(sigma),
            _nbytes(sigma), _ptr(prefix), _nbytes(prefix), _ptr(kv_out), _nbytes(kv_out), _ptr(workspace),
            _nbytes(workspace), _stream(stream)]
    return h, args


def kvc_decode(stream_bytes: torch.Tensor, mu: torch.Tensor, sigma: torch.Tensor,
               prefix: torch.Tensor | None = None, kv_out: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None, header=None) -> torch.Tensor:
    """Decode a KVC-1 stream (uint8 device tensor) back to KV bit patterns
    (int16 for bf16, uint8 for e4m3), shape [G, T, D].  header: a host copy
    of the stream's first 128 bytes; read from the device stream if None."""
    _need(stream_bytes, "stream")
    for t, nm in ((mu, "mu"), (sigma, "sigma")):
        _need(t, nm)
    if stream_bytes.numel() < HEADER_BYTES:
        raise KvcError(KVC_ERR_CORRUPT, "kvc_decode")
    h = _host_header(stream_bytes if header is None else header)
    p, _ = kvc_stream_info(h)
    shape = (p.planes, p.tokens, p.channels)
    if kv_out is None:
        kv_out = torch.empty(shape, dtype=torch.int16 if p.kv_dtype == KVC_BF16 else torch.uint8,
                             device=stream_bytes.device)
    if workspace is None:
        workspace = torch.empty(DECODE_WORKSPACE_BYTES, dtype=torch.uint8, device=stream_bytes.device)
    _, args = _decode_args(h, stream_bytes, mu, sigma, prefix, kv_out, workspace, stream)
    _check(_lib_decode(*args, None), "kvc_decode")
    return kv_out


def kvc_decode_into(stream_bytes, mu, sigma, prefix, kv_out, workspace, stream=None,
                    info: dict | None = None, header=None) -> int:
    """Decode into kv_out and return the status instead of raising (for
    timing loops and error-path tests).  header: a host copy of the stream's
    header (bytes or numpy); read from the device stream if None."""
    inf = kvc_decode_info() if info is not None else None
    try:
        _, args = _decode_args(header, stream_bytes, mu, sigma, prefix, kv_out, workspace, stream)
    except KvcError as e:                 # fewer bytes than a header
        return e.status
    st = _lib_decode(*args, ctypes.byref(inf) if inf is not None else None)
    if inf is not None:
        info["stage_ms"] = list(inf.stage_ms)
        info["fallback_symbols"] = inf.fallback_symbols
    return st


def kvc_decode_async(stream_bytes, mu, sigma, prefix, kv_out, workspace, header, stream=None) -> int:
    """Queue a decode (host checks only); kvc_decode_result gives its status."""
    _, args = _decode_args(header, stream_bytes, mu, sigma, prefix, kv_out, workspace, stream)
    return _lib_decode_async(*args)


def kvc_decode_result(workspace, stream=None, info: dict | None = None) -> int:
    inf = kvc_decode_info()
    st = _lib_decode_result(_ptr(workspace), _stream(stream), ctypes.byref(inf))
    if info is not None:
        info["fallback_symbols"] = inf.fallback_symbols
    return st


def kvc_decode_noalloc(stream_bytes, mu, sigma, prefix, kv_out, stream=None, header=None) -> int:
    """Decode into kv_out with the library's fixed device scratch (no
    workspace, nothing allocated); returns the status.  Calls on one device
    share the scratch and must not overlap."""
    try:
        h = _host_header(stream_bytes if header is None else header)
    except KvcError as e:
        return e.status
    return _lib_decode_noalloc(h.ctypes.data, _ptr(stream_bytes), stream_bytes.numel(), _ptr(mu), _nbytes(mu),
                               _ptr(sigma), _nbytes(sigma), _ptr(prefix), _nbytes(prefix), _ptr(kv_out),
                               _nbytes(kv_out), _stream(stream))


def kvc_reload(host_streams, mu: torch.Tensor, sigma: torch.Tensor, prefix, kv_out: torch.Tensor,
               staging: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None,
               copy_stream=None):
    """Decode the per-layer streams in `host_streams` (uint8 CPU tensors,
    pinned for asynchronous copies) into kv_out[l], with mu[l], sigma[l] and
    the shared prefix; copies overlap the decodes (the library's pipeline).
    Returns (status, index of the first failing layer or -1)."""
    n = len(host_streams)
    for t in host_streams:
        if t.is_cuda or t.dtype != torch.uint8 or not t.is_contiguous():
            raise ValueError("host streams must be contiguous uint8 CPU tensors")
    for t, nm in ((mu, "mu"), (sigma, "sigma"), (kv_out, "kv_out")):
        _need(t, nm)
        if t.shape[0] != n:
            raise ValueError(f"{nm} must have one entry per stream")
    dev = kv_out.device
    if staging is None:
        half = max(t.numel() for t in host_streams) + 255
        staging = torch.empty(2 * (half // 256 * 256 + 256), dtype=torch.uint8, device=dev)
    if workspace is None:
        workspace = torch.empty(n * DECODE_WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
    if copy_stream is None:
        copy_stream = torch.cuda.Stream(device=dev)
    ptrs = (ctypes.c_void_p * n)(*[t.data_ptr() for t in host_streams])
    sizes = (ctypes.c_uint64 * n)(*[t.numel() for t in host_streams])
    failed = _I64(-1)
    st = _lib_reload(n, ptrs, sizes, _ptr(mu), _nbytes(mu) // n, _ptr(sigma), _nbytes(sigma) // n, _ptr(prefix),
                     _nbytes(prefix), _ptr(kv_out), _nbytes(kv_out) // n, _ptr(staging), _nbytes(staging),
                     _ptr(workspace), _nbytes(workspace), _stream(stream), copy_stream.cuda_stream,
                     ctypes.byref(failed))
    return st, failed.value


class PagedKV:
    """A paged KV cache as the library sees it: one pool per (layer, kv),
    each [num_pages, page_tokens, heads, channels], and a block table
    [batch, max_pages] of int32 page numbers shared by every pool.  Holds
    the device array of pool pointers that the call reads."""

    def __init__(self, pools, block_table: torch.Tensor, page_tokens: int):
        pools = list(pools)
        if not pools:
            raise ValueError("no pools")
        for t in pools:
            _need(t, "pool")
        _need(block_table, "block_table")
        if block_table.dtype != torch.int32 or block_table.dim() != 2:
            raise ValueError("block_table must be int32 [batch, max_pages]")
        if pools[0].dim() != 4:
            raise ValueError("pools must be [num_pages, page_tokens, heads, channels]")
        n_pages, pt, heads, _ = pools[0].shape
        if pt != page_tokens or any(tuple(t.shape) != tuple(pools[0].shape) or t.dtype != pools[0].dtype
                                    for t in pools):
            raise ValueError("pools must all be [num_pages, page_tokens, heads, channels] of one dtype")
        self.pools = pools
        self.block_table = block_table
        self.ptrs = torch.tensor([t.data_ptr() for t in pools], dtype=torch.int64, device=block_table.device)
        self.channels = pools[0].shape[3]
        self.dtype = pools[0].dtype
        self.desc = kvc_paged_kv(self.ptrs.data_ptr(), block_table.data_ptr(), len(pools), _nbytes(pools[0]),
                                 block_table.shape[0], heads, block_table.shape[1], n_pages, page_tokens, 0)
        self.kv_dtype = _kv_dtype(pools[0])
        self.ref = ctypes.byref(self.desc)
        self._own = (torch._C._cuda_getCurrentRawStream(block_table.device.index), self.ptrs)
        self._aligned = all(t.data_ptr() % 16 == 0 for t in pools)

    def _check_pools(self):
        if not self._aligned:
            raise ValueError("the pools must be 16-byte aligned")


def kvc_decode_paged(stream_bytes, mu, sigma, prefix, paged: PagedKV, workspace, stream=None,
                     info: dict | None = None, header=None) -> int:
    """Decode straight into a paged KV cache; returns the status.  The pools'
    channels and element type must be the stream's (checked here against
    the header; the library checks the pool count and sizes)."""
    h = _host_header(stream_bytes if header is None else header)
    p, _ = kvc_stream_info(h)
    esize = 2 if p.kv_dtype == KVC_BF16 else 1
    if paged.channels != p.channels or torch.empty(0, dtype=paged.dtype).element_size() != esize:
        return KVC_ERR_INVALID
    inf = kvc_decode_info() if info is not None else None
    st = _lib_decode_paged(h.ctypes.data, _ptr(stream_bytes), stream_bytes.numel(), _ptr(mu), _nbytes(mu),
                           _ptr(sigma), _nbytes(sigma), _ptr(prefix), _nbytes(prefix), ctypes.byref(paged.desc),
                           _ptr(workspace), _nbytes(workspace), _stream(stream),
                           ctypes.byref(inf) if inf is not None else None)
    if inf is not None:
        info["stage_ms"] = list(inf.stage_ms)
        info["fallback_symbols"] = inf.fallback_symbols
    return st


def _tensor(t, name, dtype, shape, device):
    """A contiguous tensor of this type and shape (None: any extent) on this device."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if t.dtype != dtype or t.device != device or not t.is_contiguous() or t.dim() != len(shape) \
            or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on {device}")


def _rows_contiguous(t):
    """Whether the values of each t[i] [heads, channels] lie one after the other."""
    return t.numel() == 0 or t.stride(2) == 1 and (t.shape[1] == 1 or t.stride(1) == t.shape[2])


def _queue(device, stream, call, *tensors, own=()):
    """Runs call(stream pointer) with `device` current, on `stream` (the
    device's current one if None), and keeps the tensors' memory until the
    work queued there is done; so too on a current stream that is not the one
    that `own`, the caller's (stream pointer, hidden tensors) pairs, were made
    on."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(device.index)
        for home, t in own:
            if raw != home:
                t.record_stream(torch.cuda.current_stream(device))
        if torch.cuda.current_device() == device.index:
            return call(raw)
        with torch.cuda.device(device):
            return call(raw)
    if stream.device != device:
        raise ValueError(f"the stream is of {stream.device}, the tensors of {device}")
    for t in (*tensors, *(t for _, t in own)):
        if t is not None:
            t.record_stream(stream)
    with torch.cuda.device(device):
        return call(stream.cuda_stream)


def _workspace(nbytes: int, device):
    """A cleared workspace for calls on any stream, as an entry of _queue's
    `own`.  Waits for the current stream: for the clearing, and for what is
    still queued there on memory that the workspace took over.  (A capture
    orders both itself.)"""
    with torch.cuda.device(device):
        ws = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream().synchronize()
        return torch.cuda.current_stream().cuda_stream, ws


class BlockTable:
    """The pages of a batch of requests, kept on the device: the block table
    [batch, max_pages], the pages each request holds (held [batch]) and the
    stack of free pages (free_pages, its height free_count [1]), all int32 and
    the caller's; a call updates them in place, or writes held_out and
    free_count_out where they are given.  The step's rows come back in
    row_starts [batch + 1] (int32), slots [max_rows] (int64) and positions
    [max_rows] (int32; either may be None).  Holds the call's workspace, so
    that repeated calls allocate nothing."""

    def __init__(self, block_table, held, free_pages, free_count, page_tokens: int, num_pages: int, row_starts,
                 slots=None, positions=None, held_out=None, free_count_out=None):
        _need(block_table, "block_table")
        dev = block_table.device
        if block_table.dim() != 2 or block_table.dtype != torch.int32:
            raise ValueError("block_table must be int32 [batch, max_pages]")
        batch = block_table.shape[0]
        _tensor(free_pages, "free_pages", torch.int32, (None,), dev)
        for t, name in ((free_count, "free_count"), (free_count_out, "free_count_out")):
            if t is not None:
                _tensor(t, name, torch.int32, (1,), dev)
        for t, name in ((held, "held"), (held_out, "held_out")):
            if t is not None:
                _tensor(t, name, torch.int32, (batch,), dev)
        _tensor(row_starts, "row_starts", torch.int32, (batch + 1,), dev)
        given = [t for t in (slots, positions) if t is not None]
        max_rows = given[0].shape[0] if given else 0x7FFFFFFF
        if slots is not None:
            _tensor(slots, "slots", torch.int64, (max_rows,), dev)
        if positions is not None:
            _tensor(positions, "positions", torch.int32, (max_rows,), dev)
        self.device, self.batch = dev, batch
        self.block_table, self.free_pages, self.row_starts = block_table, free_pages, row_starts
        self.slots, self.positions = slots, positions
        self.held, self.free_count = held, free_count
        self.held_out = held if held_out is None else held_out
        self.free_count_out = free_count if free_count_out is None else free_count_out
        self._own = _workspace(256 + 12 * (batch + 64), dev)
        self.workspace = self._own[1]
        self.desc = kvc_block_table(
            batch, block_table.shape[1], num_pages, free_pages.numel(), max_rows, page_tokens, 0, None, None,
            _ptr(held), _ptr(self.held_out), _ptr(block_table), _ptr(free_pages), _ptr(free_count),
            _ptr(self.free_count_out), _ptr(row_starts), _ptr(slots), _ptr(positions))
        self._ref = ctypes.byref(self.desc)

    def __call__(self, cached_lens=None, new_lens=None, trim: bool = False, stream=None):
        """Queue the step of requests with cached_lens tokens that get
        new_lens more (int32 [batch]; None: no request has any); result()
        gives its outcome."""
        for t, name in ((cached_lens, "cached_lens"), (new_lens, "new_lens")):
            if t is not None:
                _tensor(t, name, torch.int32, (self.batch,), self.device)
        d = self.desc
        d.trim = 1 if trim else 0
        d.d_cached_lens, d.d_new_lens = _ptr(cached_lens), _ptr(new_lens)
        ws = self.workspace
        st = _queue(self.device, stream,
                    lambda s: _lib_block_table(self._ref, ws.data_ptr(), ws.numel(), s, None),
                    cached_lens, new_lens, self.block_table, self.held, self.held_out, self.free_pages,
                    self.free_count, self.free_count_out, self.row_starts, self.slots, self.positions, own=(self._own,))
        _check(st, "kvc_build_block_table")

    def result(self, stream=None) -> int:
        """The number of rows of the last step; raises KvcError if it failed."""
        n = _I64(0)
        st = _queue(self.device, stream,
                    lambda s: _lib_block_table_result(self.workspace.data_ptr(), s, ctypes.byref(n)))
        _check(st, "kvc_build_block_table")
        return n.value


def kvc_paged_append(paged: PagedKV, layer: int, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                     k_scale: float = 1.0, v_scale: float = 1.0, stream=None) -> None:
    """Queue the append of the rows k and v [rows, heads, channels] (views of
    wider rows allowed) to the slots [rows] (int64; -1: none) of one layer's
    pages; bf16 rows of an e4m3 cache are rounded from x / scale."""
    dev = paged.block_table.device
    paged._check_pools()
    rows = slots.shape[0]
    _tensor(slots, "slots", torch.int64, (None,), dev)
    heads, ch = paged.desc.heads, paged.channels
    for t, name in ((k, "k"), (v, "v")):
        if t.device != dev or t.shape != (rows, heads, ch) or not _rows_contiguous(t) or t.dtype != k.dtype:
            raise ValueError(f"{name} must be [{rows}, {heads}, {ch}] on {dev}, a row's values contiguous")
    st = _queue(dev, stream,
                lambda s: _lib_append(paged.ref, layer, paged.kv_dtype, ch, k.data_ptr(), v.data_ptr(), _kv_dtype(k),
                                      rows, k.stride(0), v.stride(0), slots.data_ptr(), k_scale, v_scale, s),
                k, v, slots, *(paged.pools if stream is not None else ()), own=(paged._own,))
    _check(st, "kvc_paged_append")


def _qkv_rows(t, name, shape, device):
    """The strides of a projection's rows [rows, heads, channels], bf16, views
    of wider rows allowed."""
    s = t.stride()
    if t.dtype is not torch.bfloat16 or t.shape != shape or t.device != device or (s[2] != 1 and t.numel()):
        raise ValueError(f"{name} must be bf16 {list(shape)} on {device}, channels contiguous")
    return s


class PagedQKV:
    """Norms of queries and keys, rotation by position and the append of keys
    and values to the pages, in one pass over a projection's rows.  q_norm and
    k_norm [layers, channels] (bf16 or float32, both of one type; None: no
    norm); frequencies [rotary / 2] float64, radians a position (None: no
    rotation), pairing channels i and rotary / 2 + i, or 2 i and 2 i + 1 with
    interleaved.  Threads need an object each; calls on several streams do not."""

    def __init__(self, paged: PagedKV, q_heads: int, frequencies: torch.Tensor | None = None,
                 q_norm: torch.Tensor | None = None, k_norm: torch.Tensor | None = None, eps: float = 1e-6,
                 interleaved: bool = False, k_scale: float = 1.0, v_scale: float = 1.0):
        paged._check_pools()
        self.paged, self.q_heads, self.device = paged, q_heads, paged.block_table.device
        ch, layers = paged.channels, paged.desc.n_pools // 2
        norms = [t for t in (q_norm, k_norm) if t is not None]
        dtype = norms[0].dtype if norms else torch.bfloat16
        if dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("norms must be bf16 or float32")
        for t, name in ((q_norm, "q_norm"), (k_norm, "k_norm")):
            if t is not None:
                _tensor(t, name, dtype, (layers, ch), self.device)
                if t.data_ptr() % 16:
                    raise ValueError(f"{name} must be 16-byte aligned")
        if frequencies is not None:
            _tensor(frequencies, "frequencies", torch.float64, (None,), self.device)
            if frequencies.shape[0] % 8 or not 0 < 2 * frequencies.shape[0] <= ch:
                raise ValueError(f"frequencies must be a multiple of 8, at most {ch // 2}")
        if norms and not (math.isfinite(eps) and eps >= 1e-30):
            raise ValueError("eps must be at least 1e-30")
        if not 0 <= q_heads <= 65536 or ch > 256:
            raise ValueError("q_heads must be 0 to 65536, channels at most 256")
        for x in (k_scale, v_scale):
            if not (math.isfinite(x) and x > 0) or (paged.kv_dtype == KVC_BF16 and x != 1.0):
                raise ValueError("scales must be finite and positive, and 1 for bf16 pools")
        self._norms = _ptr(q_norm), _ptr(k_norm)
        home = torch._C._cuda_getCurrentRawStream(self.device.index)
        self._own = (paged._own, *((home, t) for t in (*norms, frequencies) if t is not None))
        self._layer_bytes = ch * dtype.itemsize
        self.desc = kvc_qkv(q_heads=q_heads, channels=ch, kv_dtype=paged.kv_dtype,
                            rotary=0 if frequencies is None else 2 * frequencies.shape[0], d_frequencies=_ptr(frequencies),
                            norm_dtype=KVC_F32 if dtype == torch.float32 else KVC_BF16, neighbours=int(interleaved), eps=eps,
                            k_scale=k_scale, v_scale=v_scale)
        self._ref = ctypes.byref(self.desc)

    def __call__(self, layer: int, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                 positions: torch.Tensor | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """Queue the rows q [rows, q_heads, channels], k and v [rows, heads,
        channels] (bf16, views allowed) of one layer: keys and values to slots
        [rows] (int64; -1: none), queries to out, which may be q (returned;
        rows whose position, int32 [rows], is negative keep what it holds)."""
        d, dev, paged = self.desc, self.device, self.paged
        rows = slots.shape[0]
        _tensor(slots, "slots", torch.int64, (rows,), dev)
        if positions is not None:
            _tensor(positions, "positions", torch.int32, (rows,), dev)
            d.d_positions = positions.data_ptr()
        elif d.rotary:
            raise ValueError("a rotation needs positions")
        else:
            d.d_positions = None
        shape = (rows, self.q_heads, paged.channels)
        d.q_row_stride, d.q_head_stride, _ = _qkv_rows(q, "q", shape, dev)
        if out is None:
            with torch.cuda.stream(stream):
                out = torch.empty(shape, dtype=q.dtype, device=dev)
        d.q_out_row_stride, heads_apart, _ = _qkv_rows(out, "out", shape, dev)
        if heads_apart != shape[2] and shape[1] > 1 and rows:
            raise ValueError("out's heads must lie one after the other")
        shape = (rows, paged.desc.heads, paged.channels)
        d.k_row_stride, d.k_head_stride, _ = _qkv_rows(k, "k", shape, dev)
        d.v_row_stride, d.v_head_stride, _ = _qkv_rows(v, "v", shape, dev)
        d.rows = rows
        d.d_q, d.d_k, d.d_v, d.d_q_out = q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr()
        d.d_slots = slots.data_ptr()
        q_norm, k_norm = self._norms
        d.d_q_norm = None if q_norm is None else q_norm + layer * self._layer_bytes
        d.d_k_norm = None if k_norm is None else k_norm + layer * self._layer_bytes
        st = _queue(dev, stream, lambda s: _lib_qkv(paged.ref, layer, self._ref, s), q, k, v, slots, positions, out,
                    *(paged.pools if stream is not None else ()), own=self._own)
        _check(st, "kvc_paged_qkv")
        return out


class PagedAttention:
    """Attention of drafted tokens over a paged cache: holds the workspace of
    one shape (q_heads query heads, up to max_rows rows a call) so that
    repeated calls allocate nothing.  rows_per_sequence and max_tokens (the
    usual rows of a sequence and the longest sequence) shape the launch only;
    0: max_rows / batch and what the table can hold.  softmax_scale defaults
    to channels ** -0.5.  Calls that may run at the same time need an object
    each."""

    def __init__(self, paged: PagedKV, q_heads: int, max_rows: int, rows_per_sequence: int = 0, max_tokens: int = 0,
                 softmax_scale: float | None = None, k_scale: float = 1.0, v_scale: float = 1.0):
        paged._check_pools()
        self.paged, self.q_heads, self.max_rows = paged, q_heads, max_rows
        self.device = paged.block_table.device
        self.batch, ch = paged.desc.batch, paged.channels
        scale = ch ** -0.5 if softmax_scale is None else softmax_scale
        # fixed here: with one launch shape a call of fewer rows needs no larger workspace
        rows_per_sequence = rows_per_sequence or -(-max_rows // self.batch)
        self.desc = kvc_attention(None, q_heads * ch, ch, None, q_heads * ch, None, None, None, None, 0, max_rows,
                                  rows_per_sequence, max_tokens, q_heads, ch, paged.kv_dtype, scale, k_scale, v_scale)
        self._ref = ctypes.byref(self.desc)
        n = _U64(0)
        _check(_lib_attention_sizes(paged.ref, self._ref, ctypes.byref(n)), "kvc_paged_attention_sizes")
        self._own = _workspace(n.value, self.device)
        self.workspace = self._own[1]

    def __call__(self, layer: int, q: torch.Tensor, row_starts: torch.Tensor, context_lens: torch.Tensor | None = None,
                 tree_mask: torch.Tensor | None = None, out: torch.Tensor | None = None,
                 lse: torch.Tensor | None = None, stream=None):
        """Queue the attention of q [rows, q_heads, channels] (bf16, views
        allowed) over one layer's pages; row_starts [batch + 1] and
        context_lens [batch] int32, tree_mask [rows, words] int64 (bit j of a
        row: it sees drafted token j) or None (it sees those before it and
        itself).  Returns (out, lse); result() gives the outcome."""
        d, dev, ch = self.desc, self.device, self.paged.channels
        rows = q.shape[0]
        if q.dtype != torch.bfloat16 or q.device != dev or q.shape[1:] != (self.q_heads, ch) or \
                (rows and q.stride(2) != 1) or rows > self.max_rows:
            raise ValueError(f"q must be bf16 [up to {self.max_rows}, {self.q_heads}, {ch}] on {dev}, channels contiguous")
        _tensor(row_starts, "row_starts", torch.int32, (self.batch + 1,), dev)
        if context_lens is not None:
            _tensor(context_lens, "context_lens", torch.int32, (self.batch,), dev)
        if tree_mask is not None:
            _tensor(tree_mask, "tree_mask", torch.int64, (rows, None), dev)
            if tree_mask.shape[1] == 0:
                raise ValueError("tree_mask needs a word a row")
        if out is None or lse is None:
            with torch.cuda.stream(stream):
                out = torch.empty((rows, self.q_heads, ch), dtype=q.dtype, device=dev) if out is None else out
                lse = torch.empty((rows, self.q_heads), dtype=torch.float32, device=dev) if lse is None else lse
        if out.dtype != torch.bfloat16 or out.device != dev or out.shape != q.shape or not _rows_contiguous(out):
            raise ValueError(f"out must be bf16 {list(q.shape)} on {dev}, a row's values contiguous")
        _tensor(lse, "lse", torch.float32, (rows, self.q_heads), dev)
        d.d_q, d.q_row_stride, d.q_head_stride = q.data_ptr(), q.stride(0), q.stride(1)
        d.d_out, d.out_row_stride, d.d_lse = out.data_ptr(), out.stride(0), lse.data_ptr()
        d.d_row_starts, d.d_context_lens = row_starts.data_ptr(), _ptr(context_lens)
        d.d_tree_mask, d.mask_words = _ptr(tree_mask), tree_mask.shape[1] if tree_mask is not None and rows else 0
        d.rows = rows
        ws, paged = self.workspace, self.paged
        st = _queue(dev, stream,
                    lambda s: _lib_attention(paged.ref, layer, self._ref, ws.data_ptr(), ws.numel(), s),
                    q, out, lse, row_starts, context_lens, tree_mask, paged.block_table,
                    *(paged.pools if stream is not None else ()), own=(self._own, paged._own))
        _check(st, "kvc_paged_attention")
        return out, lse

    def result(self, stream=None) -> None:
        """Waits for the last call; raises KvcError if it met lengths or page
        numbers that do not fit."""
        st = _queue(self.device, stream, lambda s: _lib_attention_result(self.workspace.data_ptr(), s))
        _check(st, "kvc_paged_attention")


def kvc_paged_attention(paged: PagedKV, layer: int, q: torch.Tensor, row_starts: torch.Tensor,
                        context_lens: torch.Tensor | None = None, tree_mask: torch.Tensor | None = None,
                        softmax_scale: float | None = None, k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
    """One call of PagedAttention, waited for: (out [rows, q_heads, channels]
    bf16, lse [rows, q_heads] float32)."""
    with torch.cuda.stream(stream):
        att = PagedAttention(paged, q.shape[1], q.shape[0], softmax_scale=softmax_scale, k_scale=k_scale,
                             v_scale=v_scale)
    got = att(layer, q, row_starts, context_lens, tree_mask, stream=stream)
    att.result(stream)
    return got


class DraftVerifier:
    """Verification of drafted tokens of `batch` sequences, up to max_rows
    nodes a call: holds the workspace, so that repeated calls allocate nothing
    where their outputs are given.  Calls that may run at the same time need
    an object each."""

    def __init__(self, batch: int, vocab: int, max_rows: int, device="cuda"):
        self.batch, self.vocab, self.max_rows = batch, vocab, max_rows
        self.desc = kvc_drafts(batch=batch, rows=max_rows, vocab=vocab)
        self._ref = ctypes.byref(self.desc)
        n = _U64(0)
        _check(_lib_verify_sizes(self._ref, ctypes.byref(n)), "kvc_verify_drafts_sizes")
        self.device = torch.empty(0, device=device).device
        self._own = _workspace(n.value, self.device)
        self.workspace = self._own[1]

    def _rows_of(self, t, name, rows):
        s = t.stride()
        if t.dtype is not torch.float32 or t.shape != (rows, self.vocab) or t.device != self.device or \
                (s[1] != 1 and self.vocab > 1 and rows):
            raise ValueError(f"{name} must be float32 [{rows}, {self.vocab}] on {self.device}, a row's values contiguous")
        return s[0]

    def __call__(self, target: torch.Tensor, tokens: torch.Tensor, row_starts: torch.Tensor, accept: torch.Tensor,
                 sample: torch.Tensor, parents: torch.Tensor | None = None, draft: torch.Tensor | None = None,
                 kept: torch.Tensor | None = None, kept_lens: torch.Tensor | None = None,
                 out_tokens: torch.Tensor | None = None, stream=None):
        """Queue the verification of the nodes tokens [rows] (int32; of each
        sequence the first is its last token) of trees given by parents [rows]
        (int32, places in the sequence; None: chains) against the
        probabilities target [rows, vocab] behind each of them, draft those
        that its children were drawn from (float32; None: picked without);
        accept [rows] and sample [batch] float32 random numbers in [0, 1).
        Returns (kept [rows], kept_lens [batch], out_tokens [rows]), int32:
        the kept nodes' places, their number, the new tokens (-1 behind).
        result() gives the outcome."""
        d, dev = self.desc, self.device
        rows = tokens.shape[0]
        if rows > self.max_rows:
            raise ValueError(f"at most {self.max_rows} rows")
        _tensor(tokens, "tokens", torch.int32, (rows,), dev)
        _tensor(row_starts, "row_starts", torch.int32, (self.batch + 1,), dev)
        _tensor(accept, "accept", torch.float32, (rows,), dev)
        _tensor(sample, "sample", torch.float32, (self.batch,), dev)
        if parents is not None:
            _tensor(parents, "parents", torch.int32, (rows,), dev)
            d.d_parents = parents.data_ptr()
        else:
            d.d_parents = None
        d.target_row_stride = self._rows_of(target, "target", rows)
        if draft is not None:
            d.draft_row_stride = self._rows_of(draft, "draft", rows)
            d.d_draft = draft.data_ptr()
        else:
            d.d_draft = None
        if kept is None or kept_lens is None or out_tokens is None:
            with torch.cuda.stream(stream):
                make = lambda n, t: torch.empty(n, dtype=torch.int32, device=dev) if t is None else t
                kept, kept_lens, out_tokens = make(rows, kept), make(self.batch, kept_lens), make(rows, out_tokens)
        _tensor(kept, "kept", torch.int32, (rows,), dev)
        _tensor(kept_lens, "kept_lens", torch.int32, (self.batch,), dev)
        _tensor(out_tokens, "out_tokens", torch.int32, (rows,), dev)
        d.rows = rows
        d.d_row_starts, d.d_tokens, d.d_target = row_starts.data_ptr(), tokens.data_ptr(), target.data_ptr()
        d.d_accept, d.d_sample = accept.data_ptr(), sample.data_ptr()
        d.d_kept, d.d_kept_lens, d.d_out_tokens = kept.data_ptr(), kept_lens.data_ptr(), out_tokens.data_ptr()
        ws = self.workspace
        st = _queue(dev, stream, lambda s: _lib_verify(self._ref, ws.data_ptr(), ws.numel(), s), target, tokens, row_starts,
                    accept, sample, parents, draft, kept, kept_lens, out_tokens, own=(self._own,))
        _check(st, "kvc_verify_drafts")
        return kept, kept_lens, out_tokens

    def result(self, stream=None) -> None:
        """Waits for the last call; raises KvcError if it met trees, tokens or
        probabilities that do not fit."""
        st = _queue(self.device, stream, lambda s: _lib_verify_result(self.workspace.data_ptr(), s))
        _check(st, "kvc_verify_drafts")


class PagedCompaction:
    """Moves the kept ones of a step's drafted tokens together in every pool
    of a paged cache.  Calls that may run at the same time need an object
    each."""

    def __init__(self, paged: PagedKV):
        paged._check_pools()
        self.paged, self.device, self.batch = paged, paged.block_table.device, paged.desc.batch
        self._own = _workspace(256 + 4 * self.batch, self.device)
        self.workspace = self._own[1]

    def __call__(self, row_starts: torch.Tensor, context_lens: torch.Tensor | None, kept: torch.Tensor,
                 kept_lens: torch.Tensor, stream=None) -> None:
        """Queue the move: of sequence b's drafted tokens, at positions
        context_lens[b] and on, the kept_lens[b] tokens kept[row_starts[b] + j]
        (places that rise) go to context_lens[b] + j; row_starts [batch + 1],
        context_lens and kept_lens [batch], kept [rows], all int32.  result()
        gives the outcome."""
        dev, paged = self.device, self.paged
        _tensor(row_starts, "row_starts", torch.int32, (self.batch + 1,), dev)
        _tensor(kept, "kept", torch.int32, (None,), dev)
        _tensor(kept_lens, "kept_lens", torch.int32, (self.batch,), dev)
        if context_lens is not None:
            _tensor(context_lens, "context_lens", torch.int32, (self.batch,), dev)
        ws = self.workspace
        st = _queue(dev, stream,
                    lambda s: _lib_compact(paged.ref, paged.kv_dtype, paged.channels, kept.shape[0], row_starts.data_ptr(),
                                           _ptr(context_lens), kept.data_ptr(), kept_lens.data_ptr(), ws.data_ptr(),
                                           ws.numel(), s),
                    row_starts, context_lens, kept, kept_lens, paged.block_table,
                    *(paged.pools if stream is not None else ()), own=(self._own, paged._own))
        _check(st, "kvc_paged_compact")

    def result(self, stream=None) -> None:
        """Waits for the last call; raises KvcError if it met lengths, places
        or page numbers that do not fit."""
        st = _queue(self.device, stream, lambda s: _lib_compact_result(self.workspace.data_ptr(), s))
        _check(st, "kvc_paged_compact")


class SharedPages:
    """Requests that start from another's tokens and share its full pages.
    The state is BlockTable's (the table of `paged`, held [batch], free_pages,
    free_count [1]) and a count of each page's further holders, extra
    [num_pages] (0 for pages that one request holds, or none), all int32 and
    the caller's; a call updates them in place, or writes held_out and
    free_count_out where they are given.  A request whose pages were shared
    ends with release(), not with a trim, and is not trimmed below the tokens
    that it was forked from or with: BlockTable would hand out, without an
    error, pages that others hold.  Calls that may run at the same time
    need an object each."""

    def __init__(self, paged: PagedKV, held: torch.Tensor, free_pages: torch.Tensor, free_count: torch.Tensor,
                 extra: torch.Tensor, held_out: torch.Tensor | None = None, free_count_out: torch.Tensor | None = None):
        paged._check_pools()
        self.paged, self.device = paged, paged.block_table.device
        self.held, self.free_pages, self.free_count, self.extra = held, free_pages, free_count, extra
        self.held_out = held if held_out is None else held_out
        self.free_count_out = free_count if free_count_out is None else free_count_out
        batch, num_pages = paged.desc.batch, paged.desc.num_pages
        for t, name, n in ((held, "held", batch), (self.held_out, "held_out", batch), (free_pages, "free_pages", None),
                           (free_count, "free_count", 1), (self.free_count_out, "free_count_out", 1),
                           (extra, "extra", num_pages)):
            _tensor(t, name, torch.int32, (n,), self.device)
        if free_pages.shape[0] < num_pages:
            raise ValueError(f"free_pages must have room for {num_pages} pages")
        self._own = _workspace(256 + 4096 + 64 * ((num_pages + 31) // 32), self.device)
        self.workspace = self._own[1]
        self.desc = kvc_shared_pages(free_pages.numel(), _ptr(paged.block_table), _ptr(held), _ptr(self.held_out),
                                     _ptr(free_pages), _ptr(free_count), _ptr(self.free_count_out), _ptr(extra))
        self._ref = ctypes.byref(self.desc)

    def _run(self, call, where, count, stream, *tensors):
        paged, ws = self.paged, self.workspace
        args = [_ptr(t) for t in tensors]
        st = _queue(self.device, stream,
                    lambda s: call(paged.ref, paged.kv_dtype, paged.channels, self._ref, count, *args, ws.data_ptr(),
                                   ws.numel(), s),
                    *tensors, self.held, self.held_out, self.free_pages, self.free_count, self.free_count_out, self.extra,
                    paged.block_table, *(paged.pools if stream is not None else ()), own=(self._own, paged._own))
        _check(st, where)

    def fork(self, parents: torch.Tensor, children: torch.Tensor, context_lens: torch.Tensor | None, stream=None) -> None:
        """Queue the fork: request children[k], which holds no page, gets the
        context_lens[parents[k]] tokens of request parents[k] (int32, up to
        1024; a child of -1: none); context_lens int32 [batch].  result()
        gives the outcome."""
        _tensor(children, "children", torch.int32, (None,), self.device)
        _tensor(parents, "parents", torch.int32, (children.shape[0],), self.device)
        if context_lens is not None:
            _tensor(context_lens, "context_lens", torch.int32, (self.paged.desc.batch,), self.device)
        self._run(_lib_fork, "kvc_fork_pages", children.shape[0], stream, parents, children, context_lens)

    def release(self, requests: torch.Tensor, stream=None) -> None:
        """Queue the release of the requests (int32, up to 1024; -1: none):
        pages that nobody else holds go to the stack.  result() gives the
        outcome."""
        _tensor(requests, "requests", torch.int32, (None,), self.device)
        self._run(_lib_release, "kvc_release_pages", requests.shape[0], stream, requests)

    def result(self, stream=None) -> None:
        """Waits for the last call; raises KvcError if it failed."""
        st = _queue(self.device, stream, lambda s: _lib_shared_result(self.workspace.data_ptr(), s))
        _check(st, "kvc_shared_pages")


def calibrate_workspace_bytes(planes: int, channels: int) -> int:
    return planes * channels * 1024


def kvc_calibrate_sigma(kv: torch.Tensor, mu: torch.Tensor, sigma_floor: float = 2.0 ** -30,
                        out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        stream=None, block_tokens: int = 0) -> torch.Tensor:
    """kv, mu: [reps, planes, tokens, channels] -> sigma [planes, channels],
    or with block_tokens = B > 0 sigma [planes, ceil(tokens / B), channels]
    (one sigma per block of B tokens)."""
    _need(kv, "kv")
    _need(mu, "mu")
    r, g, t, d = kv.shape
    shape = sigma_shape(g, t, d, block_tokens)
    n_rows = g if block_tokens == 0 else g * shape[1]
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=kv.device)
    if workspace is None:
        workspace = torch.empty(calibrate_workspace_bytes(n_rows, d), dtype=torch.uint8, device=kv.device)
    if block_tokens == 0:
        st = _lib_calibrate(_ptr(kv), _ptr(mu), _kv_dtype(kv), _mu_dtype(mu), r, g, t, d, sigma_floor,
                            _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream))
    else:
        st = _lib_calibrate_blocks(_ptr(kv), _ptr(mu), _kv_dtype(kv), _mu_dtype(mu), r, g, t, d, block_tokens,
                                   sigma_floor, _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "kvc_calibrate_sigma")
    return out


def kvc_calibrate_sigma_rate(kv: torch.Tensor, mu: torch.Tensor, prefix: torch.Tensor | None = None,
                             weights=(9500, 300), sigma_floor: float = 2.0 ** -30, block_tokens: int = 0,
                             out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                             stream=None, narrow_dof: int = 0) -> torch.Tensor:
    """Rate-fitted sigma: of the candidates max(floor, rms * (1 - j/32)),
    j = 0..24, the one with the least integer code length of the held-out
    kv [reps, planes, tokens, channels] under the mixture the data will be
    coded with.  Shapes as kvc_calibrate_sigma."""
    _need(kv, "kv")
    _need(mu, "mu")
    r, g, t, d = kv.shape
    shape = sigma_shape(g, t, d, block_tokens)
    n_rows = g if block_tokens == 0 else g * shape[1]
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=kv.device)
    if workspace is None:
        workspace = torch.empty(n_rows * d * (1024 + 12800) + 65536, dtype=torch.uint8, device=kv.device)
    st = _lib_calibrate_rate(_ptr(kv), _ptr(mu), _kv_dtype(kv), _mu_dtype(mu), r, g, t, d, block_tokens,
                             sigma_floor, weights[0], weights[1], narrow_dof, _ptr(prefix), _ptr(out), _ptr(workspace),
                             workspace.numel(), _stream(stream))
    _check(st, "kvc_calibrate_sigma_rate")
    return out


def kvc_calibrate_split(kv: torch.Tensor, mu: torch.Tensor, sigma: torch.Tensor, prefix: torch.Tensor | None = None,
                        weights=(9500, 300), block_tokens: int = 0, narrow_dof: int = 0,
                        out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """Per-channel narrow weights: of w_j = max(w_n + w_w - 200 j, 0),
    j = 0..15, the one with the least integer code length of the held-out
    kv [reps, planes, tokens, channels] under sigma (the one the stream will
    use: [G, D], or [G, ceil(T / B), D] with block_tokens = B).  Returns
    int32 [G, D]."""
    _need(kv, "kv")
    _need(mu, "mu")
    _need(sigma, "sigma")
    r, g, t, d = kv.shape
    if out is None:
        out = torch.empty((g, d), dtype=torch.int32, device=kv.device)
    if workspace is None:
        workspace = torch.empty(g * d * 8192, dtype=torch.uint8, device=kv.device)
    st = _lib_calibrate_split(_ptr(kv), _ptr(mu), _kv_dtype(kv), _mu_dtype(mu), r, g, t, d, block_tokens, _ptr(sigma),
                              weights[0], weights[1], narrow_dof, _ptr(prefix), _ptr(out), _ptr(workspace),
                              workspace.numel(), _stream(stream))
    _check(st, "kvc_calibrate_split")
    return out


def kvc_build_marginal(samples: torch.Tensor, weights=(9500, 300), stream=None) -> torch.Tensor:
    """Prefix table of the +1-smoothed marginal; returned as int32 (all
    values are below 2^31) with N + 1 entries."""
    _need(samples, "samples")
    dt = _kv_dtype(samples)
    n_sym = 65536 if dt == KVC_BF16 else 256
    out = torch.empty(n_sym + 1, dtype=torch.int32, device=samples.device)
    st = _lib_marginal(_ptr(samples), dt, samples.numel(), weights[0], weights[1], _ptr(out), _stream(stream))
    _check(st, "kvc_build_marginal")
    return out


def kvc_estimate_bits(kv, mu, sigma, prefix=None, weights=(9500, 300), stream=None, sigma_block_tokens: int = 0,
                      chunk_tokens: int = 0, narrow_dof: int = 0, channel_split: torch.Tensor | None = None):
    """(integer-model bits/scalar, float-model bits/scalar)."""
    g, t, d = kv.shape
    if channel_split is not None:
        sigma = side_info(sigma, channel_split)
    p = make_params(_kv_dtype(kv), _mu_dtype(mu), g, t, d, weights, chunk_tokens, sigma_block_tokens, narrow_dof,
                    0 if channel_split is None else 1)
    ws = torch.empty(ESTIMATE_WORKSPACE_BYTES, dtype=torch.uint8, device=kv.device)
    out = (ctypes.c_double * 2)()
    st = _lib_estimate(ctypes.byref(p), _ptr(kv), _ptr(mu), _ptr(sigma), _ptr(prefix), ctypes.addressof(out),
                       _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "kvc_estimate_bits")
    return out[0], out[1]


def kvc_cdf_table(kv_dtype: int, mu: torch.Tensor, sigma: torch.Tensor, prefix=None, weights=(9500, 300),
                  stream=None, narrow_dof: int = 0) -> torch.Tensor:
    """C(b) for b = 0..N for each (mu, sigma) pair; int32 storage of uint32
    values (reinterpret as uint32 on the host)."""
    _need(mu, "mu")
    _need(sigma, "sigma")
    n_sym = 65536 if kv_dtype == KVC_BF16 else 256
    pairs = mu.numel()
    out = torch.empty((pairs, n_sym + 1), dtype=torch.int32, device=mu.device)
    st = _lib_cdf_table(kv_dtype, _mu_dtype(mu), weights[0], weights[1], narrow_dof, _ptr(mu), _ptr(sigma), pairs,
                        _ptr(prefix), _ptr(out), _stream(stream))
    _check(st, "kvc_cdf_table")
    return out

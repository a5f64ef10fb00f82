"""Thin Python binding of libvsamp.so, the GB300 per-row vocabulary sampling stage.

The functions carry the C-ABI names (include/vsamp.h) and only marshal arguments: torch tensors are
passed as device pointers, missing outputs are allocated with torch on the input's device, and the
call is enqueued on the current torch stream. Every step of the stage runs in the library's CUDA
kernels; there is no CPU or PyTorch fallback. If the library is missing the import still works, but
every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libvsamp.so")

VSAMP_OK = 0
VSAMP_ERR_INVALID_ARG = 1
VSAMP_ERR_UNSUPPORTED = 2
VSAMP_ERR_CUDA = 3
VSAMP_ERR_NONFINITE = 4
VSAMP_ERR_TIMEOUT = 5
VSAMP_ERR_SCRATCH_LIMIT = 6
VSAMP_STATIC_SCRATCH_BYTES = 1 << 22   # the fixed scratch array of vsamp_sample_static
VSAMP_F32 = 0
VSAMP_BF16 = 1
VSAMP_TOKEN_IGNORE = -100              # a token that is not scored and gets no gradient
VSAMP_SCORE_ALT_MAX = 128              # most alternatives of vsamp_score_tokens

EXPORTED = ("vsamp_softmax_lse", "vsamp_topk_select", "vsamp_topp_minp_mask", "vsamp_sample",
            "vsamp_sample_ws", "vsamp_sample_workspace_size", "vsamp_sample_static", "vsamp_logprob", "vsamp_topn_logprobs", "vsamp_kept_logprob",
            "vsamp_shard_pieces", "vsamp_shard_workspace_size", "vsamp_shard_partial", "vsamp_shard_merge",
            "vsamp_sample_rejection",
            "vsamp_score_workspace_size", "vsamp_score_tokens", "vsamp_score_tokens_backward",
            "vsamp_head_packed_size", "vsamp_head_pack", "vsamp_head_logits",
            "vsamp_embed", "vsamp_embed_workspace_size", "vsamp_embed_backward",
            "vsamp_status_string",
            "vsamp_device_info", "vsamp_version")


class VsampError(RuntimeError):
    def __init__(self, status: int, fn: str):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)} (status {status})")


class vsamp_cut(ctypes.Structure):
    _fields_ = [("pivot_key", ctypes.c_uint32), ("idx_cut", ctypes.c_int32), ("kept", ctypes.c_int32),
                ("status", ctypes.c_int32)]


class vsamp_limits(ctypes.Structure):
    _fields_ = [("sm_count", ctypes.c_int32), ("smem_optin_bytes", ctypes.c_int32),
                ("max_cluster", ctypes.c_int32), ("max_row_f32", ctypes.c_int64),
                ("max_row_bf16", ctypes.c_int64)]


_lib = None


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libvsamp.so (once) and declare the C signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is not built: run `python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(p)
    vp, i64, i32, st = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
    lib.vsamp_softmax_lse.argtypes = [vp, st, i64, i64, i64, vp, vp, vp, vp, vp]
    lib.vsamp_topk_select.argtypes = [vp, st, i64, i64, i64, vp, vp, i32, vp, vp, vp]
    lib.vsamp_topp_minp_mask.argtypes = [vp, st, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.vsamp_sample.argtypes = [vp, st, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.vsamp_logprob.argtypes = [vp, st, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp]
    lib.vsamp_sample_ws.argtypes = [vp, st, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                    ctypes.c_size_t, vp]
    lib.vsamp_sample_static.argtypes = [vp, st, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.vsamp_topn_logprobs.argtypes = [vp, st, i64, i64, i64, vp, i32, vp, vp, vp, vp, vp, vp]
    lib.vsamp_shard_pieces.argtypes = [st, i64]
    lib.vsamp_shard_pieces.restype = i64
    lib.vsamp_shard_workspace_size.argtypes = [st, i64, i64]
    lib.vsamp_shard_workspace_size.restype = ctypes.c_size_t
    lib.vsamp_shard_partial.argtypes = [vp, st, i64, i64, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp,
                                        ctypes.c_size_t, vp]
    lib.vsamp_shard_merge.argtypes = [vp, vp, i32, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.vsamp_shard_partial.restype = st
    lib.vsamp_sample_rejection.argtypes = [vp, st, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.vsamp_sample_rejection.restype = st
    lib.vsamp_shard_merge.restype = st
    lib.vsamp_kept_logprob.argtypes = [vp, st, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.vsamp_sample_workspace_size.argtypes = [st, i64, i64]
    lib.vsamp_sample_workspace_size.restype = ctypes.c_size_t
    for f in ("vsamp_softmax_lse", "vsamp_topk_select", "vsamp_topp_minp_mask", "vsamp_sample", "vsamp_logprob",
              "vsamp_sample_ws", "vsamp_sample_static", "vsamp_topn_logprobs", "vsamp_kept_logprob"):
        getattr(lib, f).restype = st
    sz = ctypes.c_size_t
    f32 = ctypes.c_float
    lib.vsamp_score_workspace_size.argtypes = [st, i64, i64, i32]
    lib.vsamp_score_workspace_size.restype = sz
    lib.vsamp_score_tokens.argtypes = [vp, st, i64, i64, i64, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.vsamp_score_tokens_backward.argtypes = [vp, st, i64, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp, i64, vp, vp]
    lib.vsamp_head_packed_size.argtypes = [st, i32, i64, i64, i32]
    lib.vsamp_head_packed_size.restype = sz
    lib.vsamp_head_pack.argtypes = [vp, vp, st, vp, i64, i64, i32, vp, sz, vp]
    lib.vsamp_head_logits.argtypes = [vp, st, i64, i64, vp, sz, st, i32, i64, i64, i32, vp, st, i64, vp]
    lib.vsamp_embed.argtypes = [vp, i64, vp, st, i64, i64, i64, f32, vp, st, i64, vp, vp]
    lib.vsamp_embed_workspace_size.argtypes = [i64, i64]
    lib.vsamp_embed_workspace_size.restype = sz
    lib.vsamp_embed_backward.argtypes = [vp, i64, vp, st, i64, i64, f32, i64, vp, st, i64, i32, vp, sz, vp]
    for f in ("vsamp_score_tokens", "vsamp_score_tokens_backward", "vsamp_head_pack", "vsamp_head_logits",
              "vsamp_embed", "vsamp_embed_backward"):
        getattr(lib, f).restype = st
    lib.vsamp_status_string.argtypes = [st]
    lib.vsamp_status_string.restype = ctypes.c_char_p
    lib.vsamp_device_info.argtypes = [ctypes.c_int, ctypes.POINTER(vsamp_limits)]
    lib.vsamp_device_info.restype = st
    lib.vsamp_version.argtypes = []
    lib.vsamp_version.restype = i32
    if path is None:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().vsamp_status_string(int(status)).decode()


def version() -> int:
    return int(load().vsamp_version())


def device_info(device: int = 0) -> vsamp_limits:
    out = vsamp_limits()
    _check(load().vsamp_device_info(int(device), ctypes.byref(out)), "vsamp_device_info")
    return out


# ------------------------------------------------------------------------------------------------
# marshalling helpers
# ------------------------------------------------------------------------------------------------
def _check(status: int, fn: str):
    if status != VSAMP_OK:
        raise VsampError(status, fn)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return VSAMP_F32
    if t.dtype == torch.bfloat16:
        return VSAMP_BF16
    raise TypeError(f"logits must be float32 or bfloat16, got {t.dtype}")


def _rows(x: torch.Tensor, V: Optional[int]):
    if x.dim() != 2 or not x.is_cuda:
        raise ValueError("logits must be a 2-D CUDA tensor [B, >= V]")
    if x.stride(1) != 1:
        raise ValueError("logits rows must be contiguous (stride(1) == 1)")
    B = x.shape[0]
    V = x.shape[1] if V is None else int(V)
    return B, V, x.stride(0) if B > 1 else max(x.stride(0), V)


def _ptr(t: Optional[torch.Tensor], dtype=None, dev=None, B=None, name="") -> int:
    if t is None:
        return 0
    if not t.is_cuda or (dev is not None and t.device != dev):
        raise ValueError(f"{name} must be on {dev}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if B is not None and t.numel() < B:
        raise ValueError(f"{name} needs at least {B} elements")
    return t.data_ptr()


def _param(v, B: int, dtype, dev, name):
    """Per-row parameter: None, a scalar (broadcast) or a [B] device tensor."""
    if v is None:
        return None
    if isinstance(v, torch.Tensor):
        return v.to(device=dev, dtype=dtype).contiguous()
    return torch.full((B,), v, dtype=dtype, device=dev)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


# ------------------------------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ------------------------------------------------------------------------------------------------
def vsamp_softmax_lse(logits, temperature=None, V=None, row_max=None, row_logsum=None, row_status=None,
                      stream=None):
    """Row maximum and log-sum-exp of (x - max)/T. Returns (row_max, row_logsum, row_status)."""
    B, V, ld = _rows(logits, V)
    dev = logits.device
    temperature = _param(temperature, B, torch.float32, dev, "temperature")
    row_max = torch.empty(B, dtype=torch.float32, device=dev) if row_max is None else row_max
    row_logsum = torch.empty(B, dtype=torch.float32, device=dev) if row_logsum is None else row_logsum
    row_status = torch.empty(B, dtype=torch.int32, device=dev) if row_status is None else row_status
    st = load().vsamp_softmax_lse(
        logits.data_ptr(), _dtype_code(logits), B, V, ld, _ptr(temperature, torch.float32, dev, B, "temperature"),
        _ptr(row_max, torch.float32, dev, B, "row_max"), _ptr(row_logsum, torch.float32, dev, B, "row_logsum"),
        _ptr(row_status, torch.int32, dev, B, "row_status"), _stream(stream))
    _check(st, "vsamp_softmax_lse")
    return row_max, row_logsum, row_status


def vsamp_topk_select(scores, k, k_max=None, lengths=None, max_len=None, out_idx=None, row_status=None,
                      stream=None):
    """Top-k indices per row in ascending index order, -1 padded. Returns (out_idx [B, k_max], row_status)."""
    B, max_len, ld = _rows(scores, max_len)
    dev = scores.device
    if isinstance(k, int) and k_max is None:
        k_max = k
    if k_max is None:
        raise ValueError("k_max is required when k is a tensor")
    k = _param(k, B, torch.int32, dev, "k")
    lengths = _param(lengths, B, torch.int32, dev, "lengths")
    out_idx = torch.empty((B, int(k_max)), dtype=torch.int32, device=dev) if out_idx is None else out_idx
    row_status = torch.empty(B, dtype=torch.int32, device=dev) if row_status is None else row_status
    st = load().vsamp_topk_select(
        scores.data_ptr(), _dtype_code(scores), B, max_len, ld, _ptr(lengths, torch.int32, dev, B, "lengths"),
        _ptr(k, torch.int32, dev, B, "k"), int(k_max), _ptr(out_idx, torch.int32, dev, B * int(k_max), "out_idx"),
        _ptr(row_status, torch.int32, dev, B, "row_status"), _stream(stream))
    _check(st, "vsamp_topk_select")
    return out_idx, row_status


def vsamp_topp_minp_mask(logits, temperature=None, top_k=None, top_p=None, min_p=None, V=None,
                         want_mask=True, cut=None, mask=None, stats=None, stream=None):
    """Cut descriptors [B, 4] int32 (pivot_key as int32 bits, idx_cut, kept, status), mask [B, V] uint8
    (or None) and stats [B, 4]."""
    B, V, ld = _rows(logits, V)
    dev = logits.device
    temperature = _param(temperature, B, torch.float32, dev, "temperature")
    top_k = _param(top_k, B, torch.int32, dev, "top_k")
    top_p = _param(top_p, B, torch.float32, dev, "top_p")
    min_p = _param(min_p, B, torch.float32, dev, "min_p")
    cut = torch.empty((B, 4), dtype=torch.int32, device=dev) if cut is None else cut
    if want_mask and mask is None:
        mask = torch.empty((B, V), dtype=torch.uint8, device=dev)
    stats = torch.empty((B, 4), dtype=torch.int32, device=dev) if stats is None else stats
    st = load().vsamp_topp_minp_mask(
        logits.data_ptr(), _dtype_code(logits), B, V, ld, _ptr(temperature, torch.float32, dev, B, "temperature"),
        _ptr(top_k, torch.int32, dev, B, "top_k"), _ptr(top_p, torch.float32, dev, B, "top_p"),
        _ptr(min_p, torch.float32, dev, B, "min_p"), _ptr(cut, torch.int32, dev, 4 * B, "cut"),
        _ptr(mask, torch.uint8, dev, B * V, "mask"), _ptr(stats, torch.int32, dev, 4 * B, "stats"),
        _stream(stream))
    _check(st, "vsamp_topp_minp_mask")
    return cut, mask, stats


def vsamp_sample(logits, temperature=None, top_k=None, top_p=None, min_p=None, seed=None, step=None,
                 row_id=None, V=None, token=None, logprob=None, row_status=None, stats=None,
                 want_logprob=True, want_stats=False, stream=None):
    """The fused stage. Returns (token [B] int32, logprob [B] fp32 or None, row_status [B], stats or None)."""
    B, V, ld = _rows(logits, V)
    dev = logits.device
    temperature = _param(temperature, B, torch.float32, dev, "temperature")
    top_k = _param(top_k, B, torch.int32, dev, "top_k")
    top_p = _param(top_p, B, torch.float32, dev, "top_p")
    min_p = _param(min_p, B, torch.float32, dev, "min_p")
    seed = _param(seed, B, torch.int64, dev, "seed")
    step = _param(step, B, torch.int64, dev, "step")
    row_id = _param(row_id, B, torch.int32, dev, "row_id")
    token = torch.empty(B, dtype=torch.int32, device=dev) if token is None else token
    if want_logprob and logprob is None:
        logprob = torch.empty(B, dtype=torch.float32, device=dev)
    row_status = torch.empty(B, dtype=torch.int32, device=dev) if row_status is None else row_status
    if want_stats and stats is None:
        stats = torch.empty((B, 4), dtype=torch.int32, device=dev)
    st = load().vsamp_sample(
        logits.data_ptr(), _dtype_code(logits), B, V, ld, _ptr(temperature, torch.float32, dev, B, "temperature"),
        _ptr(top_k, torch.int32, dev, B, "top_k"), _ptr(top_p, torch.float32, dev, B, "top_p"),
        _ptr(min_p, torch.float32, dev, B, "min_p"), _ptr(seed, torch.int64, dev, B, "seed"),
        _ptr(step, torch.int64, dev, B, "step"), _ptr(row_id, torch.int32, dev, B, "row_id"),
        _ptr(token, torch.int32, dev, B, "token"), _ptr(logprob, torch.float32, dev, B, "logprob"),
        _ptr(row_status, torch.int32, dev, B, "row_status"), _ptr(stats, torch.int32, dev, 4 * B, "stats"),
        _stream(stream))
    _check(st, "vsamp_sample")
    return token, logprob, row_status, stats


def vsamp_sample_rejection(logits, temperature=None, top_k=None, top_p=None, min_p=None, seed=None, step=None,
                           row_id=None, V=None, token=None, logprob=None, row_status=None, stats=None,
                           want_logprob=True, want_stats=False, stream=None):
    """The dual-pivot rejection sampler: the law of vsamp_sample from other random numbers. Returns (token,
    logprob or None, row_status, stats or None); stats rows are {passes, rounds, 0, path flags}."""
    B, V, ld = _rows(logits, V)
    dev = logits.device
    temperature = _param(temperature, B, torch.float32, dev, "temperature")
    top_k = _param(top_k, B, torch.int32, dev, "top_k")
    top_p = _param(top_p, B, torch.float32, dev, "top_p")
    min_p = _param(min_p, B, torch.float32, dev, "min_p")
    seed = _param(seed, B, torch.int64, dev, "seed")
    step = _param(step, B, torch.int64, dev, "step")
    row_id = _param(row_id, B, torch.int32, dev, "row_id")
    token = torch.empty(B, dtype=torch.int32, device=dev) if token is None else token
    if want_logprob and logprob is None:
        logprob = torch.empty(B, dtype=torch.float32, device=dev)
    row_status = torch.empty(B, dtype=torch.int32, device=dev) if row_status is None else row_status
    if want_stats and stats is None:
        stats = torch.empty((B, 4), dtype=torch.int32, device=dev)
    st = load().vsamp_sample_rejection(
        logits.data_ptr(), _dtype_code(logits), B, V, ld, _ptr(temperature, torch.float32, dev, B, "temperature"),
        _ptr(top_k, torch.int32, dev, B, "top_k"), _ptr(top_p, torch.float32, dev, B, "top_p"),
        _ptr(min_p, torch.float32, dev, B, "min_p"), _ptr(seed, torch.int64, dev, B, "seed"),
        _ptr(step, torch.int64, dev, B, "step"), _ptr(row_id, torch.int32, dev, B, "row_id"),
        _ptr(token, torch.int32, dev, B, "token"), _ptr(logprob, torch.float32, dev, B, "logprob"),
        _ptr(row_status, torch.int32, dev, B, "row_status"), _ptr(stats, torch.int32, dev, 4 * B, "stats"),
        _stream(stream))
    _check(st, "vsamp_sample_rejection")
    return token, logprob, row_status, stats


_WORKSPACES = {}


def sample_workspace(device, nbytes: int, stream=None) -> torch.Tensor:
    """A workspace of at least nbytes for vsamp_sample_ws, cached per (device, stream).

    A call writes everything it reads in the workspace, so it is reused as is; calls
    on one stream never overlap, so a workspace per stream is enough."""
    dev = torch.device(device)
    key = (dev.index if dev.index is not None else torch.cuda.current_device(), _stream(stream))
    ws = _WORKSPACES.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=dev)
        _WORKSPACES[key] = ws
    return ws


def vsamp_sample_ws(logits, temperature=None, top_k=None, top_p=None, min_p=None, seed=None, step=None,
                    row_id=None, V=None, token=None, logprob=None, row_status=None, stats=None,
                    want_logprob=True, want_stats=False, stream=None, workspace=None):
    """vsamp_sample through the split-vocabulary kernels and a workspace (cached per device and stream
    unless given). Returns (token, logprob or None, row_status, stats or None)."""
    B, V, ld = _rows(logits, V)
    dev = logits.device
    temperature = _param(temperature, B, torch.float32, dev, "temperature")
    top_k = _param(top_k, B, torch.int32, dev, "top_k")
    top_p = _param(top_p, B, torch.float32, dev, "top_p")
    min_p = _param(min_p, B, torch.float32, dev, "min_p")
    seed = _param(seed, B, torch.int64, dev, "seed")
    step = _param(step, B, torch.int64, dev, "step")
    row_id = _param(row_id, B, torch.int32, dev, "row_id")
    token = torch.empty(B, dtype=torch.int32, device=dev) if token is None else token
    if want_logprob and logprob is None:
        logprob = torch.empty(B, dtype=torch.float32, device=dev)
    row_status = torch.empty(B, dtype=torch.int32, device=dev) if row_status is None else row_status
    if want_stats and stats is None:
        stats = torch.empty((B, 4), dtype=torch.int32, device=dev)
    lib = load()
    need = int(lib.vsamp_sample_workspace_size(_dtype_code(logits), B, V))
    if workspace is None:
        workspace = sample_workspace(dev, need, stream)
    st = lib.vsamp_sample_ws(
        logits.data_ptr(), _dtype_code(logits), B, V, ld, _ptr(temperature, torch.float32, dev, B, "temperature"),
        _ptr(top_k, torch.int32, dev, B, "top_k"), _ptr(top_p, torch.float32, dev, B, "top_p"),
        _ptr(min_p, torch.float32, dev, B, "min_p"), _ptr(seed, torch.int64, dev, B, "seed"),
        _ptr(step, torch.int64, dev, B, "step"), _ptr(row_id, torch.int32, dev, B, "row_id"),
        _ptr(token, torch.int32, dev, B, "token"), _ptr(logprob, torch.float32, dev, B, "logprob"),
        _ptr(row_status, torch.int32, dev, B, "row_status"), _ptr(stats, torch.int32, dev, 4 * B, "stats"),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "vsamp_sample_ws")
    return token, logprob, row_status, stats


def vsamp_sample_static(logits, temperature=None, top_k=None, top_p=None, min_p=None, seed=None, step=None,
                        row_id=None, V=None, token=None, logprob=None, row_status=None, stats=None,
                        want_logprob=True, want_stats=False, stream=None):
    """vsamp_sample_ws on the library's fixed scratch array (no allocation by the library; calls that
    overlap on one device race). Returns (token, logprob or None, row_status, stats or None)."""
    B, V, ld = _rows(logits, V)
    dev = logits.device
    temperature = _param(temperature, B, torch.float32, dev, "temperature")
    top_k = _param(top_k, B, torch.int32, dev, "top_k")
    top_p = _param(top_p, B, torch.float32, dev, "top_p")
    min_p = _param(min_p, B, torch.float32, dev, "min_p")
    seed = _param(seed, B, torch.int64, dev, "seed")
    step = _param(step, B, torch.int64, dev, "step")
    row_id = _param(row_id, B, torch.int32, dev, "row_id")
    token = torch.empty(B, dtype=torch.int32, device=dev) if token is None else token
    if want_logprob and logprob is None:
        logprob = torch.empty(B, dtype=torch.float32, device=dev)
    row_status = torch.empty(B, dtype=torch.int32, device=dev) if row_status is None else row_status
    if want_stats and stats is None:
        stats = torch.empty((B, 4), dtype=torch.int32, device=dev)
    st = load().vsamp_sample_static(
        logits.data_ptr(), _dtype_code(logits), B, V, ld, _ptr(temperature, torch.float32, dev, B, "temperature"),
        _ptr(top_k, torch.int32, dev, B, "top_k"), _ptr(top_p, torch.float32, dev, B, "top_p"),
        _ptr(min_p, torch.float32, dev, B, "min_p"), _ptr(seed, torch.int64, dev, B, "seed"),
        _ptr(step, torch.int64, dev, B, "step"), _ptr(row_id, torch.int32, dev, B, "row_id"),
        _ptr(token, torch.int32, dev, B, "token"), _ptr(logprob, torch.float32, dev, B, "logprob"),
        _ptr(row_status, torch.int32, dev, B, "row_status"), _ptr(stats, torch.int32, dev, 4 * B, "stats"),
        _stream(stream))
    _check(st, "vsamp_sample_static")
    return token, logprob, row_status, stats


def vsamp_logprob(logits, token, temperature=None, row_max=None, row_logsum=None, V=None, out=None,
                  row_status=None, stream=None):
    """min((x_t - max)/T - log S, 0) per row. Returns (logprob, row_status)."""
    B, V, ld = _rows(logits, V)
    dev = logits.device
    temperature = _param(temperature, B, torch.float32, dev, "temperature")
    token = _param(token, B, torch.int32, dev, "token")
    out = torch.empty(B, dtype=torch.float32, device=dev) if out is None else out
    row_status = torch.empty(B, dtype=torch.int32, device=dev) if row_status is None else row_status
    st = load().vsamp_logprob(
        logits.data_ptr(), _dtype_code(logits), B, V, ld, _ptr(temperature, torch.float32, dev, B, "temperature"),
        _ptr(token, torch.int32, dev, B, "token"), _ptr(row_max, torch.float32, dev, B, "row_max"),
        _ptr(row_logsum, torch.float32, dev, B, "row_logsum"), _ptr(out, torch.float32, dev, B, "out"),
        _ptr(row_status, torch.int32, dev, B, "row_status"), _stream(stream))
    _check(st, "vsamp_logprob")
    return out, row_status


def vsamp_topn_logprobs(logits, n, temperature=None, V=None, row_max=None, row_logsum=None, out_idx=None,
                        out_lp=None, row_status=None, stream=None):
    """The n most probable tokens per row by (logit desc, index asc) with their log-probabilities.
    Returns (out_idx [B, n] int32, out_lp [B, n] fp32, row_max, row_logsum, row_status)."""
    B, V, ld = _rows(logits, V)
    dev = logits.device
    n = int(n)
    temperature = _param(temperature, B, torch.float32, dev, "temperature")
    row_max = torch.empty(B, dtype=torch.float32, device=dev) if row_max is None else row_max
    row_logsum = torch.empty(B, dtype=torch.float32, device=dev) if row_logsum is None else row_logsum
    out_idx = torch.empty((B, max(n, 1)), dtype=torch.int32, device=dev) if out_idx is None else out_idx
    out_lp = torch.empty((B, max(n, 1)), dtype=torch.float32, device=dev) if out_lp is None else out_lp
    row_status = torch.empty(B, dtype=torch.int32, device=dev) if row_status is None else row_status
    st = load().vsamp_topn_logprobs(
        logits.data_ptr(), _dtype_code(logits), B, V, ld, _ptr(temperature, torch.float32, dev, B, "temperature"),
        n, _ptr(row_max, torch.float32, dev, B, "row_max"), _ptr(row_logsum, torch.float32, dev, B, "row_logsum"),
        _ptr(out_idx, torch.int32, dev, B * max(n, 1), "out_idx"),
        _ptr(out_lp, torch.float32, dev, B * max(n, 1), "out_lp"),
        _ptr(row_status, torch.int32, dev, B, "row_status"), _stream(stream))
    _check(st, "vsamp_topn_logprobs")
    return out_idx, out_lp, row_max, row_logsum, row_status


def vsamp_kept_logprob(logits, token, temperature=None, top_k=None, top_p=None, min_p=None, V=None, out=None,
                       row_status=None, stream=None):
    """Log-probability of token[r] renormalised over the kept set of the row's cut (-inf outside it).
    Returns (out [B] fp32, row_status)."""
    B, V, ld = _rows(logits, V)
    dev = logits.device
    temperature = _param(temperature, B, torch.float32, dev, "temperature")
    top_k = _param(top_k, B, torch.int32, dev, "top_k")
    top_p = _param(top_p, B, torch.float32, dev, "top_p")
    min_p = _param(min_p, B, torch.float32, dev, "min_p")
    token = _param(token, B, torch.int32, dev, "token")
    out = torch.empty(B, dtype=torch.float32, device=dev) if out is None else out
    row_status = torch.empty(B, dtype=torch.int32, device=dev) if row_status is None else row_status
    st = load().vsamp_kept_logprob(
        logits.data_ptr(), _dtype_code(logits), B, V, ld, _ptr(temperature, torch.float32, dev, B, "temperature"),
        _ptr(top_k, torch.int32, dev, B, "top_k"), _ptr(top_p, torch.float32, dev, B, "top_p"),
        _ptr(min_p, torch.float32, dev, B, "min_p"), _ptr(token, torch.int32, dev, B, "token"),
        _ptr(out, torch.float32, dev, B, "out"), _ptr(row_status, torch.int32, dev, B, "row_status"),
        _stream(stream))
    _check(st, "vsamp_kept_logprob")
    return out, row_status


# ------------------------------------------------------------------------------------------------
# vocabulary-sharded sampling: rank-local summaries, rank-ordered exchange, the owned merge
# ------------------------------------------------------------------------------------------------
PIECE_REC_BYTES = 32
SHARD_WIN_BYTES = 16


def shard_bounds(V: int, R: int, dtype=torch.bfloat16, align_to_pieces: bool = True):
    """Split [0, V) into R contiguous shards in rank order: [(v0, V_r)]. With align_to_pieces every boundary is a
    multiple of the 4 KB piece (2048 bf16 or 1024 fp32 logits), which makes the merged outputs bit-identical to the
    unsharded streaming sampler; otherwise boundaries are multiples of the 16-byte vector (8 bf16 or 4 fp32)."""
    if R <= 0 or V <= 0:
        raise ValueError("V and R must be positive")
    unit = (2048 if dtype == torch.bfloat16 else 1024) if align_to_pieces else (8 if dtype == torch.bfloat16 else 4)
    units = -(-V // unit)
    out, start = [], 0
    for r in range(R):
        end = min(V, (units * (r + 1) // R) * unit)
        out.append((start, max(0, end - start)))
        start = end
    if any(n <= 0 for _, n in out):
        raise ValueError(f"V = {V} is too short for {R} shards of whole {unit}-logit units")
    return out


def shard_record_slots(bounds, dtype=torch.bfloat16) -> int:
    """NP: the record slots per row every shard writes (the most pieces of any shard)."""
    dt = VSAMP_F32 if dtype == torch.float32 else VSAMP_BF16
    return max(int(load().vsamp_shard_pieces(dt, n)) for _, n in bounds)


def vsamp_shard_partial(logits_shard, v0: int, NP: int, temperature=None, seed=None, step=None, row_id=None,
                        target=None, recs=None, win=None, workspace=None, stream=None):
    """Rank-local summaries of one vocabulary shard [B, V_r] starting at token v0: (recs [B, NP, 32] uint8,
    win [B, 16] uint8), as vsamp_piece_rec / vsamp_shard_win bytes."""
    B, Vr, ld = _rows(logits_shard, None)
    dev = logits_shard.device
    dt = _dtype_code(logits_shard)
    temperature = _param(temperature, B, torch.float32, dev, "temperature")
    seed = _param(seed, B, torch.int64, dev, "seed")
    step = _param(step, B, torch.int64, dev, "step")
    row_id = _param(row_id, B, torch.int32, dev, "row_id")
    target = _param(target, B, torch.int32, dev, "target")
    lib = load()
    recs = torch.empty((B, int(NP), PIECE_REC_BYTES), dtype=torch.uint8, device=dev) if recs is None else recs
    win = torch.empty((B, SHARD_WIN_BYTES), dtype=torch.uint8, device=dev) if win is None else win
    need = int(lib.vsamp_shard_workspace_size(dt, B, Vr))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    st = lib.vsamp_shard_partial(
        logits_shard.data_ptr(), dt, B, Vr, ld, int(v0), int(NP), _ptr(temperature, torch.float32, dev, B, "temperature"),
        _ptr(seed, torch.int64, dev, B, "seed"), _ptr(step, torch.int64, dev, B, "step"),
        _ptr(row_id, torch.int32, dev, B, "row_id"), _ptr(target, torch.int32, dev, B, "target"),
        _ptr(recs, torch.uint8, dev, B * int(NP) * PIECE_REC_BYTES, "recs"),
        _ptr(win, torch.uint8, dev, B * SHARD_WIN_BYTES, "win"), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "vsamp_shard_partial")
    return recs, win


def vsamp_shard_merge(recs, wins, V: int, temperature=None, seed=None, step=None, row_id=None,
                      want_target=False, stream=None):
    """The owned merge of rank-ordered records recs [R, B, NP, 32] and wins [R, B, 16] (uint8). Returns
    (row_max, row_logsum, token, logprob, target_logprob or None, row_status)."""
    if recs.dim() != 4 or wins.dim() != 3 or recs.shape[:2] != wins.shape[:2]:
        raise ValueError("recs must be [R, B, NP, 32] and wins [R, B, 16]")
    R, B, NP = int(recs.shape[0]), int(recs.shape[1]), int(recs.shape[2])
    dev = recs.device
    temperature = _param(temperature, B, torch.float32, dev, "temperature")
    seed = _param(seed, B, torch.int64, dev, "seed")
    step = _param(step, B, torch.int64, dev, "step")
    row_id = _param(row_id, B, torch.int32, dev, "row_id")
    f32 = lambda: torch.empty(B, dtype=torch.float32, device=dev)
    row_max, row_logsum, logprob = f32(), f32(), f32()
    target_lp = f32() if want_target else None
    token = torch.empty(B, dtype=torch.int32, device=dev)
    row_status = torch.empty(B, dtype=torch.int32, device=dev)
    st = load().vsamp_shard_merge(
        _ptr(recs.contiguous(), torch.uint8, dev, None, "recs"), _ptr(wins.contiguous(), torch.uint8, dev, None, "wins"),
        R, B, NP, int(V), _ptr(temperature, torch.float32, dev, B, "temperature"), _ptr(seed, torch.int64, dev, B, "seed"),
        _ptr(step, torch.int64, dev, B, "step"), _ptr(row_id, torch.int32, dev, B, "row_id"),
        row_max.data_ptr(), row_logsum.data_ptr(), token.data_ptr(), logprob.data_ptr(),
        0 if target_lp is None else target_lp.data_ptr(), row_status.data_ptr(), _stream(stream))
    _check(st, "vsamp_shard_merge")
    return row_max, row_logsum, token, logprob, target_lp, row_status


def gather_shard_records(recs, win, group=None):
    """The rank-ordered exchange: all-gather this rank's recs [B, NP, 32] and win [B, 16] into [R, B, NP, 32] and
    [R, B, 16] in rank order, with no reduction in transit (torch.distributed; any backend)."""
    import torch.distributed as dist

    R = dist.get_world_size(group)
    # concatenated along the first dimension (the form every backend accepts), then viewed rank-major
    out_r = torch.empty((R * recs.shape[0],) + tuple(recs.shape[1:]), dtype=recs.dtype, device=recs.device)
    out_w = torch.empty((R * win.shape[0],) + tuple(win.shape[1:]), dtype=win.dtype, device=win.device)
    dist.all_gather_into_tensor(out_r, recs.contiguous(), group=group)
    dist.all_gather_into_tensor(out_w, win.contiguous(), group=group)
    return out_r.view((R,) + tuple(recs.shape)), out_w.view((R,) + tuple(win.shape))


def vsamp_sample_sharded(logits, R: int, temperature=None, seed=None, step=None, row_id=None, target=None,
                         align_to_pieces: bool = True, stream=None):
    """R vocabulary shards of one device's [B, V] logits, each summarised by vsamp_shard_partial into its slice of
    the rank-ordered record arrays, then vsamp_shard_merge. Returns (row_max, row_logsum, token, logprob,
    target_logprob or None, row_status)."""
    B, V, _ = _rows(logits, None)
    bounds = shard_bounds(V, R, logits.dtype, align_to_pieces)
    NP = shard_record_slots(bounds, logits.dtype)
    dev = logits.device
    recs = torch.empty((R, B, NP, PIECE_REC_BYTES), dtype=torch.uint8, device=dev)
    wins = torch.empty((R, B, SHARD_WIN_BYTES), dtype=torch.uint8, device=dev)
    for r, (v0, n) in enumerate(bounds):
        vsamp_shard_partial(logits[:, v0:v0 + n], v0, NP, temperature=temperature, seed=seed, step=step,
                            row_id=row_id, target=target, recs=recs[r], win=wins[r], stream=stream)
    return vsamp_shard_merge(recs, wins, V, temperature=temperature, seed=seed, step=step, row_id=row_id,
                             want_target=target is not None, stream=stream)


# ------------------------------------------------------------------------------------------------
# the vocabulary's tables: token scores and their gradient, the 4-bit head, the embedding and its gradient
# ------------------------------------------------------------------------------------------------
def _elsewhere(t: torch.Tensor, stream):
    """The context a call on tensor t and `stream` has to run in, or None when the current device and stream are it.

    Everything a call allocates or converts then belongs to the stream its kernels run on."""
    index = t.get_device()
    if index < 0:
        raise ValueError(f"tensors must be on a CUDA device, got {t.device}")
    if stream is None and index == torch._C._cuda_getDevice():
        return None
    dev = t.device
    if stream is None:
        return torch.cuda.device(dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=dev) if int(stream) else torch.cuda.default_stream(dev)
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    return torch.cuda.stream(stream)


def _current(index: int) -> int:
    return torch._C._cuda_getCurrentRawStream(index)


def _at(t, dtype, index: int, n: int, name: str):
    """The address of a contiguous tensor of at least n elements of dtype on the device, None for None. The small calls
    of a decode step are bound by their argument checks, so the usual case is one line."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == index and t.is_contiguous() and t.numel() >= n:
        return t.data_ptr()
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} needs at least {n} elements")


_LOCAL = threading.local()
_SCRATCH_KEPT = 4 << 20   # bytes of the largest workspace that is kept
_SCRATCH_STREAMS = 8      # workspaces kept per host thread


def _scratch(nbytes: int, dev, index: int, stream: int) -> torch.Tensor:
    """A call's workspace. Small ones are kept per host thread, device and stream, because allocating one costs a decode
    step's call a third of its host time; nothing is kept in them, and a thread keeps those of its latest streams only. A
    stream's calls never overlap, but those of two threads may interleave on one stream. A call that is captured into a
    graph gets its own, from the graph's memory."""
    if nbytes > _SCRATCH_KEPT or torch.cuda.is_current_stream_capturing():
        return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    kept = _LOCAL.__dict__
    ws = kept.get((index, stream))
    if ws is None or ws.numel() < nbytes:
        if ws is None and len(kept) >= _SCRATCH_STREAMS:
            del kept[next(iter(kept))]   # the oldest: its stream's later calls allocate anew
        ws = kept[(index, stream)] = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    return ws


def _token_ids(v, n: int, dev):
    """Token ids as a contiguous int32 device tensor; wider ids outside its range stay outside every vocabulary."""
    if isinstance(v, torch.Tensor):
        if v.dtype is torch.int32:
            return v if v.is_contiguous() and v.device == dev else v.to(device=dev).contiguous()
        if v.is_floating_point() or v.is_complex():
            raise TypeError(f"token must hold whole numbers, got {v.dtype}")
        if v.dtype.itemsize > 2:
            v = v.to(torch.int64).clamp(-(1 << 31), (1 << 31) - 1)
        return v.to(device=dev, dtype=torch.int32).contiguous()
    return torch.full((n,), min(max(int(v), -(1 << 31)), (1 << 31) - 1), dtype=torch.int32, device=dev)


def _row_values(v, n: int, dev, name):
    """A per-row fp32 parameter: None, a scalar (broadcast) or a [n] tensor."""
    if v is None or (isinstance(v, torch.Tensor) and v.dtype is torch.float32 and v.is_contiguous() and v.device == dev):
        return v
    return _param(v, n, torch.float32, dev, name)


def _matrix(t: torch.Tensor, name: str, index: int, rows=None, cols=None):
    """Checks a row-major matrix (rows may be padded); returns its rows, columns and row stride in elements."""
    try:
        (r, c), (s0, s1) = t.shape, t.stride()
    except ValueError:
        r = None
    if r is None or t.get_device() != index or (s1 != 1 and c > 1):
        raise ValueError(f"{name} must be a 2-D tensor on cuda:{index} with contiguous rows")
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError(f"{name} must be [{rows}, {cols}], got [{r}, {c}]")
    return r, c, s0 if r > 1 or s0 > c else c


def _logits_matrix(x: torch.Tensor, V, index: int):
    B, cols, ld = _matrix(x, "logits", index)
    if V is None:
        return B, cols, ld
    if not 0 < V <= cols:
        raise ValueError(f"V = {V} is outside the rows of {cols} logits")
    return B, int(V), ld


def _alternatives(t, n_alt: int, name: str):
    """A caller's array of alternatives: rows of n_alt, which is how the library fills it."""
    if t.dim() > 1 and t.shape[-1] != n_alt:
        raise ValueError(f"{name} must have rows of {n_alt}, got {tuple(t.shape)}")
    return t


def vsamp_score_tokens(logits, token, temperature=None, n_alt=0, V=None, logprob=None, entropy=None, rank=None,
                       alt_idx=None, alt_lp=None, row_max=None, row_logsum=None, row_status=None, workspace=None,
                       stream=None):
    """Log-probability, entropy and rank of given tokens, with the n_alt most probable alternatives, in one pass over
    the logits. -inf logits are masked tokens; VSAMP_TOKEN_IGNORE as a token skips the row. Returns (logprob [B],
    entropy [B], rank [B] int32, alt_idx [B, n_alt] int32 or None, alt_lp [B, n_alt] or None, row_max [B],
    row_logsum [B], row_status [B])."""
    where = _elsewhere(logits, stream)
    if where is not None:
        with where:
            return vsamp_score_tokens(logits, token, temperature, n_alt, V, logprob, entropy, rank, alt_idx, alt_lp,
                                      row_max, row_logsum, row_status, workspace)
    dev, at = logits.device, logits.get_device()
    B, V, ld = _logits_matrix(logits, V, at)
    dt, n_alt = _dtype_code(logits), int(n_alt)
    if not 0 <= n_alt <= VSAMP_SCORE_ALT_MAX:
        raise ValueError(f"n_alt must be in [0, {VSAMP_SCORE_ALT_MAX}]")
    f32, i32, u8, empty = torch.float32, torch.int32, torch.uint8, torch.empty
    token = _token_ids(token, B, dev)
    temperature = _row_values(temperature, B, dev, "temperature")
    logprob = empty(B, dtype=f32, device=dev) if logprob is None else logprob
    entropy = empty(B, dtype=f32, device=dev) if entropy is None else entropy
    row_max = empty(B, dtype=f32, device=dev) if row_max is None else row_max
    row_logsum = empty(B, dtype=f32, device=dev) if row_logsum is None else row_logsum
    rank = empty(B, dtype=i32, device=dev) if rank is None else rank
    row_status = empty(B, dtype=i32, device=dev) if row_status is None else row_status
    if n_alt:
        alt_idx = empty((B, n_alt), dtype=i32, device=dev) if alt_idx is None else _alternatives(alt_idx, n_alt, "alt_idx")
        alt_lp = empty((B, n_alt), dtype=f32, device=dev) if alt_lp is None else _alternatives(alt_lp, n_alt, "alt_lp")
    else:
        alt_idx = alt_lp = None
    lib, on = load(), _current(at)
    if workspace is None:
        workspace = _scratch(lib.vsamp_score_workspace_size(dt, B, V, n_alt), dev, at, on)
    st = lib.vsamp_score_tokens(
        logits.data_ptr(), dt, B, V, ld, _at(temperature, f32, at, B, "temperature"), _at(token, i32, at, B, "token"),
        n_alt, _at(logprob, f32, at, B, "logprob"), _at(entropy, f32, at, B, "entropy"), _at(rank, i32, at, B, "rank"),
        _at(alt_idx, i32, at, B * n_alt, "alt_idx"), _at(alt_lp, f32, at, B * n_alt, "alt_lp"),
        _at(row_max, f32, at, B, "row_max"), _at(row_logsum, f32, at, B, "row_logsum"),
        _at(row_status, i32, at, B, "row_status"), _at(workspace, u8, at, 0, "workspace"), workspace.numel(), on)
    if st:
        _check(st, "vsamp_score_tokens")
    return logprob, entropy, rank, alt_idx, alt_lp, row_max, row_logsum, row_status


def vsamp_score_tokens_backward(logits, token, dlogprob, row_max, row_logsum, entropy=None, dentropy=None,
                                temperature=None, V=None, dlogits=None, row_status=None, stream=None):
    """Gradient of vsamp_score_tokens with respect to the logits from the gradients of the log-probabilities and of
    the entropies (either may be None) and the statistics of the forward call. dlogits may be the logits' own
    buffer. Returns (dlogits [B, V] of the logits' type, row_status [B])."""
    where = _elsewhere(logits, stream)
    if where is not None:
        with where:
            return vsamp_score_tokens_backward(logits, token, dlogprob, row_max, row_logsum, entropy, dentropy,
                                               temperature, V, dlogits, row_status)
    dev, at = logits.device, logits.get_device()
    B, V, ld = _logits_matrix(logits, V, at)
    f32, i32 = torch.float32, torch.int32
    token = _token_ids(token, B, dev)
    temperature = _row_values(temperature, B, dev, "temperature")
    dlogprob, dentropy = _row_values(dlogprob, B, dev, "dlogprob"), _row_values(dentropy, B, dev, "dentropy")
    if dlogits is None:
        dlogits = torch.empty((B, V), dtype=logits.dtype, device=dev)
    _, cols, ldd = _matrix(dlogits, "dlogits", at, B)
    if dlogits.dtype is not logits.dtype or cols < V:
        raise ValueError(f"dlogits must be [{B}, >= {V}] of {logits.dtype}")
    row_status = torch.empty(B, dtype=i32, device=dev) if row_status is None else row_status
    st = load().vsamp_score_tokens_backward(
        logits.data_ptr(), _dtype_code(logits), B, V, ld, _at(temperature, f32, at, B, "temperature"),
        _at(token, i32, at, B, "token"), _at(dlogprob, f32, at, B, "dlogprob"), _at(dentropy, f32, at, B, "dentropy"),
        _at(row_max, f32, at, B, "row_max"), _at(row_logsum, f32, at, B, "row_logsum"),
        _at(entropy, f32, at, B, "entropy"), dlogits.data_ptr(), ldd, _at(row_status, i32, at, B, "row_status"),
        _current(at))
    if st:
        _check(st, "vsamp_score_tokens_backward")
    return dlogits, row_status


class HeadWeights:
    """4-bit head weights as vsamp_head_pack laid them out: the buffer and the shape it was packed for."""

    __slots__ = ("data", "V", "D", "group", "scale_dt", "has_zeros")

    def __init__(self, data: torch.Tensor, V: int, D: int, group: int, scale_dt: int, has_zeros: bool):
        self.data, self.V, self.D, self.group = data, V, D, group
        self.scale_dt, self.has_zeros = scale_dt, has_zeros


def vsamp_head_pack(codes, scales, zeros=None, group=64, stream=None) -> HeadWeights:
    """Lays out 4-bit weights for vsamp_head_logits: codes [V, D / 2] uint8 (even elements in the low nibble), scales
    [V, D / group] fp32 or bf16, zeros [V, D / group] uint8 in 0..15 or None (8 everywhere); group 32, 64 or 128."""
    where = _elsewhere(codes, stream)
    if where is not None:
        with where:
            return vsamp_head_pack(codes, scales, zeros, group)
    dev, at, group = codes.device, codes.get_device(), int(group)
    if codes.dim() != 2 or codes.dtype != torch.uint8:
        raise ValueError("codes must be a 2-D uint8 tensor [V, D / 2]")
    V, D = int(codes.shape[0]), 2 * int(codes.shape[1])
    if group not in (32, 64, 128) or V == 0 or D == 0 or D % group:
        raise ValueError(f"group must be 32, 64 or 128 and divide D (group {group}, V {V}, D {D})")
    for t, name in ((scales, "scales"), (zeros, "zeros")):
        if t is not None and tuple(t.shape) != (V, D // group):
            raise ValueError(f"{name} must be [{V}, {D // group}], got {tuple(t.shape)}")
    lib = load()
    dt, n = _dtype_code(scales), V * D // group
    need = lib.vsamp_head_packed_size(dt, zeros is not None, V, D, group)
    data = torch.empty(need, dtype=torch.uint8, device=dev)
    st = lib.vsamp_head_pack(_at(codes, torch.uint8, at, V * D // 2, "codes"), _at(scales, scales.dtype, at, n, "scales"),
                             dt, _at(zeros, torch.uint8, at, n, "zeros"), V, D, group, data.data_ptr(), need, _current(at))
    _check(st, "vsamp_head_pack")
    return HeadWeights(data, V, D, group, dt, zeros is not None)


def vsamp_head_logits(hidden, head: HeadWeights, out=None, out_dtype=torch.float32, stream=None):
    """Logits [M, V] of hidden states [M, D] (fp32 or bf16) under 4-bit head weights, for the few rows of a decode
    step. `out` (fp32 or bf16, rows may be padded) or a new tensor of out_dtype is returned."""
    where = _elsewhere(hidden, stream)
    if where is not None:
        with where:
            return vsamp_head_logits(hidden, head, out, out_dtype)
    at, V, D = hidden.get_device(), head.V, head.D
    M, _, ldh = _matrix(hidden, "hidden", at, None, D)
    if out is None:
        out = torch.empty((M, V), dtype=out_dtype, device=hidden.device)
    ld = _matrix(out, "out", at, M, V)[2]
    data = head.data
    st = load().vsamp_head_logits(hidden.data_ptr(), _dtype_code(hidden), M, ldh, _at(data, torch.uint8, at, 0, "head"),
                                  data.numel(), head.scale_dt, head.has_zeros, V, D, head.group, out.data_ptr(),
                                  _dtype_code(out), ld, _current(at))
    if st:
        _check(st, "vsamp_head_logits")
    return out


def vsamp_embed(token, table, scale=1.0, out=None, out_dtype=None, row_status=None, stream=None):
    """scale * table[token] (token [N], table [V, D] fp32 or bf16). VSAMP_TOKEN_IGNORE gives zeros, another token
    outside the table NaN and a row status. Returns (out [N, D] of out_dtype or the table's type, row_status [N])."""
    where = _elsewhere(table, stream)
    if where is not None:
        with where:
            return vsamp_embed(token, table, scale, out, out_dtype, row_status)
    dev, at = table.device, table.get_device()
    V, D, ldt = _matrix(table, "table", at)
    N = token.numel() if isinstance(token, torch.Tensor) else 1
    token = _token_ids(token, N, dev)
    if out is None:
        out = torch.empty((N, D), dtype=out_dtype or table.dtype, device=dev)
    ldo = _matrix(out, "out", at, N, D)[2]
    row_status = torch.empty(N, dtype=torch.int32, device=dev) if row_status is None else row_status
    st = load().vsamp_embed(_at(token, torch.int32, at, N, "token"), N, table.data_ptr(), _dtype_code(table), V, D, ldt,
                            scale, out.data_ptr(), _dtype_code(out), ldo,
                            _at(row_status, torch.int32, at, N, "row_status"), _current(at))
    if st:
        _check(st, "vsamp_embed")
    return out, row_status


def vsamp_embed_backward(token, dout, V, scale=1.0, dtable=None, dtype=None, accumulate=False, workspace=None,
                         stream=None):
    """Gradient of vsamp_embed with respect to the table: scale * the sum of dout's rows (dout [N, D]) of every token.
    accumulate adds it to dtable's rows of those tokens, otherwise every row of dtable is written. Returns dtable
    [V, D] (a new one of `dtype` or dout's type if not given)."""
    where = _elsewhere(dout, stream)
    if where is not None:
        with where:
            return vsamp_embed_backward(token, dout, V, scale, dtable, dtype, accumulate, workspace)
    dev, at, V = dout.device, dout.get_device(), int(V)
    N, D, ldd = _matrix(dout, "dout", at)
    token = _token_ids(token, N, dev)
    if dtable is None:
        if accumulate:
            raise ValueError("accumulate needs the table gradient to add to")
        dtable = torch.empty((V, D), dtype=dtype or dout.dtype, device=dev)
    ldt = _matrix(dtable, "dtable", at, V, D)[2]
    lib, on = load(), _current(at)
    if workspace is None:
        workspace = _scratch(lib.vsamp_embed_workspace_size(N, D), dev, at, on)
    st = lib.vsamp_embed_backward(_at(token, torch.int32, at, N, "token"), N, dout.data_ptr(), _dtype_code(dout), D, ldd,
                                  scale, V, dtable.data_ptr(), _dtype_code(dtable), ldt, accumulate,
                                  _at(workspace, torch.uint8, at, 0, "workspace"), workspace.numel(), on)
    if st:
        _check(st, "vsamp_embed_backward")
    return dtable

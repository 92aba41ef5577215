"""Thin Python binding of libspecverify.so (ctypes). Argument marshalling only: every
step of the verification path runs in the library's CUDA kernels; there is no CPU or
PyTorch fallback, and every call raises if the library is missing or returns an error.

PyTorch supplies device memory and the current stream. Entry points mirror the C ABI in
include/specverify.h:

* ``spec_verify_attn`` -- GQA verify attention over cached prefix + draft window.
* ``spec_verify_attn_paged`` -- the same over a paged cache (block pool + block table).
* ``spec_verify_attn_host_lengths`` -- the same with host copies of the lengths (plan on
  the host, no planning kernel).
* ``spec_verify_attn_shared`` -- the paged call for groups of sequences with a common prefix,
  attended once per group.
* ``spec_pages_fork``, ``spec_pages_extend``, ``spec_pages_trim``, ``spec_pages_compact`` --
  the block tables and pages of a paged cache (shared pages, copy on write).
* ``spec_kv4_write``, ``spec_kv4_read``, ``spec_verify_attn_kv4`` -- a paged cache held in 4
  bits: rows rounded into its pages, read back, and verify attention over them.
* ``spec_attn_mass``, ``spec_kv_evict`` -- the attention weight that each cached position got,
  added up, and eviction of the positions with the least.
* ``spec_accept`` -- greedy acceptance (argmax per window row, first mismatch).
* ``spec_accept_stochastic`` -- distribution-preserving acceptance for sampled decoding.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import struct
import threading
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspecverify.so")

SV_BF16, SV_FP8_E4M3, SV_FP32, SV_KV4 = 0, 1, 2, 3
STATUS = {0: "SV_OK", 1: "SV_ERR_NULL", 2: "SV_ERR_SHAPE", 3: "SV_ERR_DTYPE",
          4: "SV_ERR_ALIGN", 5: "SV_ERR_WORKSPACE", 6: "SV_ERR_CUDA", 7: "SV_ERR_TIMEOUT",
          8: "SV_ERR_DEVICE_SHAPE", 9: "SV_ERR_NO_PAGES"}
EXPORTS = ("spec_verify_attn_workspace_size", "spec_verify_attn", "spec_verify_attn_paged",
           "spec_verify_attn_host_lengths",
           "spec_accept_workspace_size",
           "spec_accept", "spec_draft_signals_workspace_size", "spec_draft_signals",
           "sv_workspace_status", "sv_status_string", "sv_set_attn_kernel", "sv_set_unit_ctas",
           "sv_set_profile_events", "sv_version", "sv_plan_preview",
           "sv_inject_launch_failure", "sv_inject_wait_timeout", "sv_set_row_pairs",
           "sv_row_pair_mode", "sv_set_kv_rings",
           "spec_accept_stochastic_workspace_size",
           "spec_accept_stochastic",
           "spec_verify_attn_shared_workspace_size", "spec_verify_attn_shared",
           "spec_pages_workspace_size", "spec_pages_fork", "spec_pages_extend",
           "spec_pages_trim", "spec_pages_compact",
           "spec_kv4_workspace_size", "spec_kv4_write", "spec_kv4_read",
           "spec_verify_attn_kv4_workspace_size", "spec_verify_attn_kv4",
           "spec_attn_mass_workspace_size", "spec_attn_mass",
           "spec_kv_evict_workspace_size", "spec_kv_evict")


class SpecVerifyError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s failed: %s (%d)" % (where, STATUS.get(status, "?"), status))


class PlanInfo(ctypes.Structure):
    _fields_ = [("num_units", ctypes.c_int32), ("total_tiles", ctypes.c_int32),
                ("tile_keys", ctypes.c_int32), ("num_ctas", ctypes.c_int32),
                ("unit_ctas", ctypes.c_int32), ("switch_tiles", ctypes.c_int32)]


class AttnDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("max_draft_len", ctypes.c_int32), ("max_seq_len", ctypes.c_int32),
                ("q_rows", ctypes.c_int64), ("kv_rows", ctypes.c_int64),
                ("kv_dtype", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
                ("sliding_window", ctypes.c_int32)]


class PageTable(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("table_rows", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32),
                ("ref_count", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("cached_len", ctypes.c_void_p)]


class PageData(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("page_bytes", ctypes.c_int64)]


class Kv4Pages(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int64), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("kv_scale", ctypes.c_void_p)]


MAX_PAGE_POOLS = 256

_lock = threading.Lock()
_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libspecverify.so (built by ``build.build()``); raises if it is missing."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError("libspecverify.so is not built (%s); run "
                               "speculative_decoding_verification_gqa_gb300.build.build()" % path)
        lib = ctypes.CDLL(path)
        vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
        lib.spec_verify_attn_workspace_size.argtypes = [ctypes.POINTER(AttnDesc)]
        lib.spec_verify_attn_workspace_size.restype = sz
        lib.spec_verify_attn.argtypes = [ctypes.POINTER(AttnDesc), vp, vp, vp, vp, vp, vp, vp,
                                         vp, sz, vp]
        lib.spec_verify_attn.restype = ctypes.c_int
        i64 = ctypes.c_int64
        lib.spec_verify_attn_paged.argtypes = [ctypes.POINTER(AttnDesc), vp, vp, vp, i64, i32,
                                               vp, i32, vp, vp, vp, vp, vp, sz, vp]
        lib.spec_verify_attn_paged.restype = ctypes.c_int
        lib.spec_verify_attn_shared_workspace_size.argtypes = [ctypes.POINTER(AttnDesc), i32]
        lib.spec_verify_attn_shared_workspace_size.restype = sz
        lib.spec_verify_attn_shared.argtypes = [ctypes.POINTER(AttnDesc), vp, vp, vp, i64, i32,
                                                vp, i32, vp, vp, i32, vp, vp, vp, vp, vp, sz, vp]
        lib.spec_verify_attn_shared.restype = ctypes.c_int
        lib.spec_verify_attn_host_lengths.argtypes = [ctypes.POINTER(AttnDesc), vp, vp, vp, vp,
                                                      vp, vp, vp, vp, vp, vp, sz, vp]
        lib.spec_verify_attn_host_lengths.restype = ctypes.c_int
        lib.spec_accept_workspace_size.argtypes = [i32, i32, i32]
        lib.spec_accept_workspace_size.restype = sz
        lib.spec_accept.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        lib.spec_accept.restype = ctypes.c_int
        lib.spec_draft_signals_workspace_size.argtypes = [i32, i32]
        lib.spec_draft_signals_workspace_size.restype = sz
        lib.spec_draft_signals.argtypes = [i32, i32, i32, vp, vp, vp, vp, sz, vp]
        lib.spec_draft_signals.restype = ctypes.c_int
        lib.sv_workspace_status.argtypes = [vp, ctypes.c_int, vp]
        lib.sv_workspace_status.restype = ctypes.c_int
        lib.sv_status_string.argtypes = [ctypes.c_int]
        lib.sv_status_string.restype = ctypes.c_char_p
        lib.sv_set_attn_kernel.argtypes = [ctypes.c_int]
        lib.sv_set_attn_kernel.restype = ctypes.c_int
        lib.sv_set_unit_ctas.argtypes = [ctypes.c_int]
        lib.sv_set_unit_ctas.restype = ctypes.c_int
        lib.sv_set_profile_events.argtypes = [vp, vp]
        lib.sv_set_profile_events.restype = None
        lib.sv_version.restype = ctypes.c_int
        lib.sv_plan_preview.argtypes = [ctypes.POINTER(AttnDesc), i32, vp, vp, i32, i32,
                                        ctypes.POINTER(PlanInfo), vp, vp, vp, i32]
        lib.sv_plan_preview.restype = ctypes.c_int
        lib.spec_accept_stochastic_workspace_size.argtypes = [i32, i32, i32]
        lib.spec_accept_stochastic_workspace_size.restype = sz
        lib.spec_accept_stochastic.argtypes = [i32, i32, i32, i32, vp, vp, vp, vp, vp, vp,
                                               ctypes.c_float, vp, vp, vp, sz, vp]
        lib.spec_accept_stochastic.restype = ctypes.c_int
        lib.spec_pages_workspace_size.argtypes = [i32, i32]
        lib.spec_pages_workspace_size.restype = sz
        lib.spec_pages_fork.argtypes = [vp, i32, vp, vp, vp, vp, sz, vp]
        lib.spec_pages_fork.restype = ctypes.c_int
        lib.spec_pages_extend.argtypes = [vp, i32, vp, vp, i32, vp, vp, sz, vp]
        lib.spec_pages_extend.restype = ctypes.c_int
        lib.spec_pages_trim.argtypes = [vp, i32, vp, vp, vp, sz, vp]
        lib.spec_pages_trim.restype = ctypes.c_int
        lib.spec_pages_compact.argtypes = [vp, i32, vp, vp, vp, vp, sz, vp]
        lib.spec_pages_compact.restype = ctypes.c_int
        ad = ctypes.POINTER(AttnDesc)
        lib.spec_kv4_workspace_size.argtypes = [i32]
        lib.spec_kv4_workspace_size.restype = sz
        lib.spec_kv4_write.argtypes = [vp, i32, vp, i32, vp, vp, i64, vp, i64, vp, i64, vp, sz, vp]
        lib.spec_kv4_write.restype = ctypes.c_int
        lib.spec_kv4_read.argtypes = [vp, i32, vp, i32, vp, vp, i64, vp, vp, vp, sz, vp]
        lib.spec_kv4_read.restype = ctypes.c_int
        lib.spec_verify_attn_kv4_workspace_size.argtypes = [ad]
        lib.spec_verify_attn_kv4_workspace_size.restype = sz
        lib.spec_verify_attn_kv4.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, sz, vp]
        lib.spec_verify_attn_kv4.restype = ctypes.c_int
        lib.spec_attn_mass_workspace_size.argtypes = [ad]
        lib.spec_attn_mass_workspace_size.restype = sz
        lib.spec_attn_mass.argtypes = [vp, vp, vp, vp, vp, i64, i32, vp, i32, vp, vp, vp, vp, vp,
                                       i64, vp, sz, vp]
        lib.spec_attn_mass.restype = ctypes.c_int
        lib.spec_kv_evict_workspace_size.argtypes = [i32, i32, i64]
        lib.spec_kv_evict_workspace_size.restype = sz
        lib.spec_kv_evict.argtypes = [vp, i32, vp, vp, vp, i32, i32, vp, i64, vp, i64, i32, vp, vp,
                                      sz, vp]
        lib.spec_kv_evict.restype = ctypes.c_int
        lib.sv_inject_launch_failure.argtypes = [ctypes.c_int]
        lib.sv_inject_launch_failure.restype = ctypes.c_int
        lib.sv_inject_wait_timeout.argtypes = [ctypes.c_int64]
        lib.sv_inject_wait_timeout.restype = ctypes.c_int
        lib.sv_set_row_pairs.argtypes = [ctypes.c_int]
        lib.sv_set_row_pairs.restype = ctypes.c_int
        lib.sv_set_kv_rings.argtypes = [ctypes.c_int]
        lib.sv_set_kv_rings.restype = ctypes.c_int
        lib.sv_row_pair_mode.argtypes = [ctypes.POINTER(AttnDesc), i32, i32, i32]
        lib.sv_row_pair_mode.restype = ctypes.c_int
        _lib = lib
        return lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _or_placeholder(t: torch.Tensor) -> torch.Tensor:
    """t, or a small allocation of its dtype on its device when t is empty (a batch without
    drafts: the library requires the pointer when max_draft_len > 0 but never reads it)."""
    return t if t.numel() > 0 else torch.empty(16, dtype=t.dtype, device=t.device)


def _check(st: int, where: str):
    if st != 0:
        raise SpecVerifyError(st, where)


def _need(t: torch.Tensor, name: str, dtypes):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype not in dtypes:
        raise TypeError("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def attn_desc(q: torch.Tensor, k_cache: torch.Tensor, batch: int, max_draft_len: int,
              max_seq_len: int, softmax_scale: float = 0.0, sliding_window: int = 0) -> AttnDesc:
    fp8 = k_cache.dtype in (torch.uint8, torch.float8_e4m3fn)
    return AttnDesc(batch=batch, num_q_heads=q.shape[1], num_kv_heads=k_cache.shape[1],
                    head_dim=q.shape[2], max_draft_len=max_draft_len, max_seq_len=max_seq_len,
                    q_rows=q.shape[0], kv_rows=k_cache.shape[0],
                    kv_dtype=SV_FP8_E4M3 if fp8 else SV_BF16,
                    softmax_scale=float(softmax_scale), sliding_window=int(sliding_window))


def verify_workspace_bytes(desc: AttnDesc) -> int:
    n = load_library().spec_verify_attn_workspace_size(ctypes.byref(desc))
    if n == 0:
        raise SpecVerifyError(2, "spec_verify_attn_workspace_size")
    return n


def accept_workspace_bytes(batch: int, max_draft_len: int, vocab: int) -> int:
    n = load_library().spec_accept_workspace_size(batch, max_draft_len, vocab)
    if n == 0:
        raise SpecVerifyError(2, "spec_accept_workspace_size")
    return n


def signals_workspace_bytes(rows: int, vocab: int) -> int:
    n = load_library().spec_draft_signals_workspace_size(rows, vocab)
    if n == 0:
        raise SpecVerifyError(2, "spec_draft_signals_workspace_size")
    return n


def new_workspace(nbytes: int, device=None) -> torch.Tensor:
    """A zero-filled device workspace (the library's flag word must start at zero)."""
    return torch.zeros(nbytes, dtype=torch.uint8, device=device or "cuda")


def spec_verify_attn(q, k_cache, v_cache, seq_lens, draft_len, *, max_draft_len: int,
                     max_seq_len: int, kv_scale=None, out=None, workspace=None,
                     softmax_scale: float = 0.0, sliding_window: int = 0,
                     stream=None) -> torch.Tensor:
    """q [rows, Hq, d] bf16; k_cache/v_cache [kv_rows, Hkv, d] bf16, or uint8 /
    float8_e4m3fn E4M3 codes with kv_scale fp32 [2, Hkv]; seq_lens, draft_len int32 [B].
    Returns out [rows, Hq, d] bf16 (only the packed rows sum_b (1 + D_b) are written).
    ``sliding_window`` = W >= 1 restricts window row i to keys max(0, T+i-W+1) .. T+i."""
    _need(q, "q", (torch.bfloat16,))
    _need(k_cache, "k_cache", (torch.bfloat16, torch.uint8, torch.float8_e4m3fn))
    _need(v_cache, "v_cache", (k_cache.dtype,))
    _need(seq_lens, "seq_lens", (torch.int32,))
    _need(draft_len, "draft_len", (torch.int32,))
    if kv_scale is not None:
        _need(kv_scale, "kv_scale", (torch.float32,))
    if q.dim() != 3 or k_cache.dim() != 3 or v_cache.shape != k_cache.shape:
        raise ValueError("q must be [rows, Hq, d], k/v caches [kv_rows, Hkv, d]")
    desc = attn_desc(q, k_cache, seq_lens.shape[0], max_draft_len, max_seq_len, softmax_scale,
                     sliding_window)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", (torch.bfloat16,))
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if workspace is None:
        workspace = new_workspace(verify_workspace_bytes(desc), q.device)
    st = load_library().spec_verify_attn(
        ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens),
        _ptr(draft_len), _ptr(kv_scale), _ptr(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "spec_verify_attn")
    return out


def spec_verify_attn_host_lengths(q, k_cache, v_cache, seq_lens, draft_len, seq_lens_host,
                                  draft_len_host, *, max_draft_len: int, max_seq_len: int,
                                  kv_scale=None, out=None, workspace=None,
                                  softmax_scale: float = 0.0, sliding_window: int = 0,
                                  stream=None) -> torch.Tensor:
    """spec_verify_attn with the lengths also in host memory (int32 CPU tensors equal to
    seq_lens and draft_len): the work plan is made on the host and travels with the
    attention launch."""
    for t, n in ((seq_lens_host, "seq_lens_host"), (draft_len_host, "draft_len_host")):
        if t.device.type != "cpu" or t.dtype != torch.int32 or not t.is_contiguous():
            raise ValueError("%s must be a contiguous int32 CPU tensor" % n)
    _need(q, "q", (torch.bfloat16,))
    _need(k_cache, "k_cache", (torch.bfloat16, torch.uint8, torch.float8_e4m3fn))
    _need(v_cache, "v_cache", (k_cache.dtype,))
    _need(seq_lens, "seq_lens", (torch.int32,))
    _need(draft_len, "draft_len", (torch.int32,))
    if kv_scale is not None:
        _need(kv_scale, "kv_scale", (torch.float32,))
    if q.dim() != 3 or k_cache.dim() != 3 or v_cache.shape != k_cache.shape:
        raise ValueError("q must be [rows, Hq, d], k/v caches [kv_rows, Hkv, d]")
    if seq_lens_host.numel() != seq_lens.numel() or draft_len_host.numel() != draft_len.numel():
        raise ValueError("host and device length arrays differ in size")
    desc = attn_desc(q, k_cache, seq_lens.shape[0], max_draft_len, max_seq_len, softmax_scale,
                     sliding_window)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", (torch.bfloat16,))
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if workspace is None:
        workspace = new_workspace(verify_workspace_bytes(desc), q.device)
    st = load_library().spec_verify_attn_host_lengths(
        ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens),
        _ptr(draft_len), ctypes.c_void_p(seq_lens_host.data_ptr()),
        ctypes.c_void_p(draft_len_host.data_ptr()), _ptr(kv_scale), _ptr(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "spec_verify_attn_host_lengths")
    return out


def spec_verify_attn_paged(q, k_pages, v_pages, block_table, seq_lens, draft_len, *,
                           max_draft_len: int, max_seq_len: int, kv_scale=None, out=None,
                           workspace=None, softmax_scale: float = 0.0, sliding_window: int = 0,
                           stream=None) -> torch.Tensor:
    """spec_verify_attn over a paged cache. k_pages/v_pages [num_blocks, block_size, Hkv, d]
    (bf16, or uint8 / float8_e4m3fn codes with kv_scale); block_table int32 [B, max_blocks]:
    position j of sequence b is row j % block_size of block block_table[b, j // block_size]."""
    _need(q, "q", (torch.bfloat16,))
    _need(k_pages, "k_pages", (torch.bfloat16, torch.uint8, torch.float8_e4m3fn))
    _need(v_pages, "v_pages", (k_pages.dtype,))
    _need(block_table, "block_table", (torch.int32,))
    _need(seq_lens, "seq_lens", (torch.int32,))
    _need(draft_len, "draft_len", (torch.int32,))
    if kv_scale is not None:
        _need(kv_scale, "kv_scale", (torch.float32,))
    if q.dim() != 3 or k_pages.dim() != 4 or v_pages.shape != k_pages.shape:
        raise ValueError("q must be [rows, Hq, d], k/v pages [num_blocks, block_size, Hkv, d]")
    if block_table.dim() != 2 or block_table.shape[0] != seq_lens.shape[0]:
        raise ValueError("block_table must be [B, max_blocks]")
    nb, bs = k_pages.shape[0], k_pages.shape[1]
    flat = k_pages.view(nb * bs, k_pages.shape[2], k_pages.shape[3])
    desc = attn_desc(q, flat, seq_lens.shape[0], max_draft_len, max_seq_len, softmax_scale,
                     sliding_window)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", (torch.bfloat16,))
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if workspace is None:
        workspace = new_workspace(verify_workspace_bytes(desc), q.device)
    st = load_library().spec_verify_attn_paged(
        ctypes.byref(desc), _ptr(q), _ptr(k_pages), _ptr(v_pages), nb, bs, _ptr(block_table),
        block_table.shape[1], _ptr(seq_lens), _ptr(draft_len), _ptr(kv_scale), _ptr(out),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "spec_verify_attn_paged")
    return out


_I32 = (torch.int32,)
_KV = (torch.bfloat16, torch.uint8, torch.float8_e4m3fn)
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _dev(t, name, dtypes) -> int:
    """Checks a tensor as `_need` does; returns its device's index."""
    try:
        if t.dtype in dtypes and t.is_contiguous():
            d = t.get_device()
            if d >= 0:
                return d
    except AttributeError:
        pass
    _need(t, name, dtypes)
    return t.get_device()


def _one_device(devs):
    """The call's tensors lie on one device, and it is the current one: a launch goes to the
    current device's stream."""
    d = devs[0]
    for o in devs:
        if o != d:
            raise ValueError("the call's tensors lie on several devices: %s" % sorted(set(devs)))
    if d != _current_device():
        raise ValueError("the tensors lie on cuda:%d, the current device is cuda:%d"
                         % (d, _current_device()))
    return d


def _stream_on(stream, dev):
    if stream is None:
        return _raw_stream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _allocating_on(stream, dev):
    """Where a call allocates what it was not given: on the stream that it runs on, so that
    the workspace's zeros come before the call there, and memory that is used again is used
    in that stream's order."""
    raw = _stream_on(stream, dev)
    if raw == _raw_stream(dev):
        return contextlib.nullcontext()
    if raw == 0:
        return torch.cuda.stream(torch.cuda.default_stream(dev))
    return torch.cuda.stream(torch.cuda.ExternalStream(raw, device=dev))


def shared_workspace_bytes(desc: AttnDesc, num_groups: int) -> int:
    n = load_library().spec_verify_attn_shared_workspace_size(ctypes.byref(desc), num_groups)
    if n == 0:
        raise SpecVerifyError(2, "spec_verify_attn_shared_workspace_size")
    return n


def spec_verify_attn_shared(q, k_pages, v_pages, block_table, seq_lens, draft_len, group_begin,
                            prefix_len, *, max_draft_len: int, max_seq_len: int, kv_scale=None,
                            out=None, workspace=None, softmax_scale: float = 0.0,
                            stream=None) -> torch.Tensor:
    """spec_verify_attn_paged for a batch in groups that share a prefix: sequences
    group_begin[n] .. group_begin[n + 1] - 1 (int32 [groups + 1]) hold the same K/V at
    positions 0 .. prefix_len[n] - 1 (int32 [groups]), read through the block-table row of
    the group's first sequence and attended once for all of them."""
    devs = [_dev(q, "q", (torch.bfloat16,)), _dev(k_pages, "k_pages", _KV),
            _dev(v_pages, "v_pages", (k_pages.dtype,)), _dev(block_table, "block_table", _I32),
            _dev(seq_lens, "seq_lens", _I32), _dev(draft_len, "draft_len", _I32),
            _dev(group_begin, "group_begin", _I32), _dev(prefix_len, "prefix_len", _I32)]
    if q.dim() != 3 or k_pages.dim() != 4 or v_pages.shape != k_pages.shape:
        raise ValueError("q must be [rows, Hq, d], k/v pages [num_blocks, block_size, Hkv, d]")
    rows, hq, d = q.shape
    nb, bs, hkv, dk = k_pages.shape
    B, table = seq_lens.numel(), block_table.shape
    groups = prefix_len.numel()
    if dk != d:
        raise ValueError("q and the pages must have one head dimension")
    if seq_lens.dim() != 1 or len(table) != 2 or table[0] != B or draft_len.shape != (B,):
        raise ValueError("seq_lens and draft_len must be [B], block_table [B, max_blocks]")
    if prefix_len.dim() != 1 or group_begin.shape != (groups + 1,):
        raise ValueError("group_begin must be [groups + 1], prefix_len [groups]")
    fp8 = k_pages.dtype != torch.bfloat16
    scale = None
    if kv_scale is not None:
        devs.append(_dev(kv_scale, "kv_scale", (torch.float32,)))
        if kv_scale.shape != (2, hkv):
            raise ValueError("kv_scale must be [2, Hkv]")
        scale = kv_scale.data_ptr()
    desc = AttnDesc(B, hq, hkv, d, max_draft_len, max_seq_len, rows, nb * bs,
                    SV_FP8_E4M3 if fp8 else SV_BF16, softmax_scale, 0)
    if out is not None:
        devs.append(_dev(out, "out", (torch.bfloat16,)))
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if workspace is not None:
        devs.append(_dev(workspace, "workspace", (torch.uint8,)))
    dev = _one_device(devs)
    if out is None or workspace is None:
        with _allocating_on(stream, dev):
            if out is None:
                out = torch.empty_like(q)
            if workspace is None:
                workspace = new_workspace(shared_workspace_bytes(desc, groups), q.device)
    st = (_lib or load_library()).spec_verify_attn_shared(
        ctypes.byref(desc), q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), nb, bs,
        block_table.data_ptr(), table[1], seq_lens.data_ptr(), draft_len.data_ptr(), groups,
        group_begin.data_ptr(), prefix_len.data_ptr(), scale, out.data_ptr(),
        workspace.data_ptr(), workspace.numel(), _stream_on(stream, dev))
    if st:
        _check(st, "spec_verify_attn_shared")
    return out


class PagePools:
    """The pools of page data that spec_pages_extend and spec_pages_compact move pages in:
    contiguous CUDA tensors [num_blocks, block_size, ...] (K and V of each layer). Build it
    once and pass it to every call; it keeps the tensors alive."""

    def __init__(self, tensors):
        self.tensors = tuple(tensors)
        if len(self.tensors) > MAX_PAGE_POOLS:
            raise ValueError("at most %d pools" % MAX_PAGE_POOLS)
        spans = []
        for t in self.tensors:
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise TypeError("a pool must be a CUDA tensor")
            if t.dim() < 2 or not t.is_contiguous() or t.numel() == 0:
                raise ValueError("a pool must be contiguous, [num_blocks, block_size, ...]")
            if t.shape[:2] != self.tensors[0].shape[:2] or t.device != self.tensors[0].device:
                raise ValueError("the pools must have the same pages, on one device")
            spans.append((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()))
        spans.sort()
        if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
            raise ValueError("the pools must not overlap")
        self.device = self.tensors[0].get_device() if self.tensors else -1
        self.pages = tuple(self.tensors[0].shape[:2]) if self.tensors else (0, 0)
        self.heads = {t.shape[2] if t.dim() > 2 else None for t in self.tensors}
        self.array = (PageData * len(self.tensors))(*[
            PageData(t.data_ptr(), t.numel() // t.shape[0] * t.element_size())
            for t in self.tensors])

    def __len__(self):
        return len(self.tensors)


def page_pools(tensors) -> PagePools:
    """The handle of the pools of page data (see PagePools)."""
    return PagePools(tensors)


def pages_workspace_bytes(num_blocks: int, table_rows: int) -> int:
    n = load_library().spec_pages_workspace_size(num_blocks, table_rows)
    if n == 0:
        raise SpecVerifyError(2, "spec_pages_workspace_size")
    return n


# sv_page_table as bytes: packing it takes a fraction of the time of filling a ctypes structure.
_PAGE_TABLE = struct.Struct("@iiiiPPP")


def _page_table(ref_count, block_table, cached_len, block_size, lists, pools, workspace, stream):
    """The checks that the page operators share: (the C descriptor, the workspace, the
    device's index)."""
    devs = [_dev(ref_count, "ref_count", _I32), _dev(block_table, "block_table", _I32),
            _dev(cached_len, "cached_len", _I32)]
    table, blocks, rows = block_table.shape, ref_count.numel(), cached_len.numel()
    if ref_count.dim() != 1 or cached_len.dim() != 1 or len(table) != 2 or table[0] != rows:
        raise ValueError("ref_count must be [num_blocks], cached_len [rows], block_table "
                         "[rows, max_blocks]")
    n = None
    for name, t in lists:
        if t is None:
            continue
        devs.append(_dev(t, name, _I32))
        if t.dim() != 1 or (n is not None and t.numel() != n):
            raise ValueError("the call's lists must be one-dimensional and of one length")
        n = t.numel()
    if pools is not None and pools.tensors:
        devs.append(pools.device)
        if pools.pages != (blocks, block_size):
            raise ValueError("a pool must be [num_blocks, block_size, ...] of the state's pages")
    if workspace is not None:
        devs.append(_dev(workspace, "workspace", (torch.uint8,)))
    dev = _one_device(devs)
    if workspace is None:
        with _allocating_on(stream, dev):
            workspace = new_workspace(pages_workspace_bytes(blocks, rows), ref_count.device)
    try:
        packed = _PAGE_TABLE.pack(blocks, block_size, rows, table[1], ref_count.data_ptr(),
                                  block_table.data_ptr(), cached_len.data_ptr())
    except struct.error as e:
        raise ValueError("block_size: %s" % e)
    return packed, workspace, dev


def _as_pools(pools) -> PagePools:
    return pools if isinstance(pools, PagePools) else PagePools(pools)


def spec_pages_fork(ref_count, block_table, cached_len, parents, children, *, block_size: int,
                    fork_len=None, workspace=None, stream=None) -> None:
    """Rows ``children`` (unused so far) begin as copies of rows ``parents`` (int32 [n] each),
    of their first ``fork_len`` (int32 [n]) positions or whole: the same pages, each counted
    once more; no page data moves. State, changed in place: ref_count int32 [num_blocks],
    block_table int32 [rows, max_blocks], cached_len int32 [rows]."""
    t, ws, dev = _page_table(ref_count, block_table, cached_len, block_size,
                             (("parents", parents), ("children", children), ("fork_len", fork_len)),
                             None, workspace, stream)
    st = (_lib or load_library()).spec_pages_fork(
        t, parents.numel(), parents.data_ptr(), children.data_ptr(),
        None if fork_len is None else fork_len.data_ptr(), ws.data_ptr(), ws.numel(),
        _stream_on(stream, dev))
    if st:
        _check(st, "spec_pages_fork")


def spec_pages_extend(ref_count, block_table, cached_len, rows, new_len, *, block_size: int,
                      pools=(), workspace=None, stream=None) -> None:
    """Make positions cached_len[r] .. new_len[i] - 1 of row r = rows[i] writable (``rows``
    None: rows 0 .. n - 1): a shared partial last page is parted from first (its filled
    positions copied in every pool), then free pages are taken, lowest first. ``pools``: a
    PagePools (``page_pools``) or a list of pool tensors. Too few free pages: nothing
    changes and ``workspace_status`` returns 9 (SV_ERR_NO_PAGES)."""
    pools = _as_pools(pools)
    t, ws, dev = _page_table(ref_count, block_table, cached_len, block_size,
                             (("new_len", new_len), ("rows", rows)), pools, workspace, stream)
    st = (_lib or load_library()).spec_pages_extend(
        t, new_len.numel(), None if rows is None else rows.data_ptr(),
        new_len.data_ptr(), len(pools.tensors), pools.array, ws.data_ptr(), ws.numel(),
        _stream_on(stream, dev))
    if st:
        _check(st, "spec_pages_extend")


def spec_pages_trim(ref_count, block_table, cached_len, rows, new_len, *, block_size: int,
                    workspace=None, stream=None) -> None:
    """Give back the positions of row r = rows[i] from new_len[i] on (``rows`` None: rows
    0 .. n - 1): the pages past them lose a count, and their entries become -1."""
    t, ws, dev = _page_table(ref_count, block_table, cached_len, block_size,
                             (("new_len", new_len), ("rows", rows)), None, workspace, stream)
    st = (_lib or load_library()).spec_pages_trim(
        t, new_len.numel(), None if rows is None else rows.data_ptr(),
        new_len.data_ptr(), ws.data_ptr(), ws.numel(), _stream_on(stream, dev))
    if st:
        _check(st, "spec_pages_trim")


def spec_pages_compact(ref_count, block_table, cached_len, *, block_size: int, pools=(),
                       remap=None, num_live=None, workspace=None, stream=None) -> None:
    """Move the L pages in use to pages 0 .. L - 1 in every pool, with their counts, and let
    every row's entries follow. Fills ``remap`` (int32 [num_blocks]: the new page of each
    page, -1 if it was free) and ``num_live`` (int32 [1]: L) when they are given."""
    pools = _as_pools(pools)
    t, ws, dev = _page_table(ref_count, block_table, cached_len, block_size, (), pools, workspace,
                             stream)
    out = [None, None]
    for i, (o, name, n) in enumerate(((remap, "remap", ref_count.numel()), (num_live, "num_live", 1))):
        if o is not None:
            if _dev(o, name, _I32) != dev:
                raise ValueError("%s lies on another device" % name)
            if o.numel() != n:
                raise ValueError("%s must hold %d values" % (name, n))
            out[i] = o.data_ptr()
    st = (_lib or load_library()).spec_pages_compact(
        t, len(pools.tensors), pools.array, out[0], out[1], ws.data_ptr(),
        ws.numel(), _stream_on(stream, dev))
    if st:
        _check(st, "spec_pages_compact")


_U8 = (torch.uint8,)
_SCALES = (torch.uint8, torch.float8_e4m3fn)


def paged_attn_desc(q: torch.Tensor, k_pages: torch.Tensor, batch: int, max_draft_len: int,
                    max_seq_len: int, softmax_scale: float = 0.0, sliding_window: int = 0, *,
                    kv4: bool = False) -> AttnDesc:
    """The descriptor of a call over K pages [num_blocks, block_size, Hkv, d] (``kv4``: 4-bit
    codes, [num_blocks, block_size, Hkv, d / 2])."""
    nb, bs, hkv, _ = k_pages.shape
    dt = SV_KV4 if kv4 else SV_BF16 if k_pages.dtype == torch.bfloat16 else SV_FP8_E4M3
    return AttnDesc(batch, q.shape[1], hkv, q.shape[2], max_draft_len, max_seq_len, q.shape[0],
                    nb * bs, dt, float(softmax_scale), int(sliding_window))


def _workspace_bytes(name: str, *args) -> int:
    n = getattr(_lib or load_library(), name)(*args)
    if n == 0:
        raise SpecVerifyError(2, name)
    return n


def kv4_workspace_bytes(batch: int) -> int:
    return _workspace_bytes("spec_kv4_workspace_size", batch)


def verify_kv4_workspace_bytes(desc: AttnDesc) -> int:
    return _workspace_bytes("spec_verify_attn_kv4_workspace_size", ctypes.byref(desc))


def mass_workspace_bytes(desc: AttnDesc) -> int:
    return _workspace_bytes("spec_attn_mass_workspace_size", ctypes.byref(desc))


def evict_workspace_bytes(n: int, num_kv_heads: int, max_positions: int) -> int:
    """``max_positions``: positions of mass, its last dimension."""
    return _workspace_bytes("spec_kv_evict_workspace_size", n, num_kv_heads, max_positions)


# sv_kv4_pages and sv_attn_desc as bytes: packing them takes a fraction of the time of filling
# a ctypes structure, half a microsecond of a call that takes ten.
_KV4_PAGES = struct.Struct("@qiiixxxxPPPP")
_ATTN_DESC = struct.Struct("@iiiiiiqqifixxxx")


def _packed_desc(B, Hq, hkv, d, max_draft_len, max_seq_len, q_rows, dtype, scale, window) -> bytes:
    try:
        return _ATTN_DESC.pack(B, Hq, hkv, d, max_draft_len, max_seq_len, q_rows, 0, dtype, scale, window)
    except struct.error as e:
        raise ValueError("max_draft_len, max_seq_len, softmax_scale or sliding_window: %s" % e)


def _kv4_pages(k_codes, v_codes, scales, kv_scale, devs):
    """(KV heads, head dimension, C descriptor) of a 4-bit cache, its tensors' devices added to
    ``devs``."""
    devs += [_dev(k_codes, "k_codes", _U8), _dev(v_codes, "v_codes", _U8),
             _dev(scales, "scales", _SCALES), _dev(kv_scale, "kv_scale", (torch.float32,))]
    if k_codes.dim() != 4 or v_codes.shape != k_codes.shape:
        raise ValueError("k_codes and v_codes must be [num_blocks, block_size, Hkv, d / 2]")
    nb, bs, hkv, half = k_codes.shape
    if scales.shape != (nb, bs, hkv, 2, half // 8):
        raise ValueError("scales must be [num_blocks, block_size, Hkv, 2, d / 16]")
    if kv_scale.shape != (2, hkv):
        raise ValueError("kv_scale must be [2, Hkv]")
    return hkv, 2 * half, _KV4_PAGES.pack(nb, bs, hkv, 2 * half, k_codes.data_ptr(),
                                          v_codes.data_ptr(), scales.data_ptr(), kv_scale.data_ptr())


def _kv4_rows(block_table, start, count, devs, workspace, stream):
    """The checks that spec_kv4_write and spec_kv4_read share: (batch, workspace, device)."""
    devs += [_dev(block_table, "block_table", _I32), _dev(start, "start", _I32),
             _dev(count, "count", _I32)]
    B = start.numel()
    if start.dim() != 1 or count.shape != (B,) or block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("start and count must be [B], block_table [B, max_blocks]")
    if workspace is not None:
        devs.append(_dev(workspace, "workspace", _U8))
    dev = _one_device(devs)
    if workspace is None:
        with _allocating_on(stream, dev):
            workspace = new_workspace(kv4_workspace_bytes(B), start.device)
    return B, workspace, dev


def _row_stride(t, name, hkv, d, rows):
    """Elements between the rows of t [rows, Hkv, d], whose heads lie side by side."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype != torch.bfloat16:
        raise TypeError("%s has dtype %s, expected torch.bfloat16" % (name, t.dtype))
    shape = t.shape
    if len(shape) != 3 or shape != (shape[0] if rows is None else rows, hkv, d):
        raise ValueError("k and v must be [rows, Hkv, d] of the pages' heads")
    if t.is_contiguous():
        return hkv * d
    if (d > 1 and t.stride(2) != 1) or (hkv > 1 and t.stride(1) != d):
        raise ValueError("%s: a row's heads must be contiguous (rows may be apart)" % name)
    if shape[0] <= 1:
        return hkv * d
    if t.stride(0) < hkv * d:
        raise ValueError("%s: rows must not overlap" % name)
    return t.stride(0)


def spec_kv4_write(k, v, k_codes, v_codes, scales, kv_scale, block_table, start, count, *,
                   workspace=None, stream=None) -> None:
    """Round bf16 rows k, v [rows, Hkv, d] (rows may lie apart, as in a fused projection) into
    the pages of a 4-bit cache: the count[b] rows of sequence b, packed in batch order, go to
    positions start[b] .. of row b of block_table (int32 [B, max_blocks]; start, count int32
    [B]). Changed in place: k_codes, v_codes uint8 [num_blocks, block_size, Hkv, d / 2] and
    scales (uint8 or float8_e4m3fn) [num_blocks, block_size, Hkv, 2, d / 16]; kv_scale fp32
    [2, Hkv] is the caller's."""
    devs = []
    hkv, d, pages = _kv4_pages(k_codes, v_codes, scales, kv_scale, devs)
    ks = _row_stride(k, "k", hkv, d, None)
    vs = _row_stride(v, "v", hkv, d, k.shape[0])
    devs += [k.get_device(), v.get_device()]
    B, workspace, dev = _kv4_rows(block_table, start, count, devs, workspace, stream)
    st = (_lib or load_library()).spec_kv4_write(
        pages, B, block_table.data_ptr(), block_table.shape[1], start.data_ptr(),
        count.data_ptr(), k.shape[0], k.data_ptr(), ks, v.data_ptr(), vs, workspace.data_ptr(),
        workspace.numel(), _stream_on(stream, dev))
    if st:
        _check(st, "spec_kv4_write")


def spec_kv4_read(k_codes, v_codes, scales, kv_scale, block_table, start, count, *, rows=None,
                  k_out=None, v_out=None, workspace=None, stream=None):
    """The rows at positions start[b] .. start[b] + count[b] - 1 of every sequence of a 4-bit
    cache, packed in batch order: (k, v) bf16 [rows, Hkv, d]. ``rows`` (at least the sum of
    count) is needed where k_out and v_out are not given; rows past the sum are left as they
    were (zeros in outputs made here)."""
    devs = []
    *shape, pages = _kv4_pages(k_codes, v_codes, scales, kv_scale, devs)
    outs = [k_out, v_out]
    for t, name in ((k_out, "k_out"), (v_out, "v_out")):
        if t is not None:
            devs.append(_dev(t, name, (torch.bfloat16,)))
            rows = t.shape[0] if rows is None and t.dim() == 3 else rows
            if t.shape != (rows, *shape):
                raise ValueError("%s must be [rows, Hkv, d] of the pages' heads" % name)
    if rows is None:
        raise ValueError("rows, or k_out and v_out, must be given")
    B, workspace, dev = _kv4_rows(block_table, start, count, devs, workspace, stream)
    if k_out is None or v_out is None:
        with _allocating_on(stream, dev):
            for i in range(2):
                if outs[i] is None:
                    outs[i] = torch.zeros(rows, *shape, dtype=torch.bfloat16, device=k_codes.device)
    st = (_lib or load_library()).spec_kv4_read(
        pages, B, block_table.data_ptr(), block_table.shape[1], start.data_ptr(),
        count.data_ptr(), rows, outs[0].data_ptr(), outs[1].data_ptr(), workspace.data_ptr(),
        workspace.numel(), _stream_on(stream, dev))
    if st:
        _check(st, "spec_kv4_read")
    return tuple(outs)


def spec_verify_attn_kv4(q, k_codes, v_codes, scales, kv_scale, block_table, seq_lens, draft_len, *,
                         max_draft_len: int, max_seq_len: int, out=None, lse=None, workspace=None,
                         softmax_scale: float = 0.0, sliding_window: int = 0,
                         stream=None) -> torch.Tensor:
    """spec_verify_attn_paged over a 4-bit cache (see spec_kv4_write). Fills ``lse`` (fp32
    [rows, Hq]: the natural log of each row's sum of exponentials) when it is given."""
    devs = [_dev(q, "q", (torch.bfloat16,)), _dev(block_table, "block_table", _I32),
            _dev(seq_lens, "seq_lens", _I32), _dev(draft_len, "draft_len", _I32)]
    hkv, d, pages = _kv4_pages(k_codes, v_codes, scales, kv_scale, devs)
    B, shape = seq_lens.numel(), q.shape
    if len(shape) != 3 or shape[2] != d:
        raise ValueError("q must be [rows, Hq, d] with the pages' d")
    if seq_lens.dim() != 1 or draft_len.shape != (B,) or block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("seq_lens and draft_len must be [B], block_table [B, max_blocks]")
    if out is not None:
        devs.append(_dev(out, "out", (torch.bfloat16,)))
        if out.shape != shape:
            raise ValueError("out must have q's shape")
    if lse is not None:
        devs.append(_dev(lse, "lse", (torch.float32,)))
        if lse.shape != shape[:2]:
            raise ValueError("lse must be [rows, Hq]")
    if workspace is not None:
        devs.append(_dev(workspace, "workspace", _U8))
    dev = _one_device(devs)
    if out is None or workspace is None:
        with _allocating_on(stream, dev):
            if out is None:
                out = torch.empty_like(q)
            if workspace is None:
                desc = paged_attn_desc(q, k_codes, B, max_draft_len, max_seq_len, softmax_scale,
                                       sliding_window, kv4=True)
                workspace = new_workspace(verify_kv4_workspace_bytes(desc), q.device)
    desc = _packed_desc(B, shape[1], hkv, d, max_draft_len, max_seq_len, shape[0], SV_KV4,
                        softmax_scale, sliding_window)
    st = (_lib or load_library()).spec_verify_attn_kv4(
        desc, q.data_ptr(), pages, block_table.data_ptr(),
        block_table.shape[1], seq_lens.data_ptr(), draft_len.data_ptr(), out.data_ptr(),
        None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
        _stream_on(stream, dev))
    if st:
        _check(st, "spec_verify_attn_kv4")
    return out


def spec_attn_mass(q, k_pages, block_table, seq_lens, draft_len, mass, *, max_draft_len: int,
                   max_seq_len: int, kv_scale=None, scales=None, lse=None, row_count=None,
                   softmax_scale: float = 0.0, workspace=None, stream=None) -> torch.Tensor:
    """Add to mass (fp32 [B, Hkv, positions], in place) the attention weight that the first
    row_count[b] window rows of each sequence (int32 [B]: after acceptance, its accept_len;
    None: all) give to every position, summed over rows and a KV head's query heads. k_pages as
    for spec_verify_attn_paged, or 4-bit codes with their block ``scales``. ``lse`` (fp32
    [rows, Hq], as spec_verify_attn_kv4 leaves it) spares the call a pass over the keys.
    Returns mass."""
    kv4 = scales is not None
    devs = [_dev(q, "q", (torch.bfloat16,)), _dev(k_pages, "k_pages", _U8 if kv4 else _KV),
            _dev(block_table, "block_table", _I32), _dev(seq_lens, "seq_lens", _I32),
            _dev(draft_len, "draft_len", _I32), _dev(mass, "mass", (torch.float32,))]
    if q.dim() != 3 or k_pages.dim() != 4:
        raise ValueError("q must be [rows, Hq, d], k_pages [num_blocks, block_size, Hkv, d]")
    nb, bs, hkv, dk = k_pages.shape
    B, d = seq_lens.numel(), q.shape[2]
    if dk * (2 if kv4 else 1) != d:
        raise ValueError("q and the pages must have one head dimension")
    if seq_lens.dim() != 1 or draft_len.shape != (B,) or block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("seq_lens and draft_len must be [B], block_table [B, max_blocks]")
    if mass.dim() != 3 or mass.shape[:2] != (B, hkv):
        raise ValueError("mass must be [B, Hkv, positions]")
    ptr = {}
    for name, t, dt, shape in (("kv_scale", kv_scale, (torch.float32,), (2, hkv)),
                               ("scales", scales, _SCALES, (nb, bs, hkv, 2, d // 16)),
                               ("lse", lse, (torch.float32,), tuple(q.shape[:2])),
                               ("row_count", row_count, _I32, (B,))):
        ptr[name] = None
        if t is not None:
            devs.append(_dev(t, name, dt))
            if tuple(t.shape) != shape:
                raise ValueError("%s must be %s" % (name, list(shape)))
            ptr[name] = t.data_ptr()
    if workspace is not None:
        devs.append(_dev(workspace, "workspace", _U8))
    dev = _one_device(devs)
    if workspace is None:
        with _allocating_on(stream, dev):
            desc = paged_attn_desc(q, k_pages, B, max_draft_len, max_seq_len, softmax_scale, kv4=kv4)
            workspace = new_workspace(mass_workspace_bytes(desc), q.device)
    dt = SV_KV4 if kv4 else SV_BF16 if k_pages.dtype == torch.bfloat16 else SV_FP8_E4M3
    desc = _packed_desc(B, q.shape[1], hkv, d, max_draft_len, max_seq_len, q.shape[0], dt,
                        softmax_scale, 0)
    st = (_lib or load_library()).spec_attn_mass(
        desc, q.data_ptr(), k_pages.data_ptr(), ptr["scales"], ptr["kv_scale"], nb, bs,
        block_table.data_ptr(), block_table.shape[1], seq_lens.data_ptr(), draft_len.data_ptr(),
        ptr["row_count"], ptr["lse"], mass.data_ptr(), mass.shape[2], workspace.data_ptr(),
        workspace.numel(), _stream_on(stream, dev))
    if st:
        _check(st, "spec_attn_mass")
    return mass


def spec_kv_evict(ref_count, block_table, cached_len, rows, new_len, mass, *, block_size: int,
                  pools, keep_first=None, keep_last: int = 0, kept=None, workspace=None,
                  stream=None) -> None:
    """Cut row r = rows[i] (None: rows 0 .. n - 1) to new_len[i] positions, each KV head by
    itself: its first keep_first[i] (int32 [n] or None) and last keep_last stay, and of the rest
    those of largest mass (fp32 [rows, Hkv, positions]). They move to the front of the row's
    pages in every pool ([num_blocks, block_size, Hkv, ...]), and mass with them, in place.
    Fills ``kept`` (int32 [n, Hkv, k]: which position each was). Call it once a layer, then
    spec_pages_trim with the same rows and new_len."""
    if not -1 << 31 <= keep_last < 1 << 31:  # (ctypes would pass its low 32 bits)
        raise ValueError("keep_last must fit in 32 bits")
    pools = _as_pools(pools)
    if mass.dim() != 3 or mass.shape[0] != cached_len.numel():
        raise ValueError("mass must be [rows, Hkv, positions]")
    (_, hkv, positions), n = mass.shape, new_len.numel()
    if pools.tensors and pools.heads != {hkv}:
        raise ValueError("a pool must be [num_blocks, block_size, Hkv, ...] with mass's Hkv")
    devs = [_dev(mass, "mass", (torch.float32,))]
    stride = 0
    if kept is not None:
        devs.append(_dev(kept, "kept", _I32))
        if kept.dim() != 3 or kept.shape[:2] != (n, hkv):
            raise ValueError("kept must be [n, Hkv, k]")
        stride = kept.shape[2]
    if workspace is None:
        with _allocating_on(stream, _one_device(devs)):
            workspace = new_workspace(evict_workspace_bytes(n, hkv, positions), mass.device)
    t, ws, dev = _page_table(ref_count, block_table, cached_len, block_size,
                             (("new_len", new_len), ("rows", rows), ("keep_first", keep_first)),
                             pools, workspace, stream)
    if any(d != dev for d in devs):
        _one_device(devs + [dev])
    st = (_lib or load_library()).spec_kv_evict(
        t, n, None if rows is None else rows.data_ptr(), new_len.data_ptr(),
        None if keep_first is None else keep_first.data_ptr(), keep_last, hkv, mass.data_ptr(),
        positions, None if kept is None else kept.data_ptr(), stride, len(pools.tensors),
        pools.array, ws.data_ptr(), ws.numel(), _stream_on(stream, dev))
    if st:
        _check(st, "spec_kv_evict")


def spec_accept(logits, draft_tokens, draft_len, *, max_draft_len: int, accept_len=None,
                next_token=None, target_tokens=None, workspace=None, stream=None):
    """logits [sum (1 + D_b), V] bf16 or fp32; draft_tokens int32 [sum D_b]; draft_len int32
    [B]. Returns (accept_len, next_token), int32 [B] each; fills ``target_tokens`` (int32
    [sum (1 + D_b)]) with the target's greedy token per row when it is given."""
    _need(logits, "logits", (torch.bfloat16, torch.float32))
    _need(draft_tokens, "draft_tokens", (torch.int32,))
    _need(draft_len, "draft_len", (torch.int32,))
    B = draft_len.shape[0]
    V = logits.shape[-1]
    if accept_len is None:
        accept_len = torch.empty(B, dtype=torch.int32, device=logits.device)
    if next_token is None:
        next_token = torch.empty(B, dtype=torch.int32, device=logits.device)
    for t, n in ((accept_len, "accept_len"), (next_token, "next_token")):
        _need(t, n, (torch.int32,))
    if target_tokens is not None:
        _need(target_tokens, "target_tokens", (torch.int32,))
    if workspace is None:
        workspace = new_workspace(accept_workspace_bytes(B, max_draft_len, V), logits.device)
    dt = SV_BF16 if logits.dtype == torch.bfloat16 else SV_FP32
    dtok = _or_placeholder(draft_tokens)
    st = load_library().spec_accept(
        B, max_draft_len, V, dt, _ptr(logits), _ptr(dtok), _ptr(draft_len), _ptr(accept_len),
        _ptr(next_token), _ptr(target_tokens), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "spec_accept")
    return accept_len, next_token


def spec_accept_stochastic(target_logits, draft_logits, draft_tokens, draft_len, u_accept,
                           u_sample, *, max_draft_len: int, temperature: float = 1.0,
                           accept_len=None, next_token=None, workspace=None, stream=None):
    """Distribution-preserving acceptance for sampled decoding. target_logits [sum (1 + D_b),
    V] and draft_logits [sum D_b, V] (bf16 or fp32, the same); draft_tokens int32 [sum
    D_b]; draft_len int32 [B]; u_accept fp32 [sum D_b] and u_sample fp32 [B], uniform in
    [0, 1). Returns (accept_len, next_token), int32 [B] each."""
    _need(target_logits, "target_logits", (torch.bfloat16, torch.float32))
    _need(draft_logits, "draft_logits", (target_logits.dtype,))
    _need(draft_tokens, "draft_tokens", (torch.int32,))
    _need(draft_len, "draft_len", (torch.int32,))
    _need(u_accept, "u_accept", (torch.float32,))
    _need(u_sample, "u_sample", (torch.float32,))
    B = draft_len.shape[0]
    V = target_logits.shape[-1]
    if draft_logits.dim() != 2 or draft_logits.shape[1] != V:
        raise ValueError("draft_logits must be [sum D_b, V] with the target's V")
    if u_sample.numel() != B:
        raise ValueError("u_sample must hold one draw per sequence")
    if accept_len is None:
        accept_len = torch.empty(B, dtype=torch.int32, device=target_logits.device)
    if next_token is None:
        next_token = torch.empty(B, dtype=torch.int32, device=target_logits.device)
    for t, n in ((accept_len, "accept_len"), (next_token, "next_token")):
        _need(t, n, (torch.int32,))
    lib = load_library()
    if workspace is None:
        n = lib.spec_accept_stochastic_workspace_size(B, max_draft_len, V)
        if n == 0:
            raise SpecVerifyError(2, "spec_accept_stochastic_workspace_size")
        workspace = new_workspace(n, target_logits.device)
    dt = SV_BF16 if target_logits.dtype == torch.bfloat16 else SV_FP32
    dlg, dtk, ua = (_or_placeholder(t) for t in (draft_logits, draft_tokens, u_accept))
    st = lib.spec_accept_stochastic(
        B, max_draft_len, V, dt, _ptr(target_logits), _ptr(dlg), _ptr(dtk), _ptr(draft_len),
        _ptr(ua),
        _ptr(u_sample), float(temperature), _ptr(accept_len), _ptr(next_token),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "spec_accept_stochastic")
    return accept_len, next_token


def spec_draft_signals(logits, *, confidence=None, entropy=None, workspace=None, stream=None):
    """logits [rows, V] bf16 or fp32 (e.g. the draft model's logits at each drafted
    position). Returns (confidence, entropy), fp32 [rows] each: the largest probability
    and the entropy (nats) of each row's softmax."""
    _need(logits, "logits", (torch.bfloat16, torch.float32))
    rows, V = logits.shape
    if confidence is None:
        confidence = torch.empty(rows, dtype=torch.float32, device=logits.device)
    if entropy is None:
        entropy = torch.empty(rows, dtype=torch.float32, device=logits.device)
    for t, n in ((confidence, "confidence"), (entropy, "entropy")):
        _need(t, n, (torch.float32,))
    if workspace is None:
        workspace = new_workspace(signals_workspace_bytes(rows, V), logits.device)
    dt = SV_BF16 if logits.dtype == torch.bfloat16 else SV_FP32
    st = load_library().spec_draft_signals(
        rows, V, dt, _ptr(logits), _ptr(confidence), _ptr(entropy), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream))
    _check(st, "spec_draft_signals")
    return confidence, entropy


def workspace_status(workspace: torch.Tensor, clear: bool = False, stream=None) -> int:
    """Synchronises and returns the workspace's sticky device-side status (0 = ok)."""
    return load_library().sv_workspace_status(_ptr(workspace), int(clear), _stream(stream))


def set_attn_kernel(which: int) -> int:
    """0 automatic, 1 mma.sync kernel, 2 tcgen05 kernel. Returns the previous choice."""
    prev = load_library().sv_set_attn_kernel(int(which))
    if prev < 0:
        raise ValueError("attention kernel %d is not available" % which)
    return prev


def set_unit_ctas(mode: int) -> int:
    """-1 cost model (default), 0 split tile line, k >= 1 k CTAs per unit. Returns the
    previous mode."""
    prev = load_library().sv_set_unit_ctas(int(mode))
    if prev < -1:
        raise ValueError("unit-CTA mode must be in [-1, 1024]")
    return prev


def inject_launch_failure(after: int) -> int:
    """Test hook: after ``after`` more kernel launches of the library, the next one fails
    on the host, and the call that makes it raises SpecVerifyError (SV_ERR_CUDA); a
    negative ``after`` disarms. Returns the launches that were still to go before a
    pending failure, or -1."""
    return load_library().sv_inject_launch_failure(int(after))


def set_row_pairs(mode: int) -> int:
    """0 never (default), 1 whenever the row-pair kernel applies (128 < G(1 + max_draft) <=
    256, bf16, d = 128, packed, no window, B * Hkv <= SMs). Returns the previous mode."""
    prev = load_library().sv_set_row_pairs(int(mode))
    if prev < 0:
        raise ValueError("row-pair mode must be 0 or 1")
    return prev


def set_kv_rings(mode: int) -> int:
    """bf16 K/V on the tcgen05 kernel: -1 by the call's shape (default), 0 paired K + V
    stages, 1 separate K and V rings. Returns the previous mode."""
    prev = load_library().sv_set_kv_rings(int(mode))
    if prev < -1:
        raise ValueError("ring mode must be -1, 0 or 1")
    return prev


def row_pair_mode(desc, num_sms: int, attn_kernel: int = 2, block_size: int = 0) -> int:
    """1 if a call with this descriptor runs the row-pair kernel, else 0."""
    r = load_library().sv_row_pair_mode(ctypes.byref(desc), int(block_size), int(num_sms),
                                        int(attn_kernel))
    if r < 0:
        raise SpecVerifyError(2, "sv_row_pair_mode")
    return r


def inject_wait_timeout(limit_cycles: int) -> int:
    """Test hook: the next launch of the tcgen05 attention kernel waits at most
    ``limit_cycles`` clock cycles per barrier and each CTA withholds its first tile's
    loads, so the kernel gives up, sets SV_ERR_TIMEOUT in the workspace and returns. 0
    disarms.
    Returns 1 if an arming was pending, else 0."""
    return load_library().sv_inject_wait_timeout(int(limit_cycles))


def set_profile_events(start=None, stop=None):
    """Record CUDA events around the main attention kernel of later calls (None: off)."""
    lib = load_library()
    if start is None or stop is None:
        lib.sv_set_profile_events(None, None)
    else:
        lib.sv_set_profile_events(ctypes.c_void_p(start.cuda_event),
                                  ctypes.c_void_p(stop.cuda_event))


def plan_preview(desc: AttnDesc, seq_lens, draft_len, *, num_sms: int, attn_kernel: int = 2,
                 block_size: int = 0) -> dict:
    """The work plan a verify-attention call with these host lengths (int sequences) makes
    on a device of ``num_sms`` SMs, computed on the host by the library. Returns a dict:
    the sv_plan_info counts, ``units`` int32 [U, 4] (b, KV head, row tile, first cache
    position of the unit's first tile), ``unit_begin`` int32 [U + 1] and ``cta_begin``
    int32 [C + 1, 2] (first tile, its unit)."""
    import numpy as np
    T = np.ascontiguousarray(seq_lens, dtype=np.int32)
    D = np.ascontiguousarray(draft_len, dtype=np.int32)
    if T.shape != (desc.batch,) or D.shape != (desc.batch,):
        raise ValueError("seq_lens and draft_len must hold desc.batch lengths")
    lib = load_library()
    info = PlanInfo()
    st = lib.sv_plan_preview(ctypes.byref(desc), block_size, T.ctypes.data, D.ctypes.data,
                             num_sms, attn_kernel, ctypes.byref(info), None, None, None, 0)
    _check(st, "sv_plan_preview")
    U, C = info.num_units, info.num_ctas
    units = np.zeros((max(U, 1), 4), dtype=np.int32)
    ubeg = np.zeros(U + 1, dtype=np.int32)
    cta = np.zeros((C + 1, 2), dtype=np.int32)
    st = lib.sv_plan_preview(ctypes.byref(desc), block_size, T.ctypes.data, D.ctypes.data,
                             num_sms, attn_kernel, ctypes.byref(info), units.ctypes.data,
                             ubeg.ctypes.data, cta.ctypes.data, U)
    _check(st, "sv_plan_preview")
    out = {name: getattr(info, name) for name, _ in PlanInfo._fields_}
    out.update(units=units[:U], unit_begin=ubeg, cta_begin=cta)
    return out


def default_scale(head_dim: int) -> float:
    return 1.0 / math.sqrt(head_dim)

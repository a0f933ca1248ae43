"""GB300 (sm_103a) paged-KV GQA decode attention.

A thin Python binding over the C ABI in ``include/paged_attn.h``: the
functions here only marshal torch tensors into pointers, sizes and the
current CUDA stream; every step of the computation runs in the library's
CUDA kernels.  There is no fallback: if the compiled library is missing the
calls raise.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

__all__ = [
    "PagedAttnError",
    "LIB_PATH",
    "load",
    "paged_attn_decode",
    "paged_attn_decode_ws",
    "paged_attn_decode_checked",
    "paged_attn_decode_static",
    "paged_attn_append_decode",
    "paged_kv_append",
    "paged_attn_decode_fp8",
    "paged_attn_decode_xpacked",
    "paged_attn_decode_multi",
    "paged_kv_append_multi",
    "paged_attn_append_decode_multi",
    "paged_kv_append_fp8",
    "paged_attn_append_decode_fp8",
    "paged_attn_decode_mods",
    "paged_attn_decode_fp8_mods",
    "paged_attn_mods_workspace_bytes",
    "paged_attn_decode_multi_mods",
    "paged_attn_multi_mods_workspace_bytes",
    "paged_attn_decode_shared",
    "paged_attn_shared_workspace_bytes",
    "paged_kv_assign",
    "paged_kv_append_slots",
    "paged_attn_workspace_bytes",
    "paged_attn_status_string",
    "paged_attn_set_launch_flags",
    "paged_attn_set_checks",
    "paged_attn_reset_workspace",
    "FLAG_EARLY_PROLOGUE",
    "EXPORTED_SYMBOLS",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libpaged_kv_gqa_decode.so")

# Every symbol declared in include/paged_attn.h.
EXPORTED_SYMBOLS = (
    "paged_attn_decode",
    "paged_attn_workspace_bytes",
    "paged_attn_decode_ws",
    "paged_attn_decode_checked",
    "paged_attn_decode_static",
    "paged_kv_append",
    "paged_attn_append_decode",
    "paged_attn_decode_fp8",
    "paged_attn_decode_xpacked",
    "paged_attn_decode_multi",
    "paged_attn_decode_multi_ex",
    "paged_kv_append_multi",
    "paged_attn_append_decode_multi",
    "paged_kv_append_fp8",
    "paged_attn_append_decode_fp8",
    "paged_attn_decode_mods",
    "paged_attn_decode_fp8_mods",
    "paged_attn_mods_workspace_bytes",
    "paged_attn_decode_multi_mods",
    "paged_attn_multi_mods_workspace_bytes",
    "paged_attn_decode_shared",
    "paged_attn_shared_workspace_bytes",
    "paged_kv_assign",
    "paged_kv_append_slots",
    "paged_attn_status_string",
    "paged_attn_set_launch_flags",
    "paged_attn_set_checks",
    "paged_attn_reset_workspace",
    "paged_attn_last_cuda_error",
    "paged_attn_version",
)

# Launch flags (include/paged_attn.h).
FLAG_EARLY_PROLOGUE = 1

_lock = threading.Lock()
_lib = None


class PagedAttnError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"paged_attn status {status}: {message}")
        self.status = status


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load the compiled library (raises if it was not built)."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                f"{p} is missing: build it with `python -m paged_kv_gqa_decode_gb300.build` "
                "(needs nvcc from the CUDA 13 toolkit)")
        lib = ctypes.CDLL(p)
        P, I, F, LL, SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong,
                           ctypes.c_size_t)
        common = [P, P, P, P, P, P, I, I, I, I, I, I, F]
        lib.paged_attn_decode.argtypes = common + [P]
        lib.paged_attn_decode.restype = I
        lib.paged_attn_workspace_bytes.argtypes = [I, I, I, I, I, I]
        lib.paged_attn_workspace_bytes.restype = SZ
        lib.paged_attn_decode_ws.argtypes = common + [P, SZ, P]
        lib.paged_attn_decode_ws.restype = I
        lib.paged_attn_decode_checked.argtypes = common + [LL, P, P]
        lib.paged_attn_decode_checked.restype = I
        lib.paged_attn_decode_static.argtypes = common + [P]
        lib.paged_attn_decode_static.restype = I
        lib.paged_kv_append.argtypes = [P, P, P, P, P, P, I, I, I, I, I, P]
        lib.paged_kv_append.restype = I
        lib.paged_attn_append_decode.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, P]
        lib.paged_attn_append_decode.restype = I
        lib.paged_attn_decode_fp8.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, P]
        lib.paged_attn_decode_fp8.restype = I
        lib.paged_attn_decode_xpacked.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, F, P]
        lib.paged_attn_decode_xpacked.restype = I
        lib.paged_attn_decode_multi.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, F,
                                                P]
        lib.paged_attn_decode_multi.restype = I
        lib.paged_attn_decode_multi_ex.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, I,
                                                   F, I, P]
        lib.paged_attn_decode_multi_ex.restype = I
        lib.paged_kv_append_multi.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, P]
        lib.paged_kv_append_multi.restype = I
        lib.paged_attn_append_decode_multi.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I,
                                                       I, I, I, F, I, P]
        lib.paged_attn_append_decode_multi.restype = I
        lib.paged_kv_append_fp8.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, P]
        lib.paged_kv_append_fp8.restype = I
        lib.paged_attn_append_decode_fp8.argtypes = [P, P, P, P, P, P, P, P, P, P, I, I, I, I, I,
                                                     I, F, P]
        lib.paged_attn_append_decode_fp8.restype = I
        mods = [F, P, I, P, P, P, SZ, P]  # softcap .. doc_starts, workspace, stream
        lib.paged_attn_decode_mods.argtypes = common + mods
        lib.paged_attn_decode_mods.restype = I
        lib.paged_attn_decode_fp8_mods.argtypes = [P, P] + common + mods
        lib.paged_attn_decode_fp8_mods.restype = I
        lib.paged_attn_mods_workspace_bytes.argtypes = [I, I, I, I, I, I]
        lib.paged_attn_mods_workspace_bytes.restype = SZ
        lib.paged_attn_decode_multi_mods.argtypes = [P] * 7 + [I] * 7 + [F, I] + mods
        lib.paged_attn_decode_multi_mods.restype = I
        lib.paged_attn_multi_mods_workspace_bytes.argtypes = [I] * 7
        lib.paged_attn_multi_mods_workspace_bytes.restype = SZ
        lib.paged_attn_decode_shared.argtypes = ([P] * 7 + [I, I, P, P] + [I] * 6 +
                                                 [F, F, P, P, SZ, P])
        lib.paged_attn_decode_shared.restype = I
        lib.paged_attn_shared_workspace_bytes.argtypes = [I] * 7
        lib.paged_attn_shared_workspace_bytes.restype = SZ
        lib.paged_kv_assign.argtypes = [P] * 10 + [I, I, I, I, I, P]
        lib.paged_kv_assign.restype = I
        lib.paged_kv_append_slots.argtypes = [P, P, LL, LL, P, P, P, I, I, I, I, LL, P]
        lib.paged_kv_append_slots.restype = I
        lib.paged_attn_set_checks.argtypes = [LL, P]
        lib.paged_attn_set_checks.restype = I
        lib.paged_attn_reset_workspace.argtypes = [P]
        lib.paged_attn_reset_workspace.restype = I
        lib.paged_attn_status_string.argtypes = [I]
        lib.paged_attn_status_string.restype = ctypes.c_char_p
        lib.paged_attn_last_cuda_error.argtypes = []
        lib.paged_attn_last_cuda_error.restype = I
        lib.paged_attn_version.argtypes = []
        lib.paged_attn_version.restype = I
        lib.paged_attn_set_launch_flags.argtypes = [I]
        lib.paged_attn_set_launch_flags.restype = I
        if path is None:
            _lib = lib
        return lib


def paged_attn_status_string(status: int) -> str:
    return load().paged_attn_status_string(int(status)).decode()


def paged_attn_set_launch_flags(flags: int) -> None:
    """Launch flags for later decode calls from this host thread (0: the plain
    launch).  FLAG_EARLY_PROLOGUE: the caller guarantees that the work ahead in
    the stream writes none of the caches, block tables, lengths or query offsets
    (see include/paged_attn.h).  paged_kv_append and paged_attn_append_decode
    write the cache, so a launch right after one of them on the same cache must
    not use it."""
    _check(load().paged_attn_set_launch_flags(int(flags)))


def paged_attn_set_checks(num_blocks: int = 0, status=None) -> None:
    """Device-side checks for later calls from this host thread: block ids are
    validated against [0, num_blocks) and problems reported into ``status`` (an
    int32 device tensor of one element the caller zero-fills); ``(0, None)``
    turns them off (see include/paged_attn.h)."""
    _check(load().paged_attn_set_checks(int(num_blocks), _ptr(status)))


def paged_attn_reset_workspace(stream=None) -> None:
    """Zero-fill the library-owned workspace of the current device (needed only
    after a call reported a combine wait that ran out)."""
    _check(load().paged_attn_reset_workspace(_stream(stream)))


def _check(status: int) -> None:
    if status != 0:
        lib = load()
        msg = lib.paged_attn_status_string(status).decode()
        if status == -6:
            msg += f" (CUDA error {lib.paged_attn_last_cuda_error()})"
        raise PagedAttnError(status, msg)


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _stream(stream) -> int:
    import torch

    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _sizes(q, k_cache, block_tables):
    num_seqs, H_q, D = (int(x) for x in q.shape)
    _, H_kv, BS, Dk = (int(x) for x in k_cache.shape)
    if Dk != D:
        raise ValueError("q and the caches disagree on head_dim")
    maxb = int(block_tables.shape[1]) if block_tables.dim() == 2 else 0
    return num_seqs, H_q, H_kv, D, maxb, BS


def _args(q, k_cache, v_cache, out, block_tables, seq_lens, scale):
    for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache), ("out", out),
                    ("block_tables", block_tables), ("seq_lens", seq_lens)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    num_seqs, H_q, H_kv, D, maxb, BS = _sizes(q, k_cache, block_tables)
    return (_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out), _ptr(block_tables),
            _ptr(seq_lens), num_seqs, H_q, H_kv, D, maxb, BS, float(scale))


def paged_attn_decode(q, k_cache, v_cache, block_tables, seq_lens, scale: float, out=None,
                      stream=None):
    """out[s, h] = softmax(scale * q[s, h] . K^T) . V over the paged cache (see paged_attn.h)."""
    import torch

    if out is None:
        out = torch.empty_like(q)
    _check(load().paged_attn_decode(*_args(q, k_cache, v_cache, out, block_tables, seq_lens,
                                           scale), _stream(stream)))
    return out


def paged_attn_workspace_bytes(num_seqs: int, H_q: int, H_kv: int, head_dim: int,
                               max_blocks_per_seq: int, block_size: int) -> int:
    return int(load().paged_attn_workspace_bytes(num_seqs, H_q, H_kv, head_dim,
                                                 max_blocks_per_seq, block_size))


def paged_attn_decode_ws(q, k_cache, v_cache, block_tables, seq_lens, scale: float, workspace,
                         out=None, stream=None):
    """As paged_attn_decode, with a caller-owned zero-initialised uint8 device workspace."""
    import torch

    if out is None:
        out = torch.empty_like(q)
    _check(load().paged_attn_decode_ws(*_args(q, k_cache, v_cache, out, block_tables, seq_lens,
                                              scale), _ptr(workspace),
                                       int(workspace.numel() * workspace.element_size()),
                                       _stream(stream)))
    return out


def paged_attn_decode_checked(q, k_cache, v_cache, block_tables, seq_lens, scale: float,
                              status, out=None, stream=None, num_blocks: Optional[int] = None):
    """As paged_attn_decode, validating block ids and lengths on the device into ``status``
    (an int32 device tensor of one element that the caller zero-fills)."""
    import torch

    if out is None:
        out = torch.empty_like(q)
    nb = int(k_cache.shape[0]) if num_blocks is None else int(num_blocks)
    _check(load().paged_attn_decode_checked(*_args(q, k_cache, v_cache, out, block_tables,
                                                   seq_lens, scale), nb, _ptr(status),
                                            _stream(stream)))
    return out


def paged_attn_decode_static(q, k_cache, v_cache, block_tables, seq_lens, scale: float,
                             out=None, stream=None):
    """As paged_attn_decode, for callers that must not allocate device memory: the
    library's fixed 4 MiB scratch array stands in for the workspace (see paged_attn.h;
    calls that overlap on the GPU race on that array).  ``out`` should be passed in by
    such callers, since creating it here would allocate."""
    import torch

    if out is None:
        out = torch.empty_like(q)
    _check(load().paged_attn_decode_static(*_args(q, k_cache, v_cache, out, block_tables,
                                                  seq_lens, scale), _stream(stream)))
    return out


def paged_attn_decode_xpacked(q, kx, vt, block_tables, seq_lens, scale: float, out=None,
                              stream=None):
    """Decode over x-packed bf16 caches (see paged_attn.h): kx [num_blocks, H_kv,
    head_dim / 8, block_size, 8], vt [num_blocks, H_kv, head_dim, block_size]."""
    import torch

    for name, t in (("q", q), ("kx", kx), ("vt", vt), ("block_tables", block_tables),
                    ("seq_lens", seq_lens)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    num_seqs, H_q, D = (int(x) for x in q.shape)
    if kx.dim() != 5 or vt.dim() != 4:
        raise ValueError("kx must be [NB, H_kv, D/8, BS, 8] and vt [NB, H_kv, D, BS]")
    nb, H_kv, dx, BS, x = (int(v) for v in kx.shape)
    if x != 8 or dx * 8 != D or tuple(vt.shape) != (nb, H_kv, D, BS):
        raise ValueError("kx / vt shapes do not match q's head_dim")
    if out is None:
        out = torch.empty_like(q)
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    maxb = int(block_tables.shape[1]) if block_tables.dim() == 2 else 0
    _check(load().paged_attn_decode_xpacked(_ptr(q), _ptr(kx), _ptr(vt), _ptr(out),
                                            _ptr(block_tables), _ptr(seq_lens), num_seqs, H_q,
                                            H_kv, D, maxb, BS, float(scale), _stream(stream)))
    return out


def _multi_sizes(q, k_cache, qo_indptr, block_tables, seq_lens, contiguous):
    import torch

    for name, t in contiguous.items():
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    total_q, H_q, D = (int(x) for x in q.shape)
    _, H_kv, BS, Dk = (int(x) for x in k_cache.shape)
    if Dk != D:
        raise ValueError("q and the caches disagree on head_dim")
    num_seqs = int(seq_lens.shape[0])
    if tuple(qo_indptr.shape) != (num_seqs + 1,) or qo_indptr.dtype != torch.int32:
        raise ValueError("qo_indptr must be int32 [num_seqs + 1]")
    maxb = int(block_tables.shape[1]) if block_tables.dim() == 2 else 0
    return num_seqs, total_q, H_q, H_kv, D, maxb, BS


def paged_attn_decode_multi(q, k_cache, v_cache, qo_indptr, block_tables, seq_lens,
                            scale: float, max_q_len: int, out=None, stream=None,
                            causal: bool = True):
    """Multi-token decode (see paged_attn.h): q [total_q, H_q, D], sequence s owning
    rows qo_indptr[s] .. qo_indptr[s+1] - 1 (its last tokens); causal, or every
    row attending all of the sequence's tokens with ``causal=False``."""
    import torch

    num_seqs, total_q, H_q, H_kv, D, maxb, BS = _multi_sizes(
        q, k_cache, qo_indptr, block_tables, seq_lens,
        dict(q=q, k_cache=k_cache, v_cache=v_cache, qo_indptr=qo_indptr,
             block_tables=block_tables, seq_lens=seq_lens))
    if out is None:
        out = torch.empty_like(q)
    _check(load().paged_attn_decode_multi_ex(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(out),
                                             _ptr(qo_indptr), _ptr(block_tables),
                                             _ptr(seq_lens), num_seqs, total_q, int(max_q_len),
                                             H_q, H_kv, D, maxb, BS, float(scale),
                                             1 if causal else 0, _stream(stream)))
    return out


def paged_kv_append_multi(k_new, v_new, k_cache, v_cache, qo_indptr, block_tables, seq_lens,
                          stream=None):
    """Write several new tokens per sequence into the paged caches (see paged_attn.h):
    k_new, v_new [total_q, H_kv, head_dim] bf16, row qo_indptr[s] + i being token
    seq_lens[s] - q_len + i of sequence s."""
    _check_rows(k_new, v_new, None, k_cache)
    num_seqs, total_q, _, H_kv, D, maxb, BS = _multi_sizes(
        k_new, k_cache, qo_indptr, block_tables, seq_lens,
        dict(qo_indptr=qo_indptr, block_tables=block_tables, seq_lens=seq_lens))
    _check(load().paged_kv_append_multi(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                        _ptr(qo_indptr), _ptr(block_tables), _ptr(seq_lens),
                                        num_seqs, total_q, H_kv, D, maxb, BS, _stream(stream)))


def paged_attn_append_decode_multi(q, k_new, v_new, k_cache, v_cache, qo_indptr, block_tables,
                                   seq_lens, scale: float, max_q_len: int, out=None,
                                   stream=None, causal: bool = True):
    """paged_kv_append_multi then paged_attn_decode_multi (see paged_attn.h)."""
    import torch

    _check_rows(k_new, v_new, q, k_cache)
    num_seqs, total_q, H_q, H_kv, D, maxb, BS = _multi_sizes(
        q, k_cache, qo_indptr, block_tables, seq_lens,
        dict(q=q, k_cache=k_cache, v_cache=v_cache, qo_indptr=qo_indptr,
             block_tables=block_tables, seq_lens=seq_lens))
    if out is None:
        out = torch.empty_like(q)
    _check(load().paged_attn_append_decode_multi(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), _ptr(out),
        _ptr(qo_indptr), _ptr(block_tables), _ptr(seq_lens), num_seqs, total_q, int(max_q_len),
        H_q, H_kv, D, maxb, BS, float(scale), 1 if causal else 0, _stream(stream)))
    return out


def _check_rows(k_new, v_new, q_or_none, k_cache):
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    _, H_kv, _, D = (int(x) for x in k_cache.shape)
    if tuple(k_new.shape[1:]) != (H_kv, D) or k_new.shape != v_new.shape:
        raise ValueError("k_new and v_new must be [num_seqs, H_kv, head_dim]")
    if q_or_none is not None and int(k_new.shape[0]) != int(q_or_none.shape[0]):
        raise ValueError("k_new must have one row set per sequence of q")


def paged_kv_append(k_new, v_new, k_cache, v_cache, block_tables, seq_lens, stream=None):
    """Write each sequence's new token (position seq_lens[s] - 1) into the paged caches
    (see paged_attn.h).  k_new, v_new: [num_seqs, H_kv, head_dim] bf16."""
    _check_rows(k_new, v_new, None, k_cache)
    num_blocks, H_kv, BS, D = (int(x) for x in k_cache.shape)
    maxb = int(block_tables.shape[1]) if block_tables.dim() == 2 else 0
    _check(load().paged_kv_append(_ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                  _ptr(block_tables), _ptr(seq_lens), int(k_new.shape[0]), H_kv,
                                  D, maxb, BS, _stream(stream)))


def paged_attn_append_decode(q, k_new, v_new, k_cache, v_cache, block_tables, seq_lens,
                             scale: float, out=None, stream=None):
    """paged_kv_append then paged_attn_decode, fused into one launch (see paged_attn.h)."""
    import torch

    _check_rows(k_new, v_new, q, k_cache)
    if out is None:
        out = torch.empty_like(q)
    a = _args(q, k_cache, v_cache, out, block_tables, seq_lens, scale)
    # (q, k_new, v_new, k_cache, v_cache, out, tables, lens, sizes..., scale)
    _check(load().paged_attn_append_decode(a[0], _ptr(k_new), _ptr(v_new), a[1], a[2], a[3],
                                           *a[4:], _stream(stream)))
    return out


def paged_attn_decode_fp8(q, k8, v8, k_scale, v_scale, block_tables, seq_lens, scale: float,
                          out=None, stream=None):
    """Decode over FP8 caches (see paged_attn.h): k8 / v8 hold e4m3 bytes (uint8)
    [num_blocks, H_kv, block_size, head_dim], k_scale / v_scale one float32 per
    (block, KV head, slot); head_dim 128 or 256."""
    import torch

    for name, t in (("k8", k8), ("v8", v8), ("k_scale", k_scale), ("v_scale", v_scale)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if k8.dtype != torch.uint8 or v8.dtype != torch.uint8:
        raise ValueError("k8 / v8 must be uint8 (e4m3 bytes)")
    if k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32 or \
            tuple(k_scale.shape) != tuple(k8.shape[:3]) or k_scale.shape != v_scale.shape:
        raise ValueError("k_scale / v_scale must be float32 [num_blocks, H_kv, block_size]")
    if out is None:
        out = torch.empty_like(q)
    a = _args(q, k8, v8, out, block_tables, seq_lens, scale)
    # (q, k8, v8, k_scale, v_scale, out, tables, lens, sizes..., scale)
    _check(load().paged_attn_decode_fp8(a[0], a[1], a[2], _ptr(k_scale), _ptr(v_scale), a[3],
                                        *a[4:], _stream(stream)))
    return out


def _check_fp8_cache(k8, v8, k_scale, v_scale):
    import torch

    for name, t in (("k8", k8), ("v8", v8), ("k_scale", k_scale), ("v_scale", v_scale)):
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if k8.dtype != torch.uint8 or v8.dtype != torch.uint8:
        raise ValueError("k8 / v8 must be uint8 (e4m3 bytes)")
    if k_scale.dtype != torch.float32 or v_scale.dtype != torch.float32 or \
            tuple(k_scale.shape) != tuple(k8.shape[:3]) or k_scale.shape != v_scale.shape:
        raise ValueError("k_scale / v_scale must be float32 [num_blocks, H_kv, block_size]")


def paged_kv_append_fp8(k_new, v_new, k8, v8, k_scale, v_scale, block_tables, seq_lens,
                        stream=None):
    """Quantize each sequence's new K / V rows (bf16 [num_seqs, H_kv, head_dim]) to
    e4m3 with one dequant float per row and write them into the FP8 caches at
    position seq_lens[s] - 1 (see paged_attn.h)."""
    _check_fp8_cache(k8, v8, k_scale, v_scale)
    _check_rows(k_new, v_new, None, k8)
    num_blocks, H_kv, BS, D = (int(x) for x in k8.shape)
    maxb = int(block_tables.shape[1]) if block_tables.dim() == 2 else 0
    _check(load().paged_kv_append_fp8(_ptr(k_new), _ptr(v_new), _ptr(k8), _ptr(v8),
                                      _ptr(k_scale), _ptr(v_scale), _ptr(block_tables),
                                      _ptr(seq_lens), int(k_new.shape[0]), H_kv, D, maxb, BS,
                                      _stream(stream)))


def paged_attn_append_decode_fp8(q, k_new, v_new, k8, v8, k_scale, v_scale, block_tables,
                                 seq_lens, scale: float, out=None, stream=None):
    """paged_kv_append_fp8 then paged_attn_decode_fp8 (see paged_attn.h)."""
    import torch

    _check_fp8_cache(k8, v8, k_scale, v_scale)
    _check_rows(k_new, v_new, q, k8)
    if out is None:
        out = torch.empty_like(q)
    a = _args(q, k8, v8, out, block_tables, seq_lens, scale)
    # (q, k_new, v_new, k8, v8, k_scale, v_scale, out, tables, lens, sizes..., scale)
    _check(load().paged_attn_append_decode_fp8(a[0], _ptr(k_new), _ptr(v_new), a[1], a[2],
                                               _ptr(k_scale), _ptr(v_scale), a[3], *a[4:],
                                               _stream(stream)))
    return out


def _same_device(*tensors) -> int:
    """CUDA tensors must lie on the current device (whose stream the call uses); a host
    tensor must be pinned.  Returns the current device."""
    import torch

    current = torch.cuda.current_device() if tensors[0].is_cuda else -1
    for t in tensors:
        if t is None:
            continue
        if t.is_cuda:
            if t.get_device() != current:
                if current >= 0:
                    raise ValueError("every tensor must be on the current CUDA device")
                current = torch.cuda.current_device()
                if t.get_device() != current:
                    raise ValueError("every tensor must be on the current CUDA device")
        elif not t.is_pinned():
            raise ValueError("host tensors must be pinned")
    return current


def _need(name, t, dtype, shape) -> None:
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)}")


def _int32(name, x) -> int:
    """An int argument of the C ABI (whose conversion would drop the upper bits)."""
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} must fit 32 bits, got {x}")
    return x


def _softcap(x) -> float:
    """The cap as the C ABI takes it: one below float32's range is not taken for none."""
    x = float(x)
    if x != 0.0 and ctypes.c_float(x).value == 0.0:
        raise ValueError(f"softcap must be 0 or in [1e-30, 1e30], got {x}")
    return x


def _raw_stream(stream, device) -> int:
    """The stream's handle: the one given, or the device's current one."""
    if stream is not None:
        return int(stream.cuda_stream)
    import torch

    return torch.cuda.current_stream(device if device >= 0 else None).cuda_stream


def _mods_problem(q, k_cache, v_cache, block_tables, seq_lens, out, alibi_slopes, prefix_lens,
                  doc_starts, workspace, cache_dtype, rows=None):
    """Checks the tensors of a decode call with score options; returns the sizes, out and
    the device."""
    import torch

    i32 = torch.int32
    qs, ks, bs, ls = q.shape, k_cache.shape, block_tables.shape, seq_lens.shape
    if len(qs) != 3 or len(ks) != 4 or len(bs) != 2 or len(ls) != 1:
        raise ValueError("q must be [rows, H_q, D], the caches [num_blocks, H_kv, block_size, D], "
                         "block_tables [num_seqs, max_blocks] and seq_lens [num_seqs]")
    n, H_q, D = qs
    num_seqs = ls[0]
    maxb = bs[1]
    if ks[3] != D:
        raise ValueError("q and the caches disagree on head_dim")
    if rows is None and n != num_seqs:
        raise ValueError("q must have one row per sequence")
    _need("q", q, torch.bfloat16, qs)
    _need("k_cache", k_cache, cache_dtype, ks)
    _need("v_cache", v_cache, cache_dtype, ks)
    _need("block_tables", block_tables, i32, (num_seqs, maxb))
    _need("seq_lens", seq_lens, i32, ls)
    if alibi_slopes is not None:
        _need("alibi_slopes", alibi_slopes, torch.float32, (H_q,))
    if prefix_lens is not None:
        _need("prefix_lens", prefix_lens, i32, ls)
    if doc_starts is not None:
        _need("doc_starts", doc_starts, i32, (n,))
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if out is None:
        out = torch.empty_like(q)
    else:
        _need("out", out, torch.bfloat16, qs)
    device = _same_device(q, k_cache, v_cache, block_tables, seq_lens, out, alibi_slopes,
                          prefix_lens, doc_starts, workspace)
    return n, num_seqs, H_q, ks[1], D, maxb, ks[2], out, device


def _bytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def paged_attn_decode_mods(q, k_cache, v_cache, block_tables, seq_lens, scale: float, *,
                           softcap: float = 0.0, alibi_slopes=None, window: int = 0,
                           prefix_lens=None, doc_starts=None, out=None, workspace=None,
                           stream=None):
    """Decode with capped scores, a distance bias, a window, a prefix and documents (see
    paged_attn.h): a query at position L - 1 sees token t when t < prefix_lens[s], or
    when t >= doc_starts[s] and t > L - 1 - window (window 0: none), with the score
    softcap * tanh(scale * q.k / softcap) - alibi_slopes[h] * (L - 1 - t).
    ``workspace``: a zero-initialised uint8 tensor of paged_attn_mods_workspace_bytes for
    calls that do not overlap, needed while a stream is being captured; without it the
    library keeps one for each stream."""
    import torch

    softcap, window = _softcap(softcap), _int32("window", window)
    _, n, H_q, H_kv, D, maxb, BS, out, dev = _mods_problem(
        q, k_cache, v_cache, block_tables, seq_lens, out, alibi_slopes, prefix_lens, doc_starts,
        workspace, torch.bfloat16)
    _check((_lib or load()).paged_attn_decode_mods(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(),
        block_tables.data_ptr(), seq_lens.data_ptr(), n, H_q, H_kv, D, maxb, BS, float(scale),
        softcap, _ptr(alibi_slopes), window, _ptr(prefix_lens), _ptr(doc_starts),
        _ptr(workspace), _bytes(workspace), _raw_stream(stream, dev)))
    return out


def paged_attn_decode_fp8_mods(q, k8, v8, k_scale, v_scale, block_tables, seq_lens,
                               scale: float, *, softcap: float = 0.0, alibi_slopes=None,
                               window: int = 0, prefix_lens=None, doc_starts=None, out=None,
                               workspace=None, stream=None):
    """paged_attn_decode_mods over FP8 caches (as paged_attn_decode_fp8; head_dim 128 or 256)."""
    import torch

    softcap, window = _softcap(softcap), _int32("window", window)
    _, n, H_q, H_kv, D, maxb, BS, out, dev = _mods_problem(
        q, k8, v8, block_tables, seq_lens, out, alibi_slopes, prefix_lens, doc_starts, workspace,
        torch.uint8)
    _need("k_scale", k_scale, torch.float32, k8.shape[:3])
    _need("v_scale", v_scale, torch.float32, k8.shape[:3])
    _same_device(k_scale, v_scale)
    _check((_lib or load()).paged_attn_decode_fp8_mods(
        q.data_ptr(), k8.data_ptr(), v8.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
        out.data_ptr(), block_tables.data_ptr(), seq_lens.data_ptr(), n, H_q, H_kv, D, maxb, BS,
        float(scale), softcap, _ptr(alibi_slopes), window, _ptr(prefix_lens),
        _ptr(doc_starts), _ptr(workspace), _bytes(workspace), _raw_stream(stream, dev)))
    return out


def paged_attn_mods_workspace_bytes(num_seqs: int, H_q: int, H_kv: int, head_dim: int,
                                    max_blocks_per_seq: int, block_size: int) -> int:
    return int(load().paged_attn_mods_workspace_bytes(num_seqs, H_q, H_kv, head_dim,
                                                      max_blocks_per_seq, block_size))


def paged_attn_decode_multi_mods(q, k_cache, v_cache, qo_indptr, block_tables, seq_lens,
                                 scale: float, *, causal: bool = True, softcap: float = 0.0,
                                 alibi_slopes=None, window: int = 0, prefix_lens=None,
                                 doc_starts=None, out=None, workspace=None, stream=None):
    """Attention of any number of query tokens per sequence with score options (see
    paged_attn.h): q [total_q, H_q, D], sequence s owning rows qo_indptr[s] ..
    qo_indptr[s+1] - 1 (its last tokens, already in the cache); doc_starts is
    [total_q], one per query row; with ``causal=False`` a window or a document bounds the
    view on the left only, later documents are seen; the other options as paged_attn_decode_mods
    (``workspace``: paged_attn_multi_mods_workspace_bytes)."""
    import torch

    softcap, window = _softcap(softcap), _int32("window", window)
    total_q, n, H_q, H_kv, D, maxb, BS, out, dev = _mods_problem(
        q, k_cache, v_cache, block_tables, seq_lens, out, alibi_slopes, prefix_lens, doc_starts,
        workspace, torch.bfloat16, rows="many")
    _need("qo_indptr", qo_indptr, torch.int32, (n + 1,))
    _same_device(qo_indptr)
    _check((_lib or load()).paged_attn_decode_multi_mods(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(),
        qo_indptr.data_ptr(), block_tables.data_ptr(), seq_lens.data_ptr(), n, total_q, H_q, H_kv,
        D, maxb, BS, float(scale), 1 if causal else 0, softcap, _ptr(alibi_slopes),
        window, _ptr(prefix_lens), _ptr(doc_starts), _ptr(workspace), _bytes(workspace),
        _raw_stream(stream, dev)))
    return out


def paged_attn_multi_mods_workspace_bytes(num_seqs: int, total_q: int, H_q: int, H_kv: int,
                                          head_dim: int, max_blocks_per_seq: int,
                                          block_size: int) -> int:
    return int(load().paged_attn_multi_mods_workspace_bytes(num_seqs, total_q, H_q, H_kv,
                                                            head_dim, max_blocks_per_seq,
                                                            block_size))


def paged_attn_decode_shared(q, k_cache, v_cache, group_indptr, prefix_tables, prefix_lens,
                             block_tables, seq_lens, scale: float, *, softcap: float = 0.0,
                             alibi_slopes=None, out=None, workspace=None, stream=None):
    """Decode of sequences that share prefixes, each prefix read once (see paged_attn.h):
    sequences group_indptr[g] .. group_indptr[g+1] - 1 begin with the prefix_lens[g]
    tokens of prefix_tables[g] (int32 [num_groups, prefix_max_blocks]); block_tables and
    seq_lens are those of the sequences' own tokens.  ``workspace``: as
    paged_attn_decode_mods, of paged_attn_shared_workspace_bytes."""
    import torch

    softcap = _softcap(softcap)
    _, n, H_q, H_kv, D, maxb, BS, out, dev = _mods_problem(
        q, k_cache, v_cache, block_tables, seq_lens, out, alibi_slopes, None, None, workspace,
        torch.bfloat16)
    if prefix_tables.dim() != 2:
        raise ValueError("prefix_tables must be [num_groups, prefix_max_blocks]")
    groups, pmax = prefix_tables.shape
    _need("prefix_tables", prefix_tables, torch.int32, (groups, pmax))
    _need("prefix_lens", prefix_lens, torch.int32, (groups,))
    _need("group_indptr", group_indptr, torch.int32, (groups + 1,))
    _same_device(prefix_tables, prefix_lens, group_indptr)
    _check((_lib or load()).paged_attn_decode_shared(
        q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), out.data_ptr(),
        group_indptr.data_ptr(), prefix_tables.data_ptr(), prefix_lens.data_ptr(), groups, pmax,
        block_tables.data_ptr(), seq_lens.data_ptr(), n, H_q, H_kv, D, maxb, BS, float(scale),
        softcap, _ptr(alibi_slopes), _ptr(workspace), _bytes(workspace),
        _raw_stream(stream, dev)))
    return out


def paged_attn_shared_workspace_bytes(num_seqs: int, num_groups: int, H_q: int, H_kv: int,
                                      head_dim: int, max_blocks_per_seq: int,
                                      block_size: int) -> int:
    return int(load().paged_attn_shared_workspace_bytes(num_seqs, num_groups, H_q, H_kv, head_dim,
                                                        max_blocks_per_seq, block_size))


def paged_kv_assign(seq_lens, new_lens, block_tables, free_blocks, free_count, block_size: int,
                    max_new: int, *, seq_lens_out=None, qo_indptr=None, slot_map=None,
                    free_count_out=None, refused=None, stream=None):
    """Block tables, query offsets and the slot map of a serving step from request
    lengths (see paged_attn.h).  seq_lens, new_lens: int32 [num_seqs]; block_tables:
    int32 [num_seqs, max_blocks], whose entries of fresh pages are written;
    free_blocks: int32, a stack whose top is at free_count[0] - 1; max_new: rows of
    the slot map, at least the sum of new_lens.  Returns (seq_lens_out, qo_indptr,
    slot_map, free_count_out), made here unless passed; seq_lens_out may be seq_lens
    and free_count_out free_count, to update them in place.  ``refused``: an int32
    tensor of one element that receives the number of sequences refused."""
    import torch

    block_size, max_new = _int32("block_size", block_size), _int32("max_new", max_new)
    n_free = _int32("free_blocks' length", free_blocks.numel())
    n = seq_lens.shape[0]
    i32 = torch.int32
    _need("seq_lens", seq_lens, i32, (n,))
    _need("new_lens", new_lens, i32, (n,))
    if block_tables.dim() != 2:
        raise ValueError("block_tables must be [num_seqs, max_blocks]")
    _need("block_tables", block_tables, i32, (n, block_tables.shape[1]))
    _need("free_blocks", free_blocks, i32, (free_blocks.numel(),))
    _need("free_count", free_count, i32, (1,))
    where = seq_lens.device
    if seq_lens_out is None:
        seq_lens_out = torch.empty_like(seq_lens)
    else:
        _need("seq_lens_out", seq_lens_out, i32, (n,))
    if qo_indptr is None:
        qo_indptr = torch.empty(n + 1, dtype=i32, device=where)
    else:
        _need("qo_indptr", qo_indptr, i32, (n + 1,))
    if slot_map is None:
        slot_map = torch.empty(max_new, dtype=torch.int64, device=where)
    else:
        _need("slot_map", slot_map, torch.int64, (max_new,))
    if free_count_out is None:
        free_count_out = torch.empty_like(free_count)
    else:
        _need("free_count_out", free_count_out, i32, (1,))
    if refused is not None:
        _need("refused", refused, i32, (1,))
    dev = _same_device(seq_lens, new_lens, block_tables, free_blocks, free_count, seq_lens_out,
                       qo_indptr, slot_map, free_count_out, refused)
    _check((_lib or load()).paged_kv_assign(
        seq_lens.data_ptr(), new_lens.data_ptr(), block_tables.data_ptr(),
        free_blocks.data_ptr(), free_count.data_ptr(), seq_lens_out.data_ptr(),
        qo_indptr.data_ptr(), slot_map.data_ptr(), free_count_out.data_ptr(), _ptr(refused), n,
        block_tables.shape[1], block_size, n_free, max_new,
        _raw_stream(stream, dev)))
    return seq_lens_out, qo_indptr, slot_map, free_count_out


def paged_kv_append_slots(k_new, v_new, k_cache, v_cache, slot_map, stream=None):
    """Write new K and V rows into the paged caches by slot (see paged_attn.h).
    k_new, v_new: bf16 [rows, H_kv, head_dim], each row contiguous, the rows at any
    stride that is a multiple of 8 (slices of a fused projection need no copy);
    slot_map: int64 [rows], block * block_size + place, or -1 to skip the row."""
    import torch

    if k_cache.dim() != 4 or k_new.dim() != 3:
        raise ValueError("k_new must be [rows, H_kv, D], the caches [num_blocks, H_kv, "
                         "block_size, D]")
    nb, H_kv, BS, D = k_cache.shape
    rows = k_new.shape[0]
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        if t.dtype is not torch.bfloat16 or t.shape != (rows, H_kv, D):
            raise ValueError(f"{name} must be bfloat16 [rows, H_kv, head_dim]")
        if rows and (t.stride(2) != 1 or (H_kv > 1 and t.stride(1) != D)):
            raise ValueError(f"the rows of {name} must be contiguous [H_kv, head_dim]")
    _need("k_cache", k_cache, torch.bfloat16, (nb, H_kv, BS, D))
    _need("v_cache", v_cache, torch.bfloat16, (nb, H_kv, BS, D))
    _need("slot_map", slot_map, torch.int64, (rows,))
    dev = _same_device(k_new, v_new, k_cache, v_cache, slot_map)
    row = H_kv * D
    _check((_lib or load()).paged_kv_append_slots(
        k_new.data_ptr(), v_new.data_ptr(), k_new.stride(0) if rows > 1 else row,
        v_new.stride(0) if rows > 1 else row, k_cache.data_ptr(), v_cache.data_ptr(),
        slot_map.data_ptr(), rows, H_kv, D, BS, nb, _raw_stream(stream, dev)))

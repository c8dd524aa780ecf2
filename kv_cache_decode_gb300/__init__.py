"""Single-token decode attention over a KV cache on GB300 (sm_103a).

Thin ctypes binding over ``libkvdecode.so`` (C ABI declared in
``include/kvdecode.h``). Every step of the path runs in the library's CUDA
kernels; this module only checks tensor metadata and marshals pointers and
sizes. PyTorch supplies device memory and streams. There is no CPU fallback:
if the library is missing or stale, loading fails with an error.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import Optional, Tuple

import numpy as np

from . import roofline  # noqa: F401  (host-side byte model)

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkvdecode.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE_TOO_SMALL, ERR_CUDA = range(5)
OUT_BF16, OUT_F32 = 0, 1
STATUS_SEQ_LEN_CLAMPED = 0x1
STATUS_POS_OUT_OF_RANGE = 0x2
STATUS_BAD_PAGE = 0x8
STATUS_UMAX_FALLBACK = 0x10

# Every symbol include/kvdecode.h declares.
EXPORTED = (
    "kvd_decode_plan", "kvd_kv_append", "kvd_decode_attention", "kvd_split_kv_chunk",
    "kvd_split_kv_merge", "kvd_schedule_describe", "kvd_kernel_info", "kvd_status_string",
    "kvd_version", "kvd_decode_attention_static", "kvd_decode_step", "kvd_kv_append_paged",
    "kvd_decode_attention_paged", "kvd_decode_step_paged", "kvd_kv_quantize_q8", "kvd_kv_append_q8",
    "kvd_decode_attention_q8", "kvd_decode_step_q8", "kvd_decode_plan_multi", "kvd_kv_append_multi",
    "kvd_decode_attention_multi", "kvd_decode_step_multi", "kvd_decode_ex", "kvd_kv_append_q8_paged",
    "kvd_decode_attention_umax", "kvd_decode_step_umax", "kvd_step_staging_bytes", "kvd_decode_step_host",
    "kvd_kv_quantize_fp8", "kvd_kv_append_fp8", "kvd_kv_append_fp8_paged", "kvd_merge_attention",
    "kvd_probe_read", "kvd_rope_table", "kvd_rope_apply", "kvd_kv_append_rope", "kvd_fp4_block_bytes",
    "kvd_kv_quantize_fp4", "kvd_kv_read_fp4", "kvd_kv_append_fp4", "kvd_decode_plan_fp4", "kvd_decode_fp4",
)
STATIC_WORKSPACE_BYTES = 16 << 20  # KVD_STATIC_WORKSPACE_BYTES

_lock = threading.Lock()
_lib = None


class KvdError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


def load(path: str = LIB_PATH):
    """Load libkvdecode.so. Raises if it has not been built (no fallback)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with `python -m kv_cache_decode_gb300._build` "
                "(or __graft_entry__.build()); there is no CPU fallback")
        from . import _build
        if path == LIB_PATH and not _build.up_to_date():
            raise RuntimeError(f"{path} is older than its sources: rebuild it")
        _lib = _declare(ctypes.CDLL(path))
        return _lib


class _CCache(ctypes.Structure):
    """struct kvd_cache of kvdecode.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("block_table", ctypes.c_void_p), ("s_max", ctypes.c_int),
                ("max_blocks", ctypes.c_int), ("page_size", ctypes.c_int), ("num_pages", ctypes.c_int),
                ("fp8", ctypes.c_int)]


class _CRope(ctypes.Structure):
    """struct kvd_rope of kvdecode.h."""
    _fields_ = [("turns", ctypes.c_void_p), ("factor", ctypes.c_float), ("rotary_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int)]


class _CCacheFp4(ctypes.Structure):
    """struct kvd_cache_fp4 of kvdecode.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("s_max", ctypes.c_int), ("max_blocks", ctypes.c_int), ("page_size", ctypes.c_int),
                ("num_pages", ctypes.c_int)]


def _declare(lib):
    P, I, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    PI, PSZ = ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_size_t)
    lib.kvd_decode_plan.argtypes = [I, I, I, I, I, I, I, I, PI, PSZ]
    lib.kvd_kv_append.argtypes = [P, P, P, P, P, I, I, I, I, P, P]
    dec = [P, P, P, P, I, I, I, I, I, I, F, I, P, SZ, P, I, P, P, P]
    for name in ("kvd_decode_attention", "kvd_split_kv_chunk", "kvd_split_kv_merge"):
        getattr(lib, name).argtypes = dec
    lib.kvd_decode_attention_static.argtypes = [P, P, P, P, I, I, I, I, I, I, F, I, P, I, P, P, P]
    lib.kvd_decode_attention_static.restype = I
    # append arguments (k_cache, v_cache, k_new, v_new, pos), then q, seq_lens and the rest
    lib.kvd_decode_step.argtypes = [P, P, P, P, P, P, P] + dec[4:]
    lib.kvd_decode_step.restype = I
    # paged: the cache becomes (pool, block_table) and s_max becomes (max_blocks, page_size, num_pages)
    lib.kvd_kv_append_paged.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, P, P]
    lib.kvd_kv_append_paged.restype = I
    dec_paged = [P, P, P, P, P, I, I, I, I] + dec[6:]
    lib.kvd_decode_attention_paged.argtypes = dec_paged
    lib.kvd_decode_attention_paged.restype = I
    lib.kvd_decode_step_paged.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I] + dec[6:]
    lib.kvd_decode_step_paged.restype = I
    # int8: codes in place of the cache, plus the two scale arrays
    lib.kvd_kv_quantize_q8.argtypes = [P, P, P, P, I, I, I, I, I, P]
    lib.kvd_kv_quantize_q8.restype = I
    lib.kvd_kv_append_q8.argtypes = [P, P, P, P, P, P, P, I, I, I, I, P, P]
    lib.kvd_kv_append_q8.restype = I
    lib.kvd_kv_append_q8_paged.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, P, P]
    lib.kvd_kv_quantize_fp8.argtypes = lib.kvd_kv_quantize_q8.argtypes
    lib.kvd_kv_quantize_fp8.restype = I
    lib.kvd_kv_append_fp8.argtypes = lib.kvd_kv_append_q8.argtypes
    lib.kvd_kv_append_fp8.restype = I
    lib.kvd_kv_append_fp8_paged.argtypes = lib.kvd_kv_append_q8_paged.argtypes
    lib.kvd_kv_append_fp8_paged.restype = I
    lib.kvd_kv_append_q8_paged.restype = I
    # unified maximum: decode_attention / decode_step with phi after scale
    lib.kvd_decode_attention_umax.argtypes = dec[:11] + [F] + dec[11:]
    lib.kvd_decode_attention_umax.restype = I
    lib.kvd_decode_step_umax.argtypes = [P, P, P, P, P, P, P] + dec[4:11] + [F] + dec[11:]
    lib.kvd_decode_step_umax.restype = I
    lib.kvd_merge_attention.argtypes = [P, P, I, ctypes.c_longlong, I, I, P, I, P, P]
    lib.kvd_merge_attention.restype = I
    lib.kvd_probe_read.argtypes = [P, SZ, I, P, P, P]
    lib.kvd_probe_read.restype = I
    lib.kvd_step_staging_bytes.argtypes = [I, I, I, I, I]
    lib.kvd_step_staging_bytes.restype = SZ
    lib.kvd_decode_step_host.argtypes = [P, P, P, P, P, P, P, P, SZ, I, I, I, I, I, I, I, F, I, P, SZ, P, P, I, P,
                                         P, P]
    lib.kvd_decode_step_host.restype = I
    lib.kvd_decode_attention_q8.argtypes = [P, P, P, P, P] + dec[3:]
    lib.kvd_decode_attention_q8.restype = I
    lib.kvd_decode_step_q8.argtypes = [P, P, P, P, P, P, P, P, P] + dec[4:]
    lib.kvd_decode_step_q8.restype = I
    # multi-token: n_tokens after batch
    lib.kvd_decode_plan_multi.argtypes = [I, I, I, I, I, I, I, I, I, PI, PSZ]
    lib.kvd_decode_plan_multi.restype = I
    lib.kvd_kv_append_multi.argtypes = [P, P, P, P, P, I, I, I, I, I, P, P]
    lib.kvd_kv_append_multi.restype = I
    lib.kvd_decode_attention_multi.argtypes = dec[:5] + [I] + dec[5:]
    lib.kvd_decode_attention_multi.restype = I
    lib.kvd_decode_step_multi.argtypes = [P, P, P, P, P, P, P, I, I] + dec[5:]
    lib.kvd_decode_step_multi.restype = I
    lib.kvd_decode_ex.argtypes = [ctypes.POINTER(_CCache), P, P, I, I, I, I, I, I, F, I, P, SZ, P, I, P, P, P, P,
                                  P, P]
    lib.kvd_decode_ex.restype = I
    # rotary positions, rotating appends, fp4 cache
    # (structs are passed as references, or as bytes packed in their layout)
    LL, DBL, PROPE = ctypes.c_longlong, ctypes.c_double, P
    lib.kvd_rope_table.argtypes = [I, DBL, I, DBL, DBL, DBL, DBL, DBL, P, ctypes.POINTER(F)]
    lib.kvd_rope_apply.argtypes = [PROPE, P, LL, I, P, LL, I, P, LL, I, I, P]
    app = [PROPE, P, LL, P, LL, P, LL, P, LL, P, P, I, LL, I, I, I, P, P]
    lib.kvd_kv_append_rope.argtypes = [P] + app
    lib.kvd_kv_append_fp4.argtypes = [P] + app
    lib.kvd_fp4_block_bytes.argtypes = [I]
    lib.kvd_fp4_block_bytes.restype = SZ
    lib.kvd_kv_quantize_fp4.argtypes = [P, P, P, I, I, I, I, I, I, P]
    lib.kvd_kv_read_fp4.argtypes = [P, P, I, I, I, I, P, I, P, I, I, I, I, P, P]
    lib.kvd_decode_plan_fp4.argtypes = [I, I, I, I, I, I, I, I, PI, PSZ]
    lib.kvd_decode_fp4.argtypes = [P] + lib.kvd_decode_ex.argtypes[1:]
    for name in ("kvd_rope_table", "kvd_rope_apply", "kvd_kv_append_rope", "kvd_kv_append_fp4",
                 "kvd_kv_quantize_fp4", "kvd_kv_read_fp4", "kvd_decode_plan_fp4", "kvd_decode_fp4"):
        getattr(lib, name).restype = I
    lib.kvd_schedule_describe.argtypes = [P, I, I, I, I, I, I, I, I, P, I, PI, PI]
    lib.kvd_kernel_info.argtypes = [I, I, I, I, PI, PI, PI, PI, PI, PI]
    lib.kvd_status_string.argtypes = [I]
    lib.kvd_status_string.restype = ctypes.c_char_p
    lib.kvd_version.argtypes = []
    lib.kvd_version.restype = ctypes.c_char_p
    for name in EXPORTED[:7]:
        getattr(lib, name).restype = I
    return lib


def status_string(status: int) -> str:
    try:
        return load().kvd_status_string(int(status)).decode()
    except Exception:  # pragma: no cover - library missing
        return "status"


def version() -> str:
    return load().kvd_version().decode()


def _out_code(out_dtype) -> int:
    if out_dtype in (OUT_BF16, "bf16", "bfloat16"):
        return OUT_BF16
    if out_dtype in (OUT_F32, "f32", "float32", "fp32"):
        return OUT_F32
    import torch
    if out_dtype is torch.bfloat16:
        return OUT_BF16
    if out_dtype is torch.float32:
        return OUT_F32
    raise ValueError(f"unknown out_dtype {out_dtype!r}")


def _check(rc: int, what: str):
    if rc != OK:
        raise KvdError(rc, what)


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream_handle(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    h = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return h or None


# ---------------------------------------------------------------------------
# Host-only queries
# ---------------------------------------------------------------------------

def decode_plan(batch: int, n_heads_q: int, n_heads_kv: int, head_dim: int, max_seq_len: int,
                num_sms: int = 0, n_split: int = 0, out_dtype="bf16") -> Tuple[int, int]:
    """(n_split, workspace_bytes) for a decode_attention call of this shape."""
    lib = load()
    n = ctypes.c_int(0)
    ws = ctypes.c_size_t(0)
    _check(lib.kvd_decode_plan(batch, n_heads_q, n_heads_kv, head_dim, max_seq_len, num_sms,
                               n_split, _out_code(out_dtype), ctypes.byref(n), ctypes.byref(ws)),
           "kvd_decode_plan")
    return n.value, ws.value


def kernel_info(n_heads_q: int, n_heads_kv: int, head_dim: int, out_dtype="bf16") -> dict:
    lib = load()
    th, sm, tt, cps, su, sc = (ctypes.c_int(0) for _ in range(6))
    _check(lib.kvd_kernel_info(n_heads_q, n_heads_kv, head_dim, _out_code(out_dtype),
                               ctypes.byref(th), ctypes.byref(sm), ctypes.byref(tt),
                               ctypes.byref(cps), ctypes.byref(su), ctypes.byref(sc)),
           "kvd_kernel_info")
    return {"threads": th.value, "smem_bytes": sm.value, "tile_tokens": tt.value,
            "ctas_per_sm": cps.value, "seg_unit": su.value, "seg_cost": sc.value}


def schedule_describe(seq_lens, s_max: int, max_seq_len: int, n_heads_q: int, n_heads_kv: int,
                      head_dim: int, n_split: int, out_dtype="bf16"):
    """Host replica of the device schedule: (rows [n, 8] int32, n_split_eff).

    Row = (cta, b, h, tok_lo, tok_hi, kind, slot, c_last); kind 0 final,
    1 partial by owner, 2 partial by another CTA, 3 empty pair.
    """
    lib = load()
    lens = np.ascontiguousarray(seq_lens, dtype=np.int32)
    n_rows = ctypes.c_int(0)
    eff = ctypes.c_int(0)
    args = [lens.ctypes.data_as(ctypes.c_void_p), int(lens.size), s_max, max_seq_len, n_heads_q,
            n_heads_kv, head_dim, n_split, _out_code(out_dtype)]
    _check(lib.kvd_schedule_describe(*args, None, 0, ctypes.byref(n_rows), ctypes.byref(eff)),
           "kvd_schedule_describe")
    rows = np.zeros((max(n_rows.value, 1), 8), dtype=np.int32)
    _check(lib.kvd_schedule_describe(*args, rows.ctypes.data_as(ctypes.c_void_p), n_rows.value,
                                     ctypes.byref(n_rows), ctypes.byref(eff)),
           "kvd_schedule_describe")
    return rows[:n_rows.value], eff.value


# ---------------------------------------------------------------------------
# GPU entry points (torch CUDA tensors in, results written in place)
# ---------------------------------------------------------------------------

def _require(t, name, dtype=None, ndim=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


def kv_append(k_cache, v_cache, k_new, v_new, pos, status=None, stream=None):
    """k_cache[b, pos[b], h, :] = k_new[b, h, :] (and V), on the GPU."""
    import torch
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _require(t, n, torch.bfloat16, 4)
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        _require(t, n, torch.bfloat16, 3)
    _require(pos, "pos", torch.int32, 1)
    B, S, Hkv, D = k_cache.shape
    if v_cache.shape != k_cache.shape or k_new.shape != (B, Hkv, D) or v_new.shape != (B, Hkv, D) \
            or pos.shape != (B,):
        raise ValueError("kv_append: inconsistent shapes")
    _check(load().kvd_kv_append(k_cache.data_ptr(), v_cache.data_ptr(), k_new.data_ptr(),
                                v_new.data_ptr(), pos.data_ptr(), B, S, Hkv, D, _ptr(status),
                                _stream_handle(stream)), "kvd_kv_append")


def _decode_args(q, k_cache, v_cache, seq_lens, max_seq_len, scale, n_split, workspace, out,
                 lse, status, stream):
    import torch
    _require(q, "q", torch.bfloat16, 3)
    _require(k_cache, "k_cache", torch.bfloat16, 4)
    _require(v_cache, "v_cache", torch.bfloat16, 4)
    _require(seq_lens, "seq_lens", torch.int32, 1)
    _require(out, "out", None, 3)
    B, Hq, D = q.shape
    _, S, Hkv, Dk = k_cache.shape
    if k_cache.shape[0] != B or Dk != D or v_cache.shape != k_cache.shape or \
            seq_lens.shape != (B,) or out.shape != (B, Hq, D):
        raise ValueError("decode_attention: inconsistent shapes")
    if out.dtype == torch.bfloat16:
        code = OUT_BF16
    elif out.dtype == torch.float32:
        code = OUT_F32
    else:
        raise TypeError("out must be bfloat16 or float32")
    if lse is not None:
        _require(lse, "lse", torch.float32, 2)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(),
                                                           workspace.numel() * workspace.element_size())
    return [q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), seq_lens.data_ptr(), B, S,
            int(max_seq_len), Hq, Hkv, D, float(scale), int(n_split), ws_ptr, ws_bytes,
            out.data_ptr(), code, _ptr(lse), _ptr(status), _stream_handle(stream)]


def alloc_workspace(q, k_cache, max_seq_len: int, n_split: int = 0, out_dtype="bf16"):
    """A device workspace big enough for decode_attention with these arguments."""
    import torch
    B, Hq, D = q.shape
    Hkv = k_cache.shape[2]
    with torch.cuda.device(q.device):
        _, nbytes = decode_plan(B, Hq, Hkv, D, max_seq_len, 0, n_split, out_dtype)
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=q.device)


def decode_attention(q, k_cache, v_cache, seq_lens, max_seq_len: int, scale: float, out,
                     workspace=None, n_split: int = 0, lse=None, status=None, stream=None):
    """out[b, h] = softmax(scale * q[b, h] . K[b, :L_b, h // G]) V[b, :L_b, h // G]."""
    args = _decode_args(q, k_cache, v_cache, seq_lens, max_seq_len, scale, n_split, workspace,
                        out, lse, status, stream)
    _check(load().kvd_decode_attention(*args), "kvd_decode_attention")


def decode_attention_static(q, k_cache, v_cache, seq_lens, max_seq_len: int, scale: float, out,
                            n_split: int = 0, lse=None, status=None, stream=None):
    """decode_attention using the library's own static scratch array (no workspace
    argument, nothing allocated). Calls that overlap on the GPU share that array."""
    a = _decode_args(q, k_cache, v_cache, seq_lens, max_seq_len, scale, n_split, None, out, lse,
                     status, stream)
    args = a[:12] + a[14:]  # drop workspace pointer and size
    _check(load().kvd_decode_attention_static(*args), "kvd_decode_attention_static")


def _paged_args(k_pages, v_pages, block_table, B, what):
    import torch
    _require(k_pages, "k_pages", torch.bfloat16, 4)
    _require(v_pages, "v_pages", torch.bfloat16, 4)
    _require(block_table, "block_table", torch.int32, 2)
    num_pages, page, Hkv, D = k_pages.shape
    if v_pages.shape != k_pages.shape or block_table.shape[0] != B:
        raise ValueError(f"{what}: inconsistent shapes")
    return block_table.shape[1], page, num_pages, Hkv, D


def kv_append_paged(k_pages, v_pages, k_new, v_new, block_table, pos, status=None, stream=None):
    """Paged kv_append: the new rows go to row pos[b] % page of page
    block_table[b, pos[b] // page] of the pools [num_pages, page, Hkv, D]."""
    import torch
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        _require(t, n, torch.bfloat16, 3)
    _require(pos, "pos", torch.int32, 1)
    B = k_new.shape[0]
    max_blocks, page, num_pages, Hkv, D = _paged_args(k_pages, v_pages, block_table, B, "kv_append_paged")
    if k_new.shape != (B, Hkv, D) or v_new.shape != (B, Hkv, D) or pos.shape != (B,):
        raise ValueError("kv_append_paged: inconsistent shapes")
    _check(load().kvd_kv_append_paged(k_pages.data_ptr(), v_pages.data_ptr(), k_new.data_ptr(),
                                      v_new.data_ptr(), block_table.data_ptr(), pos.data_ptr(), B,
                                      max_blocks, page, num_pages, Hkv, D, _ptr(status),
                                      _stream_handle(stream)), "kvd_kv_append_paged")


def _decode_paged_args(q, k_pages, v_pages, block_table, seq_lens, max_seq_len, scale, n_split,
                       workspace, out, lse, status, stream):
    B = q.shape[0]
    max_blocks, page, num_pages, _, _ = _paged_args(k_pages, v_pages, block_table, B, "decode_attention_paged")
    import torch
    _require(q, "q", torch.bfloat16, 3)
    _require(seq_lens, "seq_lens", torch.int32, 1)
    _require(out, "out", None, 3)
    _, Hq, D = q.shape
    Hkv = k_pages.shape[2]
    if k_pages.shape[3] != D or seq_lens.shape != (B,) or out.shape != (B, Hq, D):
        raise ValueError("decode_attention_paged: inconsistent shapes")
    if out.dtype == torch.bfloat16:
        code = OUT_BF16
    elif out.dtype == torch.float32:
        code = OUT_F32
    else:
        raise TypeError("out must be bfloat16 or float32")
    if lse is not None:
        _require(lse, "lse", torch.float32, 2)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(),
                                                           workspace.numel() * workspace.element_size())
    head = [B, max_blocks, page, num_pages]
    tail = [int(max_seq_len), Hq, Hkv, D, float(scale), int(n_split), ws_ptr, ws_bytes, out.data_ptr(),
            code, _ptr(lse), _ptr(status), _stream_handle(stream)]
    return head, tail


def decode_attention_paged(q, k_pages, v_pages, block_table, seq_lens, max_seq_len: int, scale: float,
                           out, workspace=None, n_split: int = 0, lse=None, status=None, stream=None):
    """decode_attention over a paged cache: pools [num_pages, page, Hkv, D] and
    block_table [B, max_blocks] (token t of sequence b is row t % page of page
    block_table[b, t // page]). Workspace as for decode_attention."""
    head, tail = _decode_paged_args(q, k_pages, v_pages, block_table, seq_lens, max_seq_len, scale,
                                    n_split, workspace, out, lse, status, stream)
    _check(load().kvd_decode_attention_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                             block_table.data_ptr(), seq_lens.data_ptr(), *head, *tail),
           "kvd_decode_attention_paged")


def decode_step_paged(q, k_pages, v_pages, k_new, v_new, pos, block_table, seq_lens, max_seq_len: int,
                      scale: float, out, workspace=None, n_split: int = 0, lse=None, status=None,
                      stream=None):
    """kv_append_paged then decode_attention_paged as one call (kvd_decode_step_paged)."""
    import torch
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        _require(t, n, torch.bfloat16, 3)
    _require(pos, "pos", torch.int32, 1)
    B = q.shape[0]
    Hkv, D = k_pages.shape[2], k_pages.shape[3]
    if k_new.shape != (B, Hkv, D) or v_new.shape != (B, Hkv, D) or pos.shape != (B,):
        raise ValueError("decode_step_paged: inconsistent shapes")
    head, tail = _decode_paged_args(q, k_pages, v_pages, block_table, seq_lens, max_seq_len, scale,
                                    n_split, workspace, out, lse, status, stream)
    _check(load().kvd_decode_step_paged(k_pages.data_ptr(), v_pages.data_ptr(), k_new.data_ptr(),
                                        v_new.data_ptr(), pos.data_ptr(), q.data_ptr(),
                                        block_table.data_ptr(), seq_lens.data_ptr(), *head, *tail),
           "kvd_decode_step_paged")


def _code_dtypes(fmt):
    """Tensor dtypes an 8-bit cache's codes may have: int8, or for fp8 E4M3
    bytes (uint8) or torch's float8_e4m3fn (the same bits)."""
    import torch
    if fmt == "int8":
        return (torch.int8,)
    if fmt == "fp8":
        return (torch.uint8, torch.float8_e4m3fn)
    raise ValueError(f"unknown 8-bit cache format {fmt!r}")


def _is_fp8(codes) -> bool:
    import torch
    return codes.dtype in (torch.uint8, torch.float8_e4m3fn)


def _q8_args(k_codes, v_codes, k_scales, v_scales, fmt="int8"):
    import torch
    _require(k_codes, "k_codes", _code_dtypes(fmt), 4)
    _require(v_codes, "v_codes", _code_dtypes(fmt), 4)
    _require(k_scales, "k_scales", torch.float32, 3)
    _require(v_scales, "v_scales", torch.float32, 3)
    if v_codes.shape != k_codes.shape or k_scales.shape != k_codes.shape[:3] or v_scales.shape != k_scales.shape:
        raise ValueError(f"{fmt} cache: codes [B, S_max, Hkv, D] and scales [B, S_max, Hkv] disagree")


def _quantize8(cache, codes, scales, seq_lens, max_seq_len, stream, fmt):
    import torch
    _require(cache, "cache", torch.bfloat16, 4)
    _require(codes, "codes", _code_dtypes(fmt), 4)
    _require(scales, "scales", torch.float32, 3)
    _require(seq_lens, "seq_lens", torch.int32, 1)
    B, S, Hkv, D = cache.shape
    if codes.shape != cache.shape or scales.shape != (B, S, Hkv) or seq_lens.shape != (B,):
        raise ValueError(f"kv_quantize_{fmt}: inconsistent shapes")
    name = "kvd_kv_quantize_q8" if fmt == "int8" else "kvd_kv_quantize_fp8"
    _check(getattr(load(), name)(cache.data_ptr(), codes.data_ptr(), scales.data_ptr(), seq_lens.data_ptr(), B, S,
                                 int(max_seq_len), Hkv, D, _stream_handle(stream)), name)


def kv_quantize_q8(cache, codes, scales, seq_lens, max_seq_len: int, stream=None):
    """int8 codes/scales of rows t < seq_lens[b] of a bf16 cache [B, S_max, Hkv, D]."""
    _quantize8(cache, codes, scales, seq_lens, max_seq_len, stream, "int8")


def kv_quantize_fp8(cache, codes, scales, seq_lens, max_seq_len: int, stream=None):
    """fp8 E4M3 codes (uint8 or float8_e4m3fn) and scales of rows t < seq_lens[b]
    of a bf16 cache [B, S_max, Hkv, D] (kvd_kv_quantize_fp8)."""
    _quantize8(cache, codes, scales, seq_lens, max_seq_len, stream, "fp8")


def _append8(k_codes, v_codes, k_scales, v_scales, k_new, v_new, pos, status, stream, fmt):
    import torch
    _q8_args(k_codes, v_codes, k_scales, v_scales, fmt)
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        _require(t, n, torch.bfloat16, 3)
    _require(pos, "pos", torch.int32, 1)
    B, S, Hkv, D = k_codes.shape
    if k_new.shape != (B, Hkv, D) or v_new.shape != (B, Hkv, D) or pos.shape != (B,):
        raise ValueError(f"kv_append_{fmt}: inconsistent shapes")
    name = "kvd_kv_append_q8" if fmt == "int8" else "kvd_kv_append_fp8"
    _check(getattr(load(), name)(k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                                 k_new.data_ptr(), v_new.data_ptr(), pos.data_ptr(), B, S, Hkv, D, _ptr(status),
                                 _stream_handle(stream)), name)


def kv_append_q8(k_codes, v_codes, k_scales, v_scales, k_new, v_new, pos, status=None, stream=None):
    """The new bf16 rows quantized and written at pos[b] of the int8 cache."""
    _append8(k_codes, v_codes, k_scales, v_scales, k_new, v_new, pos, status, stream, "int8")


def kv_append_fp8(k_codes, v_codes, k_scales, v_scales, k_new, v_new, pos, status=None, stream=None):
    """The new bf16 rows quantized to fp8 E4M3 and written at pos[b] (kvd_kv_append_fp8)."""
    _append8(k_codes, v_codes, k_scales, v_scales, k_new, v_new, pos, status, stream, "fp8")


def _append8_paged(k_code_pages, v_code_pages, k_scale_pages, v_scale_pages, k_new, v_new, block_table, pos,
                   status, stream, fmt):
    import torch
    _q8_args(k_code_pages, v_code_pages, k_scale_pages, v_scale_pages, fmt)
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        _require(t, n, torch.bfloat16, 3)
    _require(pos, "pos", torch.int32, 1)
    _require(block_table, "block_table", torch.int32, 2)
    num_pages, page, Hkv, D = k_code_pages.shape
    B = k_new.shape[0]
    if (k_new.shape != (B, Hkv, D) or v_new.shape != (B, Hkv, D) or pos.shape != (B,)
            or block_table.shape[0] != B):
        raise ValueError(f"kv_append_{fmt}_paged: inconsistent shapes")
    name = "kvd_kv_append_q8_paged" if fmt == "int8" else "kvd_kv_append_fp8_paged"
    _check(getattr(load(), name)(k_code_pages.data_ptr(), v_code_pages.data_ptr(), k_scale_pages.data_ptr(),
                                 v_scale_pages.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), block_table.data_ptr(),
                                 pos.data_ptr(), B, block_table.shape[1], page, num_pages, Hkv, D, _ptr(status),
                                 _stream_handle(stream)), name)


def kv_append_q8_paged(k_code_pages, v_code_pages, k_scale_pages, v_scale_pages, k_new, v_new, block_table, pos,
                       status=None, stream=None):
    """The new bf16 rows quantized and written, as kv_append_paged places them,
    into int8 page pools: codes [num_pages, page, Hkv, D], scales
    [num_pages, page, Hkv]."""
    _append8_paged(k_code_pages, v_code_pages, k_scale_pages, v_scale_pages, k_new, v_new, block_table, pos,
                   status, stream, "int8")


def kv_append_fp8_paged(k_code_pages, v_code_pages, k_scale_pages, v_scale_pages, k_new, v_new, block_table, pos,
                        status=None, stream=None):
    """kv_append_q8_paged for fp8 E4M3 page pools (kvd_kv_append_fp8_paged)."""
    _append8_paged(k_code_pages, v_code_pages, k_scale_pages, v_scale_pages, k_new, v_new, block_table, pos,
                   status, stream, "fp8")


def _decode_q8_args(q, k_codes, v_codes, k_scales, v_scales, seq_lens, max_seq_len, scale, n_split, workspace,
                    out, lse, status, stream):
    """(seq_lens pointer, batch, s_max, ...) as for kvd_decode_attention, after the int8 cache."""
    import torch
    _q8_args(k_codes, v_codes, k_scales, v_scales)
    _require(q, "q", torch.bfloat16, 3)
    _require(seq_lens, "seq_lens", torch.int32, 1)
    _require(out, "out", None, 3)
    B, Hq, D = q.shape
    _, S, Hkv, Dk = k_codes.shape
    if k_codes.shape[0] != B or Dk != D or seq_lens.shape != (B,) or out.shape != (B, Hq, D):
        raise ValueError("decode_attention_q8: inconsistent shapes")
    if out.dtype == torch.bfloat16:
        code = OUT_BF16
    elif out.dtype == torch.float32:
        code = OUT_F32
    else:
        raise TypeError("out must be bfloat16 or float32")
    if lse is not None:
        _require(lse, "lse", torch.float32, 2)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(),
                                                           workspace.numel() * workspace.element_size())
    return [seq_lens.data_ptr(), B, S, int(max_seq_len), Hq, Hkv, D, float(scale), int(n_split), ws_ptr, ws_bytes,
            out.data_ptr(), code, _ptr(lse), _ptr(status), _stream_handle(stream)]


def decode_attention_q8(q, k_codes, v_codes, k_scales, v_scales, seq_lens, max_seq_len: int, scale: float, out,
                        workspace=None, n_split: int = 0, lse=None, status=None, stream=None):
    """decode_attention over an int8 cache (codes [B, S_max, Hkv, D] int8, scales
    [B, S_max, Hkv] float32; a row reads back as scale * code). Any group."""
    tail = _decode_q8_args(q, k_codes, v_codes, k_scales, v_scales, seq_lens, max_seq_len, scale, n_split,
                           workspace, out, lse, status, stream)
    _check(load().kvd_decode_attention_q8(q.data_ptr(), k_codes.data_ptr(), v_codes.data_ptr(),
                                          k_scales.data_ptr(), v_scales.data_ptr(), *tail),
           "kvd_decode_attention_q8")


def decode_step_q8(q, k_codes, v_codes, k_scales, v_scales, k_new, v_new, pos, seq_lens, max_seq_len: int,
                   scale: float, out, workspace=None, n_split: int = 0, lse=None, status=None, stream=None):
    """kv_append_q8 then decode_attention_q8 as one call (kvd_decode_step_q8)."""
    import torch
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        _require(t, n, torch.bfloat16, 3)
    _require(pos, "pos", torch.int32, 1)
    B, S, Hkv, D = k_codes.shape
    if k_new.shape != (B, Hkv, D) or v_new.shape != (B, Hkv, D) or pos.shape != (B,):
        raise ValueError("decode_step_q8: inconsistent shapes")
    tail = _decode_q8_args(q, k_codes, v_codes, k_scales, v_scales, seq_lens, max_seq_len, scale, n_split,
                           workspace, out, lse, status, stream)
    _check(load().kvd_decode_step_q8(k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(),
                                     v_scales.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), pos.data_ptr(),
                                     q.data_ptr(), *tail), "kvd_decode_step_q8")


def decode_plan_multi(batch: int, n_tokens: int, n_heads_q: int, n_heads_kv: int, head_dim: int,
                      max_seq_len: int, num_sms: int = 0, n_split: int = 0, out_dtype="bf16") -> Tuple[int, int]:
    """(n_split, workspace_bytes) for a multi-token call of this shape."""
    lib = load()
    n = ctypes.c_int(0)
    ws = ctypes.c_size_t(0)
    _check(lib.kvd_decode_plan_multi(batch, n_tokens, n_heads_q, n_heads_kv, head_dim, max_seq_len, num_sms,
                                     n_split, _out_code(out_dtype), ctypes.byref(n), ctypes.byref(ws)),
           "kvd_decode_plan_multi")
    return n.value, ws.value


def kv_append_multi(k_cache, v_cache, k_new, v_new, pos, status=None, stream=None):
    """The T new rows of each sequence (k_new [B, T, Hkv, D]) at pos[b] + i."""
    import torch
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _require(t, n, torch.bfloat16, 4)
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        _require(t, n, torch.bfloat16, 4)
    _require(pos, "pos", torch.int32, 1)
    B, S, Hkv, D = k_cache.shape
    T = k_new.shape[1]
    if v_cache.shape != k_cache.shape or k_new.shape != (B, T, Hkv, D) or v_new.shape != k_new.shape \
            or pos.shape != (B,):
        raise ValueError("kv_append_multi: inconsistent shapes")
    _check(load().kvd_kv_append_multi(k_cache.data_ptr(), v_cache.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
                                      pos.data_ptr(), B, T, S, Hkv, D, _ptr(status), _stream_handle(stream)),
           "kvd_kv_append_multi")


def _decode_multi_args(q, k_cache, v_cache, seq_lens, max_seq_len, scale, n_split, workspace, out, lse, status,
                       stream):
    import torch
    _require(q, "q", torch.bfloat16, 4)
    _require(out, "out", None, 4)
    B, T, Hq, D = q.shape
    if out.shape != q.shape:
        raise ValueError("decode_attention_multi: out must be [B, T, Hq, D]")
    if lse is not None:
        _require(lse, "lse", torch.float32, 3)
        if lse.shape != (B, T, Hq):
            raise ValueError("decode_attention_multi: lse must be [B, T, Hq]")
    # the single-token checks on [B, T*Hq, D] views (rows of one sequence are contiguous)
    a = _decode_args(q.view(B, T * Hq, D), k_cache, v_cache, seq_lens, max_seq_len, scale, n_split, workspace,
                     out.view(B, T * Hq, D), None if lse is None else lse.view(B, T * Hq), status, stream)
    a[7] = Hq  # n_heads_q proper
    return a[:5] + [T] + a[5:]


def decode_attention_multi(q, k_cache, v_cache, seq_lens, max_seq_len: int, scale: float, out, workspace=None,
                           n_split: int = 0, lse=None, status=None, stream=None):
    """T query tokens per sequence (q, out [B, T, Hq, D]); token i attends to the
    first seq_lens[b] - T + 1 + i cached tokens. T from 1 to 64."""
    args = _decode_multi_args(q, k_cache, v_cache, seq_lens, max_seq_len, scale, n_split, workspace, out, lse,
                              status, stream)
    _check(load().kvd_decode_attention_multi(*args), "kvd_decode_attention_multi")


def decode_step_multi(q, k_cache, v_cache, k_new, v_new, pos, seq_lens, max_seq_len: int, scale: float, out,
                      workspace=None, n_split: int = 0, lse=None, status=None, stream=None):
    """kv_append_multi then decode_attention_multi as one call (kvd_decode_step_multi)."""
    import torch
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        _require(t, n, torch.bfloat16, 4)
    _require(pos, "pos", torch.int32, 1)
    a = _decode_multi_args(q, k_cache, v_cache, seq_lens, max_seq_len, scale, n_split, workspace, out, lse,
                           status, stream)
    B, T, Hq, D = q.shape
    if k_new.shape != (B, T, k_cache.shape[2], D) or v_new.shape != k_new.shape or pos.shape != (B,):
        raise ValueError("decode_step_multi: inconsistent shapes")
    # (k_cache, v_cache, k_new, v_new, pos, q, seq_lens, batch, T, ...)
    args = [a[1], a[2], k_new.data_ptr(), v_new.data_ptr(), pos.data_ptr(), a[0], a[3], a[4], a[5]] + a[6:]
    _check(load().kvd_decode_step_multi(*args), "kvd_decode_step_multi")


def decode_ex(q, k, v, seq_lens, max_seq_len: int, scale: float, out, *, k_scales=None, v_scales=None,
              block_table=None, k_new=None, v_new=None, pos=None, workspace=None, n_split: int = 0, lse=None,
              status=None, stream=None):
    """Any supported combination in one call (kvd_decode_ex): q [B, Hq, D] or
    [B, T, Hq, D]; k, v a contiguous cache [B, S_max, Hkv, D] (bf16, or 8-bit
    codes with k_scales/v_scales [B, S_max, Hkv]: int8 codes, or fp8 E4M3 codes
    as uint8 or float8_e4m3fn) or, with block_table [B, max_blocks], page pools
    [num_pages, page, Hkv, D] (bf16, or 8-bit codes with scale pools
    [num_pages, page, Hkv]); k_new, v_new ([B, Hkv, D] or [B, T, Hkv, D]) and pos
    to append first. Workspace: decode_plan_multi."""
    import torch
    T = q.shape[1] if q.dim() == 4 else 1
    B, Hq, D = q.shape[0], q.shape[-2], q.shape[-1]
    Hkv = k.shape[2]
    c = _CCache()
    c.k, c.v = k.data_ptr(), v.data_ptr()
    c.k_scales, c.v_scales = _ptr(k_scales), _ptr(v_scales)
    c.fp8 = 1 if (k_scales is not None and _is_fp8(k)) else 0
    if block_table is not None:
        _require(block_table, "block_table", torch.int32, 2)
        c.block_table, c.max_blocks, c.page_size, c.num_pages = (block_table.data_ptr(), block_table.shape[1],
                                                                   k.shape[1], k.shape[0])
    else:
        c.s_max = k.shape[1]
    if out.shape != q.shape or k.shape[3] != D or v.shape != k.shape:
        raise ValueError("decode_ex: inconsistent shapes")
    code = OUT_BF16 if out.dtype == torch.bfloat16 else OUT_F32 if out.dtype == torch.float32 else None
    if code is None:
        raise TypeError("out must be bfloat16 or float32")
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(),
                                                           workspace.numel() * workspace.element_size())
    _check(load().kvd_decode_ex(ctypes.byref(c), q.data_ptr(), seq_lens.data_ptr(), B, T, int(max_seq_len), Hq,
                                Hkv, D, float(scale), int(n_split), ws_ptr, ws_bytes, out.data_ptr(), code,
                                _ptr(lse), _ptr(k_new), _ptr(v_new), _ptr(pos), _ptr(status),
                                _stream_handle(stream)), "kvd_decode_ex")


def decode_step(q, k_cache, v_cache, k_new, v_new, pos, seq_lens, max_seq_len: int, scale: float,
                out, workspace=None, n_split: int = 0, lse=None, status=None, stream=None):
    """kv_append(k_cache, v_cache, k_new, v_new, pos) then decode_attention(...), as one
    call whose attention launch starts while the append runs (kvd_decode_step)."""
    import torch
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        _require(t, n, torch.bfloat16, 3)
    _require(pos, "pos", torch.int32, 1)
    B, S, Hkv, D = k_cache.shape
    if k_new.shape != (B, Hkv, D) or v_new.shape != (B, Hkv, D) or pos.shape != (B,):
        raise ValueError("decode_step: inconsistent shapes")
    a = _decode_args(q, k_cache, v_cache, seq_lens, max_seq_len, scale, n_split, workspace, out,
                     lse, status, stream)
    args = [a[1], a[2], k_new.data_ptr(), v_new.data_ptr(), pos.data_ptr(), a[0], a[3]] + a[4:]
    _check(load().kvd_decode_step(*args), "kvd_decode_step")


def decode_attention_umax(q, k_cache, v_cache, seq_lens, max_seq_len: int, scale: float, phi: float, out,
                          workspace=None, n_split: int = 0, lse=None, status=None, stream=None):
    """decode_attention with the unified-maximum softmax: every split's partial
    softmax is taken against phi (logit units) while a row's scores allow,
    so the merge is a plain sum (kvd_decode_attention_umax)."""
    a = _decode_args(q, k_cache, v_cache, seq_lens, max_seq_len, scale, n_split, workspace, out, lse, status,
                     stream)
    _check(load().kvd_decode_attention_umax(*(a[:11] + [float(phi)] + a[11:])), "kvd_decode_attention_umax")


def decode_step_umax(q, k_cache, v_cache, k_new, v_new, pos, seq_lens, max_seq_len: int, scale: float, phi: float,
                     out, workspace=None, n_split: int = 0, lse=None, status=None, stream=None):
    """decode_step with the unified-maximum softmax (kvd_decode_step_umax)."""
    import torch
    for t, n in ((k_new, "k_new"), (v_new, "v_new")):
        _require(t, n, torch.bfloat16, 3)
    _require(pos, "pos", torch.int32, 1)
    B, S, Hkv, D = k_cache.shape
    if k_new.shape != (B, Hkv, D) or v_new.shape != (B, Hkv, D) or pos.shape != (B,):
        raise ValueError("decode_step_umax: inconsistent shapes")
    a = _decode_args(q, k_cache, v_cache, seq_lens, max_seq_len, scale, n_split, workspace, out, lse, status,
                     stream)
    args = [a[1], a[2], k_new.data_ptr(), v_new.data_ptr(), pos.data_ptr(), a[0], a[3]] + a[4:11] + [float(phi)] + a[11:]
    _check(load().kvd_decode_step_umax(*args), "kvd_decode_step_umax")


def merge_attention(outs, lses, out, lse=None, stream=None):
    """Results over disjoint token shards combined by their normalisers
    (kvd_merge_attention): outs [n, ..., D] bf16 or fp32 and lses [n, ...] fp32
    as the attention calls return out and lse; out [..., D] bf16 or fp32."""
    import torch
    _require(outs, "outs", (torch.bfloat16, torch.float32))
    _require(lses, "lses", torch.float32)
    _require(out, "out", (torch.bfloat16, torch.float32))
    n, D = outs.shape[0], outs.shape[-1]
    if lses.shape != outs.shape[:-1] or out.shape != outs.shape[1:]:
        raise ValueError("merge_attention: outs [n, ..., D], lses [n, ...] and out [..., D] disagree")
    if lse is not None:
        _require(lse, "lse", torch.float32)
        if lse.shape != lses.shape[1:]:
            raise ValueError("merge_attention: lse must be shaped like lses[0]")
    rows = out.numel() // D
    code = lambda t: OUT_BF16 if t.dtype == torch.bfloat16 else OUT_F32
    _check(load().kvd_merge_attention(outs.data_ptr(), lses.data_ptr(), n, rows, D, code(outs), out.data_ptr(),
                                      code(out), _ptr(lse), _stream_handle(stream)), "kvd_merge_attention")


def probe_read(src, nbytes: int = 0, ctas: int = 0, sink=None, status=None, stream=None):
    """One read-only streaming pass over a device tensor's bytes (kvd_probe_read):
    a measurement aid giving the read ceiling of a kernel that reads those
    bytes once. nbytes = 0 reads the whole tensor."""
    n = nbytes or src.numel() * src.element_size()
    _check(load().kvd_probe_read(src.data_ptr(), n, ctas, _ptr(sink), _ptr(status), _stream_handle(stream)),
           "kvd_probe_read")


def step_staging_bytes(batch: int, n_tokens: int, n_heads_q: int, n_heads_kv: int, head_dim: int) -> int:
    """Device staging bytes decode_step_host needs (kvd_step_staging_bytes)."""
    return int(load().kvd_step_staging_bytes(batch, n_tokens, n_heads_q, n_heads_kv, head_dim))


class HostStep:
    """A step from host inputs to a host result (kvd_decode_step_host) with its
    buffers bound once: the CPU tensors q_host [B, Hq, D] or [B, T, Hq, D]
    (bf16), k_new_host, v_new_host ([B, Hkv, D] or [B, T, Hkv, D]), pos_host,
    seq_lens_host (int32 [B]), the device cache, the device buffer `staging`
    (step_staging_bytes), `out` and its CPU copy out_host. Each call copies the
    host inputs' current contents in, runs the step and copies `out` back, on
    `stream` (pin the host tensors for asynchronous copies); nothing is
    synchronised. With out=None the kernels write the result straight into the
    pinned out_host. Arguments are checked here and by the library on every call."""

    def __init__(self, q_host, k_new_host, v_new_host, pos_host, seq_lens_host, k_cache, v_cache, staging,
                 max_seq_len: int, scale: float, out, out_host, workspace=None, n_split: int = 0, lse=None,
                 status=None, stream=None):
        import torch
        for t, n in ((q_host, "q_host"), (k_new_host, "k_new_host"), (v_new_host, "v_new_host")):
            if t.dtype != torch.bfloat16 or t.device.type != "cpu" or not t.is_contiguous():
                raise TypeError(f"{n} must be a contiguous bfloat16 CPU tensor")
        for t, n in ((pos_host, "pos_host"), (seq_lens_host, "seq_lens_host")):
            if t.dtype != torch.int32 or t.device.type != "cpu" or not t.is_contiguous():
                raise TypeError(f"{n} must be a contiguous int32 CPU tensor")
        # out None: the kernels write the result straight into out_host (pinned)
        if out is None and not out_host.is_pinned():
            raise ValueError("out=None needs a pinned out_host")
        like = out if out is not None else out_host
        if out_host.device.type != "cpu" or out_host.dtype != like.dtype or out_host.shape != like.shape:
            raise TypeError("out_host must be a CPU tensor like out")
        _require(k_cache, "k_cache", torch.bfloat16, 4)
        _require(v_cache, "v_cache", torch.bfloat16, 4)
        T = q_host.shape[1] if q_host.dim() == 4 else 1
        B, Hq, D = q_host.shape[0], q_host.shape[-2], q_host.shape[-1]
        S, Hkv = k_cache.shape[1], k_cache.shape[2]
        code = OUT_BF16 if like.dtype == torch.bfloat16 else OUT_F32 if like.dtype == torch.float32 else None
        if code is None or like.shape != q_host.shape:
            raise TypeError("out must be bfloat16 or float32, shaped like q")
        ws_ptr, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(),
                                                               workspace.numel() * workspace.element_size())
        self._keep = (q_host, k_new_host, v_new_host, pos_host, seq_lens_host, k_cache, v_cache, staging, out,
                      out_host, workspace, lse, status)
        self._fn = load().kvd_decode_step_host
        self._args = (k_cache.data_ptr(), v_cache.data_ptr(), q_host.data_ptr(), k_new_host.data_ptr(),
                      v_new_host.data_ptr(), pos_host.data_ptr(), seq_lens_host.data_ptr(), staging.data_ptr(),
                      staging.numel() * staging.element_size(), B, T, S, int(max_seq_len), Hq, Hkv, D,
                      float(scale), int(n_split), ws_ptr, ws_bytes, None if out is None else out.data_ptr(),
                      out_host.data_ptr(), code,
                      _ptr(lse), _ptr(status), _stream_handle(stream))

    def __call__(self):
        _check(self._fn(*self._args), "kvd_decode_step_host")


def alloc_host_packet(batch: int, n_tokens: int, n_heads_q: int, n_heads_kv: int, head_dim: int):
    """One pinned host buffer laid out like decode_step_host's staging buffer,
    and its views (q, k_new, v_new, pos, seq_lens; shapes as decode_step_host
    takes them). A HostStep over these views copies its inputs in one copy."""
    import torch
    B, T = batch, n_tokens
    al = lambda n: -(-n // 256) * 256
    nq, nk, ni = B * T * n_heads_q * head_dim * 2, B * T * n_heads_kv * head_dim * 2, B * 4
    packet = torch.empty(step_staging_bytes(B, T, n_heads_q, n_heads_kv, head_dim), dtype=torch.uint8).pin_memory()
    offs = [0, al(nq), al(nq) + al(nk), al(nq) + 2 * al(nk), al(nq) + 2 * al(nk) + al(ni)]
    qs = (B, n_heads_q, head_dim) if T == 1 else (B, T, n_heads_q, head_dim)
    ks = (B, n_heads_kv, head_dim) if T == 1 else (B, T, n_heads_kv, head_dim)
    q = packet[offs[0]:offs[0] + nq].view(torch.bfloat16).view(qs)
    kn = packet[offs[1]:offs[1] + nk].view(torch.bfloat16).view(ks)
    vn = packet[offs[2]:offs[2] + nk].view(torch.bfloat16).view(ks)
    pos = packet[offs[3]:offs[3] + ni].view(torch.int32)
    lens = packet[offs[4]:offs[4] + ni].view(torch.int32)
    return packet, q, kn, vn, pos, lens


def decode_step_host(q_host, k_new_host, v_new_host, pos_host, seq_lens_host, k_cache, v_cache, staging,
                     max_seq_len: int, scale: float, out, out_host, workspace=None, n_split: int = 0, lse=None,
                     status=None, stream=None):
    """One HostStep call: copy the host inputs in, run the step, copy out back."""
    HostStep(q_host, k_new_host, v_new_host, pos_host, seq_lens_host, k_cache, v_cache, staging, max_seq_len,
             scale, out, out_host, workspace, n_split, lse, status, stream)()


def split_kv_chunk(q, k_cache, v_cache, seq_lens, max_seq_len: int, scale: float, out,
                   workspace=None, n_split: int = 0, lse=None, status=None, stream=None):
    """First launch of decode_attention only (the split-KV chunk kernel)."""
    args = _decode_args(q, k_cache, v_cache, seq_lens, max_seq_len, scale, n_split, workspace,
                        out, lse, status, stream)
    _check(load().kvd_split_kv_chunk(*args), "kvd_split_kv_chunk")


def split_kv_merge(q, k_cache, v_cache, seq_lens, max_seq_len: int, scale: float, out,
                   workspace=None, n_split: int = 0, lse=None, status=None, stream=None):
    """Second launch of decode_attention only (the log-sum-exp merge kernel)."""
    args = _decode_args(q, k_cache, v_cache, seq_lens, max_seq_len, scale, n_split, workspace,
                        out, lse, status, stream)
    _check(load().kvd_split_kv_merge(*args), "kvd_split_kv_merge")


# ---------------------------------------------------------------------------
# Rotary positions, appends that apply them, and the fp4 cache
# ---------------------------------------------------------------------------

ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3, "wavelength": 4}
#: Default (slow, fast) turns in the original context between which a scaling mixes.
_ROPE_TURNS = {"parts": (1.0, 32.0), "wavelength": (1.0, 4.0)}


def rope_table(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               original_len: float = 0.0, slow: Optional[float] = None, fast: Optional[float] = None,
               attn_factor: float = 0.0):
    """(turns, factor): the pairs' frequencies as uint64 fractions of a turn per
    position [rotary_dim / 2] (numpy, on the host) and what multiplies cosine
    and sine (kvd_rope_table)."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}, got {scaling!r}")
    dslow, dfast = _ROPE_TURNS.get(scaling, (0.0, 0.0))
    turns = np.zeros(max(int(rotary_dim) // 2, 1), np.uint64)
    out = ctypes.c_float(0.0)
    _check(load().kvd_rope_table(int(rotary_dim), float(base), ROPE_SCALINGS[scaling], float(factor),
                                 float(original_len), float(dslow if slow is None else slow),
                                 float(dfast if fast is None else fast), float(attn_factor),
                                 turns.ctypes.data_as(ctypes.c_void_p), ctypes.byref(out)), "kvd_rope_table")
    return turns, out.value


class RopeTable:
    """Rotary positions of one model, made once: the frequencies of rope_table
    (same arguments) on `device`, adjacent pairs when `interleaved`, else halves."""

    def __init__(self, rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                 original_len: float = 0.0, slow: Optional[float] = None, fast: Optional[float] = None,
                 attn_factor: float = 0.0, interleaved: bool = False, device="cuda"):
        import torch
        turns, self.factor = rope_table(rotary_dim, base, scaling, factor, original_len, slow, fast, attn_factor)
        self.rotary_dim, self.interleaved = int(rotary_dim), bool(interleaved)
        self.turns = torch.from_numpy(turns.view(np.int64)).to(device)
        self._device = self.turns.get_device()  # -1 on the CPU
        self._struct = _CRope(self.turns.data_ptr(), self.factor, self.rotary_dim, 1 if self.interleaved else 0)
        self._ref = ctypes.byref(self._struct)


# The calls below are made once a layer and step, so what they check is written to cost a few microseconds: a
# chain of comparisons that a right call passes, and, when it does not, _explain, which names the tensor that is
# wrong. The device is only switched to when it is not the current one.

_torch = None
_raw_stream = _current_device = None
_pack_cache = struct.Struct("PPPPPiiiii0P").pack   # struct kvd_cache (0P: padded to its full size)
_pack_fp4 = struct.Struct("PPPiiii0P").pack        # struct kvd_cache_fp4


def _import_torch():
    global _torch, _raw_stream, _current_device
    import torch
    _raw_stream, _current_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    _torch = torch
    return torch


def _explain(what, *named):
    """Raises for the first tensor that is not as asked: (tensor, name, dtypes, dims or None); None passed over."""
    import torch
    dev = None
    for t, name, dtypes, ndim in named:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{what}: {name} must be a torch.Tensor")
        i = t.get_device()
        if i < 0:
            raise ValueError(f"{what}: {name} must be on a CUDA device")
        if dev is not None and i != dev:
            raise ValueError(f"{what}: {name} is on cuda:{i}, other tensors on cuda:{dev}")
        dev = i
        if dtypes is not None and t.dtype not in dtypes:
            raise TypeError(f"{what}: {name} must be {dtypes}, got {t.dtype}")
        if ndim is not None and t.dim() != ndim:
            raise ValueError(f"{what}: {name} must have {ndim} dims, got {t.dim()}")
        if ndim is not None and not t.is_contiguous():
            raise ValueError(f"{what}: {name} must be contiguous")


def _is(t, dtype, dev):
    """A tensor of this type on this device (negative: the CPU, never)."""
    return t.dtype is dtype and t.get_device() == dev >= 0


def _whole(t, dtype, dev, ndim):
    """The same, contiguous, of so many dimensions."""
    return t.dtype is dtype and t.get_device() == dev >= 0 and t.dim() == ndim and t.is_contiguous()


def _rope_on(rope, dev, what):
    if rope.__class__ is RopeTable and rope._device == dev:
        return rope._ref
    if not isinstance(rope, RopeTable):
        raise TypeError(f"{what}: rope must be a RopeTable")
    if rope._device != dev:
        raise ValueError(f"{what}: the rope table is on {rope.turns.device}, the tensors on cuda:{dev}")
    return rope._ref


def _launch(fn, what, dev, stream, *args):
    """Calls fn(*args, stream handle) with device `dev` current; without a stream, on that device's current one."""
    if stream is None:
        h = _raw_stream(dev)
    elif hasattr(stream, "cuda_stream"):
        if stream.device_index != dev:
            raise ValueError(f"{what}: a stream of cuda:{stream.device_index}, tensors on cuda:{dev}")
        h = stream.cuda_stream
    else:
        h = int(stream)
    if _current_device() == dev:
        rc = fn(*args, h)
    else:
        with _torch.cuda.device(dev):
            rc = fn(*args, h)
    if rc:
        raise KvdError(rc, what)


def _rows(t, name, what):
    """[N, H, D] rows, or [B, T, H, D] as B * T of them, whose heads are contiguous:
    (rows, heads, head_dim, elements between rows)."""
    s, st = t.shape, t.stride()
    if len(s) == 3:
        N, H, D = s
        step, inner, last = st
        if last == 1 and inner == D and N > 1 and H:  # the usual rows, at once
            return N, H, D, step
        even = True
    elif len(s) == 4:
        B, T, H, D = s
        N = B * T
        outer, step, inner, last = st
        if last == 1 and inner == D and T > 1 and outer == T * step and N and H:
            return N, H, D, step
        if T <= 1:
            step = outer
        even = B <= 1 or T <= 1 or outer == T * step
    else:
        raise ValueError(f"{what}: {name} must be [N, H, D] or [B, T, H, D]")
    if N == 0 or H == 0 or D == 0:
        return N, H, D, H * D
    if (last != 1 and D > 1) or (inner != D and H > 1):
        raise ValueError(f"{what}: {name}'s heads must be contiguous")
    if not even:
        raise ValueError(f"{what}: {name}'s rows must be evenly spaced")
    return N, H, D, step if N > 1 else H * D


def _alike(t, name, what, N, H, D):
    """Elements between the rows of t, which has as many rows, heads and columns."""
    n, h, d, step = _rows(t, name, what)
    if n != N or h != H or d != D:
        raise ValueError(f"{what}: inconsistent shapes")
    return step


def _same_batch(what, *shapes):
    """Refuses [B, T] shapes of as many rows that are not alike; one with a 1 in it is the rows in order."""
    two = {tuple(s) for s in shapes if len(s) == 2 and 1 not in s}
    if len(two) > 1:
        raise ValueError(f"{what}: inconsistent shapes")


def rope_apply(rope: RopeTable, x, positions, out, stream=None):
    """out = x's rows turned by their positions: x, out [N, H, D] or [B, T, H, D],
    bf16 or fp32 each, rows evenly spaced (slices of a fused projection may be
    passed as they are); positions int32, one a row: [N] or [B, T]. out may be x."""
    torch = _torch or _import_torch()
    what, bf, f32 = "rope_apply", torch.bfloat16, torch.float32
    try:
        dev = x.get_device()
        xt, ot = x.dtype, out.dtype
        xc, oc = xt is f32, ot is f32
        ok = (dev >= 0 and (xc or xt is bf) and (oc or ot is bf) and out.get_device() == dev
              and positions.dtype is torch.int32 and positions.get_device() == dev and positions.is_contiguous())
    except AttributeError:
        ok = False
    if not ok:
        _explain(what, (x, "x", (bf, f32), None), (out, "out", (bf, f32), None), (positions, "positions", (torch.int32,), None))
        raise ValueError(f"{what}: positions must be contiguous")
    N, H, D, xs = _rows(x, "x", what)
    ys = xs if out is x else _alike(out, "out", what, N, H, D)
    if positions.numel() != N:
        raise ValueError(f"{what}: inconsistent shapes")
    if positions.dim() > 1 or (out is not x and x.dim() == 4):
        _same_batch(what, positions.shape, x.shape[:-2], out.shape[:-2])
    ref = _rope_on(rope, dev, what)
    if N == 0:
        return
    _launch((_lib or load()).kvd_rope_apply, "kvd_rope_apply", dev, stream, ref, x.data_ptr(), xs,
            OUT_F32 if xc else OUT_BF16, out.data_ptr(), ys, OUT_F32 if oc else OUT_BF16, positions.data_ptr(), N, H, D)


def _append_rows(what, rope, q, q_out, k_new, v_new, pos, row_offsets, dev, torch):
    """(batch, rows, KV heads, head_dim, the arguments of kvd_kv_append_rope between the cache and the status word)."""
    bf, i32 = torch.bfloat16, torch.int32
    if (q is None) != (q_out is None):
        raise ValueError(f"{what}: q and q_out go together")
    try:
        ok = (dev >= 0 and k_new.dtype is bf and k_new.get_device() == dev and v_new.dtype is bf and v_new.get_device() == dev
              and pos.dtype is i32 and pos.get_device() == dev and pos.dim() == 1 and pos.is_contiguous()
              and (q is None or (q.dtype is bf and q.get_device() == dev and q_out.dtype is bf and q_out.get_device() == dev))
              and (row_offsets is None or _whole(row_offsets, i32, dev, 1)))
    except AttributeError:
        ok = False
    if not ok:
        _explain(what, (k_new, "k_new", (bf,), None), (v_new, "v_new", (bf,), None), (pos, "pos", (i32,), 1), (q, "q", (bf,), None),
                 (q_out, "q_out", (bf,), None), (row_offsets, "row_offsets", (i32,), 1))
        raise ValueError(f"{what}: the new rows are on cuda:{pos.get_device()}, the cache on cuda:{dev}")
    N, Hkv, D, ks = _rows(k_new, "k_new", what)
    vs = _alike(v_new, "v_new", what, N, Hkv, D)
    B = pos.numel()
    lead = B  # the first of four dimensions
    if row_offsets is not None:
        if row_offsets.numel() != B + 1:
            raise ValueError(f"{what}: row_offsets must be [batch + 1]")
        off, lead = row_offsets.data_ptr(), 1
    else:
        if (N % B if B else N):
            raise ValueError(f"{what}: {N} new rows for {B} sequences")
        off = None
    if ((k_new.dim() == 4 and k_new.shape[0] != lead) or (v_new.dim() == 4 and v_new.shape[0] != lead)
            or (q is not None and ((q.dim() == 4 and q.shape[0] != lead) or (q_out.dim() == 4 and q_out.shape[0] != lead)))):
        raise ValueError(f"{what}: new rows must be [batch, T, H, D]" if row_offsets is None
                         else f"{what}: rows with row_offsets must be packed, [N, H, D]")
    ref = None if rope is None else _rope_on(rope, dev, what)
    if q is None:
        qp = op = None
        Hq = qs = os_ = 0
    else:
        if rope is None:
            raise ValueError(f"{what}: q needs a rope")
        Nq, Hq, Dq, qs = _rows(q, "q", what)
        os_ = qs if q_out is q else _alike(q_out, "q_out", what, N, Hq, D)
        if Nq != N or Dq != D:
            raise ValueError(f"{what}: inconsistent shapes")
        qp, op = q.data_ptr(), q_out.data_ptr()
    return B, N, Hkv, D, (ref, qp, qs, op, os_, k_new.data_ptr(), ks, v_new.data_ptr(), vs, pos.data_ptr(), off, B, N, Hq,
                          Hkv, D)


def _status_ptr(status, dev, what, torch):
    if status is None:
        return None
    if not isinstance(status, torch.Tensor) or not _is(status, torch.int32, dev):
        raise TypeError(f"{what}: status must be an int32 tensor on cuda:{dev}")
    return status.data_ptr()


def kv_append_rope(rope: RopeTable, k, v, k_new, v_new, pos, *, q=None, q_out=None, k_scales=None, v_scales=None,
                   block_table=None, row_offsets=None, status=None, stream=None):
    """New rows into a cache as decode_ex takes it (k, v contiguous [B, S_max, Hkv,
    D], or pools with block_table; bf16, or 8-bit codes with scales), keys
    turned by their positions, and q turned into q_out (kvd_kv_append_rope).
    k_new, v_new, q: [B, T, H, D] or [B * T, H, D] at pos[b] + i, or with row_offsets
    int32 [B + 1] the packed rows [N, H, D] of prompts of any lengths; rows evenly
    spaced, so slices of a fused projection may be passed as they are."""
    torch = _torch or _import_torch()
    what, bf, i32, f32 = "kv_append_rope", torch.bfloat16, torch.int32, torch.float32
    if rope is None:
        raise TypeError(f"{what}: rope must be a RopeTable")
    if (k_scales is None) != (v_scales is None):
        raise ValueError(f"{what}: k_scales and v_scales go together")
    quant = k_scales is not None
    dts = (torch.int8, torch.uint8, torch.float8_e4m3fn) if quant else (bf,)
    try:
        dev, dt = k.get_device(), k.dtype
        ok = (dev >= 0 and (dt is bf if not quant else dt in dts) and k.dim() == 4 and k.is_contiguous()
              and v.dtype is dt and v.get_device() == dev and v.is_contiguous()
              and (block_table is None or _whole(block_table, i32, dev, 2))
              and (not quant or (_whole(k_scales, f32, dev, 3) and _whole(v_scales, f32, dev, 3))))
    except AttributeError:
        ok = False
    if not ok:
        _explain(what, (k, "k", dts, 4), (v, "v", dts, 4), (block_table, "block_table", (i32,), 2),
                 (k_scales, "k_scales", (f32,), 3), (v_scales, "v_scales", (f32,), 3))
        raise TypeError(f"{what}: k is {k.dtype}, v {v.dtype}")
    B, N, Hkv, D, args = _append_rows(what, rope, q, q_out, k_new, v_new, pos, row_offsets, dev, torch)
    n, cap, heads, width = shape = k.shape
    if v.shape != shape or heads != Hkv or width != D:
        raise ValueError(f"{what}: inconsistent shapes")
    ksp = vsp = fp8 = 0
    if quant:
        if k_scales.shape != shape[:3] or v_scales.shape != shape[:3]:
            raise ValueError(f"{what}: codes [B, S_max, Hkv, D] and scales [B, S_max, Hkv] disagree")
        ksp, vsp, fp8 = k_scales.data_ptr(), v_scales.data_ptr(), 0 if dt is torch.int8 else 1
    if block_table is not None:
        rows, blocks = block_table.shape
        if rows != B:
            raise ValueError(f"{what}: inconsistent shapes")
        c = _pack_cache(k.data_ptr(), v.data_ptr(), ksp, vsp, block_table.data_ptr(), 0, blocks, cap, n, fp8)
    else:
        if n != B:
            raise ValueError(f"{what}: inconsistent shapes")
        c = _pack_cache(k.data_ptr(), v.data_ptr(), ksp, vsp, 0, cap, 0, 0, 0, fp8)
    if N == 0:
        return
    _launch((_lib or load()).kvd_kv_append_rope, "kvd_kv_append_rope", dev, stream, c, *args,
            None if status is None else _status_ptr(status, dev, what, torch))


def fp4_block_bytes(head_dim: int) -> int:
    """Bytes of an fp4 cache's block of 16 tokens of one KV head: 9 * head_dim + 16."""
    n = int(load().kvd_fp4_block_bytes(int(head_dim)))
    if n == 0:
        raise ValueError(f"fp4 cache: head_dim must be 64, 128 or 256, got {head_dim}")
    return n


def alloc_cache_fp4(batch_or_pages: int, n_heads_kv: int, head_dim: int, tokens: int, device="cuda"):
    """One fp4 tensor (K or V), zeroed: a contiguous cache of `tokens` (a multiple
    of 16) per sequence, or a pool of pages of `tokens` each."""
    import torch
    if tokens < 16 or tokens % 16:
        raise ValueError("fp4 cache: tokens must be a multiple of 16")
    return torch.zeros(batch_or_pages, n_heads_kv, tokens // 16, fp4_block_bytes(head_dim), dtype=torch.uint8,
                       device=device)


def _fp4_cache(what, k, v, D, B, block_table, torch):
    """(the packed struct kvd_cache_fp4, KV heads, capacity of a sequence, device) of the blocks k and v (v may be None)."""
    u8, i32 = torch.uint8, torch.int32
    try:
        dev = k.get_device()
        ok = (dev >= 0 and k.dtype is u8 and k.dim() == 4 and k.is_contiguous()
              and (v is None or (v.dtype is u8 and v.get_device() == dev and v.is_contiguous()))
              and (block_table is None or _whole(block_table, i32, dev, 2)))
    except AttributeError:
        ok = False
    if not ok:
        _explain(what, (k, "k" if v is not None else "blocks", (u8,), 4), (v, "v", (u8,), 4), (block_table, "block_table", (i32,), 2))
        raise ValueError(f"{what}: the fp4 cache must be on a CUDA device")
    n, heads, blks, width = shape = k.shape
    if width != 9 * D + 16 or D not in (64, 128, 256):
        raise ValueError(f"{what}: blocks of {width} bytes at head_dim {D}")
    vp = 0
    if v is not None:
        if v.shape != shape:
            raise ValueError(f"{what}: inconsistent shapes")
        vp = v.data_ptr()
    if block_table is not None:
        rows, per = block_table.shape
        if rows != B:
            raise ValueError(f"{what}: inconsistent shapes")
        return _pack_fp4(k.data_ptr(), vp, block_table.data_ptr(), 0, per, 16 * blks, n), heads, 16 * blks * per, dev
    if n != B:
        raise ValueError(f"{what}: inconsistent shapes")
    return _pack_fp4(k.data_ptr(), vp, 0, 16 * blks, 0, 0, 0), heads, 16 * blks, dev


def kv_append_fp4(k, v, k_new, v_new, pos, *, rope: Optional[RopeTable] = None, q=None, q_out=None, block_table=None,
                  row_offsets=None, status=None, stream=None):
    """kv_append_rope for an fp4 cache (k, v uint8 [B, Hkv, S_max / 16, 9 D + 16], or
    pools [pages, Hkv, page / 16, 9 D + 16] with block_table); rope None appends
    the rows as they are (kvd_kv_append_fp4)."""
    torch = _torch or _import_torch()
    what = "kv_append_fp4"
    if v is None:
        raise TypeError(f"{what}: v must be a torch.Tensor")
    if not isinstance(k, torch.Tensor):
        raise TypeError(f"{what}: k must be a torch.Tensor")
    B, N, Hkv, D, args = _append_rows(what, rope, q, q_out, k_new, v_new, pos, row_offsets, k.get_device(), torch)
    c, heads, _, dev = _fp4_cache(what, k, v, D, B, block_table, torch)
    if heads != Hkv:
        raise ValueError(f"{what}: inconsistent shapes")
    if N == 0:
        return
    _launch((_lib or load()).kvd_kv_append_fp4, "kvd_kv_append_fp4", dev, stream, c, *args,
            None if status is None else _status_ptr(status, dev, what, torch))


def _bf16_rows_and_lens(what, cache, name, seq_lens, torch):
    """(B, S, Hkv, D, device) of a contiguous bf16 cache [B, S, Hkv, D] and its lengths."""
    bf, i32 = torch.bfloat16, torch.int32
    try:
        dev = cache.get_device()
        ok = (dev >= 0 and cache.dtype is bf and cache.dim() == 4 and cache.is_contiguous()
              and seq_lens.dtype is i32 and seq_lens.get_device() == dev and seq_lens.dim() == 1 and seq_lens.is_contiguous())
    except AttributeError:
        ok = False
    if not ok:
        _explain(what, (cache, name, (bf,), 4), (seq_lens, "seq_lens", (i32,), 1))
        raise ValueError(f"{what}: {name} must be on a CUDA device")
    B, S, Hkv, D = cache.shape
    if seq_lens.numel() != B:
        raise ValueError(f"{what}: inconsistent shapes")
    return B, S, Hkv, D, dev


def kv_quantize_fp4(cache, blocks, seq_lens, max_seq_len: int, stream=None):
    """Rows t < seq_lens[b] of a bf16 cache [B, S_max, Hkv, D] (K or V) into the blocks
    of a contiguous fp4 cache (kvd_kv_quantize_fp4)."""
    torch = _torch or _import_torch()
    what = "kv_quantize_fp4"
    B, S, Hkv, D, dev = _bf16_rows_and_lens(what, cache, "cache", seq_lens, torch)
    _, heads, cap, on = _fp4_cache(what, blocks, None, D, B, None, torch)
    if heads != Hkv:
        raise ValueError(f"{what}: inconsistent shapes")
    if on != dev:
        raise ValueError(f"{what}: cache on cuda:{dev}, blocks on cuda:{on}")
    if B == 0:
        return
    _launch((_lib or load()).kvd_kv_quantize_fp4, "kvd_kv_quantize_fp4", dev, stream, cache.data_ptr(), blocks.data_ptr(),
            seq_lens.data_ptr(), B, S, cap, int(max_seq_len), Hkv, D)


def kv_read_fp4(blocks, out, seq_lens, max_seq_len: int, block_table=None, status=None, stream=None):
    """Rows t < seq_lens[b] of an fp4 cache's K or V blocks (contiguous, or a pool
    with block_table) back to bf16 out [B, S, Hkv, D], exactly (kvd_kv_read_fp4)."""
    torch = _torch or _import_torch()
    what = "kv_read_fp4"
    B, S, Hkv, D, dev = _bf16_rows_and_lens(what, out, "out", seq_lens, torch)
    _, heads, cap, on = _fp4_cache(what, blocks, None, D, B, block_table, torch)
    if heads != Hkv:
        raise ValueError(f"{what}: inconsistent shapes")
    if on != dev:
        raise ValueError(f"{what}: out on cuda:{dev}, blocks on cuda:{on}")
    if B == 0:
        return
    if block_table is None:
        table = (None, cap, 0, 0, 0)
    else:
        table = (block_table.data_ptr(), 0, block_table.shape[1], 16 * blocks.shape[2], blocks.shape[0])
    _launch((_lib or load()).kvd_kv_read_fp4, "kvd_kv_read_fp4", dev, stream, blocks.data_ptr(), *table, out.data_ptr(), S,
            seq_lens.data_ptr(), B, int(max_seq_len), Hkv, D,
            None if status is None else _status_ptr(status, dev, what, torch))


def decode_plan_fp4(batch: int, n_tokens: int, n_heads_q: int, n_heads_kv: int, head_dim: int, max_seq_len: int,
                    num_sms: int = 0, n_split: int = 0) -> Tuple[int, int]:
    """(n_split, workspace_bytes) for a decode_fp4 call of this shape."""
    n = ctypes.c_int(0)
    ws = ctypes.c_size_t(0)
    _check(load().kvd_decode_plan_fp4(batch, n_tokens, n_heads_q, n_heads_kv, head_dim, max_seq_len, num_sms, n_split,
                                      ctypes.byref(n), ctypes.byref(ws)), "kvd_decode_plan_fp4")
    return n.value, ws.value


def decode_fp4(q, k, v, seq_lens, max_seq_len: int, scale: float, out, *, block_table=None, k_new=None, v_new=None,
               pos=None, workspace=None, n_split: int = 0, lse=None, status=None, stream=None):
    """decode_ex over an fp4 cache (kvd_decode_fp4): q, out [B, Hq, D] or [B, T, Hq, D];
    k, v uint8 [B, Hkv, S_max / 16, 9 D + 16], or pools [pages, Hkv, page / 16, 9 D + 16] with
    block_table [B, max_blocks]; k_new, v_new ([B, Hkv, D] or [B, T, Hkv, D]) and
    pos to append first. Workspace: decode_plan_fp4."""
    torch = _torch or _import_torch()
    what, bf, i32, f32 = "decode_fp4", torch.bfloat16, torch.int32, torch.float32
    try:
        dev = q.get_device()
        ot = out.dtype
        f32_out = ot is f32
        ok = (dev >= 0 and q.dtype is bf and q.is_contiguous() and (f32_out or ot is bf) and out.get_device() == dev
              and out.is_contiguous() and seq_lens.dtype is i32 and seq_lens.get_device() == dev and seq_lens.dim() == 1
              and seq_lens.is_contiguous()
              and (lse is None or (_is(lse, f32, dev) and lse.is_contiguous()))
              and (workspace is None or (workspace.get_device() == dev and workspace.is_contiguous())))
    except AttributeError:
        ok = False
    if not ok:
        _explain(what, (q, "q", (bf,), None), (out, "out", (bf, f32), None), (seq_lens, "seq_lens", (i32,), 1),
                 (lse, "lse", (f32,), None), (workspace, "workspace", None, None))
        raise ValueError(f"{what}: q, out, lse and workspace must be contiguous")
    shape = q.shape
    if len(shape) == 3:
        (B, Hq, D), T = shape, 1
    elif len(shape) == 4:
        B, T, Hq, D = shape
    else:
        raise ValueError(f"{what}: q must be [B, Hq, D] or [B, T, Hq, D]")
    if out.shape != shape or seq_lens.numel() != B or (lse is not None and lse.shape != shape[:-1]):
        raise ValueError(f"{what}: inconsistent shapes")
    if v is None:
        raise TypeError(f"{what}: v must be a torch.Tensor")
    c, Hkv, _, on = _fp4_cache(what, k, v, D, B, block_table, torch)
    if on != dev:
        raise ValueError(f"{what}: q on cuda:{dev}, the cache on cuda:{on}")
    kp = vp = pp = None
    if k_new is not None or v_new is not None or pos is not None:
        if k_new is None or v_new is None or pos is None:
            raise ValueError(f"{what}: k_new, v_new and pos go together")
        n = len(shape)
        if not (_whole(k_new, bf, dev, n) and _whole(v_new, bf, dev, n) and _whole(pos, i32, dev, 1)):
            _explain(what, (q, "q", (bf,), None), (k_new, "k_new", (bf,), n), (v_new, "v_new", (bf,), n), (pos, "pos", (i32,), 1))
        if k_new.shape != shape[:-2] + (Hkv, D) or v_new.shape != k_new.shape or pos.numel() != B:
            raise ValueError(f"{what}: inconsistent shapes")
        kp, vp, pp = k_new.data_ptr(), v_new.data_ptr(), pos.data_ptr()
    wp, wb = None, 0
    if workspace is not None:
        wp, wb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if B == 0:
        return
    _launch((_lib or load()).kvd_decode_fp4, "kvd_decode_fp4", dev, stream, c, q.data_ptr(), seq_lens.data_ptr(), B, T,
            int(max_seq_len), Hq, Hkv, D, float(scale), int(n_split), wp, wb, out.data_ptr(),
            OUT_F32 if f32_out else OUT_BF16, None if lse is None else lse.data_ptr(), kp, vp, pp,
            None if status is None else _status_ptr(status, dev, what, torch))

"""ctypes binding of libtq_gb300.so (include/tq.h): argument marshalling only.

Every computation runs in the library's CUDA kernels (or, for the rotation signs
and the codebook, in its host C++).  If the library has not been built these
functions raise: there is no fallback path.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading
from typing import NamedTuple

import torch

from .build import LIB_PATH

TQ_OK = 0
TQ_ERR_INVALID_ARG = 1
TQ_ERR_UNSUPPORTED = 2
TQ_ERR_SLOT_OUT_OF_RANGE = 3
TQ_ERR_BLOCK_OUT_OF_RANGE = 4
TQ_ERR_CUDA = 5
TQ_ERR_TIMEOUT = 6
TQ_ERR_OUT_OF_BLOCKS = 7

STATUS_NAMES = {
    TQ_OK: "TQ_OK",
    TQ_ERR_INVALID_ARG: "TQ_ERR_INVALID_ARG",
    TQ_ERR_UNSUPPORTED: "TQ_ERR_UNSUPPORTED",
    TQ_ERR_SLOT_OUT_OF_RANGE: "TQ_ERR_SLOT_OUT_OF_RANGE",
    TQ_ERR_BLOCK_OUT_OF_RANGE: "TQ_ERR_BLOCK_OUT_OF_RANGE",
    TQ_ERR_CUDA: "TQ_ERR_CUDA",
    TQ_ERR_TIMEOUT: "TQ_ERR_TIMEOUT",
    TQ_ERR_OUT_OF_BLOCKS: "TQ_ERR_OUT_OF_BLOCKS",
}

_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}

TQ_RECIPE_TURBOQUANT25 = 25
TQ_RECIPE_TURBOQUANT35 = 35
RECIPES = {"turboquant25": TQ_RECIPE_TURBOQUANT25, "turboquant35": TQ_RECIPE_TURBOQUANT35}
RECIPE_ROTATION_SEED = 42
RECIPE_SKETCH_SEED = 43

# Every symbol include/tq.h declares, with (restype, argtypes).
_c_int, _c_i64, _c_u64, _c_f, _c_p, _c_sz = (ctypes.c_int, ctypes.c_int64, ctypes.c_uint64, ctypes.c_float,
                                            ctypes.c_void_p, ctypes.c_size_t)
SIGNATURES = {
    "tq_last_error": (ctypes.c_char_p, []),
    "tq_set_wait_limit": (_c_i64, [_c_i64]),
    "tq_launch_count": (ctypes.c_uint64, []),
    "tq_row_bytes": (_c_i64, [_c_int, _c_int]),
    "tq_build_rotation": (_c_int, [_c_int, _c_u64, _c_p]),
    "tq_codebook": (_c_int, [_c_int, _c_int, _c_p, _c_p]),
    "tq_write_kv": (_c_int, [_c_p, _c_int, _c_i64, _c_int, _c_int, _c_int, _c_p, _c_p, _c_i64, _c_int,
                             _c_p, _c_p, _c_p, _c_p]),
    "tq_dequant_rows": (_c_int, [_c_p, _c_int, _c_i64, _c_int, _c_int, _c_int, _c_p, _c_i64, _c_p, _c_p, _c_p,
                                 _c_int, _c_p, _c_p]),
    "tq_paged_decode_workspace": (_c_sz, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "tq_paged_prefill_workspace": (_c_sz, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "tq_paged_prefill": (_c_int, [_c_p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_p, _c_int, _c_p, _c_int, _c_i64,
                                  _c_int, _c_p, _c_int, _c_int, _c_p, _c_p, _c_p, _c_p, _c_p, _c_f, _c_p, _c_int,
                                  _c_p, _c_sz, _c_p, _c_p]),
    "tq_paged_decode": (_c_int, [_c_p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_p, _c_int, _c_p, _c_int,
                                 _c_i64, _c_int, _c_p, _c_int, _c_p, _c_p, _c_p, _c_p, _c_f, _c_p, _c_int,
                                 _c_p, _c_sz, _c_p, _c_p]),
    "tq_paged_decode_static": (_c_int, [_c_p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_p, _c_int, _c_p,
                                        _c_int, _c_i64, _c_int, _c_p, _c_int, _c_p, _c_p, _c_p, _c_p, _c_f,
                                        _c_p, _c_int, _c_p, _c_p]),
    "tq_prod_row_bytes": (_c_i64, [_c_int, _c_int]),
    "tq_build_qjl_matrix": (_c_int, [_c_int, _c_u64, _c_p]),
    "tq_write_kv_prod": (_c_int, [_c_p, _c_int, _c_i64, _c_int, _c_int, _c_int, _c_p, _c_p, _c_i64, _c_int,
                                  _c_p, _c_p, _c_p, _c_p, _c_p]),
    "tq_paged_decode_prod_workspace": (_c_sz, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "tq_paged_decode_prod": (_c_int, [_c_p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_p, _c_int, _c_p, _c_int,
                                      _c_i64, _c_int, _c_p, _c_int, _c_p, _c_p, _c_p, _c_p, _c_p, _c_f, _c_p,
                                      _c_int, _c_p, _c_sz, _c_p, _c_p]),
    "tq_quantize_queries_int8": (_c_int, [_c_p, _c_int, _c_i64, _c_int, _c_int, _c_p, _c_p, _c_p]),
    "tq_paged_prefill_int8q": (_c_int, [_c_p, _c_p, _c_int, _c_int, _c_int, _c_int, _c_p, _c_int, _c_p, _c_int,
                                        _c_i64, _c_int, _c_p, _c_int, _c_int, _c_p, _c_p, _c_p, _c_p, _c_p, _c_f,
                                        _c_p, _c_int, _c_p, _c_sz, _c_p, _c_p]),
    "tq_recipe_row_bytes": (_c_i64, [_c_int, _c_int]),
    "tq_recipe_channel_order": (_c_int, [_c_int, _c_int, _c_int, _c_p, _c_p]),
    "tq_recipe_calibrate": (_c_int, [_c_int, _c_int, _c_int, _c_p, _c_i64, _c_p]),
    "tq_write_kv_recipe": (_c_int, [_c_p, _c_int, _c_i64, _c_int, _c_int, _c_int, _c_p, _c_p, _c_i64, _c_int, _c_p,
                                    _c_p, _c_p, _c_p, _c_p, _c_p, _c_p]),
    "tq_paged_decode_recipe_workspace": (_c_sz, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "tq_paged_decode_recipe": (_c_int, [_c_p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_p, _c_p, _c_int, _c_i64,
                                        _c_int, _c_p, _c_int, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_f, _c_p, _c_int,
                                        _c_p, _c_sz, _c_p, _c_p]),
    "tq_plan_step": (_c_int, [_c_p, _c_p, _c_p, _c_int, _c_p, _c_int, _c_p, _c_p, _c_i64, _c_int, _c_i64, _c_p, _c_p,
                              _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p]),
    "tq_commit_tree": (_c_int, [_c_p, _c_i64, _c_p, _c_i64, _c_i64, _c_int, _c_int, _c_p, _c_int, _c_int, _c_p, _c_p,
                                _c_p, _c_int, _c_p, _c_p, _c_p]),
    "tq_paged_tree_workspace": (_c_sz, [_c_int, _c_int, _c_int, _c_int]),
    "tq_paged_tree": (_c_int, [_c_p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_p, _c_int, _c_p, _c_int, _c_i64,
                               _c_int, _c_p, _c_int, _c_int, _c_p, _c_p, _c_p, _c_int, _c_p, _c_p, _c_p, _c_f, _c_f,
                               _c_p, _c_int, _c_p, _c_sz, _c_p, _c_p]),
    "tq_paged_prefill_biased": (_c_int, [_c_p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_p, _c_int, _c_p, _c_int,
                                         _c_i64, _c_int, _c_p, _c_int, _c_int, _c_p, _c_p, _c_p, _c_p, _c_int, _c_p,
                                         _c_p, _c_p, _c_p, _c_f, _c_f, _c_p, _c_int, _c_p, _c_sz, _c_p, _c_p]),
    "tq_build_rope": (_c_int, [_c_int, _c_i64, ctypes.c_double, _c_p, _c_p]),
    "tq_norm_rope": (_c_int, [_c_p, _c_i64, _c_int, _c_p, _c_i64, _c_int, _c_int, _c_i64, _c_int, _c_p, _c_int, _c_p,
                              _c_i64, _c_int, _c_int, _c_p, _c_p, _c_f, _c_p, _c_i64, _c_p, _c_i64, _c_p, _c_p]),
    "tq_append_kv": (_c_int, [_c_p, _c_i64, _c_int, _c_p, _c_i64, _c_p, _c_i64, _c_p, _c_i64, _c_int, _c_i64, _c_int,
                              _c_int, _c_p, _c_p, _c_int, _c_p, _c_int, _c_i64, _c_int, _c_p, _c_p, _c_p, _c_p, _c_int,
                              _c_p, _c_i64, _c_int, _c_int, _c_p, _c_p, _c_f, _c_p, _c_p]),
    "tq_verify_tree_workspace": (_c_sz, [_c_int, _c_int, _c_int]),
    "tq_verify_tree": (_c_int, [_c_p, _c_int, _c_i64, _c_int, _c_int, _c_p, _c_int, _c_i64, _c_p, _c_int, _c_p, _c_p,
                                _c_p, _c_p, _c_p, _c_p, _c_int, _c_p, _c_p, _c_p, _c_sz, _c_p, _c_p]),
}

_lib = None
_lock = threading.Lock()


class TQError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(f"{LIB_PATH} is missing: build it first "
                                       "(python -m quantized_kv_cache_06_gb300.build, needs nvcc for sm_103a)")
                handle = ctypes.CDLL(LIB_PATH)
                for name, (res, args) in SIGNATURES.items():
                    fn = getattr(handle, name)
                    fn.restype = res
                    fn.argtypes = args
                _lib = handle
    return _lib


def _check(status: int) -> None:
    if status != TQ_OK:
        msg = lib().tq_last_error().decode(errors="replace")
        raise TQError(status, msg)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _need_cuda(name: str, *tensors: torch.Tensor) -> torch.device:
    dev = tensors[0].device
    for t in tensors:
        if t.device.type != "cuda" or t.device != dev:
            raise ValueError(f"{name}: all tensors must be on the same CUDA device")
        if not t.is_contiguous():
            raise ValueError(f"{name}: tensors must be contiguous")
    return dev


_status_bufs: dict = {}


def _status_buffer(device: torch.device) -> torch.Tensor:
    key = (device.index, torch.cuda.current_stream(device).cuda_stream)
    buf = _status_bufs.get(key)
    if buf is None:
        buf = torch.zeros(1, dtype=torch.int32, device=device)
        _status_bufs[key] = buf
    return buf


def raise_for_device_status(status: torch.Tensor) -> None:
    """Synchronises on `status` (a device int32 the library wrote) and raises on a non-zero code."""
    code = int(status.item())
    if code != TQ_OK:
        raise TQError(code, "reported by the device status word")


# ---------------------------------------------------------------- host set-up

def tq_set_wait_limit(tries: int) -> int:
    """Failure-path testing hook: tries of the decode's bounded device waits for later
    launches (>= 0), or the default (< 0).  Returns the previous value."""
    return int(lib().tq_set_wait_limit(int(tries)))


def tq_launch_count() -> int:
    """Kernel launches the library has enqueued in this process so far."""
    return int(lib().tq_launch_count())


def tq_row_bytes(head_dim: int, bits: int) -> int:
    n = lib().tq_row_bytes(int(head_dim), int(bits))
    if n < 0:
        raise TQError(TQ_ERR_UNSUPPORTED, f"head_dim {head_dim} / bits {bits} unsupported")
    return int(n)


def tq_build_rotation(head_dim: int, seed: int = 42, device=None) -> torch.Tensor:
    """RHT signs (float32 [head_dim], +-1) for build_rotation(dim, RHT, seed)."""
    out = torch.empty(int(head_dim), dtype=torch.float32)
    _check(lib().tq_build_rotation(int(head_dim), int(seed) & ((1 << 64) - 1), out.data_ptr()))
    return out if device is None else out.to(device)


def tq_codebook(head_dim: int, bits: int, device=None):
    """(centroids float32 [2^bits], boundaries float32 [2^bits - 1])."""
    n = 1 << int(bits)
    c = torch.empty(n, dtype=torch.float32)
    b = torch.empty(n - 1, dtype=torch.float32)
    _check(lib().tq_codebook(int(head_dim), int(bits), c.data_ptr(), b.data_ptr()))
    if device is not None:
        c, b = c.to(device), b.to(device)
    return c, b


def _need_f32(name: str, head_dim: int, signs: torch.Tensor, *others: torch.Tensor) -> None:
    """The rotation signs, codebooks and sketch matrix are read by the kernels as fp32 arrays
    of known length: another dtype, or fewer than head_dim signs, would make them read past
    the buffer."""
    for t in (signs, *others):
        if t.dtype != torch.float32:
            raise ValueError(f"{name}: signs, codebooks and the sketch matrix must be float32, got {t.dtype}")
    if signs.numel() != head_dim:
        raise ValueError(f"{name}: signs must hold head_dim = {head_dim} values, got {signs.numel()}")


def _need_out(name: str, out: torch.Tensor, shape: tuple, device: torch.device) -> None:
    """A caller-supplied output must have exactly the rows the kernels write."""
    if tuple(out.shape) != tuple(shape) or out.dtype not in _DTYPES:
        raise ValueError(f"{name}: out must be {list(shape)} f32/f16/bf16, got {list(out.shape)} {out.dtype}")
    _need_cuda(name, out)
    if out.device != device:
        raise ValueError(f"{name}: out must be on {device}")


def _need_status(name: str, status: torch.Tensor | None, device: torch.device | None = None) -> None:
    """A caller-supplied status word: one int32 (at least) on the call's device."""
    if status is None:
        return
    if status.dtype != torch.int32 or status.numel() < 1 or status.device.type != "cuda" or \
            (device is not None and status.device != device):
        raise ValueError(f"{name}: status must be an int32 tensor of at least one element on the call's device")


def _bits_from_centroids(centroids: torch.Tensor) -> int:
    n = centroids.numel()
    bits = n.bit_length() - 1
    if n < 4 or (1 << bits) != n:
        raise ValueError(f"centroids must hold 2^bits values, got {n}")
    return bits


# ---------------------------------------------------------------- writer

def tq_write_kv(raw: torch.Tensor, pages: torch.Tensor, slots: torch.Tensor, signs: torch.Tensor,
                centroids: torch.Tensor, status: torch.Tensor | None = None, check: bool = True) -> torch.Tensor:
    """write_tq4_kv(raw, pages, slots, rotation, centroids): encode raw[T, H, D] into pages[NB, bs, H, RB].

    Returns the device status word.  With check=True the call synchronises on it and
    raises TQError(TQ_ERR_SLOT_OUT_OF_RANGE) when a slot was out of range (then no row
    was written).
    """
    dev = _need_cuda("tq_write_kv", raw, pages, slots, signs, centroids)
    if raw.dim() != 3 or pages.dim() != 4 or slots.dim() != 1 or slots.numel() != raw.shape[0]:
        raise ValueError("tq_write_kv: raw [T, H, D], pages [NB, bs, H, RB], slots [T] expected")
    if raw.dtype not in _DTYPES or pages.dtype != torch.uint8 or slots.dtype != torch.int64:
        raise ValueError("tq_write_kv: raw f32/f16/bf16, pages uint8, slots int64 expected")
    t, h, d = raw.shape
    bits = _bits_from_centroids(centroids)
    _need_f32("tq_write_kv", d, signs, centroids)
    if pages.shape[2] != h or pages.shape[3] != tq_row_bytes(d, bits):
        raise ValueError(f"tq_write_kv: pages {tuple(pages.shape)} do not match H={h}, RB={tq_row_bytes(d, bits)}")
    _need_status("tq_write_kv", status, dev)
    if status is None:
        status = _status_buffer(dev)
    with torch.cuda.device(dev):
        _check(lib().tq_write_kv(_ptr(raw), _DTYPES[raw.dtype], t, h, d, bits, _ptr(slots), _ptr(pages),
                                 pages.shape[0], pages.shape[1], _ptr(signs), _ptr(centroids), _ptr(status),
                                 _stream(dev)))
    if check:
        raise_for_device_status(status)
    return status


# ---------------------------------------------------------------- readback

def tq_dequant_rows(pages: torch.Tensor, slots: torch.Tensor, signs: torch.Tensor, centroids: torch.Tensor,
                    out: torch.Tensor | None = None, out_dtype: torch.dtype = torch.float16,
                    status: torch.Tensor | None = None, check: bool = True) -> torch.Tensor:
    """Dense readback (tq4_decompress) of the rows written at `slots`: out[T, H, D] =
    nu * R^T c[idx] for slot >= 0, zeros for slot < 0.  pages [NB, bs, H, RB] uint8,
    slots [T] int64.  With check=True the call synchronises and raises
    TQError(TQ_ERR_SLOT_OUT_OF_RANGE) when a slot lies past the pages.  Returns `out`."""
    index = pages.get_device()
    if pages.dim() != 4 or slots.dim() != 1 or pages.dtype is not torch.uint8 or slots.dtype is not torch.int64:
        raise ValueError("tq_dequant_rows: pages uint8 [NB, bs, H, RB] and slots int64 [T] expected")
    nb, bs, h, rb = pages.shape
    d, t = signs.numel(), slots.numel()
    bits = _bits_from_centroids(centroids)
    if not (index >= 0 and slots.get_device() == index and signs.get_device() == index and
            centroids.get_device() == index and pages.is_contiguous() and slots.is_contiguous() and
            signs.is_contiguous() and centroids.is_contiguous()):
        _need_cuda("tq_dequant_rows", pages, slots, signs, centroids)
    if signs.dtype is not torch.float32 or centroids.dtype is not torch.float32:
        _need_f32("tq_dequant_rows", d, signs, centroids)
    if d % 16 or rb * 8 != d * bits + 32 or not 2 <= bits <= 5:  # as tq_row_bytes has it for its head dims
        if rb != tq_row_bytes(d, bits):
            raise ValueError(f"tq_dequant_rows: pages row bytes {rb} != RB({d}, {bits})")
    if out is None:
        out = torch.empty((t, h, d), dtype=out_dtype, device=pages.device)
    if out.shape != (t, h, d) or out.dtype not in _DTYPES:
        raise ValueError(f"tq_dequant_rows: out must be [{t}, {h}, {d}] f32/f16/bf16")
    if out.get_device() != index or not out.is_contiguous():
        _need_cuda("tq_dequant_rows", pages, out)
    _need_status("tq_dequant_rows", status, pages.device)
    if status is None and check:
        status = _status_buffer(pages.device)
    with _on(index):
        code = lib().tq_dequant_rows(pages.data_ptr(), bits, nb, bs, h, d, slots.data_ptr(), t, signs.data_ptr(),
                                     centroids.data_ptr(), out.data_ptr(), _DTYPES[out.dtype], _ptr(status),
                                     _stream_ptr(index))
    if code != TQ_OK:
        _check(code)
    if check:
        raise_for_device_status(status)
    return out


# ---------------------------------------------------------------- decode

def tq_paged_decode_workspace(batch: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                              max_blocks_per_seq: int, block_size: int) -> int:
    return int(lib().tq_paged_decode_workspace(batch, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                                               block_size))


def tq_paged_decode(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                    seq_lens: torch.Tensor, signs: torch.Tensor, k_centroids: torch.Tensor,
                    v_centroids: torch.Tensor, scale: float | None = None, out: torch.Tensor | None = None,
                    out_dtype: torch.dtype | None = None, workspace: torch.Tensor | None = None,
                    status: torch.Tensor | None = None, check: bool = False) -> torch.Tensor:
    """decode_tq4_paged: attention of q[B, Hq, D] over packed K/V pages through block_table[B, maxblk]."""
    dev = _need_cuda("tq_paged_decode", q, k_pages, v_pages, block_table, seq_lens, signs, k_centroids,
                     v_centroids)
    if q.dim() != 3 or k_pages.dim() != 4 or v_pages.dim() != 4 or block_table.dim() != 2:
        raise ValueError("tq_paged_decode: q [B, Hq, D], pages [NB, bs, H, RB], block_table [B, maxblk] expected")
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32 or q.dtype not in _DTYPES:
        raise ValueError("tq_paged_decode: block_table / seq_lens int32, q f32/f16/bf16 expected")
    b, hq, d = q.shape
    nb, bs, h, _ = k_pages.shape
    kb, vb = _bits_from_centroids(k_centroids), _bits_from_centroids(v_centroids)
    _need_f32("tq_paged_decode", d, signs, k_centroids, v_centroids)
    if k_pages.shape[3] != tq_row_bytes(d, kb) or v_pages.shape[3] != tq_row_bytes(d, vb) or \
            tuple(v_pages.shape[:3]) != (nb, bs, h) or block_table.shape[0] != b or seq_lens.numel() != b:
        raise ValueError("tq_paged_decode: page / table shapes inconsistent with q and the codebooks")
    out_dtype = out_dtype or q.dtype
    if out is None:
        out = torch.empty((b, hq, d), dtype=out_dtype, device=dev)
    _need_out("tq_paged_decode", out, (b, hq, d), dev)
    _need_status("tq_paged_decode", status, dev)
    maxb = block_table.shape[1]
    need = tq_paged_decode_workspace(b, hq, h, d, maxb, bs)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        _check(lib().tq_paged_decode(_ptr(q), _DTYPES[q.dtype], b, hq, h, d, _ptr(k_pages), kb, _ptr(v_pages), vb,
                                     nb, bs, _ptr(block_table), maxb, _ptr(seq_lens), _ptr(signs),
                                     _ptr(k_centroids), _ptr(v_centroids), float(scale or 0.0), _ptr(out),
                                     _DTYPES[out.dtype], _ptr(workspace), workspace.numel(), _ptr(status),
                                     _stream(dev)))
    if check and status is not None:
        raise_for_device_status(status)
    return out


def tq_paged_prefill(q: torch.Tensor, q_seq: torch.Tensor, q_len: torch.Tensor, k_pages: torch.Tensor,
                     v_pages: torch.Tensor, block_table: torch.Tensor, signs: torch.Tensor, k_centroids: torch.Tensor,
                     v_centroids: torch.Tensor, scale: float | None = None, out: torch.Tensor | None = None,
                     out_dtype: torch.dtype | None = None, workspace: torch.Tensor | None = None,
                     status: torch.Tensor | None = None, check: bool = False) -> torch.Tensor:
    """Mixed prefill/decode over the packed pages: row i of q[T, Hq, D] is a query of sequence
    q_seq[i] that sees that sequence's first q_len[i] tokens (block_table[S, maxblk])."""
    dev = _need_cuda("tq_paged_prefill", q, q_seq, q_len, k_pages, v_pages, block_table, signs, k_centroids,
                     v_centroids)
    if q.dim() != 3 or k_pages.dim() != 4 or v_pages.dim() != 4 or block_table.dim() != 2:
        raise ValueError("tq_paged_prefill: q [T, Hq, D], pages [NB, bs, H, RB], block_table [S, maxblk] expected")
    if block_table.dtype != torch.int32 or q_seq.dtype != torch.int32 or q_len.dtype != torch.int32 or \
            q.dtype not in _DTYPES:
        raise ValueError("tq_paged_prefill: block_table / q_seq / q_len int32, q f32/f16/bf16 expected")
    t, hq, d = q.shape
    nb, bs, h, _ = k_pages.shape
    kb, vb = _bits_from_centroids(k_centroids), _bits_from_centroids(v_centroids)
    _need_f32("tq_paged_prefill", d, signs, k_centroids, v_centroids)
    if k_pages.shape[3] != tq_row_bytes(d, kb) or v_pages.shape[3] != tq_row_bytes(d, vb) or \
            tuple(v_pages.shape[:3]) != (nb, bs, h) or q_seq.numel() != t or q_len.numel() != t:
        raise ValueError("tq_paged_prefill: page / row shapes inconsistent with q and the codebooks")
    out_dtype = out_dtype or q.dtype
    if out is None:
        out = torch.empty((t, hq, d), dtype=out_dtype, device=dev)
    _need_out("tq_paged_prefill", out, (t, hq, d), dev)
    _need_status("tq_paged_prefill", status, dev)
    s_rows, maxb = block_table.shape
    need = int(lib().tq_paged_prefill_workspace(t, hq, h, d, maxb, bs))
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        _check(lib().tq_paged_prefill(_ptr(q), _DTYPES[q.dtype], t, hq, h, d, _ptr(k_pages), kb, _ptr(v_pages), vb,
                                      nb, bs, _ptr(block_table), s_rows, maxb, _ptr(q_seq), _ptr(q_len), _ptr(signs),
                                      _ptr(k_centroids), _ptr(v_centroids), float(scale or 0.0), _ptr(out),
                                      _DTYPES[out.dtype], _ptr(workspace), workspace.numel(), _ptr(status),
                                      _stream(dev)))
    if check and status is not None:
        raise_for_device_status(status)
    return out


def tq_quantize_queries_int8(q: torch.Tensor):
    """int8 codes [T, Hq, D] and fp32 scales [T, Hq] of queries q[T, Hq, D] (one symmetric
    scale per (row, q head))."""
    dev = _need_cuda("tq_quantize_queries_int8", q)
    if q.dim() != 3 or q.dtype not in _DTYPES or not q.is_contiguous():
        raise ValueError("tq_quantize_queries_int8: contiguous q [T, Hq, D] f32/f16/bf16 expected")
    t, hq, d = q.shape
    codes = torch.empty((t, hq, d), dtype=torch.int8, device=dev)
    scales = torch.empty((t, hq), dtype=torch.float32, device=dev)
    with torch.cuda.device(dev):
        _check(lib().tq_quantize_queries_int8(_ptr(q), _DTYPES[q.dtype], t, hq, d, _ptr(codes), _ptr(scales),
                                              _stream(dev)))
    return codes, scales


def tq_paged_prefill_int8q(q_codes: torch.Tensor, q_scales: torch.Tensor, q_seq: torch.Tensor, q_len: torch.Tensor,
                           k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                           signs: torch.Tensor, k_centroids: torch.Tensor, v_centroids: torch.Tensor,
                           scale: float | None = None, out: torch.Tensor | None = None,
                           out_dtype: torch.dtype = torch.float16, workspace: torch.Tensor | None = None,
                           status: torch.Tensor | None = None, check: bool = False) -> torch.Tensor:
    """tq_paged_prefill with int8 query codes [T, Hq, D] and their fp32 scales [T, Hq]."""
    dev = _need_cuda("tq_paged_prefill_int8q", q_codes, q_scales, q_seq, q_len, k_pages, v_pages, block_table, signs,
                     k_centroids, v_centroids)
    if q_codes.dim() != 3 or q_codes.dtype != torch.int8 or q_scales.dtype != torch.float32 or \
            tuple(q_scales.shape) != tuple(q_codes.shape[:2]) or not q_codes.is_contiguous() or \
            not q_scales.is_contiguous():
        raise ValueError("tq_paged_prefill_int8q: contiguous int8 codes [T, Hq, D] and float32 scales [T, Hq] "
                         "expected")
    if block_table.dtype != torch.int32 or q_seq.dtype != torch.int32 or q_len.dtype != torch.int32:
        raise ValueError("tq_paged_prefill_int8q: block_table / q_seq / q_len int32 expected")
    t, hq, d = q_codes.shape
    nb, bs, h, _ = k_pages.shape
    kb, vb = _bits_from_centroids(k_centroids), _bits_from_centroids(v_centroids)
    _need_f32("tq_paged_prefill_int8q", d, signs, k_centroids, v_centroids)
    if k_pages.shape[3] != tq_row_bytes(d, kb) or v_pages.shape[3] != tq_row_bytes(d, vb) or \
            tuple(v_pages.shape[:3]) != (nb, bs, h) or q_seq.numel() != t or q_len.numel() != t:
        raise ValueError("tq_paged_prefill_int8q: page / row shapes inconsistent with q and the codebooks")
    if out is None:
        out = torch.empty((t, hq, d), dtype=out_dtype, device=dev)
    _need_out("tq_paged_prefill_int8q", out, (t, hq, d), dev)
    _need_status("tq_paged_prefill_int8q", status, dev)
    s_rows, maxb = block_table.shape
    need = int(lib().tq_paged_prefill_workspace(t, hq, h, d, maxb, bs))
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        _check(lib().tq_paged_prefill_int8q(_ptr(q_codes), _ptr(q_scales), t, hq, h, d, _ptr(k_pages), kb,
                                            _ptr(v_pages), vb, nb, bs, _ptr(block_table), s_rows, maxb, _ptr(q_seq),
                                            _ptr(q_len), _ptr(signs), _ptr(k_centroids), _ptr(v_centroids),
                                            float(scale or 0.0), _ptr(out), _DTYPES[out.dtype], _ptr(workspace),
                                            workspace.numel(), _ptr(status), _stream(dev)))
    if check and status is not None:
        raise_for_device_status(status)
    return out


def tq_paged_decode_static(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                           seq_lens: torch.Tensor, signs: torch.Tensor, k_centroids: torch.Tensor,
                           v_centroids: torch.Tensor, out: torch.Tensor, scale: float | None = None,
                           status: torch.Tensor | None = None) -> torch.Tensor:
    """Allocation-free decode for callers that cannot allocate device memory: the caller
    passes `out`, and the split-K partials go to the library's fixed 16 MiB device array
    (so concurrent calls on different streams race; serialise them)."""
    dev = _need_cuda("tq_paged_decode_static", q, k_pages, v_pages, block_table, seq_lens, signs, k_centroids,
                     v_centroids, out)
    b, hq, d = q.shape
    nb, bs, h, _ = k_pages.shape
    kb, vb = _bits_from_centroids(k_centroids), _bits_from_centroids(v_centroids)
    _need_f32("tq_paged_decode_static", d, signs, k_centroids, v_centroids)
    if out.shape != q.shape or out.dtype not in _DTYPES:
        raise ValueError("tq_paged_decode_static: out must be [B, Hq, D] f32/f16/bf16")
    _need_status("tq_paged_decode_static", status, dev)
    with torch.cuda.device(dev):
        _check(lib().tq_paged_decode_static(_ptr(q), _DTYPES[q.dtype], b, hq, h, d, _ptr(k_pages), kb,
                                            _ptr(v_pages), vb, nb, bs, _ptr(block_table), block_table.shape[1],
                                            _ptr(seq_lens), _ptr(signs), _ptr(k_centroids), _ptr(v_centroids),
                                            float(scale or 0.0), _ptr(out), _DTYPES[out.dtype], _ptr(status),
                                            _stream(dev)))
    return out


# ---------------------------------------------------------------- product-quantised keys

def tq_prod_row_bytes(head_dim: int, bits: int) -> int:
    """Bytes of one product-quantised key row: (bits-1)-bit indices, D sign bits, nu, gamma."""
    n = lib().tq_prod_row_bytes(int(head_dim), int(bits))
    if n < 0:
        raise TQError(TQ_ERR_UNSUPPORTED, f"head_dim {head_dim} / bits {bits} unsupported")
    return int(n)


def tq_build_qjl_matrix(head_dim: int, seed: int, device=None) -> torch.Tensor:
    """The N(0, 1) sketch matrix S, float32 [head_dim, head_dim] (host, or moved to `device`)."""
    out = torch.empty(int(head_dim), int(head_dim), dtype=torch.float32)
    _check(lib().tq_build_qjl_matrix(int(head_dim), int(seed) & ((1 << 64) - 1), out.data_ptr()))
    return out if device is None else out.to(device)


def tq_write_kv_prod(raw: torch.Tensor, pages: torch.Tensor, slots: torch.Tensor, signs: torch.Tensor,
                     mse_centroids: torch.Tensor, qjl_matrix: torch.Tensor, status: torch.Tensor | None = None,
                     check: bool = True) -> torch.Tensor:
    """Product-quantised key rows: encode raw[T, H, D] into pages[NB, bs, H, RBP] at
    bits = log2(len(mse_centroids)) + 1.  Same slot rules and status as tq_write_kv."""
    dev = _need_cuda("tq_write_kv_prod", raw, pages, slots, signs, mse_centroids, qjl_matrix)
    if raw.dim() != 3 or pages.dim() != 4 or slots.dim() != 1 or slots.numel() != raw.shape[0]:
        raise ValueError("tq_write_kv_prod: raw [T, H, D], pages [NB, bs, H, RBP], slots [T] expected")
    if raw.dtype not in _DTYPES or pages.dtype != torch.uint8 or slots.dtype != torch.int64 or \
            qjl_matrix.dtype != torch.float32:
        raise ValueError("tq_write_kv_prod: raw f32/f16/bf16, pages uint8, slots int64, qjl_matrix f32 expected")
    t, h, d = raw.shape
    n = mse_centroids.numel()
    bits = n.bit_length()
    if n < 2 or (1 << (bits - 1)) != n:
        raise ValueError(f"tq_write_kv_prod: mse_centroids must hold 2^(bits-1) values, got {n}")
    if tuple(qjl_matrix.shape) != (d, d):
        raise ValueError(f"tq_write_kv_prod: qjl_matrix must be [{d}, {d}]")
    _need_f32("tq_write_kv_prod", d, signs, mse_centroids)
    if pages.shape[2] != h or pages.shape[3] != tq_prod_row_bytes(d, bits):
        raise ValueError(f"tq_write_kv_prod: pages {tuple(pages.shape)} do not match H={h}, "
                         f"RBP={tq_prod_row_bytes(d, bits)}")
    _need_status("tq_write_kv_prod", status, dev)
    if status is None:
        status = _status_buffer(dev)
    with torch.cuda.device(dev):
        _check(lib().tq_write_kv_prod(_ptr(raw), _DTYPES[raw.dtype], t, h, d, bits, _ptr(slots), _ptr(pages),
                                      pages.shape[0], pages.shape[1], _ptr(signs), _ptr(mse_centroids),
                                      _ptr(qjl_matrix), _ptr(status), _stream(dev)))
    if check:
        raise_for_device_status(status)
    return status


def tq_paged_decode_prod(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                         seq_lens: torch.Tensor, signs: torch.Tensor, k_mse_centroids: torch.Tensor,
                         v_centroids: torch.Tensor, qjl_matrix: torch.Tensor, scale: float | None = None,
                         out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                         workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                         check: bool = False) -> torch.Tensor:
    """tq_paged_decode with product-quantised key pages (k_bits = log2(len(k_mse_centroids)) + 1)."""
    dev = _need_cuda("tq_paged_decode_prod", q, k_pages, v_pages, block_table, seq_lens, signs, k_mse_centroids,
                     v_centroids, qjl_matrix)
    if q.dim() != 3 or k_pages.dim() != 4 or v_pages.dim() != 4 or block_table.dim() != 2:
        raise ValueError("tq_paged_decode_prod: q [B, Hq, D], pages [NB, bs, H, RB], block_table [B, maxblk] expected")
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32 or q.dtype not in _DTYPES:
        raise ValueError("tq_paged_decode_prod: block_table / seq_lens int32, q f32/f16/bf16 expected")
    b, hq, d = q.shape
    nb, bs, h, _ = k_pages.shape
    n = k_mse_centroids.numel()
    kb = n.bit_length()
    if n < 2 or (1 << (kb - 1)) != n:
        raise ValueError(f"tq_paged_decode_prod: k_mse_centroids must hold 2^(k_bits-1) values, got {n}")
    vb = _bits_from_centroids(v_centroids)
    _need_f32("tq_paged_decode_prod", d, signs, k_mse_centroids, v_centroids, qjl_matrix)
    if k_pages.shape[3] != tq_prod_row_bytes(d, kb) or v_pages.shape[3] != tq_row_bytes(d, vb) or \
            tuple(v_pages.shape[:3]) != (nb, bs, h) or block_table.shape[0] != b or seq_lens.numel() != b or \
            tuple(qjl_matrix.shape) != (d, d):
        raise ValueError("tq_paged_decode_prod: page / table / matrix shapes inconsistent with q and the codebooks")
    out_dtype = out_dtype or q.dtype
    if out is None:
        out = torch.empty((b, hq, d), dtype=out_dtype, device=dev)
    _need_out("tq_paged_decode_prod", out, (b, hq, d), dev)
    _need_status("tq_paged_decode_prod", status, dev)
    maxb = block_table.shape[1]
    need = int(lib().tq_paged_decode_prod_workspace(b, hq, h, d, maxb, bs))
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        _check(lib().tq_paged_decode_prod(_ptr(q), _DTYPES[q.dtype], b, hq, h, d, _ptr(k_pages), kb, _ptr(v_pages),
                                          vb, nb, bs, _ptr(block_table), maxb, _ptr(seq_lens), _ptr(signs),
                                          _ptr(k_mse_centroids), _ptr(v_centroids), _ptr(qjl_matrix),
                                          float(scale or 0.0), _ptr(out), _DTYPES[out.dtype], _ptr(workspace),
                                          workspace.numel(), _ptr(status), _stream(dev)))
    if check and status is not None:
        raise_for_device_status(status)
    return out


# ---------------------------------------------------------------- recipe modes

def _recipe_id(recipe) -> int:
    if isinstance(recipe, str):
        if recipe not in RECIPES:
            raise ValueError(f"unknown recipe {recipe!r}")
        return RECIPES[recipe]
    return int(recipe)


def tq_recipe_row_bytes(recipe, head_dim: int) -> int:
    rb = int(lib().tq_recipe_row_bytes(_recipe_id(recipe), int(head_dim)))
    if rb < 0:
        raise ValueError(f"recipe {recipe!r} at head_dim {head_dim} is not supported")
    return rb


def tq_recipe_channel_order(recipe, head_dim: int, high) -> torch.Tensor:
    """Checks the metadata's high groups [H, head_dim / 2] and returns the channel order
    int32 [H, head_dim] (high group, then the rest ascending) on the host."""
    high = torch.as_tensor(high).to(torch.int32).contiguous().cpu()
    if high.dim() != 2 or high.shape[1] * 2 != int(head_dim):
        raise ValueError(f"tq_recipe_channel_order: high groups must be [H, {int(head_dim) // 2}], got "
                         f"{tuple(high.shape)}")
    order = torch.empty(high.shape[0], int(head_dim), dtype=torch.int32)
    _check(lib().tq_recipe_channel_order(_recipe_id(recipe), int(head_dim), high.shape[0], high.data_ptr(),
                                         order.data_ptr()))
    return order


def tq_recipe_calibrate(recipe, samples) -> torch.Tensor:
    """High groups int32 [H, D / 2] from calibration rows samples[N, H, D] (host)."""
    x = torch.as_tensor(samples).to(torch.float32).contiguous().cpu()
    if x.dim() != 3:
        raise ValueError("tq_recipe_calibrate: samples must be [N, H, D]")
    n, h, d = x.shape
    high = torch.empty(h, d // 2, dtype=torch.int32)
    _check(lib().tq_recipe_calibrate(_recipe_id(recipe), d, h, x.data_ptr(), n, high.data_ptr()))
    return high


class RecipeCodec:
    """The shared group codec of a recipe at one head_dim, on a device: the signs of R_d
    (seed 42), the MSE codebooks of both groups and S_d (seed 43), d = head_dim / 2."""

    def __init__(self, recipe, head_dim: int, device=None):
        rid = _recipe_id(recipe)
        bits = {TQ_RECIPE_TURBOQUANT25: (3, 2), TQ_RECIPE_TURBOQUANT35: (4, 3)}.get(rid)
        if bits is None:
            raise ValueError(f"unknown recipe {recipe!r}")
        self.recipe, self.head_dim, self.d, self.bits = rid, int(head_dim), int(head_dim) // 2, bits
        self.row_bytes = tq_recipe_row_bytes(rid, head_dim)
        self.signs = tq_build_rotation(self.d, RECIPE_ROTATION_SEED, device)
        self.mse_high = tq_codebook(self.d, bits[0] - 1, device)[0]
        self.mse_low = tq_codebook(self.d, bits[1] - 1, device)[0]
        self.smat = tq_build_qjl_matrix(self.d, RECIPE_SKETCH_SEED, device)


def _need_order(name: str, order: torch.Tensor, h: int, d: int, device) -> None:
    if order.dtype != torch.int32 or tuple(order.shape) != (h, d) or not order.is_contiguous() or \
            order.device != device:
        raise ValueError(f"{name}: channel order must be contiguous int32 [{h}, {d}] on {device}")


def tq_write_kv_recipe(raw: torch.Tensor, pages: torch.Tensor, slots: torch.Tensor, order: torch.Tensor,
                       codec: RecipeCodec, status: torch.Tensor | None = None, check: bool = True) -> torch.Tensor:
    """Encode raw[T, H, D] into recipe pages[NB, bs, H, RB] (tq_write_kv's slot rules)."""
    dev = _need_cuda("tq_write_kv_recipe", raw, pages, slots, order, codec.signs, codec.smat)
    if raw.dim() != 3 or pages.dim() != 4 or slots.dim() != 1 or slots.numel() != raw.shape[0]:
        raise ValueError("tq_write_kv_recipe: raw [T, H, D], pages [NB, bs, H, RB], slots [T] expected")
    if raw.dtype not in _DTYPES or pages.dtype != torch.uint8 or slots.dtype != torch.int64:
        raise ValueError("tq_write_kv_recipe: raw f32/f16/bf16, pages uint8, slots int64 expected")
    t, h, d = raw.shape
    if d != codec.head_dim or pages.shape[2] != h or pages.shape[3] != codec.row_bytes:
        raise ValueError("tq_write_kv_recipe: raw / pages do not match the codec's head_dim and row bytes")
    _need_order("tq_write_kv_recipe", order, h, d, dev)
    _need_status("tq_write_kv_recipe", status, dev)
    if status is None:
        status = _status_buffer(dev)
    with torch.cuda.device(dev):
        _check(lib().tq_write_kv_recipe(_ptr(raw), _DTYPES[raw.dtype], t, h, d, codec.recipe, _ptr(slots),
                                        _ptr(pages), pages.shape[0], pages.shape[1], _ptr(order), _ptr(codec.signs),
                                        _ptr(codec.mse_high), _ptr(codec.mse_low), _ptr(codec.smat), _ptr(status),
                                        _stream(dev)))
    if check:
        raise_for_device_status(status)
    return status


def tq_paged_decode_recipe(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                           seq_lens: torch.Tensor, order: torch.Tensor, codec: RecipeCodec,
                           scale: float | None = None, out: torch.Tensor | None = None,
                           out_dtype: torch.dtype | None = None, workspace: torch.Tensor | None = None,
                           status: torch.Tensor | None = None, check: bool = False) -> torch.Tensor:
    """tq_paged_decode over recipe K and V pages."""
    dev = _need_cuda("tq_paged_decode_recipe", q, k_pages, v_pages, block_table, seq_lens, order, codec.signs)
    if q.dim() != 3 or k_pages.dim() != 4 or v_pages.dim() != 4 or block_table.dim() != 2:
        raise ValueError("tq_paged_decode_recipe: q [B, Hq, D], pages [NB, bs, H, RB], block_table [B, maxblk] "
                         "expected")
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32 or q.dtype not in _DTYPES:
        raise ValueError("tq_paged_decode_recipe: block_table / seq_lens int32, q f32/f16/bf16 expected")
    b, hq, d = q.shape
    nb, bs, h, rb = k_pages.shape
    if d != codec.head_dim or rb != codec.row_bytes or tuple(v_pages.shape) != tuple(k_pages.shape) or \
            block_table.shape[0] != b or seq_lens.numel() != b:
        raise ValueError("tq_paged_decode_recipe: page / table shapes inconsistent with q and the codec")
    _need_order("tq_paged_decode_recipe", order, h, d, dev)
    out_dtype = out_dtype or q.dtype
    if out is None:
        out = torch.empty((b, hq, d), dtype=out_dtype, device=dev)
    _need_out("tq_paged_decode_recipe", out, (b, hq, d), dev)
    _need_status("tq_paged_decode_recipe", status, dev)
    maxb = block_table.shape[1]
    need = int(lib().tq_paged_decode_recipe_workspace(b, hq, h, d, maxb, bs))
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    with torch.cuda.device(dev):
        _check(lib().tq_paged_decode_recipe(_ptr(q), _DTYPES[q.dtype], b, hq, h, d, _ptr(k_pages), _ptr(v_pages),
                                            codec.recipe, nb, bs, _ptr(block_table), maxb, _ptr(seq_lens),
                                            _ptr(order), _ptr(codec.signs), _ptr(codec.mse_high),
                                            _ptr(codec.mse_low), _ptr(codec.smat), float(scale or 0.0), _ptr(out),
                                            _DTYPES[out.dtype], _ptr(workspace), workspace.numel(), _ptr(status),
                                            _stream(dev)))
    if check and status is not None:
        raise_for_device_status(status)
    return out


# ---------------------------------------------------------------- serving steps

class StepPlan(NamedTuple):
    """Outputs of tq_plan_step: the rows of the step and the state after it."""
    slots: torch.Tensor       # int64 [max_rows]
    q_seq: torch.Tensor       # int32 [max_rows]
    q_len: torch.Tensor       # int32 [max_rows]
    row_start: torch.Tensor   # int32 [S + 1]
    seq_lens: torch.Tensor    # int32 [S]
    seq_blocks: torch.Tensor  # int32 [S]
    free_state: torch.Tensor  # int32 [2]


def _need_like(name: str, index: int, **want) -> None:
    """Every named (tensor, dtype, shape) is a contiguous tensor of that dtype and shape on CUDA
    device `index`."""
    for what, (t, dtype, shape) in want.items():
        if t.get_device() != index or index < 0:
            raise ValueError(f"{name}: all tensors must be on the same CUDA device ({what} is on {t.device})")
        if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name}: {what} must be a contiguous {dtype} {list(shape)}, got {t.dtype} "
                             f"{list(t.shape)}")


_NO_SWITCH = contextlib.nullcontext()


def _on(index: int):
    """Makes device `index` current for a call (nothing to do where it is)."""
    return _NO_SWITCH if torch.cuda.current_device() == index else torch.cuda.device(index)


# The current stream of a device, as the library takes it (without the Stream object where torch
# gives the pointer itself).
_stream_ptr = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _plain(t: torch.Tensor, dtype: torch.dtype, shape: tuple, index: int) -> bool:
    """Whether _need_like would let `t` pass."""
    return t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous()


def tq_plan_step(seq_lens: torch.Tensor, new_lens: torch.Tensor, seq_blocks: torch.Tensor, block_table: torch.Tensor,
                 free_blocks: torch.Tensor, free_state: torch.Tensor, block_size: int, max_rows: int,
                 out: StepPlan | None = None, status: torch.Tensor | None = None, check: bool = False) -> StepPlan:
    """Plans a step on the device: appends new_lens[s] tokens to each sequence (negative:
    finished, its blocks are returned), taking new blocks from the ring free_blocks[NB] whose
    {head, count} is free_state[2].  block_table[S, W] and free_blocks are updated in place; the
    state after the step is in the result, whose seq_lens / seq_blocks / free_state may be the
    inputs themselves (pass them in `out`).  With check=True the call synchronises and raises
    TQError(TQ_ERR_OUT_OF_BLOCKS / TQ_ERR_INVALID_ARG), with nothing planned."""
    name = "tq_plan_step"
    dev, i32, index = seq_lens.device, torch.int32, seq_lens.get_device()
    if block_table.dim() != 2 or free_blocks.dim() != 1:
        raise ValueError(f"{name}: block_table [S, W] and free_blocks [NB] expected")
    s, w = block_table.shape
    max_rows = int(max_rows)
    if max_rows < 0:
        raise ValueError(f"{name}: max_rows {max_rows} < 0")
    if out is None:
        if index < 0:
            raise ValueError(f"{name}: all tensors must be on the same CUDA device (seq_lens is on {dev})")
        slots = torch.empty(max_rows, dtype=torch.int64, device=dev)
        q_seq, q_len, row_start, lens, blocks, state = torch.empty(2 * max_rows + 3 * s + 3, dtype=i32, device=dev).split(
            [max_rows, max_rows, s + 1, s, s, 2])
        out = StepPlan(slots, q_seq, q_len, row_start, lens, blocks, state)
    else:
        _need_like(name, index, slots=(out.slots, torch.int64, (max_rows,)), q_seq=(out.q_seq, i32, (max_rows,)),
                   q_len=(out.q_len, i32, (max_rows,)), row_start=(out.row_start, i32, (s + 1,)),
                   seq_lens_out=(out.seq_lens, i32, (s,)), seq_blocks_out=(out.seq_blocks, i32, (s,)),
                   free_state_out=(out.free_state, i32, (2,)))
    _need_like(name, index, seq_lens=(seq_lens, i32, (s,)), new_lens=(new_lens, i32, (s,)),
               seq_blocks=(seq_blocks, i32, (s,)), block_table=(block_table, i32, (s, w)),
               free_blocks=(free_blocks, i32, (free_blocks.numel(),)), free_state=(free_state, i32, (2,)))
    _need_status(name, status, dev)
    if status is None and check:
        status = _status_buffer(dev)
    with _on(index):
        code = lib().tq_plan_step(seq_lens.data_ptr(), new_lens.data_ptr(), seq_blocks.data_ptr(), s,
                                  block_table.data_ptr(), w, free_blocks.data_ptr(), free_state.data_ptr(),
                                  free_blocks.numel(), int(block_size), max_rows, out.slots.data_ptr(),
                                  out.q_seq.data_ptr(), out.q_len.data_ptr(), out.row_start.data_ptr(),
                                  out.seq_lens.data_ptr(), out.seq_blocks.data_ptr(), out.free_state.data_ptr(),
                                  _ptr(status), _stream_ptr(index))
    if code != TQ_OK:
        _check(code)
    if check:
        raise_for_device_status(status)
    return out


def tq_commit_tree(k_pages: torch.Tensor | None, v_pages: torch.Tensor | None, block_table: torch.Tensor,
                   ctx_lens: torch.Tensor, path: torch.Tensor, path_lens: torch.Tensor,
                   seq_lens: torch.Tensor | None = None, status: torch.Tensor | None = None,
                   check: bool = False) -> torch.Tensor:
    """Moves the accepted rows of a verified tree: token ctx + path[s, j] to token ctx + j for
    j < path_lens[s] (path[S, P] strictly ascending), in both page tensors [NB, bs, H, RB].
    Returns the new lengths ctx + path_lens (written to `seq_lens`, which may be ctx_lens)."""
    name = "tq_commit_tree"
    pages = k_pages if k_pages is not None else v_pages
    if pages is None or pages.dim() != 4 or block_table.dim() != 2 or path.dim() != 2:
        raise ValueError(f"{name}: pages [NB, bs, H, RB], block_table [S, W] and path [S, P] expected")
    nb, bs, h, _ = pages.shape
    s, w = block_table.shape
    dev, i32, index = pages.device, torch.int32, pages.get_device()
    if seq_lens is None:
        seq_lens = torch.empty(s, dtype=i32, device=dev)
    rb = [0, 0]
    for i, (what, t) in enumerate((("k_pages", k_pages), ("v_pages", v_pages))):
        if t is not None:
            rb[i] = t.shape[-1]
            _need_like(name, index, **{what: (t, torch.uint8, (nb, bs, h, rb[i]))})
    _need_like(name, index, block_table=(block_table, i32, (s, w)), ctx_lens=(ctx_lens, i32, (s,)),
               path=(path, i32, (s, path.shape[1])), path_lens=(path_lens, i32, (s,)), seq_lens=(seq_lens, i32, (s,)))
    _need_status(name, status, dev)
    if status is None and check:
        status = _status_buffer(dev)
    with _on(index):
        code = lib().tq_commit_tree(_ptr(k_pages), rb[0], _ptr(v_pages), rb[1], nb, bs, h, block_table.data_ptr(), s, w,
                                    ctx_lens.data_ptr(), path.data_ptr(), path_lens.data_ptr(), path.shape[1],
                                    seq_lens.data_ptr(), _ptr(status), _stream_ptr(index))
    if code != TQ_OK:
        _check(code)
    if check:
        raise_for_device_status(status)
    return seq_lens


_TREE_WORKSPACE: dict = {}


def tq_paged_tree_workspace(num_q_rows: int, num_q_heads: int, num_kv_heads: int, head_dim: int) -> int:
    """Workspace bytes of tq_paged_tree and tq_paged_prefill_biased on the current device."""
    key = (torch.cuda.current_device(), num_q_rows, num_q_heads, num_kv_heads, head_dim)
    need = _TREE_WORKSPACE.get(key)
    if need is None:
        need = int(lib().tq_paged_tree_workspace(num_q_rows, num_q_heads, num_kv_heads, head_dim))
        if len(_TREE_WORKSPACE) > 4096:
            _TREE_WORKSPACE.clear()
        _TREE_WORKSPACE[key] = need
    return need


def _attn_call(name: str, q, q_seq, k_pages, v_pages, block_table, signs, k_centroids, v_centroids, out, out_dtype,
               workspace, status, check, more, middle, tail, fn):
    """Checks shared by tq_paged_tree and tq_paged_prefill_biased, and the call: `more` their
    own tensors for _need_like (given the sizes), `middle` and `tail` their arguments."""
    if q.dim() != 3 or k_pages.dim() != 4 or v_pages.dim() != 4 or block_table.dim() != 2:
        raise ValueError(f"{name}: q [T, Hq, D], pages [NB, bs, H, RB], block_table [S, W] expected")
    if q.dtype not in _DTYPES:
        raise ValueError(f"{name}: q f32/f16/bf16 expected")
    t, hq, d = q.shape
    nb, bs, h, rbk = k_pages.shape
    rbv = v_pages.shape[3]
    s, w = block_table.shape
    dev, i32, f32, u8, index = q.device, torch.int32, torch.float32, torch.uint8, q.get_device()
    kb, vb = _bits_from_centroids(k_centroids), _bits_from_centroids(v_centroids)
    if rbk * 8 != d * kb + 32 or rbv * 8 != d * vb + 32:  # head dims are multiples of 16
        raise ValueError(f"{name}: page rows of {rbk} / {rbv} bytes do not match head_dim {d} at {kb} / {vb} bits")
    if out is None:
        out = torch.empty((t, hq, d), dtype=out_dtype or q.dtype, device=dev)
    elif out.dtype not in _DTYPES:
        raise ValueError(f"{name}: out must be f32/f16/bf16, got {out.dtype}")
    else:
        _need_like(name, index, out=(out, out.dtype, (t, hq, d)))
    _need_like(name, index, q=(q, q.dtype, (t, hq, d)), k_pages=(k_pages, u8, (nb, bs, h, rbk)),
               v_pages=(v_pages, u8, (nb, bs, h, rbv)), block_table=(block_table, i32, (s, w)), q_seq=(q_seq, i32, (t,)),
               signs=(signs, f32, (d,)), k_centroids=(k_centroids, f32, (1 << kb,)),
               v_centroids=(v_centroids, f32, (1 << vb,)), **more(t, hq, s, i32))
    _need_status(name, status, dev)
    with _on(index):
        need = tq_paged_tree_workspace(t, hq, h, d)
        if workspace is None:
            workspace = torch.empty(max(need, 256), dtype=u8, device=dev)
        elif workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError(f"{name}: workspace must be contiguous on {dev}")
        if status is None and check:
            status = _status_buffer(dev)
        code = fn(q.data_ptr(), _DTYPES[q.dtype], t, hq, h, d, k_pages.data_ptr(), kb, v_pages.data_ptr(), vb, nb, bs,
                  block_table.data_ptr(), s, w, q_seq.data_ptr(), *middle, signs.data_ptr(), k_centroids.data_ptr(),
                  v_centroids.data_ptr(), *tail, out.data_ptr(), _DTYPES[out.dtype], workspace.data_ptr(),
                  workspace.numel() * workspace.element_size(), _ptr(status), _stream_ptr(index))
    if code != TQ_OK:
        _check(code)
    if check:
        raise_for_device_status(status)
    return out


def tq_paged_tree(q: torch.Tensor, q_seq: torch.Tensor, ctx_lens: torch.Tensor, tree_mask: torch.Tensor,
                  k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor, signs: torch.Tensor,
                  k_centroids: torch.Tensor, v_centroids: torch.Tensor, scale: float | None = None,
                  softcap: float = 0.0, out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                  workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                  check: bool = False) -> torch.Tensor:
    """Attention of drafted tokens: row i of q[T, Hq, D] sees the first ctx_lens[q_seq[i]]
    tokens of its sequence and, behind them, token ctx + j for every set bit j of its mask
    (bit j % 32 of tree_mask[i, j // 32], int32 [T, words]).  q_seq -1 is a padding row."""
    if tree_mask.dim() != 2:
        raise ValueError("tq_paged_tree: tree_mask [T, words] expected")
    words = tree_mask.shape[1]
    return _attn_call("tq_paged_tree", q, q_seq, k_pages, v_pages, block_table, signs, k_centroids, v_centroids, out,
                      out_dtype, workspace, status, check,
                      lambda t, hq, s, i32: dict(ctx_lens=(ctx_lens, i32, (s,)), tree_mask=(tree_mask, i32, (t, words))),
                      (ctx_lens.data_ptr(), tree_mask.data_ptr(), words), (float(scale or 0.0), float(softcap)),
                      lib().tq_paged_tree)


def tq_paged_prefill_biased(q: torch.Tensor, q_seq: torch.Tensor, q_len: torch.Tensor, k_pages: torch.Tensor,
                            v_pages: torch.Tensor, block_table: torch.Tensor, signs: torch.Tensor,
                            k_centroids: torch.Tensor, v_centroids: torch.Tensor, scale: float | None = None,
                            softcap: float = 0.0, window: int = 0, alibi_slopes: torch.Tensor | None = None,
                            prefix_lens: torch.Tensor | None = None, doc_starts: torch.Tensor | None = None,
                            out: torch.Tensor | None = None, out_dtype: torch.dtype | None = None,
                            workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                            check: bool = False) -> torch.Tensor:
    """tq_paged_prefill with modified scores and visible sets: scores capped at `softcap` by a
    tanh, minus alibi_slopes[Hq] times the distance; row i sees tokens t >= doc_starts[i] with
    t < prefix_lens[q_seq[i]] or q_len[i] - window <= t < q_len[i] (window 0: all before it)."""
    def more(t, hq, s, i32):
        want = dict(q_len=(q_len, i32, (t,)))
        if alibi_slopes is not None:
            want["alibi_slopes"] = (alibi_slopes, torch.float32, (hq,))
        if prefix_lens is not None:
            want["prefix_lens"] = (prefix_lens, i32, (s,))
        if doc_starts is not None:
            want["doc_starts"] = (doc_starts, i32, (t,))
        return want

    return _attn_call("tq_paged_prefill_biased", q, q_seq, k_pages, v_pages, block_table, signs, k_centroids,
                      v_centroids, out, out_dtype, workspace, status, check, more,
                      (q_len.data_ptr(), _ptr(prefix_lens), _ptr(doc_starts), int(window), _ptr(alibi_slopes)),
                      (float(scale or 0.0), float(softcap)), lib().tq_paged_prefill_biased)


# ---------------------------------------------------------------- norms, position rotation, append

def tq_build_rope(rot_dim: int, num_positions: int, base: float = 10000.0, inv_freq: torch.Tensor | None = None,
                  device=None) -> torch.Tensor:
    """cos / sin table float32 [num_positions, rot_dim]: rot_dim / 2 cosines of position *
    inv_freq[i] (base^(-2 i / rot_dim) by default), then the sines."""
    if inv_freq is not None:
        inv_freq = torch.as_tensor(inv_freq).to(torch.float64).contiguous().cpu()
        if inv_freq.numel() * 2 != int(rot_dim):
            raise ValueError(f"tq_build_rope: inv_freq must hold rot_dim / 2 = {int(rot_dim) // 2} values")
    rot_dim = _i32("tq_build_rope", "rot_dim", rot_dim)
    out = torch.empty(max(0, int(num_positions)), max(0, rot_dim), dtype=torch.float32)
    _check(lib().tq_build_rope(rot_dim, int(num_positions), float(base), _ptr(inv_freq), out.data_ptr()))
    return out if device is None else out.to(device)


def _i32(name: str, what: str, value: int) -> int:
    """A number that the library takes in 32 bits (ctypes would cut it off)."""
    value = int(value)
    if not -1 << 31 <= value < 1 << 31:
        raise ValueError(f"{name}: {what} {value} does not fit 32 bits")
    return value


# Codebook sizes and their bits.
_BITS = {4: 2, 8: 3, 16: 4, 32: 5}


def _rows(t: torch.Tensor, dtype: torch.dtype, shape: tuple, index: int) -> bool:
    """Whether t is head rows [T, heads, D] whose heads are contiguous."""
    st = t.stride()
    return t.dtype is dtype and t.shape == shape and st[2] == 1 and (st[1] == shape[2] or shape[1] == 1) and \
        t.get_device() == index


def _explain_rows(name: str, what: str, t: torch.Tensor, dtype: torch.dtype, shape: tuple, index: int) -> None:
    """The error of a tensor that _rows does not let pass (none where it does)."""
    if t.get_device() != index or index < 0:
        raise ValueError(f"{name}: all tensors must be on the same CUDA device ({what} is on {t.device})")
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: {what} must be {dtype} {list(shape)}, got {t.dtype} {list(t.shape)}")
    if not _rows(t, dtype, shape, index):
        raise ValueError(f"{name}: the heads of a token of {what} must be contiguous")


def _rope_args(name: str, index: int, tokens: int, d: int, positions, position_offset, cos_sin, interleaved, q_weight,
               k_weight, eps):
    """Checks and arguments of the position rotation and the norms."""
    f32, rows, rot, pp, cp = torch.float32, 0, 0, None, None
    if positions is not None:
        if not _plain(positions, torch.int32, (tokens,), index):
            _need_like(name, index, positions=(positions, torch.int32, (tokens,)))
        pp = positions.data_ptr()
    if cos_sin is not None:
        if cos_sin.dim() != 2 or positions is None:
            raise ValueError(f"{name}: cos_sin [P, rot_dim] comes with positions [T]")
        rows, rot = cos_sin.shape
        if not _plain(cos_sin, f32, (rows, rot), index):
            _need_like(name, index, cos_sin=(cos_sin, f32, (rows, rot)))
        if rows * rot == 0:
            raise ValueError(f"{name}: cos_sin {[rows, rot]} is empty")
        cp = cos_sin.data_ptr()
    qw = kw = None
    if q_weight is not None:
        if not _plain(q_weight, f32, (d,), index):
            _need_like(name, index, q_weight=(q_weight, f32, (d,)))
        qw = q_weight.data_ptr()
    if k_weight is not None:
        if not _plain(k_weight, f32, (d,), index):
            _need_like(name, index, k_weight=(k_weight, f32, (d,)))
        kw = k_weight.data_ptr()
    return pp, _i32(name, "position_offset", position_offset), cp, rows, rot, 1 if interleaved else 0, qw, kw, float(eps)


def tq_norm_rope(q: torch.Tensor | None, k: torch.Tensor | None, positions: torch.Tensor | None = None,
                 cos_sin: torch.Tensor | None = None, q_weight: torch.Tensor | None = None,
                 k_weight: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False,
                 position_offset: int = 0, q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                 status: torch.Tensor | None = None, check: bool = False):
    """Norm (weights [D], or none) of every head of q[T, Hq, D] and k[T, H, D], then the rotation by
    the table row of positions[t] + position_offset.  q and k may be slices of one projection's output
    (any token stride), q_out and k_out q and k themselves.  A token at a negative position is left
    out.  Returns (q_out, k_out)."""
    name = "tq_norm_rope"
    x = q if q is not None else k
    if x is None or x.dim() != 3 or x.dtype not in _DTYPES:
        raise ValueError(f"{name}: q [T, Hq, D] or k [T, H, D], f32/f16/bf16, expected")
    t, h, d = x.shape
    dtype, index = x.dtype, x.get_device()
    if index < 0:
        raise ValueError(f"{name}: all tensors must be on the same CUDA device (got {x.device})")
    qp = qo = kp = ko = None
    qs = qos = ks = kos = hq = 0
    if q is not None:
        hq = h
        shape = (t, hq, d)
        if q_out is None:
            q_out = torch.empty(shape, dtype=dtype, device=q.device)
        if not (_rows(q, dtype, shape, index) and _rows(q_out, dtype, shape, index)):
            _explain_rows(name, "q", q, dtype, shape, index)
            _explain_rows(name, "q_out", q_out, dtype, shape, index)
        qp, qo = q.data_ptr(), q_out.data_ptr()
        qs, qos = (q.stride(0), q_out.stride(0)) if t > 1 else (hq * d, hq * d)
    if k is not None:
        if k.dim() != 3:
            raise ValueError(f"{name}: k [T, H, D] expected")
        h = k.shape[1]
        shape = (t, h, d)
        if k_out is None:
            k_out = torch.empty(shape, dtype=dtype, device=x.device)
        if not (_rows(k, dtype, shape, index) and _rows(k_out, dtype, shape, index)):
            _explain_rows(name, "k", k, dtype, shape, index)
            _explain_rows(name, "k_out", k_out, dtype, shape, index)
        kp, ko = k.data_ptr(), k_out.data_ptr()
        ks, kos = (k.stride(0), k_out.stride(0)) if t > 1 else (h * d, h * d)
    rope = _rope_args(name, index, t, d, positions, position_offset, cos_sin, interleaved, q_weight, k_weight, eps)
    if status is not None:
        _need_status(name, status, x.device)
    elif check:
        status = _status_buffer(x.device)
    with _on(index):
        code = lib().tq_norm_rope(qp, qs, hq, kp, ks, h if kp is not None else 0, _DTYPES[dtype], t, d, *rope, qo, qos, ko,
                                  kos, None if status is None else status.data_ptr(), _stream_ptr(index))
    if code != TQ_OK:
        _check(code)
    if check:
        raise_for_device_status(status)
    return (q_out if q is not None else None), (k_out if k is not None else None)


def _pages_like(name: str, what: str, rows: torch.Tensor, pages, cents, t: int, d: int, dtype: torch.dtype, index: int):
    """(pointer, token stride, page pointer, bits, centroids pointer, (blocks, block size, heads)) of one
    packed side, checked."""
    if pages is None or cents is None or rows.dim() != 3 or pages.dim() != 4:
        raise ValueError(f"{name}: {what} [T, H, D] comes with its pages [NB, bs, H, RB] and centroids")
    nb, bs, h, rb = pages.shape
    bits = _BITS.get(cents.numel(), 0)
    if rb * 8 != d * bits + 32 or h != rows.shape[1]:  # head dims are multiples of 16
        bits = _bits_from_centroids(cents)
        raise ValueError(f"{name}: {what}_pages {list(pages.shape)} do not match {what} {list(rows.shape)} at {bits} bits")
    if not (_rows(rows, dtype, (t, h, d), index) and pages.dtype is torch.uint8 and pages.get_device() == index and
            pages.is_contiguous() and cents.dtype is torch.float32 and cents.get_device() == index and
            cents.is_contiguous()):
        _explain_rows(name, what, rows, dtype, (t, h, d), index)
        _need_like(name, index, **{what + "_pages": (pages, torch.uint8, (nb, bs, h, rb)),
                                   what + "_centroids": (cents, torch.float32, (1 << bits,))})
    return rows.data_ptr(), (rows.stride(0) if t > 1 else h * d), pages.data_ptr(), bits, cents.data_ptr(), (nb, bs, h)


def tq_append_kv(q: torch.Tensor | None, k: torch.Tensor | None, v: torch.Tensor | None,
                 k_pages: torch.Tensor | None, v_pages: torch.Tensor | None, slots: torch.Tensor, signs: torch.Tensor,
                 k_centroids: torch.Tensor | None, v_centroids: torch.Tensor | None,
                 positions: torch.Tensor | None = None, cos_sin: torch.Tensor | None = None,
                 q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None, eps: float = 1e-6,
                 interleaved: bool = False, position_offset: int = 0, q_out: torch.Tensor | None = None,
                 status: torch.Tensor | None = None, check: bool = False) -> torch.Tensor | None:
    """tq_norm_rope of q[T, Hq, D] and k[T, H, D] with the keys and the values v[T, H, D] encoded into
    pages[NB, bs, H, RB] at slots[T] (negative: not written), one launch.  q, k or v may be None
    (with its pages and centroids).  Returns q_out.  With check=True the call synchronises and raises
    TQError for a slot or a position out of range (other tokens have been written)."""
    name = "tq_append_kv"
    x = q if q is not None else k if k is not None else v
    if x is None or x.dim() != 3 or x.dtype not in _DTYPES:
        raise ValueError(f"{name}: q [T, Hq, D], k, v [T, H, D], f32/f16/bf16, expected")
    t, hq, d = x.shape
    dtype, index = x.dtype, x.get_device()
    if index < 0:
        raise ValueError(f"{name}: all tensors must be on the same CUDA device (got {x.device})")
    if not (_plain(slots, torch.int64, (t,), index) and _plain(signs, torch.float32, (d,), index)):
        _need_like(name, index, slots=(slots, torch.int64, (t,)), signs=(signs, torch.float32, (d,)))
    if q is not None:
        shape = (t, hq, d)
        if q_out is None:
            q_out = torch.empty(shape, dtype=dtype, device=q.device)
        if not (_rows(q, dtype, shape, index) and _rows(q_out, dtype, shape, index)):
            _explain_rows(name, "q", q, dtype, shape, index)
            _explain_rows(name, "q_out", q_out, dtype, shape, index)
        qp, qo = q.data_ptr(), q_out.data_ptr()
        qs, qos = (q.stride(0), q_out.stride(0)) if t > 1 else (hq * d, hq * d)
    else:
        qp = qo = q_out = None
        qs = qos = hq = 0
    kp = kpg = kc = vp = vpg = vc = shape = None
    ks = kb = vs = vb = 0
    if k is not None:
        kp, ks, kpg, kb, kc, shape = _pages_like(name, "k", k, k_pages, k_centroids, t, d, dtype, index)
    if v is not None:
        vp, vs, vpg, vb, vc, other = _pages_like(name, "v", v, v_pages, v_centroids, t, d, dtype, index)
        if shape is not None and shape != other:
            raise ValueError(f"{name}: k_pages {list(k_pages.shape)} and v_pages {list(v_pages.shape)} hold different tokens")
        shape = other
    nb, bs, h = shape or (0, 1, 1)
    rope = _rope_args(name, index, t, d, positions, position_offset, cos_sin, interleaved, q_weight, k_weight, eps)
    if status is not None:
        _need_status(name, status, x.device)
    elif check:
        status = _status_buffer(x.device)
    with _on(index):
        code = lib().tq_append_kv(qp, qs, hq, qo, qos, kp, ks, vp, vs, _DTYPES[dtype], t, h, d, slots.data_ptr(), kpg, kb,
                                  vpg, vb, nb, bs, signs.data_ptr(), kc, vc, *rope,
                                  None if status is None else status.data_ptr(), _stream_ptr(index))
    if code != TQ_OK:
        _check(code)
    if check:
        raise_for_device_status(status)
    return q_out


# ---------------------------------------------------------------- verification of drafted tokens

class Verified(NamedTuple):
    """Outputs of tq_verify_tree."""
    path: torch.Tensor        # int32 [S, max_path]: kept nodes, then -1
    path_lens: torch.Tensor   # int32 [S]
    next_token: torch.Tensor  # int32 [S]


@functools.lru_cache(maxsize=4096)
def tq_verify_tree_workspace(num_rows: int, vocab_size: int, num_seqs: int) -> int:
    """Workspace bytes of tq_verify_tree; 0 when the arguments are invalid."""
    if max(num_rows, vocab_size, num_seqs) >= 1 << 31:
        return 0
    return int(lib().tq_verify_tree_workspace(num_rows, vocab_size, num_seqs))


def _vocab_rows(name: str, what: str, t: torch.Tensor, index: int, shape: tuple):
    """(pointer, row stride) of rows t[R, V] with contiguous elements."""
    if t.get_device() != index:
        raise ValueError(f"{name}: all tensors must be on the same CUDA device ({what} is on {t.device})")
    if t.dtype not in _DTYPES or t.shape != shape or (shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: {what} must be f32/f16/bf16 rows {list(shape)} of contiguous elements, got {t.dtype} "
                         f"{list(t.shape)}")
    return t.data_ptr(), (t.stride(0) if shape[0] > 1 else shape[1])


def tq_verify_tree(logits: torch.Tensor, row_start: torch.Tensor, tokens: torch.Tensor, u_sample: torch.Tensor,
                   max_path: int, parents: torch.Tensor | None = None, temperature: torch.Tensor | None = None,
                   draft_probs: torch.Tensor | None = None, u_accept: torch.Tensor | None = None,
                   out: Verified | None = None, workspace: torch.Tensor | None = None,
                   status: torch.Tensor | None = None, check: bool = False) -> Verified:
    """Keeps or refuses drafted tokens by the target's logits[R, V].  Rows row_start[s] ..
    row_start[s + 1] - 1 are sequence s's nodes: node 0 its last token, the others drafted behind
    parents (None: a chain).  temperature[S] 0: largest logits.  Without draft_probs a token is drawn
    from every row with u_sample[R] and the path follows it; with draft_probs[R, V] (row i: what node
    i's children were drawn from) a child is kept by u_accept[R], refused ones are subtracted.  The
    result's path and path_lens are tq_commit_tree's; next_token follows the path."""
    name = "tq_verify_tree"
    if logits.dim() != 2 or row_start.dim() != 1 or row_start.numel() < 1:
        raise ValueError(f"{name}: logits [R, V] and row_start [S + 1] expected")
    r, vocab = logits.shape
    s, max_path = row_start.numel() - 1, _i32(name, "max_path", max_path)
    dev, i32, f32, index = logits.device, torch.int32, torch.float32, logits.get_device()
    if index < 0:
        raise ValueError(f"{name}: all tensors must be on the same CUDA device (got {dev})")
    if max_path < 1:
        raise ValueError(f"{name}: max_path {max_path} < 1")
    if max(r, vocab, s) >= 1 << 31:
        raise ValueError(f"{name}: logits {[r, vocab]} of {s} sequences: counts of 2^31 and more are not taken")
    if (draft_probs is None) != (u_accept is None):
        raise ValueError(f"{name}: draft_probs and u_accept come together")
    lp, ls = _vocab_rows(name, "logits", logits, index, (r, vocab))
    qp, qs, qt = None, 0, 0
    if draft_probs is not None:
        qp, qs = _vocab_rows(name, "draft_probs", draft_probs, index, (r, vocab))
        qt = _DTYPES[draft_probs.dtype]
        if not _plain(u_accept, f32, (r,), index):
            _need_like(name, index, u_accept=(u_accept, f32, (r,)))
    if not (_plain(row_start, i32, (s + 1,), index) and _plain(tokens, i32, (r,), index) and
            _plain(u_sample, f32, (r,), index)):
        _need_like(name, index, row_start=(row_start, i32, (s + 1,)), tokens=(tokens, i32, (r,)),
                   u_sample=(u_sample, f32, (r,)))
    if parents is not None and not _plain(parents, i32, (r,), index):
        _need_like(name, index, parents=(parents, i32, (r,)))
    if temperature is not None and not _plain(temperature, f32, (s,), index):
        _need_like(name, index, temperature=(temperature, f32, (s,)))
    if out is None:
        out = Verified(torch.empty((s, max_path), dtype=i32, device=dev), torch.empty(s, dtype=i32, device=dev),
                       torch.empty(s, dtype=i32, device=dev))
    else:
        _need_like(name, index, path=(out.path, i32, (s, max_path)), path_lens=(out.path_lens, i32, (s,)),
                   next_token=(out.next_token, i32, (s,)))
    _need_status(name, status, dev)
    if status is None and check:
        status = _status_buffer(dev)
    with _on(index):
        if workspace is None:
            workspace = torch.empty(tq_verify_tree_workspace(r, vocab, s), dtype=torch.uint8, device=dev)
        elif workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError(f"{name}: workspace must be contiguous on {dev}")
        code = lib().tq_verify_tree(lp, _DTYPES[logits.dtype], ls, r, vocab, qp, qt, qs, row_start.data_ptr(), s,
                                    tokens.data_ptr(), _ptr(parents), _ptr(temperature), _ptr(u_accept),
                                    u_sample.data_ptr(), out.path.data_ptr(), max_path, out.path_lens.data_ptr(),
                                    out.next_token.data_ptr(), workspace.data_ptr(),
                                    workspace.numel() * workspace.element_size(), _ptr(status), _stream_ptr(index))
    if code != TQ_OK:
        _check(code)
    if check:
        raise_for_device_status(status)
    return out

"""Thin ctypes binding of libcsa2 (declared in include/csa2.h).

Argument marshalling only: each function checks dtypes/devices/shapes of the
torch tensors it is given, passes raw device pointers and the current CUDA
stream to the C entry point of the same name, and raises ``Csa2Error`` on a
non-zero status. Every step of the computation runs in libcsa2's kernels.
Importing this module loads the library and raises if it is missing.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import List, Optional, Sequence

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libcsa2.so")

POOL_BLOCKS = 2048
BLOCK_TOKENS = 8
TOPK = 512
N_WIN = 128
# Rows of at most this many candidates are selected by one single-CTA kernel
# inside the decode step; longer rows take a compaction and a finishing kernel.
TOPK_SHORT_ROW = 65536
# csa2_full_select holds a row of block scores (and of pooled token scores) in
# shared memory: at most this many of each.
FULL_SELECT_MAX = 16384
# The decode stack launches the attention of a layer group (a Full or Reindex
# layer and the Reuse layers after it, up to ATTN_GROUP_MAX layers) as one
# kernel when the tensor-core cluster kernel takes the shape (512 channels, 64
# heads, fewer than ATTN_ROWS_MIN query rows); otherwise one kernel per layer.
ATTN_GROUP_MAX = 8
ATTN_ROWS_MIN = 64
MODE_FULL, MODE_REINDEX, MODE_REUSE = 0, 1, 2


class Csa2Error(RuntimeError):
    def __init__(self, fn: str, status: int, text: str):
        super().__init__(f"{fn} failed with status {status}: {text}")
        self.status = status


if not os.path.exists(_LIB_PATH):
    raise ImportError(f"libcsa2.so is not built ({_LIB_PATH}); build it with "
                      "`python -m sparse_attention_fp4_kv_b200.build`")

lib = ctypes.CDLL(_LIB_PATH)

_P = ctypes.c_void_p
_I = ctypes.c_int
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_F = ctypes.c_float
_D = ctypes.c_double


class csa2_layer(ctypes.Structure):
    _fields_ = [("mode", _I), ("q_idx", _P), ("q", _P), ("swa", _P), ("out", _P), ("topk", _P)]


class csa2_page_buf(ctypes.Structure):
    _fields_ = [("base", _P), ("page_bytes", _I64)]


_SIGS = {
    "csa2_status_string": (ctypes.c_char_p, [_I]),
    "csa2_abi_version": (_I, []),
    "csa2_device_status": (_I, [_I]),
    "csa2_selftest_wait_timeout": (_I, [_I, _P]),
    "csa2_kv_append_fp4": (_I, [_P, _I, _I, _I, _P, _I64, _P, _P, _P]),
    "csa2_kv_append_mxfp4": (_I, [_P, _I, _I, _I, _P, _I64, _P, _P, _P]),
    "csa2_index_full": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I64, _P, _P, _P, _P]),
    "csa2_topk_workspace_size": (_SZ, [_I, _I64, _I]),
    "csa2_topk": (_I, [_P, _P, _P, _I, _I64, _I, _P, _P, _SZ, _P]),
    "csa2_pool_gather": (_I, [_P, _P, _P, _P, _I, _I, _I, _I64, _P, _P, _P]),
    "csa2_full_select": (_I, [_P, _P, _P, _P, _P, _I, _I, _I64, _I, _I, _P, _P, _P]),
    "csa2_index_reindex": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I64, _I, _P, _P, _P]),
    "csa2_sparse_attn_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "csa2_sparse_attn_decode": (_I, [_P, _P, _P, _I64, _P, _I, _P, _P, _I, _P, _I, _I, _I, _I,
                                     _I, _F, _P, _P, _SZ, _P]),
    "csa2_sparse_attn_decode_mxfp4": (_I, [_P, _P, _P, _I64, _P, _I, _P, _P, _I, _P, _I, _I, _I,
                                           _I, _I, _F, _P, _P, _SZ, _P]),
    "csa2_decode_stack_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I64]),
    "csa2_decode_stack": (_I, [ctypes.POINTER(csa2_layer), _I, _P, _P, _P, _P, _P, _I64, _P, _P,
                               _I, _I, _I, _I, _I, _I, _F, _P, _I, _P, _P, _SZ, _P]),
    "csa2_decode_stack_noalloc": (_I, [ctypes.POINTER(csa2_layer), _I, _P, _P, _P, _P, _P, _I64,
                                       _P, _P, _I, _I, _I, _I, _I, _I, _F, _P, _I, _P]),
    "csa2_attn_resident_clusters": (_I, [_I]),
    "csa2_rope": (_I, [_P, _P, _I, _P, _P, _I64, _I, _I, _I, _I, _I, _I, _F, _I64, _I64, _I64, _I64,
                       _P]),
    "csa2_rope_freqs": (_I, [_I, _D, _I, _D, _I64, _D, _D, _P, _P]),
    "csa2_paged_kv_append_fp4": (_I, [_P, _I, _I, _I, _P, _P, _P, _I, _I, _I, _P, _P, _P]),
    "csa2_paged_kv_append_mxfp4": (_I, [_P, _I, _I, _I, _P, _P, _P, _I, _I, _I, _P, _P, _P]),
    "csa2_paged_kv_gather_fp4": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _I, _I, _I, _P, _P]),
    "csa2_paged_kv_gather_mxfp4": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _I, _I, _I, _P, _P]),
    "csa2_pages_workspace_size": (_SZ, [_I, _I]),
    "csa2_pages_extend": (_I, [_P, _I, _I, _P, _I, _I, _P, _P, _P, _SZ, _P]),
    "csa2_pages_fork": (_I, [_P, _I, _I, _P, _I, _I, _P, _P, _P, _I, _P, _P, _P, _SZ, _P]),
    "csa2_pages_free": (_I, [_P, _I, _I, _P, _I, _I, _P, _P, _I, _P]),
    "csa2_pages_copy": (_I, [_P, _I, ctypes.POINTER(csa2_page_buf), _I, _I, _P]),
    "csa2_pages_compact": (_I, [_P, _I, _I, _P, _I, ctypes.POINTER(csa2_page_buf), _I, _P, _P, _P,
                                _P, _SZ, _P]),
    "csa2_paged_attn_workspace_size": (_SZ, [_I, _I, _I]),
    "csa2_paged_attn_decode": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _I64, _I64, _I, _I, _I, _F, _P,
                                    _P, _P, _SZ, _P]),
    "csa2_paged_attn_decode_mxfp4": (_I, [_P, _P, _P, _P, _I, _I, _I, _P, _I64, _I64, _I, _I, _I, _F,
                                          _P, _P, _P, _SZ, _P]),
    "csa2_workspace_status": (_I, [_P, _I, _P]),
    "csa2_selftest_workspace_timeout": (_I, [_I, _P, _P]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def exported_symbols() -> List[str]:
    return list(_SIGS)


def status_string(status: int) -> str:
    return lib.csa2_status_string(status).decode()


def _check(name: str, st: int):
    if st != 0:
        raise Csa2Error(name, st, status_string(st))


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libcsa2 must be contiguous")
    return _P(t.data_ptr())


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return _P(stream.cuda_stream)


def _want(t: torch.Tensor, dtype, name: str):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


# ----------------------------------------------------------------------------- calls
def csa2_kv_append_fp4(kv_bf16: torch.Tensor, start_pos: torch.Tensor, kv_fp4: torch.Tensor,
                       kv_sf: torch.Tensor, stream=None, mx: bool = False) -> None:
    """kv_bf16 [B][n_new][C] bf16; start_pos [B] int64; kv_fp4 [B][cap][C/2] uint8;
    kv_sf [B][cap][C/16] uint8 (E4M3), or with mx the MXFP4 variant's
    [B][cap][C/32] E8M0 (csa2_kv_append_mxfp4)."""
    _want(kv_bf16, torch.bfloat16, "kv_bf16")
    _want(start_pos, torch.int64, "start_pos")
    _want(kv_fp4, torch.uint8, "kv_fp4")
    _want(kv_sf, torch.uint8, "kv_sf")
    B, n, C = kv_bf16.shape
    cap = kv_fp4.shape[1]
    assert kv_fp4.shape == (B, cap, C // 2) and kv_sf.shape == (B, cap, C // (32 if mx else 16))
    name = "csa2_kv_append_mxfp4" if mx else "csa2_kv_append_fp4"
    _check(name, getattr(lib, name)(
        _ptr(kv_bf16), B, n, C, _ptr(start_pos), cap, _ptr(kv_fp4), _ptr(kv_sf), _stream(stream)))


def csa2_index_full(q_idx, k_idx, k_scale, ctx_len, blk_score, tok_score=None, n_blk=None,
                    q_pos=None, stream=None) -> None:
    """q_idx [B][Nq][H][D] int8; k_idx [B][cap][H][D] int8; k_scale [B][cap] fp32;
    ctx_len [B] int64; blk_score [B][Nq][ceil(cap/8)] fp32; tok_score [B][Nq][cap]
    fp32 or None; n_blk [B][Nq] int32 or None; q_pos [B][Nq] int64 or None."""
    _want(q_idx, torch.int8, "q_idx")
    _want(k_idx, torch.int8, "k_idx")
    B, Nq, H, D = q_idx.shape
    cap = k_idx.shape[1]
    assert k_idx.shape == (B, cap, H, D) and k_scale.shape == (B, cap)
    assert blk_score.shape == (B, Nq, (cap + 7) // 8)
    if tok_score is not None:
        assert tok_score.shape == (B, Nq, cap)
    _check("csa2_index_full", lib.csa2_index_full(
        _ptr(q_idx), _ptr(k_idx), _ptr(k_scale), _ptr(ctx_len), _ptr(q_pos), B, Nq, H, D, cap,
        _ptr(tok_score), _ptr(blk_score), _ptr(n_blk), _stream(stream)))


def csa2_topk(score, k: int, out, cand_pos=None, n_valid=None, ws=None, stream=None) -> None:
    """score [R][n] fp32; out [R][k] int32; cand_pos [R][n] int32 or None;
    n_valid [R] int32 or None."""
    _want(score, torch.float32, "score")
    _want(out, torch.int32, "out")
    R, n = score.shape
    assert out.shape == (R, k)
    need = lib.csa2_topk_workspace_size(R, n, k)
    wsb = 0
    if need:
        if ws is None:
            raise ValueError(f"csa2_topk needs {need} workspace bytes")
        wsb = ws.numel() * ws.element_size()
    _check("csa2_topk", lib.csa2_topk(_ptr(score), _ptr(cand_pos), _ptr(n_valid), R, n, k,
                                      _ptr(out), _ptr(ws) if need else None, wsb, _stream(stream)))


def csa2_pool_gather(tok_score, pool, ctx_len, pool_score, pool_pos, q_pos=None,
                     stream=None) -> None:
    """tok_score [B][Nq][cap] fp32; pool [B][Nq][P] int32; pool_score/pool_pos [B][Nq][8P]."""
    B, Nq, cap = tok_score.shape
    P = pool.shape[2]
    assert pool_score.shape == (B, Nq, 8 * P) and pool_pos.shape == (B, Nq, 8 * P)
    _check("csa2_pool_gather", lib.csa2_pool_gather(
        _ptr(tok_score), _ptr(pool), _ptr(ctx_len), _ptr(q_pos), B, Nq, P, cap,
        _ptr(pool_score), _ptr(pool_pos), _stream(stream)))


def workspace_status(ws: torch.Tensor, clear: bool = False, stream=None) -> int:
    """Status of the call whose workspace is ws (its error word): 0, or
    CSA2_ERR_DEVICE_TIMEOUT (-7) if a kernel of that call gave up a wait."""
    return lib.csa2_workspace_status(_ptr(ws), int(clear), _stream(stream))


def attn_resident_clusters(heads_per_cluster: int) -> int:
    """8-CTA attention clusters that fit on the current device at once with
    heads_per_cluster (16, 32 or 64) query heads each."""
    return lib.csa2_attn_resident_clusters(heads_per_cluster)


def device_status(clear: bool = False) -> int:
    """CSA2_OK, or CSA2_ERR_DEVICE_TIMEOUT if a kernel gave up a bounded wait
    (synchronizes the device; clear resets the flags)."""
    return lib.csa2_device_status(1 if clear else 0)


def selftest_wait_timeout(limit_us: int = 1000, stream=None) -> None:
    """Launch one CTA whose wait nothing completes; it records a timeout."""
    _check("csa2_selftest_wait_timeout", lib.csa2_selftest_wait_timeout(limit_us, _stream(stream)))


def csa2_full_select(blk_score, n_blk, tok_score, ctx_len, pool, top, q_pos=None,
                     stream=None) -> None:
    """blk_score [B][Nq][ceil(cap/8)] fp32; n_blk [B][Nq] int32; tok_score [B][Nq][cap] fp32;
    pool [B][Nq][P] int32; top [B][Nq][K] int32."""
    _want(blk_score, torch.float32, "blk_score")
    _want(tok_score, torch.float32, "tok_score")
    _want(n_blk, torch.int32, "n_blk")
    B, Nq, cap = tok_score.shape
    P, K = pool.shape[2], top.shape[2]
    assert blk_score.shape == (B, Nq, (cap + 7) // 8) and n_blk.shape == (B, Nq)
    assert pool.shape[:2] == (B, Nq) and top.shape[:2] == (B, Nq)
    _check("csa2_full_select", lib.csa2_full_select(
        _ptr(blk_score), _ptr(n_blk), _ptr(tok_score), _ptr(ctx_len), _ptr(q_pos), B, Nq, cap, P, K,
        _ptr(pool), _ptr(top), _stream(stream)))


def csa2_index_reindex(q_idx, k_idx, k_scale, pool, ctx_len, pool_score, pool_pos, q_pos=None,
                       stream=None) -> None:
    """q_idx [B][Nq][H][D] int8; pool [B][Nq][P] int32; pool_score/pool_pos [B][Nq][8P]."""
    _want(q_idx, torch.int8, "q_idx")
    B, Nq, H, D = q_idx.shape
    cap = k_idx.shape[1]
    P = pool.shape[2]
    assert pool_score.shape == (B, Nq, 8 * P) and pool_pos.shape == (B, Nq, 8 * P)
    _check("csa2_index_reindex", lib.csa2_index_reindex(
        _ptr(q_idx), _ptr(k_idx), _ptr(k_scale), _ptr(pool), _ptr(ctx_len), _ptr(q_pos), B, Nq,
        H, D, cap, P, _ptr(pool_score), _ptr(pool_pos), _stream(stream)))


def sparse_attn_workspace_size(B, Nq, Hq, C, K, n_win=N_WIN) -> int:
    return lib.csa2_sparse_attn_workspace_size(B, Nq, Hq, C, K, n_win)


def csa2_sparse_attn_decode(q_bf16, kv_fp4, kv_sf, topk, swa_bf16, swa_pos0, out, softmax_scale,
                            q_pos=None, n_win=N_WIN, ws=None, stream=None, mx: bool = False) -> None:
    """q_bf16 [B][Nq][Hq][C]; topk [B][Nq][K] int32; swa_bf16 [B][rows][C] bf16;
    swa_pos0 [B] int64; out [B][Nq][Hq][C] fp32; with mx the cache is the MXFP4
    variant (csa2_sparse_attn_decode_mxfp4)."""
    _want(q_bf16, torch.bfloat16, "q_bf16")
    _want(out, torch.float32, "out")
    B, Nq, Hq, C = q_bf16.shape
    cap = kv_fp4.shape[1]
    K = topk.shape[2]
    rows = swa_bf16.shape[1] if swa_bf16 is not None else 0
    need = sparse_attn_workspace_size(B, Nq, Hq, C, K, n_win)
    if need and ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=q_bf16.device)
    wsb = ws.numel() * ws.element_size() if ws is not None else 0
    name = "csa2_sparse_attn_decode_mxfp4" if mx else "csa2_sparse_attn_decode"
    _check(name, getattr(lib, name)(
        _ptr(q_bf16), _ptr(kv_fp4), _ptr(kv_sf), cap, _ptr(topk), K, _ptr(swa_bf16),
        _ptr(swa_pos0), rows, _ptr(q_pos), n_win, B, Nq, Hq, C, float(softmax_scale), _ptr(out),
        _ptr(ws), wsb, _stream(stream)))


def decode_stack_workspace_size(B, Hq, C, H, D, cap) -> int:
    return lib.csa2_decode_stack_workspace_size(B, Hq, C, H, D, cap)


class DecodeStack:
    """Pre-marshalled arguments of csa2_decode_stack for a fixed set of device
    buffers, so that a decode step is one C call."""

    def __init__(self, modes: Sequence[int], q_idx: Sequence[Optional[torch.Tensor]],
                 q: Sequence[torch.Tensor], swa: Sequence[torch.Tensor],
                 out: Sequence[torch.Tensor], topk: Sequence[Optional[torch.Tensor]],
                 k_idx: torch.Tensor, k_scale: torch.Tensor, kv_fp4: torch.Tensor,
                 kv_sf: torch.Tensor, ctx_len: torch.Tensor, swa_pos0: torch.Tensor,
                 pool: torch.Tensor, softmax_scale: float, ws: Optional[torch.Tensor] = None,
                 kv_new: Optional[torch.Tensor] = None, pool_ready: bool = False):
        n = len(modes)
        self.layers = (csa2_layer * n)()
        self._keep = [q_idx, q, swa, out, topk, k_idx, k_scale, kv_fp4, kv_sf, ctx_len, swa_pos0,
                      pool, kv_new]
        for l in range(n):
            self.layers[l] = csa2_layer(int(modes[l]), _ptr(q_idx[l]), _ptr(q[l]), _ptr(swa[l]),
                                        _ptr(out[l]), _ptr(topk[l]))
        B, cap, H, D = k_idx.shape
        Hq, C = q[0].shape[-2], q[0].shape[-1]
        self.dims = (B, Hq, C, H, D, cap)
        need = decode_stack_workspace_size(B, Hq, C, H, D, cap)
        if ws is None:
            ws = torch.empty(need, dtype=torch.uint8, device=k_idx.device)
        assert ws.numel() >= need
        self.ws = ws
        self.args = (self.layers, n, _ptr(kv_new), _ptr(k_idx), _ptr(k_scale), _ptr(kv_fp4), _ptr(kv_sf), cap,
                     _ptr(ctx_len), _ptr(swa_pos0), swa[0].shape[1], B, Hq, C, H, D,
                     float(softmax_scale), _ptr(pool), int(bool(pool_ready)))
        self.ws_args = (_ptr(ws), ws.numel())

    def call_noalloc(self, stream=None) -> int:
        """The same decode step through csa2_decode_stack_noalloc, which uses
        the library's own scratch array instead of self.ws (for callers that
        cannot allocate). Returns the C status code."""
        return lib.csa2_decode_stack_noalloc(*self.args, _stream(stream))

    def __call__(self, stream=None, scan_events=None) -> None:
        """One decode step. scan_events: optional (start, end) torch.cuda.Event
        pair recorded around the first Full layer's indexer scan."""
        ev = None
        if scan_events is not None:
            ev = (_P * 2)(_P(scan_events[0].cuda_event), _P(scan_events[1].cuda_event))
        _check("csa2_decode_stack", lib.csa2_decode_stack(*self.args, ev, *self.ws_args,
                                                          _stream(stream)))


# ----------------------------------------------------------------------------- paged FP4 cache
ROPE_PLAIN, ROPE_LINEAR, ROPE_YARN = 0, 1, 2


# These calls are a few microseconds each on the device, so the marshalling counts:
# one check per tensor, and raw pointers and stream handles go to ctypes as plain
# integers.
def _device(t, dtype, name: str) -> int:
    """The device of a call's first tensor, on which the others have to be too."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _arg(t, dtype, name: str, dev: int) -> int:
    """The address of a contiguous tensor of this type on this device."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the call runs on cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _handle(stream, dev: int) -> int:
    """The stream handle of a call on `dev`, which has to be the current device."""
    if torch.cuda.current_device() != dev:
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    if stream.device.index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on cuda:{dev}")
    return stream.cuda_stream


def _scratch(nbytes: int, device, stream):
    """Workspace of a call that was given none: allocated on the call's stream,
    so that it is not handed out again before the call's kernels have run."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def csa2_rope_freqs(inv_freq, theta: float = 10000.0, scaling: int = ROPE_PLAIN, factor: float = 1.0,
                    orig_ctx: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                    stream=None) -> None:
    """inv_freq [rot_dim / 2] fp64: the table csa2_rope reads."""
    dev = _device(inv_freq, torch.float64, "inv_freq")
    table = _arg(inv_freq, torch.float64, "inv_freq", dev)
    _check("csa2_rope_freqs", lib.csa2_rope_freqs(
        2 * inv_freq.numel(), float(theta), scaling, float(factor), orig_ctx, float(beta_fast),
        float(beta_slow), table, _handle(stream, dev)))


def csa2_rope(x, pos, inv_freq, out, rot_start: int = 0, interleaved: bool = True,
              inverse: bool = False, mscale: float = 1.0, stream=None) -> None:
    """x, out [T][H][D] bf16 or fp32 (out may be x; channels contiguous, any token
    and head strides); pos [T] int64; inv_freq [rot_dim / 2] fp64. Rotates the
    channels [rot_start, rot_start + rot_dim) of every head."""
    f32 = x.dtype is torch.float32
    if not f32 and x.dtype is not torch.bfloat16:
        raise TypeError(f"x must be torch.bfloat16 or torch.float32, got {x.dtype}")
    dev = _device(x, x.dtype, "x")
    if _device(out, x.dtype, "out") != dev:
        raise ValueError("x and out must be on one device")
    at = _arg(pos, torch.int64, "pos", dev)
    table = _arg(inv_freq, torch.float64, "inv_freq", dev)
    T, H, D = x.shape
    assert out.shape == x.shape and pos.shape == (T,) and inv_freq.dim() == 1
    (xt, xh, xc), (ot, oh, oc) = x.stride(), out.stride()
    if D > 1 and (xc != 1 or oc != 1):
        raise ValueError("the channels of x and out must be contiguous")
    _check("csa2_rope", lib.csa2_rope(
        x.data_ptr(), out.data_ptr(), int(f32), at, table,
        T, H, D, rot_start, 2 * inv_freq.shape[0], 0 if interleaved else 1, int(inverse),
        float(mscale), xt, xh, ot, oh, _handle(stream, dev)))


def _pool(kv_fp4, kv_sf, C: int, mx: bool, dev: int):
    """(codes, scales, page_size, n_pages) of a pool kv_fp4 [n_pages][page_size][C/2]."""
    n_pages, page_size, half = kv_fp4.shape
    assert half == C // 2 and kv_sf.shape == (n_pages, page_size, C // (32 if mx else 16))
    return _arg(kv_fp4, torch.uint8, "kv_fp4", dev), _arg(kv_sf, torch.uint8, "kv_sf", dev), page_size, n_pages


def _counts(n_valid, B: int, dev: int):
    if n_valid is None:
        return None
    assert n_valid.shape == (B,)
    return _arg(n_valid, torch.int32, "n_valid", dev)


def _table(page_table, S: int, dev: int):
    """(address, max_pages) of a page table [S][max_pages]."""
    rows, max_pages = page_table.shape
    assert rows == S
    return _arg(page_table, torch.int32, "page_table", dev), max_pages


def csa2_paged_kv_append_fp4(kv_bf16, start_pos, page_table, kv_fp4, kv_sf, n_valid=None, stream=None,
                             mx: bool = False) -> None:
    """kv_bf16 [B][n_new][C] bf16; start_pos [B] int64; page_table [B][max_pages]
    int32; kv_fp4 [n_pages][page_size][C/2] and kv_sf [..][C/16] (mx: [..][C/32])
    uint8; n_valid [B] int32 or None."""
    dev = _device(kv_bf16, torch.bfloat16, "kv_bf16")
    rows = _arg(kv_bf16, torch.bfloat16, "kv_bf16", dev)
    at = _arg(start_pos, torch.int64, "start_pos", dev)
    B, n, C = kv_bf16.shape
    table, max_pages = _table(page_table, B, dev)
    codes, scales, page_size, n_pages = _pool(kv_fp4, kv_sf, C, mx, dev)
    assert start_pos.shape == (B,)
    valid = _counts(n_valid, B, dev)
    name = "csa2_paged_kv_append_mxfp4" if mx else "csa2_paged_kv_append_fp4"
    _check(name, getattr(lib, name)(
        rows, B, n, C, at, valid, table, max_pages, page_size, n_pages, codes, scales, _handle(stream, dev)))


def csa2_paged_kv_gather(kv_fp4, kv_sf, page_table, start_pos, out, n_valid=None, stream=None,
                         mx: bool = False) -> None:
    """out [B][n][C] bf16 receives the rows at positions start_pos[b] + i; rows
    with i >= n_valid[b] or no page are left as they were."""
    dev = _device(out, torch.bfloat16, "out")
    rows = _arg(out, torch.bfloat16, "out", dev)
    at = _arg(start_pos, torch.int64, "start_pos", dev)
    B, n, C = out.shape
    table, max_pages = _table(page_table, B, dev)
    codes, scales, page_size, n_pages = _pool(kv_fp4, kv_sf, C, mx, dev)
    assert start_pos.shape == (B,)
    valid = _counts(n_valid, B, dev)
    name = "csa2_paged_kv_gather_mxfp4" if mx else "csa2_paged_kv_gather_fp4"
    _check(name, getattr(lib, name)(
        codes, scales, table, max_pages, page_size, n_pages, at, valid, B, n, C, rows, _handle(stream, dev)))


@functools.lru_cache(maxsize=256)
def pages_workspace_size(n_pages: int, n: int = 0) -> int:
    return lib.csa2_pages_workspace_size(n_pages, n)


def _workspace(ws, nbytes: int, dev: int, stream):
    """(tensor, address, bytes) of a call's workspace; nbytes of it are allocated if it was given none."""
    if ws is None:
        ws = _scratch(nbytes, dev, stream)
    return ws, _arg(ws, ws.dtype, "ws", dev), ws.numel() * ws.element_size()


def _pages(page_table, ref):
    """(device, table, S, max_pages, counts, n_pages)"""
    dev = _device(page_table, torch.int32, "page_table")
    S, max_pages = page_table.shape
    n_pages, = ref.shape
    return (dev, _arg(page_table, torch.int32, "page_table", dev), S, max_pages,
            _arg(ref, torch.int32, "ref", dev), n_pages)


def csa2_pages_extend(page_table, ref, want_len, page_size: int, n_failed, ws=None, stream=None) -> None:
    """page_table [S][max_pages] int32; ref [n_pages] int32; want_len [S] int64;
    n_failed [1] int32."""
    dev, table, S, M, counts, n_pages = _pages(page_table, ref)
    want = _arg(want_len, torch.int64, "want_len", dev)
    failed = _arg(n_failed, torch.int32, "n_failed", dev)
    assert want_len.shape == (S,)
    st = _handle(stream, dev)
    ws, wsp, wsb = _workspace(ws, pages_workspace_size(n_pages, S), dev, stream)
    _check("csa2_pages_extend", lib.csa2_pages_extend(
        table, S, M, counts, n_pages, page_size, want, failed, wsp, wsb, st))


def csa2_pages_fork(page_table, ref, seq_len, src, dst, page_size: int, pairs, n_failed, ws=None,
                    stream=None) -> None:
    """seq_len [S] int64; src, dst [F] int32; pairs [F][2] int32; n_failed [1] int32."""
    dev, table, S, M, counts, n_pages = _pages(page_table, ref)
    lens = _arg(seq_len, torch.int64, "seq_len", dev)
    of, to = _arg(src, torch.int32, "src", dev), _arg(dst, torch.int32, "dst", dev)
    copies = _arg(pairs, torch.int32, "pairs", dev)
    failed = _arg(n_failed, torch.int32, "n_failed", dev)
    F, = src.shape
    assert seq_len.shape == (S,) and dst.shape == (F,) and pairs.shape == (F, 2)
    st = _handle(stream, dev)
    ws, wsp, wsb = _workspace(ws, pages_workspace_size(n_pages, F), dev, stream)
    _check("csa2_pages_fork", lib.csa2_pages_fork(
        table, S, M, counts, n_pages, page_size, lens, of, to, F, copies, failed, wsp, wsb, st))


def csa2_pages_free(page_table, ref, seq, page_size: int, keep_len=None, stream=None) -> None:
    """seq [F] int32; keep_len [F] int64 or None (nothing is kept)."""
    dev, table, S, M, counts, n_pages = _pages(page_table, ref)
    which = _arg(seq, torch.int32, "seq", dev)
    F, = seq.shape
    keep = None
    if keep_len is not None:
        assert keep_len.shape == (F,)
        keep = _arg(keep_len, torch.int64, "keep_len", dev)
    _check("csa2_pages_free", lib.csa2_pages_free(
        table, S, M, counts, n_pages, page_size, which, keep, F, _handle(stream, dev)))


def _page_bufs(bufs, n_pages: int, dev: int):
    """Tensors [n_pages][...] of one cache -> the C array of their bases and page sizes."""
    arr = (csa2_page_buf * max(1, len(bufs)))()
    for a, t in zip(arr, bufs):
        assert t.shape[0] == n_pages
        a.base = _arg(t, t.dtype, "a cache buffer", dev)
        a.page_bytes = t.numel() // n_pages * t.element_size()
    return arr


def csa2_pages_copy(pairs, bufs: Sequence[torch.Tensor], stream=None) -> None:
    """pairs [F][2] int32 (from, onto); bufs: tensors [n_pages][...] of any dtype."""
    dev = _device(pairs, torch.int32, "pairs")
    copies = _arg(pairs, torch.int32, "pairs", dev)
    F, two = pairs.shape
    assert two == 2 and len(bufs) >= 1
    n_pages = bufs[0].shape[0]
    _check("csa2_pages_copy", lib.csa2_pages_copy(
        copies, F, _page_bufs(bufs, n_pages, dev), len(bufs), n_pages, _handle(stream, dev)))


def csa2_pages_compact(page_table, ref, bufs: Sequence[torch.Tensor], page_table_out, ref_out, n_live,
                       ws=None, stream=None) -> None:
    """page_table, page_table_out [S][max_pages] int32 and ref, ref_out [n_pages]
    int32 (the outputs may be the inputs); bufs: tensors [n_pages][...]; n_live [1]
    int32."""
    dev, table, S, M, counts, n_pages = _pages(page_table, ref)
    table_out = _arg(page_table_out, torch.int32, "page_table_out", dev)
    counts_out = _arg(ref_out, torch.int32, "ref_out", dev)
    live = _arg(n_live, torch.int32, "n_live", dev)
    assert page_table_out.shape == (S, M) and ref_out.shape == (n_pages,)
    st = _handle(stream, dev)
    ws, wsp, wsb = _workspace(ws, pages_workspace_size(n_pages, 0), dev, stream)
    _check("csa2_pages_compact", lib.csa2_pages_compact(
        table, S, M, counts, n_pages, _page_bufs(bufs, n_pages, dev), len(bufs), table_out, counts_out, live,
        wsp, wsb, st))


@functools.lru_cache(maxsize=256)
def _paged_attn_ws(device: int, B: int, Hq: int, C: int) -> int:
    return lib.csa2_paged_attn_workspace_size(B, Hq, C)


def paged_attn_workspace_size(B: int, Hq: int, C: int) -> int:
    return lib.csa2_paged_attn_workspace_size(B, Hq, C)


def csa2_paged_attn_decode(q_bf16, kv_fp4, kv_sf, page_table, ctx_len, out, softmax_scale,
                           n_win: int = 0, n_sink: int = 0, lse=None, ws=None, stream=None,
                           mx: bool = False) -> None:
    """q_bf16, out [B][Hq][C] bf16; kv_fp4 [n_pages][page_size][C/2] and kv_sf uint8;
    page_table [B][max_pages] int32; ctx_len [B] int64; lse [B][Hq] fp32 or None;
    n_win = 0 attends every position, else the last n_win and the first n_sink."""
    dev = _device(q_bf16, torch.bfloat16, "q_bf16")
    q = _arg(q_bf16, torch.bfloat16, "q_bf16", dev)
    o = _arg(out, torch.bfloat16, "out", dev)
    lens = _arg(ctx_len, torch.int64, "ctx_len", dev)
    B, Hq, C = shape = q_bf16.shape
    table, max_pages = _table(page_table, B, dev)
    codes, scales, page_size, n_pages = _pool(kv_fp4, kv_sf, C, mx, dev)
    assert out.shape == shape and ctx_len.shape == (B,)
    lse_at = None
    if lse is not None:
        assert lse.shape == (B, Hq)
        lse_at = _arg(lse, torch.float32, "lse", dev)
    st = _handle(stream, dev)
    ws, wsp, wsb = _workspace(ws, _paged_attn_ws(dev, B, Hq, C), dev, stream)
    name = "csa2_paged_attn_decode_mxfp4" if mx else "csa2_paged_attn_decode"
    _check(name, getattr(lib, name)(
        q, codes, scales, table, max_pages, page_size, n_pages, lens, n_win, n_sink, B, Hq, C,
        float(softmax_scale), o, lse_at, wsp, wsb, st))

"""KaLM-Reranker-V1 FBNL scoring hot path on B200: thin PyTorch binding of libkalm.

Every function here marshals torch tensors (device memory owned by the caller)
into the C ABI of ``include/kalm.h``; all arithmetic runs in the CUDA kernels of
``libkalm.so``.  Functions keep the C names.  There is no CPU fallback: without
the built library or an sm_100 device they raise ``KalmError``.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from ._abi import KalmError, call, load, library_path  # noqa: F401

__all__ = [
    "KalmError", "load", "library_path", "kalm_version", "kalm_device_check", "kalm_check_device_errors",
    "kalm_ragged_offsets", "kalm_chunk_pool", "kalm_linear", "kalm_linear_chain", "kalm_linear_chain_sync_len",
    "kalm_linear_chain_rope",
    "kalm_cross_kv_proj", "kalm_merged_attention",
    "kalm_merged_attention_out_proj", "kalm_merged_attention_out_proj_static", "kalm_attention_out_proj_sync_len",
    "kalm_yes_no_score", "kalm_broadcast_rows", "kalm_selftest_wait_timeout", "kalm_attention_items",
    "kalm_attention_schedule", "kalm_rope", "kalm_rope_table", "kalm_linear_rope",
    "kalm_cache_write", "kalm_cache_read", "kalm_merged_attention_cache",
    "kalm_merged_attention_cache_rows", "kalm_rms_norm", "kalm_norm_residual",
]

HEAD_DIM = 256
MAX_QUERY_TOKENS = 512  # KALM_MAX_QUERY_TOKENS
CACHE_GROUP = 32  # KALM_CACHE_GROUP: columns of a cached row that share a scale
CACHE_FEW_ROWS = 8  # KALM_CACHE_FEW_ROWS: packed rows up to which the cache attention takes no workspace


# The current device and a device's current stream handle as torch keeps them, without the checks and the Stream
# object around them (0.1 us instead of 3 us a call); called with a CUDA tensor in hand, so CUDA is initialised.  They
# are torch's own, not public: where a version lacks one, the public call takes its place.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _stream(stream: Optional[torch.cuda.Stream], dev: Optional[int] = None) -> int:
    """Handle of a stream, or of the current one of `dev` (None: the current device)."""
    if stream is not None:
        return stream.cuda_stream
    return _current_stream(torch.cuda.current_device() if dev is None else dev)


def _p(t: Optional[torch.Tensor], dtype: Optional[torch.dtype] = None) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise KalmError(1, "binding", "tensors must live on the CUDA device")
    if dtype is not None and t.dtype != dtype:
        raise KalmError(1, "binding", f"expected {dtype}, got {t.dtype}")
    return t.data_ptr()


def _ld(t: torch.Tensor) -> int:
    """Row stride (elements) of a 2-D view whose last dimension is contiguous."""
    if t.dim() != 2 or t.stride(1) != 1:
        raise KalmError(1, "binding", "expected a 2-D tensor with contiguous rows")
    return t.stride(0)


def _refuse(where: str, name: str, t: torch.Tensor, dtype: torch.dtype, dev: int, what: str) -> None:
    """Raise for a tensor that is not `what` of this type on the current device."""
    if t.dtype is not dtype:
        what = f"expected {dtype}, got {t.dtype}"
    elif t.get_device() != dev:
        what = f"tensor on {t.device}, current device is cuda:{dev}"
    raise KalmError(1, where, f"{name}: {what}")


def _device(where: str, t: torch.Tensor) -> int:
    """The current device, on which the call's tensors must live."""
    if not t.is_cuda:
        raise KalmError(1, where, "tensors must live on the CUDA device")
    return _current_device()


def _mat(where: str, name: str, t: torch.Tensor, dtype: torch.dtype, dev: int, rows: int = -1, width: int = -1) -> int:
    """Row stride (elements) of a 2-D view with contiguous rows, after checking type, device and sizes."""
    shape = t.shape
    if t.dtype is not dtype or t.get_device() != dev or len(shape) != 2 or (rows >= 0 and shape[0] != rows) or \
            (width >= 0 and shape[1] != width):
        _refuse(where, name, t, dtype, dev, f"shape {tuple(shape)}, expected ({'rows' if rows < 0 else rows}, "
                                            f"{'columns' if width < 0 else width})")
    ld, step = t.stride()
    if step != 1 and shape[1] > 1:
        _refuse(where, name, t, dtype, dev, "expected contiguous rows")
    # the stride of a single row is arbitrary in torch; any that covers the row will do
    return ld if shape[0] > 1 else -(-shape[1] // 16) * 16


def _pair(where: str, name: str, k: torch.Tensor, v: torch.Tensor) -> None:
    """The V tensor of a K / V pair is laid out as its (checked) K (the stride of a single row is arbitrary in torch)."""
    if v.shape != k.shape or v.dtype is not k.dtype or v.get_device() != k.get_device() or \
            (v.stride() != k.stride() and (k.size(0) > 1 or v.stride(1) != 1)):
        raise KalmError(1, where, f"{name}: K is {k.dtype} {tuple(k.shape)} with strides {k.stride()} on {k.device}, V "
                                  f"{v.dtype} {tuple(v.shape)} with strides {v.stride()} on {v.device}")


def _vec(where: str, name: str, t: Optional[torch.Tensor], dtype: torch.dtype, dev: int, n: int) -> Optional[int]:
    """Address of a contiguous vector of n values (None passes)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != dev or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        _refuse(where, name, t, dtype, dev, f"shape {tuple(t.shape)}, expected a contiguous vector of {n}")
    return t.data_ptr()


def kalm_version() -> int:
    return load().kalm_version()


def kalm_device_check() -> None:
    call("kalm_device_check")


def kalm_check_device_errors(stream: Optional[torch.cuda.Stream] = None) -> int:
    """Synchronise the stream and raise if a kernel recorded a device error."""
    word = ctypes.c_uint32(0)
    call("kalm_check_device_errors", _stream(stream), ctypes.byref(word))
    return word.value


def kalm_ragged_offsets(length: torch.Tensor, tok_off: Optional[torch.Tensor], pool_off: Optional[torch.Tensor],
                        chunk: int = 4, stream=None) -> None:
    call("kalm_ragged_offsets", _p(length, torch.int32), length.numel(), chunk, _p(tok_off, torch.int64),
         _p(pool_off, torch.int64), _stream(stream))


def kalm_chunk_pool(enc: torch.Tensor, tok_off: torch.Tensor, length: torch.Tensor, pooled: torch.Tensor,
                    pool_off: torch.Tensor, total_pooled: int, chunk: int = 4, stream=None) -> None:
    call("kalm_chunk_pool", _p(enc, torch.bfloat16), _ld(enc), _p(tok_off, torch.int64), _p(length, torch.int32),
         length.numel(), enc.shape[1], chunk, _p(pooled, torch.bfloat16), _ld(pooled), _p(pool_off, torch.int64),
         int(total_pooled), _stream(stream))


def kalm_linear(x: torch.Tensor, w: torch.Tensor, y: torch.Tensor, residual: Optional[torch.Tensor] = None,
                stream=None) -> None:
    """y = x . w^T (+ residual); w is [out][in]."""
    m, k = x.shape
    n = w.shape[0]
    if w.shape[1] != k or y.shape[0] != m or y.shape[1] != n:
        raise KalmError(1, "kalm_linear", f"shapes x{tuple(x.shape)} w{tuple(w.shape)} y{tuple(y.shape)}")
    call("kalm_linear", _p(x, torch.bfloat16), _ld(x), _p(w, torch.bfloat16), _ld(w),
         _p(residual, torch.bfloat16), _ld(residual) if residual is not None else 0,
         _p(y, torch.bfloat16), _ld(y), m, n, k, _stream(stream))


def kalm_linear_chain_sync_len(m: int) -> int:
    return int(load().kalm_linear_chain_sync_len(m))


def kalm_linear_chain(x1: torch.Tensor, w1: torch.Tensor, y1: torch.Tensor, w2: torch.Tensor, y2: torch.Tensor,
                      sync: Optional[torch.Tensor], stream=None) -> None:
    """y1 = x1 . w1^T + y1 (in place), then y2 = y1 . w2^T, in one launch; ``sync`` is an
    int32 tensor of ``kalm_linear_chain_sync_len(m)`` entries, zero before the first call
    (every call leaves it zero)."""
    m, k1 = x1.shape
    n1, n2 = w1.shape[0], w2.shape[0]
    if w1.shape[1] != k1 or y1.shape != (m, n1) or w2.shape[1] != n1 or y2.shape != (m, n2):
        raise KalmError(1, "kalm_linear_chain", f"shapes x1{tuple(x1.shape)} w1{tuple(w1.shape)} y1{tuple(y1.shape)} "
                                                f"w2{tuple(w2.shape)} y2{tuple(y2.shape)}")
    call("kalm_linear_chain", _p(x1, torch.bfloat16), _ld(x1), _p(w1, torch.bfloat16), _ld(w1),
         _p(y1, torch.bfloat16), _ld(y1), _p(w2, torch.bfloat16), _ld(w2), _p(y2, torch.bfloat16), _ld(y2), m, n1, k1,
         n2, _p(sync, torch.int32), sync.numel() if sync is not None else 0, _stream(stream))


def kalm_linear_chain_rope(x1: torch.Tensor, w1: torch.Tensor, y1: torch.Tensor, w2: torch.Tensor, y2: torch.Tensor,
                           q_off: torch.Tensor, rot_heads: int, table: torch.Tensor, sync: Optional[torch.Tensor],
                           head_dim: int = HEAD_DIM, stream=None) -> None:
    """kalm_linear_chain with the first rot_heads head vectors of every row of y2 rotated
    by the row's decoder position (angles from kalm_rope_table), as kalm_linear_rope."""
    m, k1 = x1.shape
    n1, n2 = w1.shape[0], w2.shape[0]
    if w1.shape[1] != k1 or y1.shape != (m, n1) or w2.shape[1] != n1 or y2.shape != (m, n2):
        raise KalmError(1, "kalm_linear_chain_rope", f"shapes x1{tuple(x1.shape)} w1{tuple(w1.shape)} "
                                                     f"y1{tuple(y1.shape)} w2{tuple(w2.shape)} y2{tuple(y2.shape)}")
    if table.numel() != MAX_QUERY_TOKENS * head_dim or not table.is_contiguous():
        raise KalmError(1, "kalm_linear_chain_rope", "table must be a contiguous kalm_rope_table output")
    call("kalm_linear_chain_rope", _p(x1, torch.bfloat16), _ld(x1), _p(w1, torch.bfloat16), _ld(w1),
         _p(y1, torch.bfloat16), _ld(y1), _p(w2, torch.bfloat16), _ld(w2), _p(y2, torch.bfloat16), _ld(y2), m, n1, k1,
         n2, rot_heads * head_dim, head_dim, _p(q_off, torch.int64), q_off.numel() - 1, _p(table, torch.float32),
         _p(sync, torch.int32), sync.numel() if sync is not None else 0, _stream(stream))


def kalm_cross_kv_proj(pooled: torch.Tensor, w_kv: torch.Tensor, kv_cross: torch.Tensor, n_kv: int,
                       head_dim: int = HEAD_DIM, stream=None) -> None:
    """w_kv: [n_layers][2*n_kv*D][hidden]; kv_cross: [rows][n_layers*2*n_kv*D]."""
    n_layers = w_kv.shape[0]
    if not w_kv.is_contiguous() or not kv_cross.is_contiguous():
        raise KalmError(1, "kalm_cross_kv_proj", "w_kv and kv_cross must be contiguous")
    call("kalm_cross_kv_proj", _p(pooled, torch.bfloat16), _ld(pooled), pooled.shape[0], pooled.shape[1],
         _p(w_kv, torch.bfloat16), n_layers, n_kv, head_dim, _p(kv_cross, torch.bfloat16), _stream(stream))


def kalm_merged_attention(q: torch.Tensor, k_self: torch.Tensor, v_self: torch.Tensor, k_cross: torch.Tensor,
                          v_cross: torch.Tensor, q_off: torch.Tensor, pool_off: torch.Tensor, max_q: int,
                          n_q: int, n_kv: int, out: torch.Tensor, scale: Optional[float] = None,
                          lse: Optional[torch.Tensor] = None, head_dim: int = HEAD_DIM,
                          in_off: Optional[torch.Tensor] = None, last_tile_only: bool = False,
                          total_q: Optional[int] = None, order: Optional[torch.Tensor] = None, stream=None) -> None:
    """2-D row views: q/k/v self [input rows][...], out [q_off[-1] rows][>= n_q*D],
    k/v cross [pooled rows][>= n_kv*D].  ``in_off`` (optional) gives each document's
    first input row; by default it is q_off.  ``order`` (optional) is a work order
    from ``kalm_attention_schedule`` for the same offsets and sizes."""
    if scale is None:
        scale = head_dim ** -0.5
    if _ld(k_self) != _ld(v_self) or _ld(k_cross) != _ld(v_cross):
        raise KalmError(1, "kalm_merged_attention", "K and V views must share a row stride")
    n_docs = q_off.numel() - 1
    total_q = out.shape[0] if total_q is None else total_q
    call("kalm_merged_attention", _p(q, torch.bfloat16), _ld(q), _p(k_self, torch.bfloat16),
         _p(v_self, torch.bfloat16), _ld(k_self), _p(k_cross, torch.bfloat16), _p(v_cross, torch.bfloat16),
         _ld(k_cross), _p(q_off, torch.int64), _p(in_off, torch.int64), q.shape[0], _p(pool_off, torch.int64),
         n_docs, int(max_q), int(total_q), k_cross.shape[0], n_q, n_kv, head_dim, float(scale),
         1 if last_tile_only else 0, _p(order, torch.int32), _p(out, torch.bfloat16), _ld(out), _p(lse, torch.float32),
         _stream(stream))


def kalm_merged_attention_out_proj(q: torch.Tensor, k_self: torch.Tensor, v_self: torch.Tensor,
                                   k_cross: torch.Tensor, v_cross: torch.Tensor, q_off: torch.Tensor,
                                   pool_off: torch.Tensor, max_q: int, n_q: int, n_kv: int, out: torch.Tensor,
                                   w_o: torch.Tensor, x: torch.Tensor, sync: torch.Tensor,
                                   scale: Optional[float] = None, head_dim: int = HEAD_DIM,
                                   in_off: Optional[torch.Tensor] = None, total_q: Optional[int] = None,
                                   order: Optional[torch.Tensor] = None, stream=None) -> None:
    """Merged attention into ``out`` and then ``x[rows of d] += out[rows of d] . w_o^T`` for
    every document, in one launch.  ``sync``: int32 device tensor of at least
    ``kalm_attention_out_proj_sync_len(n_docs, max_q, hidden)`` entries, zero before the first call
    (every call leaves it zero)."""
    if scale is None:
        scale = head_dim ** -0.5
    if _ld(k_self) != _ld(v_self) or _ld(k_cross) != _ld(v_cross):
        raise KalmError(1, "kalm_merged_attention_out_proj", "K and V views must share a row stride")
    n_docs = q_off.numel() - 1
    total_q = out.shape[0] if total_q is None else total_q
    call("kalm_merged_attention_out_proj", _p(q, torch.bfloat16), _ld(q), _p(k_self, torch.bfloat16),
         _p(v_self, torch.bfloat16), _ld(k_self), _p(k_cross, torch.bfloat16), _p(v_cross, torch.bfloat16),
         _ld(k_cross), _p(q_off, torch.int64), _p(in_off, torch.int64), q.shape[0], _p(pool_off, torch.int64),
         n_docs, int(max_q), int(total_q), k_cross.shape[0], n_q, n_kv, head_dim, float(scale),
         _p(order, torch.int32), _p(out, torch.bfloat16), _ld(out), _p(w_o, torch.bfloat16), _ld(w_o),
         _p(x, torch.bfloat16), _ld(x), x.shape[1], _p(sync, torch.int32), sync.numel(), _stream(stream))


def kalm_merged_attention_out_proj_static(q: torch.Tensor, k_self: torch.Tensor, v_self: torch.Tensor,
                                          k_cross: torch.Tensor, v_cross: torch.Tensor, q_off: torch.Tensor,
                                          pool_off: torch.Tensor, max_q: int, n_q: int, n_kv: int,
                                          out: torch.Tensor, w_o: torch.Tensor, x: torch.Tensor,
                                          scale: Optional[float] = None, head_dim: int = HEAD_DIM,
                                          in_off: Optional[torch.Tensor] = None, total_q: Optional[int] = None,
                                          order: Optional[torch.Tensor] = None, stream=None) -> None:
    """kalm_merged_attention_out_proj with the library's built-in counters (no counter
    array from the caller): for callers that cannot allocate device memory.  At most
    KALM_OUT_PROJ_STATIC_MAX_DOCS (4096) documents and KALM_OUT_PROJ_STATIC_MAX_TILES (49152)
    projection tiles; calls that overlap on the GPU race."""
    if scale is None:
        scale = head_dim ** -0.5
    if _ld(k_self) != _ld(v_self) or _ld(k_cross) != _ld(v_cross):
        raise KalmError(1, "kalm_merged_attention_out_proj_static", "K and V views must share a row stride")
    n_docs = q_off.numel() - 1
    total_q = out.shape[0] if total_q is None else total_q
    call("kalm_merged_attention_out_proj_static", _p(q, torch.bfloat16), _ld(q), _p(k_self, torch.bfloat16),
         _p(v_self, torch.bfloat16), _ld(k_self), _p(k_cross, torch.bfloat16), _p(v_cross, torch.bfloat16),
         _ld(k_cross), _p(q_off, torch.int64), _p(in_off, torch.int64), q.shape[0], _p(pool_off, torch.int64),
         n_docs, int(max_q), int(total_q), k_cross.shape[0], n_q, n_kv, head_dim, float(scale),
         _p(order, torch.int32), _p(out, torch.bfloat16), _ld(out), _p(w_o, torch.bfloat16), _ld(w_o),
         _p(x, torch.bfloat16), _ld(x), x.shape[1], _stream(stream))


def kalm_attention_out_proj_sync_len(n_docs: int, max_q: int, hidden: int) -> int:
    """Entries of the sync array kalm_merged_attention_out_proj needs (-1 for bad sizes)."""
    return int(load().kalm_attention_out_proj_sync_len(n_docs, max_q, hidden))


def kalm_attention_items(n_docs: int, max_q: int, n_q: int, n_kv: int, last_tile_only: bool = False) -> int:
    """Work items of one kalm_merged_attention call (-1 for rejected sizes)."""
    return int(load().kalm_attention_items(n_docs, max_q, n_q, n_kv, 1 if last_tile_only else 0))


def kalm_attention_schedule(q_off: torch.Tensor, pool_off: torch.Tensor, max_q: int, n_q: int, n_kv: int,
                            order: torch.Tensor, last_tile_only: bool = False, stream=None) -> None:
    """Write a balanced work order for kalm_merged_attention into ``order`` (int32)."""
    call("kalm_attention_schedule", _p(q_off, torch.int64), _p(pool_off, torch.int64), q_off.numel() - 1, int(max_q),
         n_q, n_kv, 1 if last_tile_only else 0, _p(order, torch.int32), order.numel(), _stream(stream))


def kalm_yes_no_score(hidden: torch.Tensor, q_off: torch.Tensor, w_yes: torch.Tensor, w_no: torch.Tensor,
                      yes: torch.Tensor, no: torch.Tensor, score: torch.Tensor,
                      margin: Optional[torch.Tensor] = None, stream=None) -> None:
    call("kalm_yes_no_score", _p(hidden, torch.bfloat16), _ld(hidden), _p(q_off, torch.int64), q_off.numel() - 1,
         hidden.shape[1], _p(w_yes, torch.bfloat16), _p(w_no, torch.bfloat16), _p(yes, torch.float32),
         _p(no, torch.float32), _p(margin, torch.float32), _p(score, torch.float32), _stream(stream))


def kalm_broadcast_rows(src: torch.Tensor, q_off: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    call("kalm_broadcast_rows", _p(src, torch.bfloat16), _ld(src), src.shape[0], src.shape[1],
         _p(q_off, torch.int64), q_off.numel() - 1, _p(dst, torch.bfloat16), _ld(dst), _stream(stream))


def kalm_rope(x: torch.Tensor, q_off: torch.Tensor, n_heads: int, theta: float, head_dim: int = HEAD_DIM,
              stream=None) -> None:
    """Rotate the first n_heads head vectors of every row of x in place by the row's
    decoder position (row - q_off[d] for the document d owning the row)."""
    call("kalm_rope", _p(x, torch.bfloat16), _ld(x), x.shape[0], n_heads, head_dim, _p(q_off, torch.int64),
         q_off.numel() - 1, float(theta), _stream(stream))


def kalm_rope_table(theta: float, head_dim: int = HEAD_DIM, stream=None) -> torch.Tensor:
    """(cos, sin) of every rotary angle: float32 [head_dim/4][KALM_MAX_QUERY_TOKENS][4],
    entry [q][pos] = (cos, sin) of pair 2q then of pair 2q + 1."""
    table = torch.empty(head_dim // 4, MAX_QUERY_TOKENS, 4, dtype=torch.float32, device="cuda")
    call("kalm_rope_table", float(theta), head_dim, _p(table, torch.float32), _stream(stream))
    return table


def kalm_linear_rope(x: torch.Tensor, w: torch.Tensor, y: torch.Tensor, q_off: torch.Tensor, rot_heads: int,
                     table: torch.Tensor, head_dim: int = HEAD_DIM, stream=None) -> None:
    """y = x . w^T with the first rot_heads head vectors of every row rotated by the
    row's decoder position, in the projection's epilogue (angles from kalm_rope_table)."""
    m, k = x.shape
    n = w.shape[0]
    if w.shape[1] != k or y.shape[0] != m or y.shape[1] != n:
        raise KalmError(1, "kalm_linear_rope", f"shapes x{tuple(x.shape)} w{tuple(w.shape)} y{tuple(y.shape)}")
    if table.numel() != MAX_QUERY_TOKENS * head_dim or not table.is_contiguous():
        raise KalmError(1, "kalm_linear_rope", "table must be a contiguous kalm_rope_table output")
    call("kalm_linear_rope", _p(x, torch.bfloat16), _ld(x), _p(w, torch.bfloat16), _ld(w), _p(y, torch.bfloat16),
         _ld(y), m, n, k, rot_heads * head_dim, head_dim, _p(q_off, torch.int64), q_off.numel() - 1,
         _p(table, torch.float32), _stream(stream))


def _cache_args(where: str, dev: int, row_off: torch.Tensor, page_table: torch.Tensor, page_rows: int,
                codes: torch.Tensor, scales: torch.Tensor, width: int):
    """Checks what the calls on a document cache share; (n_docs, ld_table, n_pages, ld_codes, ld_scales)."""
    if row_off.dtype is not torch.int64 or row_off.get_device() != dev or row_off.dim() != 1 or \
            not row_off.is_contiguous():
        _refuse(where, "offsets", row_off, torch.int64, dev, "expected a contiguous vector")
    n_docs = row_off.size(0) - 1
    if n_docs < 0:
        raise KalmError(1, where, "the offsets are empty")
    shape = page_table.shape
    if page_table.dtype is not torch.int32 or page_table.get_device() != dev or len(shape) != 2 or \
            shape[0] != n_docs or not page_table.is_contiguous():
        _refuse(where, "page_table", page_table, torch.int32, dev, f"expected a contiguous [{n_docs}][pages] tensor")
    ld_codes = _mat(where, "codes", codes, torch.uint8, dev, -1, width)
    cached = codes.size(0)
    if page_rows <= 0 or cached % page_rows:
        raise KalmError(1, where, f"{cached} cache rows are not whole pages of {page_rows}")
    ld_scales = _mat(where, "scales", scales, torch.uint8, dev, cached, width // CACHE_GROUP)
    return n_docs, shape[1], cached // page_rows, ld_codes, ld_scales


def kalm_cache_write(src: torch.Tensor, row_off: torch.Tensor, page_table: torch.Tensor, page_rows: int,
                     codes: torch.Tensor, scales: torch.Tensor, first_row: Optional[torch.Tensor] = None,
                     stream=None) -> None:
    """Quantise packed bf16 rows into the pages of an 8-bit document cache.

    src [rows][width]: document d's rows are row_off[d] .. row_off[d+1] - 1 and become rows
    first_row[d] .. of the document (first_row None: from its row 0).  page_table int32
    [n_docs][pages]; codes uint8 [n_pages * page_rows][width]; scales uint8 [same rows][width / 32].
    No two rows may have the same place."""
    where = "kalm_cache_write"
    page_rows = int(page_rows)
    dev = _device(where, src)
    ld_src = _mat(where, "src", src, torch.bfloat16, dev)
    rows, width = src.shape
    n_docs, ld_table, n_pages, ld_codes, ld_scales = _cache_args(where, dev, row_off, page_table, page_rows, codes,
                                                                 scales, width)
    call(where, src.data_ptr(), ld_src, row_off.data_ptr(), n_docs, rows, width,
         _vec(where, "first_row", first_row, torch.int32, dev, n_docs), page_table.data_ptr(), ld_table, page_rows,
         n_pages, codes.data_ptr(), ld_codes, scales.data_ptr(), ld_scales, _stream(stream, dev))


def kalm_cache_read(codes: torch.Tensor, scales: torch.Tensor, row_off: torch.Tensor, page_table: torch.Tensor,
                    page_rows: int, dst: torch.Tensor, first_row: Optional[torch.Tensor] = None, stream=None) -> None:
    """Read cached rows back into packed bf16 rows: dst[row_off[d] + i] = row first_row[d] + i of
    document d (the stored values exactly).  Arguments as kalm_cache_write."""
    where = "kalm_cache_read"
    page_rows = int(page_rows)
    dev = _device(where, dst)
    ld_dst = _mat(where, "dst", dst, torch.bfloat16, dev)
    rows, width = dst.shape
    n_docs, ld_table, n_pages, ld_codes, ld_scales = _cache_args(where, dev, row_off, page_table, page_rows, codes,
                                                                 scales, width)
    call(where, codes.data_ptr(), ld_codes, scales.data_ptr(), ld_scales, row_off.data_ptr(), n_docs, rows, width,
         _vec(where, "first_row", first_row, torch.int32, dev, n_docs), page_table.data_ptr(), ld_table, page_rows,
         n_pages, dst.data_ptr(), ld_dst, _stream(stream, dev))


def kalm_merged_attention_cache(q: torch.Tensor, k_self: torch.Tensor, v_self: torch.Tensor, k_codes: torch.Tensor,
                                k_scales: torch.Tensor, v_codes: torch.Tensor, v_scales: torch.Tensor,
                                page_table: torch.Tensor, page_rows: int, q_off: torch.Tensor, pool_off: torch.Tensor,
                                max_q: int, n_q: int, n_kv: int, out: torch.Tensor, scale: Optional[float] = None,
                                lse: Optional[torch.Tensor] = None, head_dim: int = HEAD_DIM,
                                in_off: Optional[torch.Tensor] = None, last_tile_only: bool = False,
                                total_q: Optional[int] = None, order: Optional[torch.Tensor] = None,
                                workspace: Optional[torch.Tensor] = None, stream=None,
                                total_pool: Optional[int] = None) -> None:
    """kalm_merged_attention with the cross K/V of an 8-bit document cache: document d attends to its
    first pool_off[d+1] - pool_off[d] cached rows.  k/v codes uint8 [cache rows][n_kv * head_dim]
    (column views of the cached rows are fine), k/v scales uint8 [cache rows][n_kv * head_dim / 32];
    the other arguments as kalm_merged_attention.

    workspace: bf16 scratch [>= kalm_merged_attention_cache_rows(cached rows, n_docs)][2 * n_kv * head_dim];
    None allocates one for this call: for `total_pool` cached rows (pool_off[-1] - pool_off[0], where the
    caller has it on the host), or else for as many as the page table has places, which is far more where
    one document is much longer than the rest.  Calls of at most CACHE_FEW_ROWS packed rows a KV head
    (max_q * n_q / n_kv) use none."""
    where = "kalm_merged_attention_cache"
    bf16 = torch.bfloat16
    max_q, page_rows = int(max_q), int(page_rows)
    dev = _device(where, q)
    width, rows = n_kv * head_dim, q.size(0)
    n_docs, ld_table, n_pages, ld_codes, ld_scales = _cache_args(where, dev, pool_off, page_table, page_rows, k_codes,
                                                                 k_scales, width)
    ld_self = _mat(where, "k_self", k_self, bf16, dev, rows, width)
    _pair(where, "self rows", k_self, v_self)
    _pair(where, "codes", k_codes, v_codes)
    _pair(where, "scales", k_scales, v_scales)
    ldq = _mat(where, "q", q, bf16, dev, rows, n_q * head_dim)
    ldo = _mat(where, "out", out, bf16, dev, -1, n_q * head_dim)
    out_rows = out.size(0)
    total_q = out_rows if total_q is None else int(total_q)
    if total_q > out_rows or (in_off is None and total_q > rows):
        raise KalmError(1, where, f"total_q={total_q} exceeds the rows of out ({out_rows}) or q ({rows})")
    if lse is not None and (lse.dtype is not torch.float32 or lse.get_device() != dev or lse.dim() != 2 or
                            lse.shape[0] < total_q or lse.shape[1] != n_q or not lse.is_contiguous()):
        _refuse(where, "lse", lse, torch.float32, dev, f"expected a contiguous [{total_q}][{n_q}] tensor")
    if order is not None:
        tile = max(128 * n_kv // n_q, 1) if n_q > 0 else 1  # positions of a query tile, as in kalm_attention_items
        items = n_docs * n_kv * (1 if last_tile_only else -(-max_q // tile))
        if order.dtype is not torch.int32 or order.get_device() != dev or order.numel() < items or \
                not order.is_contiguous():
            _refuse(where, "order", order, torch.int32, dev, f"expected at least the call's {items} work items")
    ws, ws_rows = None, 0
    if workspace is None and max_q * n_q > CACHE_FEW_ROWS * n_kv:
        if total_pool is None:
            total_pool = n_docs * ld_table * page_rows  # every place of the table
        elif total_pool < 0:
            raise KalmError(1, where, f"total_pool={total_pool}")
        shape = (total_pool + 64 * n_docs, 2 * width)  # kalm_merged_attention_cache_rows
        if stream is None:
            workspace = q.new_empty(shape)
        else:
            with torch.cuda.stream(stream):  # the allocator hands memory out per stream
                workspace = q.new_empty(shape)
    elif workspace is not None and _mat(where, "workspace", workspace, bf16, dev, -1, 2 * width) != 2 * width:
        raise KalmError(1, where, "the workspace must be contiguous")
    if workspace is not None:
        ws, ws_rows = workspace.data_ptr(), workspace.size(0)
    call(where, q.data_ptr(), ldq, k_self.data_ptr(), v_self.data_ptr(), ld_self, k_codes.data_ptr(),
         v_codes.data_ptr(), ld_codes, k_scales.data_ptr(), v_scales.data_ptr(), ld_scales, page_table.data_ptr(),
         ld_table, page_rows, n_pages, _vec(where, "q_off", q_off, torch.int64, dev, n_docs + 1),
         _vec(where, "in_off", in_off, torch.int64, dev, n_docs), rows, pool_off.data_ptr(), n_docs, max_q, total_q,
         n_q, n_kv, head_dim, head_dim ** -0.5 if scale is None else float(scale), 1 if last_tile_only else 0,
         None if order is None else order.data_ptr(), ws, ws_rows, out.data_ptr(), ldo,
         None if lse is None else lse.data_ptr(), _stream(stream, dev))


def kalm_merged_attention_cache_rows(total_pool: int, n_docs: int) -> int:
    """Rows of kalm_merged_attention_cache's workspace (-1 for negative sizes)."""
    return int(load().kalm_merged_attention_cache_rows(total_pool, n_docs))


def kalm_rms_norm(x: torch.Tensor, w: torch.Tensor, h: torch.Tensor, eps: float = 1e-6, weight_offset: float = 0.0,
                  stream=None) -> None:
    """h = x / sqrt(mean(x^2) + eps) * (w + weight_offset), row by row; h may be x."""
    where = "kalm_rms_norm"
    dev = _device(where, x)
    ldx = _mat(where, "x", x, torch.bfloat16, dev)
    rows, width = x.shape
    call(where, x.data_ptr(), ldx, _vec(where, "w", w, torch.bfloat16, dev, width), h.data_ptr(),
         _mat(where, "h", h, torch.bfloat16, dev, rows, width), rows, width, float(eps), float(weight_offset),
         _stream(stream, dev))


def kalm_norm_residual(y: torch.Tensor, x: torch.Tensor, x_out: torch.Tensor, h: Optional[torch.Tensor] = None,
                       w_post: Optional[torch.Tensor] = None, w_pre: Optional[torch.Tensor] = None,
                       gate: Optional[torch.Tensor] = None, q_off: Optional[torch.Tensor] = None,
                       residual_scale: float = 1.0, eps: float = 1e-6, weight_offset: float = 0.0,
                       stream=None) -> None:
    """Between two blocks: t = residual_scale * x + gate * norm(y, w_post), x_out = t, h = norm(t, w_pre).

    gate: None, one vector [width], or one per document [n_docs][width] (with q_off, the documents'
    row offsets).  With q_off only the documents' rows are computed.  w_post None: y enters without a
    norm; h and w_pre go together.  x_out may be x."""
    where = "kalm_norm_residual"
    bf16 = torch.bfloat16
    dev = _device(where, x)
    ldx = _mat(where, "x", x, bf16, dev)
    rows, width = x.shape
    n_docs = 0 if q_off is None else q_off.numel() - 1
    if n_docs < 0:
        raise KalmError(1, where, "the offsets are empty")
    ld_gate, gate_at = 0, None
    if gate is not None and gate.dim() == 2:
        if q_off is None:
            raise KalmError(1, where, "a gate per document needs q_off")
        ld_gate, gate_at = _mat(where, "gate", gate, bf16, dev, n_docs, width), gate.data_ptr()
    else:
        gate_at = _vec(where, "gate", gate, bf16, dev, width)
    call(where, y.data_ptr(), _mat(where, "y", y, bf16, dev, rows, width), x.data_ptr(), ldx,
         _vec(where, "w_post", w_post, bf16, dev, width), gate_at, ld_gate,
         _vec(where, "q_off", q_off, torch.int64, dev, n_docs + 1), n_docs, float(residual_scale), x_out.data_ptr(),
         _mat(where, "x_out", x_out, bf16, dev, rows, width), _vec(where, "w_pre", w_pre, bf16, dev, width),
         None if h is None else h.data_ptr(), 0 if h is None else _mat(where, "h", h, bf16, dev, rows, width), rows,
         width, float(eps), float(weight_offset), _stream(stream, dev))


def kalm_selftest_wait_timeout(wait_ns: int, stream=None) -> None:
    call("kalm_selftest_wait_timeout", int(wait_ns), _stream(stream))

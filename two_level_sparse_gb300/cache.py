"""ctypes binding of the paged key-value cache (include/ci_cache.h), same entry-point names.

Argument marshalling only, like ``ci``: tensors become device pointers and
sizes, the current torch stream becomes the cudaStream_t, and a non-zero
status becomes a ``ci.CIError``.  The cache format and the head size follow
from the tensors' shapes.

A pool is a uint8 tensor [num_pages, kv_heads, page_bytes(format, head_dim)];
``page_table`` int32 [requests, max_pages], ``ref_count`` int32 [num_pages].
"""
from __future__ import annotations

import ctypes
from array import array

import torch

from .ci import (CI_OK, DEVERR_LEN, DEVERR_PAGE, DEVERR_POS, DEVERR_REQ, LAYOUT_DECODE, LAYOUT_PREFILL,  # noqa: F401
                 LAYOUT_VARLEN, CIError, lib)

CACHE_BF16, CACHE_FP8 = 0, 1
PAGE = 64
MAX_POOLS = 160

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_F32 = ctypes.c_float

_TABLE = [_P, _I32, _I32, _P, _I64]  # page_table, num_req, max_pages, ref_count, num_pages
SIGNATURES = {
    "ci_cache_page_bytes": [_I32, _I32],
    "ci_attn_workspace_bytes": [_I32, _I32, _I32, _I32],
    "ci_attn_decode": [_P, _I64, _I32, _I32, _I32, _I32, _F32, _P, _P, _I64, _I32, _P, _I32, _I32, _I32, _P, _P, _I32,
                       _P, _I64, _I32, _P, _I64, _P, _P, _I64, _P, _P],
    "ci_qk_norm_rope_append": [_P, _I64, _P, _I64, _P, _I64, _I32, _I32, _I32, _I32, _P, _P, _F32, _P, _I32, _I32,
                               _I32, _P, _P, _P, _I64, _P, _P, _I64, _I32, _P, _I32, _I32, _I32, _P, _P, _P],
    "ci_pages_alloc": [*_TABLE, _P, _P, _P, _P],
    "ci_pages_fork": [*_TABLE, _P, _P, _P, _I32, _P, _P, _P, _P],
    "ci_pages_free": [*_TABLE, _P, _I32, _P, _P],
    "ci_pages_compact": [*_TABLE, _P, _P, _P, _P, _P, _P],
    "ci_pages_copy": [_P, _P, _I32, _I64, _P, _P, _I32, _P, _P, _P],
}
for _name, _argtypes in SIGNATURES.items():
    _fn = getattr(lib, _name)
    _fn.argtypes = _argtypes
    _fn.restype = _I64 if _name.endswith("_bytes") else ctypes.c_int


_U8, _BF16, _F32T, _I32T = torch.uint8, torch.bfloat16, torch.float32, torch.int32


def _dev(t, dtype, name):
    """The device pointer of a contiguous GPU tensor of the type (None: NULL)."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _ints(t, name):
    """_dev for an int32 tensor that is there."""
    if t.dtype is not _I32T or not t.is_cuda or not t.is_contiguous():
        return _dev(t, _I32T, name)  # says what is wrong
    return t.data_ptr()


def _heads(t, name):
    """Pointer, row stride and shape of a bf16 [rows, heads, head_dim] tensor whose rows may lie apart."""
    if t.dtype is not _BF16:
        raise TypeError(f"{name} must be {_BF16}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU")
    shape = t.shape
    rows, heads, dim = shape
    stride, head_stride, one = t.stride()
    if dim > 1 and one != 1 or heads > 1 and head_stride != dim:
        raise ValueError(f"{name} must be contiguous within a row")
    return t.data_ptr(), (stride if rows > 1 else heads * dim), shape


def _numel(t, n, name):
    if t is not None and t.numel() < n:
        raise ValueError(f"{name} needs {n} entries, got {t.numel()}")


_current_stream = torch._C._cuda_getCurrentRawStream  # torch.cuda.current_stream(device).cuda_stream, without the object


def _on(stream, like):
    return stream.cuda_stream if stream is not None else _current_stream(like.get_device())


def empty_on(stream, shape, dtype, device):
    """torch.empty of the memory of the stream that is to use it (None: the
    current one): what another stream had there, or gets there once the tensor
    is dropped, may not be ordered with the work on ``stream``."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _check(fn, status):
    if status != CI_OK:
        raise CIError(fn, status)


def page_bytes(cache_format: int, head_dim: int) -> int:
    """Bytes of one (page, key-value head) of a pool."""
    n = lib.ci_cache_page_bytes(cache_format, head_dim)
    if n < 0:
        raise CIError("ci_cache_page_bytes", n)
    return n


def cache_format(pool, head_dim: int) -> int:
    """The format of a pool, from the bytes of its pages."""
    return _format(pool.shape, head_dim)


def _format(shape, head_dim):
    if len(shape) == 3:
        n = shape[2]
        if n == PAGE * head_dim * 2:
            return CACHE_BF16
        if n == PAGE * head_dim + PAGE * 4:
            return CACHE_FP8
    raise ValueError(f"a pool must be [num_pages, kv_heads, {PAGE * head_dim * 2}] (bf16) or "
                     f"[num_pages, kv_heads, {PAGE * head_dim + PAGE * 4}] (FP8) for heads of {head_dim}, got "
                     f"{tuple(shape)}")


def _pools(k_pool, v_pool, head_dim):
    shape = k_pool.shape
    if shape != v_pool.shape:
        raise ValueError("k_pool and v_pool must have the same shape")
    fmt = _format(shape, head_dim)
    return _dev(k_pool, _U8, "k_pool"), _dev(v_pool, _U8, "v_pool"), shape[0], shape[1], fmt


def attn_workspace_bytes(rows: int, num_q_heads: int, num_kv_heads: int, head_dim: int) -> int:
    n = lib.ci_attn_workspace_bytes(rows, num_q_heads, num_kv_heads, head_dim)
    if n < 0:
        raise CIError("ci_attn_workspace_bytes", n)
    return n


def ci_attn_decode(q, k_pool, v_pool, page_table, layout, seq_len, max_len, scale, out, lse=None, pos=None,
                   workspace=None, dev_err=None, stream=None, req_start=None):
    """Attention of q [rows, q_heads, head_dim] over the cache, or over the
    positions ``pos`` [rows, n] of it (see include/ci_cache.h).  ``workspace``:
    uint8, attn_workspace_bytes() of it; allocated here, from the memory of the
    call's stream, if None."""
    qp, q_stride, shape = _heads(q, "q")
    op, out_stride, out_shape = _heads(out, "out")
    if out_shape != shape:
        raise ValueError("out must have q's shape")
    rows, hq, d = shape
    kp, vp, num_pages, hkv, fmt = _pools(k_pool, v_pool, d)
    _numel(seq_len, rows, "seq_len")
    _numel(lse, rows * hq, "lse")
    pp, pos_stride = None, 0
    if pos is not None:
        if pos.dim() != 2 or pos.shape[0] < rows:
            raise ValueError("pos must be [rows, n]")
        pos_stride = pos.shape[1]
        # an empty tensor has a null pointer, which would mean "every position": any other one does, it is not read
        pp = _ints(pos, "pos") if pos_stride else qp
    if workspace is None:
        workspace = empty_on(stream, (attn_workspace_bytes(rows, hq, hkv, d),), _U8, q.device)
    num_req, max_pages = page_table.shape
    starts = None
    if layout == LAYOUT_VARLEN:
        _numel(req_start, num_req + 1, "req_start")
        starts = _dev(req_start, _I32T, "req_start")
    status = lib.ci_attn_decode(
        qp, q_stride, rows, hq, hkv, d, scale, kp, vp, num_pages, fmt, _ints(page_table, "page_table"), num_req,
        max_pages, layout, starts, _ints(seq_len, "seq_len"), max_len, pp, pos_stride, pos_stride, op, out_stride,
        _dev(lse, _F32T, "lse"), _dev(workspace, _U8, "workspace"), workspace.numel(), _dev(dev_err, _I32T, "dev_err"),
        _on(stream, q))
    if status:
        _check("ci_attn_decode", status)


def ci_qk_norm_rope_append(q, k, v, q_norm, k_norm, eps, cos_sin, is_neox, positions, q_out, k_pool, v_pool,
                           page_table, layout, dev_err=None, stream=None, req_start=None, cache_pos=None):
    """Norm and rotation of the new tokens' queries and keys; keys and values
    into their pages (see include/ci_cache.h)."""
    qp, q_stride, shape = _heads(q, "q")
    kp, k_stride, k_shape = _heads(k, "k")
    vp, v_stride, v_shape = _heads(v, "v")
    op, o_stride, o_shape = _heads(q_out, "q_out")
    tokens, hq, d = shape
    kpool, vpool, num_pages, hkv, fmt = _pools(k_pool, v_pool, d)
    if o_shape != shape or k_shape != v_shape or k_shape != (tokens, hkv, d):
        raise ValueError("q_out must have q's shape, k and v [tokens, the pools' kv_heads, head_dim]")
    _numel(positions, tokens, "positions")
    _numel(cache_pos, tokens, "cache_pos")
    _numel(q_norm, d, "q_norm")
    _numel(k_norm, d, "k_norm")
    max_pos, rot = cos_sin.shape
    num_req, max_pages = page_table.shape
    starts = None
    if layout == LAYOUT_VARLEN:
        _numel(req_start, num_req + 1, "req_start")
        starts = _dev(req_start, _I32T, "req_start")
    status = lib.ci_qk_norm_rope_append(
        qp, q_stride, kp, k_stride, vp, v_stride, tokens, hq, hkv, d, _dev(q_norm, _F32T, "q_norm"),
        _dev(k_norm, _F32T, "k_norm"), eps, _dev(cos_sin, _F32T, "cos_sin"), max_pos, rot, is_neox,
        _ints(positions, "positions"), _dev(cache_pos, _I32T, "cache_pos"), op, o_stride, kpool, vpool, num_pages, fmt,
        _ints(page_table, "page_table"), num_req, max_pages, layout, starts, _dev(dev_err, _I32T, "dev_err"),
        _on(stream, q))
    if status:
        _check("ci_qk_norm_rope_append", status)


def _table(page_table, ref_count):
    num_req, max_pages = page_table.shape
    return _ints(page_table, "page_table"), num_req, max_pages, _ints(ref_count, "ref_count"), ref_count.shape[0]


def ci_pages_alloc(page_table, ref_count, old_len, new_len, dev_err=None, stream=None):
    """Pages for every request's growth from old_len to new_len positions (see include/ci_cache.h)."""
    _numel(old_len, page_table.shape[0], "old_len")
    _numel(new_len, page_table.shape[0], "new_len")
    _check("ci_pages_alloc", lib.ci_pages_alloc(
        *_table(page_table, ref_count), _ints(old_len, "old_len"), _ints(new_len, "new_len"),
        _dev(dev_err, _I32T, "dev_err"), _on(stream, page_table)))


def ci_pages_fork(page_table, ref_count, parent, child, length, copy_src, copy_dst, dev_err=None, stream=None):
    """Children that share their parents' full pages; the pairs still to be copied (see include/ci_cache.h)."""
    n = parent.shape[0]
    if min(child.numel(), length.numel(), copy_src.numel(), copy_dst.numel()) < n:
        raise ValueError(f"child, length, copy_src and copy_dst need {n} entries each")
    _check("ci_pages_fork", lib.ci_pages_fork(
        *_table(page_table, ref_count), _ints(parent, "parent"), _ints(child, "child"), _ints(length, "length"), n,
        _ints(copy_src, "copy_src"), _ints(copy_dst, "copy_dst"), _dev(dev_err, _I32T, "dev_err"),
        _on(stream, page_table)))


def ci_pages_free(page_table, ref_count, req, dev_err=None, stream=None):
    """The pages of the requests ``req`` released, their rows -1 (see include/ci_cache.h)."""
    _check("ci_pages_free", lib.ci_pages_free(
        *_table(page_table, ref_count), _ints(req, "req"), req.shape[0], _dev(dev_err, _I32T, "dev_err"),
        _on(stream, page_table)))


def ci_pages_compact(page_table, ref_count, remap, copy_src, copy_dst, count, dev_err=None, stream=None):
    """Live pages into the lowest ids; the pairs to be copied and their count (see include/ci_cache.h)."""
    n = ref_count.shape[0]
    if min(remap.numel(), copy_src.numel(), copy_dst.numel()) < n:
        raise ValueError(f"remap, copy_src and copy_dst need {n} entries each")
    _numel(count, 1, "count")
    _check("ci_pages_compact", lib.ci_pages_compact(
        *_table(page_table, ref_count), _ints(remap, "remap"), _ints(copy_src, "copy_src"),
        _ints(copy_dst, "copy_dst"), _ints(count, "count"), _dev(dev_err, _I32T, "dev_err"), _on(stream, page_table)))


def ci_pages_copy(pools, copy_src, copy_dst, count=None, dev_err=None, stream=None):
    """The pairs' pages copied in every pool (see include/ci_cache.h).
    ``pools``: one uint8 tensor [pools, num_pages, ...] or a sequence of
    tensors [num_pages, ...], such as every layer's key, value and index pools."""
    n = len(pools)
    if not 1 <= n <= MAX_POOLS:
        raise ValueError(f"1 to {MAX_POOLS} pools per call")
    if isinstance(pools, torch.Tensor):
        base, num_pages = _dev(pools, _U8, "pools"), pools.shape[1]
        step = pools.numel() // n  # (the first stride of one pool may be anything)
        ptrs = array("Q", [base + i * step for i in range(n)])
        sizes = array("q", [step // num_pages if num_pages else 0]) * n
    else:
        num_pages = pools[0].shape[0]
        if any(p.shape[0] != num_pages for p in pools):
            raise ValueError("every pool needs the same number of pages")
        ptrs = array("Q", [_dev(p, _U8, "pools") for p in pools])
        sizes = array("q", [p.numel() // num_pages if num_pages else 0 for p in pools])
    m = copy_src.shape[0]
    _numel(copy_dst, m, "copy_dst")
    _check("ci_pages_copy", lib.ci_pages_copy(
        ptrs.buffer_info()[0], sizes.buffer_info()[0], n, num_pages, _ints(copy_src, "copy_src"),
        _ints(copy_dst, "copy_dst"), m, _dev(count, _I32T, "count"), _dev(dev_err, _I32T, "dev_err"),
        _on(stream, copy_src)))

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


def _dev(t, dtype, name):
    """The device pointer of a contiguous GPU tensor of the type (None: NULL)."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _heads(t, name):
    """Pointer, row stride and shape of a bf16 [rows, heads, head_dim] tensor whose rows may lie apart."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on the GPU")
    rows, heads, dim = t.shape
    stride, head_stride, one = t.stride()
    if dim > 1 and one != 1 or heads > 1 and head_stride != dim:
        raise ValueError(f"{name} must be contiguous within a row")
    return t.data_ptr(), (stride if rows > 1 else heads * dim), rows, heads, dim


def _numel(t, n, name):
    if t is not None and t.numel() < n:
        raise ValueError(f"{name} needs {n} entries, got {t.numel()}")


_current_stream = torch._C._cuda_getCurrentRawStream  # torch.cuda.current_stream(device).cuda_stream, without the object


def _on(stream, like):
    return stream.cuda_stream if stream is not None else _current_stream(like.get_device())


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
    if pool.dim() == 3:
        n = pool.shape[2]
        if n == PAGE * head_dim * 2:
            return CACHE_BF16
        if n == PAGE * head_dim + PAGE * 4:
            return CACHE_FP8
    raise ValueError(f"a pool must be [num_pages, kv_heads, {PAGE * head_dim * 2}] (bf16) or "
                     f"[num_pages, kv_heads, {PAGE * head_dim + PAGE * 4}] (FP8) for heads of {head_dim}, got "
                     f"{tuple(pool.shape)}")


def _pools(k_pool, v_pool, head_dim):
    if k_pool.shape != v_pool.shape:
        raise ValueError("k_pool and v_pool must have the same shape")
    return (_dev(k_pool, torch.uint8, "k_pool"), _dev(v_pool, torch.uint8, "v_pool"), k_pool.shape[0],
            cache_format(k_pool, head_dim))


def attn_workspace_bytes(rows: int, num_q_heads: int, num_kv_heads: int, head_dim: int) -> int:
    n = lib.ci_attn_workspace_bytes(rows, num_q_heads, num_kv_heads, head_dim)
    if n < 0:
        raise CIError("ci_attn_workspace_bytes", n)
    return n


def ci_attn_decode(q, k_pool, v_pool, page_table, layout, seq_len, max_len, scale, out, lse=None, pos=None,
                   workspace=None, dev_err=None, stream=None, req_start=None):
    """Attention of q [rows, q_heads, head_dim] over the cache, or over the
    positions ``pos`` [rows, n] of it (see include/ci_cache.h).  ``workspace``:
    uint8, attn_workspace_bytes() of it; allocated here if None."""
    qp, q_stride, rows, hq, d = _heads(q, "q")
    op, out_stride, *shape = _heads(out, "out")
    if shape != [rows, hq, d]:
        raise ValueError("out must have q's shape")
    kp, vp, num_pages, fmt = _pools(k_pool, v_pool, d)
    hkv = k_pool.shape[1]
    _numel(seq_len, rows, "seq_len")
    _numel(lse, rows * hq, "lse")
    pos_stride = npos = 0
    if pos is not None:
        if pos.dim() != 2 or pos.shape[0] < rows:
            raise ValueError("pos must be [rows, n]")
        npos = pos_stride = pos.shape[1]
    # an empty tensor has a null pointer, which would mean "every position": any other one does, it is not read
    pp = qp if pos is not None and npos == 0 else _dev(pos, torch.int32, "pos")
    if workspace is None:
        workspace = torch.empty(attn_workspace_bytes(rows, hq, hkv, d), dtype=torch.uint8, device=q.device)
    num_req, max_pages = page_table.shape
    if layout == LAYOUT_VARLEN:
        _numel(req_start, num_req + 1, "req_start")
    _check("ci_attn_decode", lib.ci_attn_decode(
        qp, q_stride, rows, hq, hkv, d, scale, kp, vp, num_pages, fmt, _dev(page_table, torch.int32, "page_table"),
        num_req, max_pages, layout, _dev(req_start, torch.int32, "req_start"), _dev(seq_len, torch.int32, "seq_len"),
        max_len, pp, pos_stride, npos, op, out_stride, _dev(lse, torch.float32, "lse"),
        _dev(workspace, torch.uint8, "workspace"), workspace.numel(), _dev(dev_err, torch.int32, "dev_err"),
        _on(stream, q)))


def ci_qk_norm_rope_append(q, k, v, q_norm, k_norm, eps, cos_sin, is_neox, positions, q_out, k_pool, v_pool,
                           page_table, layout, dev_err=None, stream=None, req_start=None, cache_pos=None):
    """Norm and rotation of the new tokens' queries and keys; keys and values
    into their pages (see include/ci_cache.h)."""
    qp, q_stride, tokens, hq, d = _heads(q, "q")
    kp, k_stride, *ks = _heads(k, "k")
    vp, v_stride, *vs = _heads(v, "v")
    op, o_stride, *os_ = _heads(q_out, "q_out")
    hkv = k_pool.shape[1]
    if os_ != [tokens, hq, d] or ks != [tokens, hkv, d] or vs != [tokens, hkv, d]:
        raise ValueError("q_out must have q's shape, k and v [tokens, the pools' kv_heads, head_dim]")
    kpool, vpool, num_pages, fmt = _pools(k_pool, v_pool, d)
    _numel(positions, tokens, "positions")
    _numel(cache_pos, tokens, "cache_pos")
    _numel(q_norm, d, "q_norm")
    _numel(k_norm, d, "k_norm")
    max_pos, rot = cos_sin.shape
    num_req, max_pages = page_table.shape
    if layout == LAYOUT_VARLEN:
        _numel(req_start, num_req + 1, "req_start")
    f32, i32 = torch.float32, torch.int32
    _check("ci_qk_norm_rope_append", lib.ci_qk_norm_rope_append(
        qp, q_stride, kp, k_stride, vp, v_stride, tokens, hq, hkv, d, _dev(q_norm, f32, "q_norm"),
        _dev(k_norm, f32, "k_norm"), eps, _dev(cos_sin, f32, "cos_sin"), max_pos, rot, is_neox,
        _dev(positions, i32, "positions"), _dev(cache_pos, i32, "cache_pos"), op, o_stride, kpool, vpool, num_pages,
        fmt, _dev(page_table, i32, "page_table"), num_req, max_pages, layout, _dev(req_start, i32, "req_start"),
        _dev(dev_err, i32, "dev_err"), _on(stream, q)))


def _table(page_table, ref_count):
    num_req, max_pages = page_table.shape
    return (_dev(page_table, torch.int32, "page_table"), num_req, max_pages,
            _dev(ref_count, torch.int32, "ref_count"), ref_count.shape[0])


def ci_pages_alloc(page_table, ref_count, old_len, new_len, dev_err=None, stream=None):
    """Pages for every request's growth from old_len to new_len positions (see include/ci_cache.h)."""
    _numel(old_len, page_table.shape[0], "old_len")
    _numel(new_len, page_table.shape[0], "new_len")
    i32 = torch.int32
    _check("ci_pages_alloc", lib.ci_pages_alloc(
        *_table(page_table, ref_count), _dev(old_len, i32, "old_len"), _dev(new_len, i32, "new_len"),
        _dev(dev_err, i32, "dev_err"), _on(stream, page_table)))


def ci_pages_fork(page_table, ref_count, parent, child, length, copy_src, copy_dst, dev_err=None, stream=None):
    """Children that share their parents' full pages; the pairs still to be copied (see include/ci_cache.h)."""
    n = parent.shape[0]
    for t, name in ((child, "child"), (length, "length"), (copy_src, "copy_src"), (copy_dst, "copy_dst")):
        _numel(t, n, name)
    i32 = torch.int32
    _check("ci_pages_fork", lib.ci_pages_fork(
        *_table(page_table, ref_count), _dev(parent, i32, "parent"), _dev(child, i32, "child"),
        _dev(length, i32, "length"), n, _dev(copy_src, i32, "copy_src"), _dev(copy_dst, i32, "copy_dst"),
        _dev(dev_err, i32, "dev_err"), _on(stream, page_table)))


def ci_pages_free(page_table, ref_count, req, dev_err=None, stream=None):
    """The pages of the requests ``req`` released, their rows -1 (see include/ci_cache.h)."""
    _check("ci_pages_free", lib.ci_pages_free(
        *_table(page_table, ref_count), _dev(req, torch.int32, "req"), req.shape[0],
        _dev(dev_err, torch.int32, "dev_err"), _on(stream, page_table)))


def ci_pages_compact(page_table, ref_count, remap, copy_src, copy_dst, count, dev_err=None, stream=None):
    """Live pages into the lowest ids; the pairs to be copied and their count (see include/ci_cache.h)."""
    n = ref_count.shape[0]
    for t, name in ((remap, "remap"), (copy_src, "copy_src"), (copy_dst, "copy_dst")):
        _numel(t, n, name)
    _numel(count, 1, "count")
    i32 = torch.int32
    _check("ci_pages_compact", lib.ci_pages_compact(
        *_table(page_table, ref_count), _dev(remap, i32, "remap"), _dev(copy_src, i32, "copy_src"),
        _dev(copy_dst, i32, "copy_dst"), _dev(count, i32, "count"), _dev(dev_err, i32, "dev_err"),
        _on(stream, page_table)))


def ci_pages_copy(pools, copy_src, copy_dst, count=None, dev_err=None, stream=None):
    """The pairs' pages copied in every pool (see include/ci_cache.h).
    ``pools``: one uint8 tensor [pools, num_pages, ...] or a sequence of
    tensors [num_pages, ...], such as every layer's key, value and index pools."""
    n = len(pools)
    if not 1 <= n <= MAX_POOLS:
        raise ValueError(f"1 to {MAX_POOLS} pools per call")
    if isinstance(pools, torch.Tensor):
        base, num_pages = _dev(pools, torch.uint8, "pools"), pools.shape[1]
        step = pools.stride(0)
        ptrs = (_P * n)(*range(base, base + n * step, step)) if step else (_P * n)(*[base] * n)
        sizes = (_I64 * n)(*[step // num_pages if num_pages else 0] * n)
    else:
        num_pages = pools[0].shape[0]
        if any(p.shape[0] != num_pages for p in pools):
            raise ValueError("every pool needs the same number of pages")
        ptrs = (_P * n)(*[_dev(p, torch.uint8, "pools") for p in pools])
        sizes = (_I64 * n)(*[p.numel() // num_pages if num_pages else 0 for p in pools])
    _numel(copy_dst, copy_src.shape[0], "copy_dst")
    i32 = torch.int32
    _check("ci_pages_copy", lib.ci_pages_copy(
        ptrs, sizes, n, num_pages, _dev(copy_src, i32, "copy_src"), _dev(copy_dst, i32, "copy_dst"),
        copy_src.shape[0], _dev(count, i32, "count"), _dev(dev_err, i32, "dev_err"), _on(stream, copy_src)))

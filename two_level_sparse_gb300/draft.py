"""ctypes binding of drafted steps over the paged cache (include/ci_draft.h), same entry-point names.

Argument marshalling only, like ``cache``, whose conventions hold: pools are
uint8 [num_pages, kv_heads, bytes], ids and lengths int32, and a call runs on
``stream`` (None: the current one of its tensors' device, which has to be the
current device).

Trees are ``parent`` [requests, nodes] (None: chains); node 0 of a request is
the token that it goes on with.
"""
from __future__ import annotations

import ctypes
from array import array

import torch

from .cache import (_F32, _F32T, _I32, _I32T, _I64, _P, _U8, MAX_POOLS, PAGE, _check, _dev, _heads, _on, _pools,
                    empty_on)
from .ci import CIError, lib

MAX_NODES = 256

SIGNATURES = {
    "ci_draft_plan": [_P, _P, _P, _P, _I32, _I32, _P, _I32, _I64, _I32, _P, _P, _P, _P, _I32, _P, _P, _P],
    "ci_attn_draft_workspace_bytes": [_I32, _I32, _I32, _I32],
    "ci_attn_draft": [_P, _I64, _I32, _I32, _I32, _I32, _F32, _P, _P, _I64, _I32, _P, _I32, _I32, _P, _P, _I32, _I32,
                      _P, _I32, _P, _I64, _P, _P, _I64, _P, _P],
    "ci_draft_accept": [_P, _P, _P, _I32, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P],
    "ci_slots_move": [_P, _P, _P, _P, _I32, _I64, _P, _I32, _I32, _P, _P, _I32, _P, _P, _P],
    "ci_pages_trim": [_P, _I32, _I32, _P, _I64, _P, _P, _P, _P],
}
for _name, _argtypes in SIGNATURES.items():
    _fn = getattr(lib, _name)
    _fn.argtypes = _argtypes
    _fn.restype = _I64 if _name.endswith("_bytes") else ctypes.c_int


_current_device = torch._C._cuda_getDevice  # torch.cuda.current_device(), without the check that CUDA is up


def _at(t, name):
    """The device of a call's first tensor: the current one, which the launch goes to.  The others are compared with it."""
    at = t.get_device()
    if at < 0:
        raise ValueError(f"{name} must live on the GPU")
    if at != _current_device():
        raise ValueError(f"{name} must live on the current device")
    return at


def _here(t, at, dtype, name):
    """The device pointer of a contiguous tensor of the type on device ``at`` (None: NULL)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != at or not t.is_contiguous():
        _dev(t, dtype, name)  # says what is wrong
        raise ValueError(f"{name} must live on the current device")
    return t.data_ptr()


def _shape(t, shape, at, name):
    """_here for an int32 tensor of the shape."""
    if t is None:
        return None
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype is not _I32T or t.get_device() != at or not t.is_contiguous():
        return _here(t, at, _I32T, name)
    return t.data_ptr()


def ci_draft_plan(length, count, parent, page_table, num_pages, req_start, positions, cache_pos, mask=None, token=None,
                  row_token=None, max_nodes=None, dev_err=None, stream=None):
    """The rows of a drafted step (see include/ci_draft.h).  ``positions`` has
    as many rows as the step can have; ``max_nodes`` is ``parent``'s or
    ``token``'s second size where one is given."""
    num_req, max_pages = page_table.shape
    rows = positions.shape[0]
    of = parent if parent is not None else token
    if of is not None:
        max_nodes = of.shape[1]
    if max_nodes is None:
        raise ValueError("chains without tokens need max_nodes")
    if (token is None) != (row_token is None):
        raise ValueError("token and row_token come together")
    words = 0 if mask is None else mask.shape[1]
    at, of_rows = _at(page_table, "page_table"), (rows,)
    args = [_shape(length, (num_req,), at, "length"), _shape(count, (num_req,), at, "count"),
            _shape(parent, (num_req, max_nodes), at, "parent"), _shape(token, (num_req, max_nodes), at, "token"), num_req,
            max_nodes, _here(page_table, at, _I32T, "page_table"), max_pages, num_pages, rows,
            _shape(req_start, (num_req + 1,), at, "req_start"), _shape(positions, of_rows, at, "positions"),
            _shape(cache_pos, of_rows, at, "cache_pos"), _shape(mask, (rows, words), at, "mask"), words,
            _shape(row_token, of_rows, at, "row_token"), _here(dev_err, at, _I32T, "dev_err"), _on(stream, page_table)]
    _check("ci_draft_plan", lib.ci_draft_plan(*args))


def attn_draft_workspace_bytes(max_rows: int, num_q_heads: int, num_kv_heads: int, head_dim: int) -> int:
    """Of ci_attn_draft.  It goes by ``head_dim`` alone; the others are checked."""
    n = lib.ci_attn_draft_workspace_bytes(max_rows, num_q_heads, num_kv_heads, head_dim)
    if n < 0:
        raise CIError("ci_attn_draft_workspace_bytes", n)
    return n


def ci_attn_draft(q, k_pool, v_pool, page_table, req_start, length, max_len, max_rows, scale, out, mask=None, lse=None,
                  workspace=None, dev_err=None, stream=None):
    """Attention of q [rows, q_heads, head_dim] over each row's request and
    over the nodes of ``mask`` [rows, words] (None: every node up to the row's
    own; see include/ci_draft.h).  ``max_len``: no request's length and nodes
    are more; ``max_rows``: no request has more rows.  ``workspace``: uint8,
    attn_draft_workspace_bytes() of it; allocated here, from the memory of the
    call's stream, if None."""
    qp, q_stride, shape = _heads(q, "q")
    op, out_stride, out_shape = _heads(out, "out")
    if out_shape != shape:
        raise ValueError("out must have q's shape")
    rows, hq, d = shape
    kp, vp, num_pages, hkv, fmt = _pools(k_pool, v_pool, d)
    num_req, max_pages = page_table.shape
    words = 0 if mask is None else mask.shape[1]
    at = _at(q, "q")
    for t, name in ((out, "out"), (k_pool, "k_pool"), (v_pool, "v_pool")):
        if t.get_device() != at:
            raise ValueError(f"{name} must live on the current device")
    mp = _shape(mask, (rows, words), at, "mask")
    if mask is not None and rows and not words:
        raise ValueError("mask needs a word per row")
    starts = _shape(req_start, (num_req + 1,), at, "req_start")
    lens = _shape(length, (num_req,), at, "length")
    if lse is not None and tuple(lse.shape) != (rows, hq):
        raise ValueError(f"lse must be [{rows}, {hq}]")
    if workspace is None:
        workspace = empty_on(stream, (attn_draft_workspace_bytes(max_rows, hq, hkv, d),), _U8, q.device)
    status = lib.ci_attn_draft(
        qp, q_stride, rows, hq, hkv, d, scale, kp, vp, num_pages, fmt, _here(page_table, at, _I32T, "page_table"), num_req,
        max_pages, starts, lens, max_len, max_rows, mp, words, op, out_stride, _here(lse, at, _F32T, "lse"),
        _here(workspace, at, _U8, "workspace"), workspace.numel(), _here(dev_err, at, _I32T, "dev_err"), _on(stream, q))
    if status:
        _check("ci_attn_draft", status)


def ci_draft_accept(req_start, length, parent, row_token, target, path, accepted, next, new_len, cache_pos=None,
                    dev_err=None, stream=None):
    """The path of every tree that the model agrees with: ``target`` [rows] is
    its choice behind each row (see include/ci_draft.h)."""
    num_req, max_nodes = path.shape
    rows = row_token.shape[0]
    at, of_rows, of_req = _at(path, "path"), (rows,), (num_req,)
    args = [_shape(req_start, (num_req + 1,), at, "req_start"), _shape(length, of_req, at, "length"),
            _shape(parent, (num_req, max_nodes), at, "parent"), num_req, max_nodes, rows,
            _shape(row_token, of_rows, at, "row_token"), _shape(target, of_rows, at, "target"),
            _shape(cache_pos, of_rows, at, "cache_pos"), _here(path, at, _I32T, "path"),
            _shape(accepted, of_req, at, "accepted"), _shape(next, of_req, at, "next"),
            _shape(new_len, of_req, at, "new_len"), _here(dev_err, at, _I32T, "dev_err"), _on(stream, path)]
    _check("ci_draft_accept", lib.ci_draft_accept(*args))


def ci_slots_move(pools, row_bytes, scale_bytes, page_table, length, path, count, dev_err=None, stream=None):
    """Position length + d of every request becomes what length + path[d] was,
    d < count, in every pool (see include/ci_draft.h).  ``pools``: one uint8
    tensor [pools, num_pages, heads, bytes] or a sequence of tensors
    [num_pages, heads, bytes] or [num_pages, bytes]; ``row_bytes`` and
    ``scale_bytes`` of one position and head: a number, or one for each pool."""
    n = len(pools)
    if not 1 <= n <= MAX_POOLS:
        raise ValueError(f"1 to {MAX_POOLS} pools per call")
    rows = array("i", [row_bytes]) * n if isinstance(row_bytes, int) else array("i", row_bytes)
    scales = array("i", [scale_bytes]) * n if isinstance(scale_bytes, int) else array("i", scale_bytes)
    if len(rows) != n or len(scales) != n:
        raise ValueError("row_bytes and scale_bytes: a number, or one for each pool")
    num_req, max_pages = page_table.shape
    if path.dim() != 2 or path.shape[0] != num_req:
        raise ValueError(f"path must be [{num_req}, n]")
    at = _at(path, "path")
    if isinstance(pools, torch.Tensor):
        base, shapes = _here(pools, at, _U8, "pools"), [pools.shape[1:]]
        step = pools.numel() // n
        ptrs = array("Q", range(base, base + n * step, step) if step else [base] * n)
    else:
        shapes = [p.shape for p in pools]
        ptrs = array("Q", [_here(p, at, _U8, "pools") for p in pools])
    num_pages = shapes[0][0]
    heads = array("i")
    for shape, row, scale in {(shape, row, scale): None for shape, row, scale in
                              zip(shapes * (n // len(shapes)), rows, scales)}:
        if len(shape) not in (2, 3) or shape[0] != num_pages or shape[-1] != PAGE * (row + scale):
            raise ValueError(f"a pool must be [{num_pages}, heads, {PAGE * (row + scale)}], got {list(shape)}")
    heads.extend([shape[1] if len(shape) == 3 else 1 for shape in shapes] * (n // len(shapes)))
    _check("ci_slots_move", lib.ci_slots_move(
        ptrs.buffer_info()[0], heads.buffer_info()[0], rows.buffer_info()[0], scales.buffer_info()[0], n, num_pages,
        _here(page_table, at, _I32T, "page_table"), num_req, max_pages, _shape(length, (num_req,), at, "length"),
        _here(path, at, _I32T, "path"), path.shape[1], _shape(count, (num_req,), at, "count"),
        _here(dev_err, at, _I32T, "dev_err"), _on(stream, path)))


def ci_pages_trim(page_table, ref_count, old_len, new_len, dev_err=None, stream=None):
    """The pages behind new_len released, where a request had old_len positions (see include/ci_draft.h)."""
    num_req, max_pages = page_table.shape
    at = _at(page_table, "page_table")
    _check("ci_pages_trim", lib.ci_pages_trim(
        _here(page_table, at, _I32T, "page_table"), num_req, max_pages, _here(ref_count, at, _I32T, "ref_count"),
        ref_count.shape[0], _shape(old_len, (num_req,), at, "old_len"), _shape(new_len, (num_req,), at, "new_len"),
        _here(dev_err, at, _I32T, "dev_err"), _on(stream, page_table)))

"""The drafted step's part of the C ABI: exported symbols, the refusals of the
host-side checks and of the binding (no GPU needed: they run before any CUDA
call), and the oracle's own pins."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from oracle import draft_oracle as D

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ci_draft.h")
OK, NULL, SHAPE, ALIGN, RANGE, UNSUPPORTED = 0, -1, -2, -3, -4, -5
P = 0x1000  # never dereferenced: the host checks fail first


@pytest.fixture(scope="module")
def draft():
    from two_level_sparse_gb300 import build

    if not os.path.exists(os.path.join(ROOT, "two_level_sparse_gb300", "libci.so")):
        build.build()
    from two_level_sparse_gb300 import draft as mod

    return mod


def test_header_binding_and_library_agree(draft):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = re.findall(r"CI_API\s+\w+\s+(ci_\w+)\s*\(([^;]*)\)\s*;", text)
    assert sorted(n for n, _ in declared) == sorted(draft.SIGNATURES)
    for name, args in declared:
        assert len(args.split(",")) == len(draft.SIGNATURES[name]), name
        assert hasattr(ctypes.CDLL(draft.lib._name), name)
    assert f"#define CI_DRAFT_MAX_NODES {draft.MAX_NODES}\n" in open(HEADER).read()


PLAN = dict(length=P, count=P, parent=P, token=P, req=2, nodes=16, pt=P, mp=4, pages=8, rows=32, starts=P, at=P, cp=P,
            mask=P, words=1, rt=P, err=None, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(req=-1), SHAPE), (dict(req=0), RANGE), (dict(req=4097), RANGE), (dict(nodes=0), SHAPE),
    (dict(nodes=257, words=8), RANGE), (dict(nodes=33), SHAPE), (dict(words=0), SHAPE), (dict(words=9), SHAPE),
    (dict(rows=-1), SHAPE), (dict(length=None), NULL), (dict(count=None), NULL), (dict(starts=None), NULL),
    (dict(at=None), NULL), (dict(cp=None), NULL), (dict(pt=None), NULL), (dict(token=None), NULL),
    (dict(rt=None), NULL), (dict(mp=1 << 30), RANGE), (dict(pages=1 << 40), RANGE),
])
def test_plan_refusals(draft, change, want):
    assert draft.lib.ci_draft_plan(*dict(PLAN, **change).values()) == want


ATTN = dict(q=P, q_stride=1024, rows=6, hq=8, hkv=2, d=128, scale=1.0, k=P, v=P, pages=4, fmt=0, pt=P, req=2, mp=2,
            starts=P, length=P, max_len=128, max_rows=4, mask=P, words=1, out=P, out_stride=1024, lse=None, ws=P,
            ws_bytes=1 << 40, err=None, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(rows=0, q=None, k=None), OK),
    (dict(rows=0, max_rows=0, words=0), OK),
    (dict(rows=-1), SHAPE), (dict(max_len=-1), SHAPE), (dict(max_rows=-1), SHAPE), (dict(words=0), SHAPE),
    (dict(fmt=2), UNSUPPORTED), (dict(d=32), UNSUPPORTED), (dict(hq=7), SHAPE), (dict(hkv=0), SHAPE),
    (dict(hq=258), RANGE), (dict(req=0), RANGE), (dict(req=4097), RANGE),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(pt=None), NULL), (dict(length=None), NULL),
    (dict(starts=None), NULL), (dict(ws=None), NULL), (dict(out=None), NULL),
    (dict(pages=0), RANGE), (dict(pages=2 ** 25), RANGE), (dict(max_len=129), SHAPE),
    (dict(q_stride=1016), SHAPE), (dict(out_stride=1028), ALIGN), (dict(q=P + 8), ALIGN), (dict(v=P + 4), ALIGN),
    (dict(ws_bytes=0), SHAPE),
    (dict(rows=1 << 30, max_rows=1 << 30, mp=1 << 24, max_len=1 << 30), RANGE),
])
def test_attn_refusals(draft, change, want):
    assert draft.lib.ci_attn_draft(*dict(ATTN, **change).values()) == want


def test_workspace_refusals(draft):
    f = draft.lib.ci_attn_draft_workspace_bytes
    assert f(4, 64, 8, 128) > 0
    assert f(0, 64, 8, 128) > 0  # a step in which nobody drafts
    assert f(-1, 64, 8, 128) == SHAPE
    assert f(4, 65, 8, 128) == SHAPE
    assert f(4, 129, 1, 128) == RANGE
    assert f(4, 64, 8, 100) == UNSUPPORTED


ACCEPT = dict(starts=P, length=P, parent=P, req=2, nodes=16, rows=32, rt=P, target=P, cp=P, path=P, acc=P, nxt=P, new=P,
              err=None, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(req=0, starts=None), OK), (dict(req=-1), SHAPE), (dict(req=4097), RANGE), (dict(nodes=0), SHAPE),
    (dict(nodes=257), RANGE), (dict(rows=-1), SHAPE), (dict(starts=None), NULL), (dict(length=None), NULL),
    (dict(rt=None), NULL), (dict(target=None), NULL), (dict(path=None), NULL), (dict(acc=None), NULL),
    (dict(nxt=None), NULL), (dict(new=None), NULL),
])
def test_accept_refusals(draft, change, want):
    assert draft.lib.ci_draft_accept(*dict(ACCEPT, **change).values()) == want


def test_move_and_trim_refusals(draft):
    one = (ctypes.c_void_p * 1)
    n = lambda v: (ctypes.c_int32 * 1)(v)  # noqa: E731
    good = dict(pools=one(P), heads=n(2), rows=n(256), scales=n(4), num=1, pages=8, pt=P, req=2, mp=4, length=P, path=P,
                stride=16, count=P, err=None, stream=None)
    for change, want in [
            (dict(req=0, length=None), OK), (dict(req=-1), SHAPE), (dict(req=4097), RANGE), (dict(num=0), RANGE),
            (dict(num=161), RANGE), (dict(stride=0), SHAPE), (dict(stride=257), RANGE), (dict(pools=one(None)), NULL),
            (dict(pools=None), NULL), (dict(pools=one(P + 8)), ALIGN), (dict(rows=n(24)), ALIGN),
            (dict(rows=n(0)), RANGE), (dict(heads=n(0)), RANGE), (dict(scales=n(2)), UNSUPPORTED),
            (dict(length=None), NULL), (dict(path=None), NULL), (dict(count=None), NULL), (dict(pt=None), NULL)]:
        assert draft.lib.ci_slots_move(*dict(good, **change).values()) == want, change
    trim = draft.lib.ci_pages_trim
    assert trim(None, 0, 0, None, 0, None, None, None, None) == OK
    assert trim(P, 2, 4, P, 8, None, P, None, None) == NULL
    assert trim(P, 2, 4, None, 8, P, P, None, None) == NULL
    assert trim(None, 2, 4, P, 8, P, P, None, None) == NULL
    assert trim(P, 5000, 4, P, 8, P, P, None, None) == RANGE
    assert trim(P, -1, 4, P, 8, P, P, None, None) == SHAPE


def test_move_refuses_pools_that_share_bytes(draft):
    page = 2 * 64 * (256 + 4)  # of a pool of two heads
    i32 = ctypes.c_int32
    def status(*starts, pages=8):  # noqa: E306
        n = len(starts)
        return draft.lib.ci_slots_move((ctypes.c_void_p * n)(*starts), (i32 * n)(*[2] * n), (i32 * n)(*[256] * n),
                                       (i32 * n)(*[4] * n), n, pages, P, 0, 4, None, P, 16, None, None, None)

    assert status(P, P + 8 * page, P + 16 * page) == OK
    assert status(P + 16 * page, P, P + 8 * page) == OK
    assert status(P, P) == SHAPE
    assert status(P + 8 * page, P, P + 8 * page) == SHAPE
    assert status(P, P + 8 * page - 16) == SHAPE
    assert status(P + 8 * page - 16, P + 32 * page, P) == SHAPE
    assert status(*[P + 8 * page * i for i in range(160)]) == OK
    assert status(*[P + 8 * page * (i % 159) for i in range(160)]) == SHAPE
    assert status(P, P + 8 * page, pages=2 ** 31 - 1) == SHAPE


def test_binding_refuses_what_it_can_see(draft):
    i32 = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):  # not on the GPU
        draft.ci_pages_trim(i32.view(4, 1), i32, i32, i32)
    with pytest.raises(ValueError):  # a length per request
        draft.ci_pages_trim(i32.view(2, 2), i32, i32, i32)
    with pytest.raises(ValueError):
        draft.ci_slots_move([], 128, 4, i32.view(2, 2), i32, i32.view(2, 2), i32)
    with pytest.raises(ValueError, match="max_nodes"):
        draft.ci_draft_plan(i32, i32, None, i32.view(4, 1), 3, i32, i32, i32)
    with pytest.raises(ValueError, match="together"):
        draft.ci_draft_plan(i32, i32, i32.view(4, 1), i32.view(4, 1), 3, i32, i32, i32, token=i32.view(4, 1))
    with pytest.raises(TypeError):
        draft.ci_attn_draft(torch.zeros(1, 8, 128), None, None, None, None, None, 0, 1, 1.0, None)
    with pytest.raises(draft.CIError) as e:
        draft.attn_draft_workspace_bytes(1, 7, 2, 128)
    assert e.value.status == SHAPE


# ------------------------------------------------------------------ the oracle, by hand
def test_oracle_trees():
    #      0
    #    1   2
    #    3   4 5
    parent = [-1, 0, 0, 1, 2, 2]
    assert D.ancestors(parent) == [{0}, {0, 1}, {0, 2}, {0, 1, 3}, {0, 2, 4}, {0, 2, 5}]
    assert D.ancestors([-1, 1, 0, -2]) == [{0}, None, {0, 2}, None]
    table = np.array([[7, 5], [3, -1]])
    start, at, slot, mask, tok = D.plan([62, 63], [6, 2], [parent, [-1, 0] + [-1] * 4], np.arange(12).reshape(2, 6),
                                        table, 8, 10, 6, 1)
    assert start.tolist() == [0, 6, 8]
    assert at.tolist() == [62, 63, 63, 64, 64, 64, 63, 64, 0, 0]
    assert slot.tolist() == [62, 63, 64, 65, 66, 67, 63, -1, -1, -1]  # the second request has one page
    assert mask[:, 0].tolist() == [1, 3, 5, 11, 21, 37, 1, 3, 0, 0]
    assert tok.tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 0, 0]
    assert D.sees(2, 6, 4, mask[4], 8, table[0]) == [0, 1, 2, 4, 6]
    assert D.sees(2, 6, 2, None, 8, table[0]) == [0, 1, 2, 3, 4]


def test_oracle_path_and_moves():
    parent = [[-1, 0, 0, 1, 2, 2]]
    token, target = [9, 4, 5, 1, 6, 6], [5, 0, 6, 0, 8, 0]  # 0 -> 2 (5), 2 -> 4 (the lower 6)
    path, n, after, new = D.accept([0, 6], [62], parent, token, target, None, 6)
    assert path[0].tolist() == [0, 2, 4, -1, -1, -1] and (n, after, new) == ([3], [8], [65])
    path, n, after, new = D.accept([0, 6], [62], parent, token, target, [1, 1, -1, 1, 1, 1], 6)
    assert (n, after, new) == ([1], [5], [63])
    pool = np.zeros((3, 1, 64 * 2), np.uint8)
    table = np.array([[2, 0]])
    for i in range(6):  # node i holds 10 + i at position 62 + i
        pool[table[0, (62 + i) // 64], 0, 2 * ((62 + i) % 64):][:2] = 10 + i
    out = D.move(pool, 2, 0, table, [62], [[0, 2, 4]], [3])
    assert [int(out[table[0, s // 64], 0, 2 * (s % 64)]) for s in (62, 63, 64, 65)] == [10, 12, 14, 13]
    t, ref = D.trim(np.array([[2, 0, 1]]), np.array([1, 1, 2]), [190], [64])
    assert t.tolist() == [[2, -1, -1]] and ref.tolist() == [0, 0, 2]


def test_workspace_goes_by_the_head_size(draft):
    """Two blocks (of 256 rows; 128 with D = 256) of sums and two statistics per SM, whatever the rows and heads."""
    n = draft.attn_draft_workspace_bytes
    for d, rows in ((64, 256), (128, 256), (256, 128)):
        got = {n(m, hq, hkv, d) for m in (0, 1, 77, 10 ** 6) for hq, hkv in ((1, 1), (64, 8), (128, 1))}
        assert len(got) == 1
        block = 2 * rows * (d + 2) * 4
        sms = got.pop() // block
        assert 0 <= n(1, 8, 8, d) - sms * block <= 16 * sms + 16

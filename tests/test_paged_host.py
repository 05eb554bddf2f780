"""PagedCache's bookkeeping without a GPU: the page calls are replaced by plain
statements of their contract over host tensors."""
import os

import numpy as np
import pytest
import torch

from oracle import cache_oracle as C

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def i32(*v):
    return torch.tensor(v, dtype=torch.int32)


@pytest.fixture
def make(monkeypatch):
    from two_level_sparse_gb300 import build

    if not os.path.exists(os.path.join(ROOT, "two_level_sparse_gb300", "libci.so")):
        build.build()
    from two_level_sparse_gb300 import paged

    ops = paged.ops

    def pages(table, ref):
        return C.Pages(table.numpy(), ref.numpy(), np.zeros((0, 0)))

    def put(o, table, ref):
        table.copy_(torch.from_numpy(o.table)), ref.copy_(torch.from_numpy(o.ref))

    def ok_len(table, n):
        return 0 <= n <= 64 * table.shape[1]

    def alloc(table, ref, old, new, dev_err):
        o, pairs = pages(table, ref), []
        for a, b in zip(old.tolist(), new.tolist()):
            good = ok_len(table, a) and ok_len(table, b) and a <= b
            dev_err |= 0 if good else ops.DEVERR_LEN
            pairs.append((a, b) if good else (0, 0))
        before = (o.table < 0).sum()
        o.alloc(*zip(*pairs))
        asked = sum(-(-b // 64) - -(-a // 64) for a, b in pairs)
        dev_err |= ops.DEVERR_PAGE if before - (o.table < 0).sum() < asked else 0
        put(o, table, ref)

    def free(table, ref, req, dev_err):
        o = pages(table, ref)
        for r in req.tolist():
            if 0 <= r < len(o.table):
                o.free([r])
            else:
                dev_err |= ops.DEVERR_REQ
        put(o, table, ref)

    def fork(table, ref, parent, child, length, src, dst, dev_err):
        o, do = pages(table, ref), []
        for i, (p, c, n) in enumerate(zip(parent.tolist(), child.tolist(), length.tolist())):
            src[i] = dst[i] = -1
            if not (0 <= p < len(o.table) and 0 <= c < len(o.table) and p != c):
                dev_err |= ops.DEVERR_REQ
            elif not ok_len(table, n):
                dev_err |= ops.DEVERR_LEN
            else:
                do.append((i, p, c, n))
        if do:
            s, d = o.fork(*zip(*[x[1:] for x in do]))
            for (i, _, _, n), a, b in zip(do, s, d):
                src[i], dst[i] = int(a), int(b)
                dev_err |= ops.DEVERR_PAGE if n % 64 and b < 0 else 0
        put(o, table, ref)

    monkeypatch.setattr(ops, "ci_pages_alloc", alloc)
    monkeypatch.setattr(ops, "ci_pages_free", free)
    monkeypatch.setattr(ops, "ci_pages_fork", fork)
    monkeypatch.setattr(ops, "ci_pages_copy", lambda *a, **k: None)
    return lambda requests=4, max_pages=4, num_pages=12: paged.PagedCache(1, requests, max_pages, num_pages, 1, 64,
                                                                          device="cpu")


def consistent(c):
    """Every reference is an entry of the table, and every length has its pages."""
    entries = c.page_table[c.page_table >= 0].long()
    assert torch.equal(torch.bincount(entries, minlength=len(c.ref_count)), c.ref_count.long())
    for row, n in zip(c.page_table.tolist(), c.length.tolist()):
        assert all(p >= 0 for p in row[:-(-n // 64)]) and all(p < 0 for p in row[-(-n // 64):])


@pytest.mark.parametrize("req", [[-1], [4], [-4, 2 ** 31 - 1], [4, 1, -1]])
def test_free_of_requests_that_are_not_there(make, req):
    from two_level_sparse_gb300.cache import DEVERR_REQ

    c = make()
    c.grow(i32(100, 64, 0, 130))
    c.free(i32(*req))
    want = [100, 64, 0, 130]
    for r in req:
        if 0 <= r < 4:
            want[r] = 0
    assert c.length.tolist() == want and int(c.dev_err) == DEVERR_REQ
    consistent(c)


@pytest.mark.parametrize("parent,child,length,err", [
    ([0], [4], [100], "REQ"), ([0], [-1], [100], "REQ"), ([4], [1], [100], "REQ"), ([-1], [1], [64], "REQ"),
    ([0], [0], [100], "REQ"), ([0], [1], [257], "LEN"), ([0], [1], [-1], "LEN"),
    ([0, 3, 0], [4, 1, 2], [100, 130, 70], "REQ")])
def test_fork_that_is_refused_changes_nothing(make, parent, child, length, err):
    from two_level_sparse_gb300 import cache as ops

    c = make()
    lens = [100, 64, 0, 130]
    c.grow(i32(*lens))
    table = c.page_table.clone()
    c.fork(i32(*parent), i32(*child), i32(*length))
    assert int(c.dev_err) == getattr(ops, "DEVERR_" + err)
    if len(parent) == 1:
        assert c.length.tolist() == lens and torch.equal(c.page_table, table)
    else:  # the forks beside it are carried out
        assert c.length.tolist() == [100, 130, 70, 130] and c.page_table[1, :2].tolist() == table[3, :2].tolist()
    consistent(c)


def test_growth_that_runs_out_goes_as_far_as_the_pages(make):
    from two_level_sparse_gb300 import cache as ops

    c = make(num_pages=5)
    c.grow(i32(100, 70, 200, 1))
    assert c.length.tolist() == [100, 70, 64, 0] and c.short.tolist() == [0, 0, 1, 1]
    assert int(c.dev_err) == ops.DEVERR_PAGE
    consistent(c)
    c.free(i32(0))
    c.grow(i32(0, 70, 200, 1))  # what was short is asked for again
    assert c.length.tolist() == [0, 70, 192, 0] and c.short.tolist() == [0, 0, 1, 1]
    consistent(c)
    c.free(i32(1))
    assert c.short.tolist() == [0, 0, 1, 1]
    c.free(i32(2, 3))
    assert c.short.tolist() == [0] * 4 and c.length.tolist() == [0] * 4
    c.grow(i32(0, 128, 0, 192))
    assert c.length.tolist() == [0, 128, 0, 192] and c.short.tolist() == [0] * 4
    consistent(c)


def test_growth_that_is_refused_changes_nothing(make):
    from two_level_sparse_gb300 import cache as ops

    c = make()
    c.grow(i32(100, 64, 5, 0))
    c.grow(i32(99, 257, -1, 130))
    assert c.length.tolist() == [100, 64, 5, 130] and c.short.tolist() == [1, 1, 1, 0]
    assert int(c.dev_err) == ops.DEVERR_LEN
    consistent(c)
    c.grow(i32(101, 65, 5, 130))
    assert c.length.tolist() == [101, 65, 5, 130] and c.short.tolist() == [0] * 4
    consistent(c)


def test_fork_without_a_page_for_its_end(make):
    from two_level_sparse_gb300 import cache as ops

    c = make(num_pages=5)
    c.grow(i32(100, 0, 65, 0))
    c.fork(i32(0, 2), i32(1, 3), i32(100, 65))
    assert c.length.tolist() == [100, 100, 65, 64] and c.short.tolist() == [0, 0, 0, 1]
    assert int(c.dev_err) == ops.DEVERR_PAGE
    consistent(c)
    c.fork(i32(2), i32(1), i32(65))  # the page that the child before it had
    assert c.length.tolist() == [100, 65, 65, 64] and c.short.tolist() == [0, 0, 0, 1]
    consistent(c)


def test_a_step_writes_no_token_that_has_no_place(make, monkeypatch):
    """Where a request's growth was cut, its last position is an older token's: it stays as it is."""
    from types import SimpleNamespace

    from two_level_sparse_gb300 import paged

    c = make(num_pages=3)
    c.grow(i32(64, 63, 0, 64))
    c.grow(i32(65, 64, 0, 65))
    assert c.length.tolist() == [64, 64, 0, 64] and c.short.tolist() == [1, 0, 0, 1]
    seen = []
    monkeypatch.setattr(paged.ops, "ci_qk_norm_rope_append",
                        lambda *a, cache_pos, **k: seen.append((a[8].tolist(), cache_pos.tolist())))
    monkeypatch.setattr(paged.PagedCache, "attend", lambda self, j, q, *a, **k: q)
    step = SimpleNamespace(run=lambda: None, max_len=256, pos=[None])
    paged.sparse_decode_step(c, step, [torch.zeros(4, 6, 64)], None, None, 1e-6, None)
    assert seen == [([63, 63, 0, 63], [-1, 63, -1, -1])]

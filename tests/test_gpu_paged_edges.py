"""PagedCache where calls are refused or pages run out, on the device (without
one: test_paged_host.py)."""
import pytest
import torch

from test_gpu_cache import i32

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def make(requests=4, max_pages=4, num_pages=12):
    from two_level_sparse_gb300.paged import PagedCache

    return PagedCache(1, requests, max_pages, num_pages, 1, 64)


def test_requests_that_are_not_there():
    from two_level_sparse_gb300 import cache as ops

    c = make()
    c.grow(i32([100, 64, 0, 130]))
    table = c.page_table.clone()
    c.free(i32([4, -1]))
    c.fork(i32([0, 4, 0, 0]), i32([5, 1, 0, -2]), i32([100, 64, 100, 64]))
    assert c.length.tolist() == [100, 64, 0, 130] and torch.equal(c.page_table, table)
    assert int(c.dev_err) == ops.DEVERR_REQ
    c.dev_err.zero_()
    c.fork(i32([0, 3]), i32([1, 2]), i32([257, 70]))
    assert c.length.tolist() == [100, 64, 70, 130] and int(c.dev_err) == ops.DEVERR_LEN
    assert c.ref_count.sum() == (c.page_table >= 0).sum()


def test_pages_run_out_and_come_back():
    from two_level_sparse_gb300 import cache as ops

    c = make(num_pages=5)
    c.grow(i32([100, 70, 200, 1]))
    assert c.length.tolist() == [100, 70, 64, 0] and c.short.tolist() == [0, 0, 1, 1]
    assert int(c.dev_err) == ops.DEVERR_PAGE
    c.free(i32([0]))
    c.grow(i32([0, 70, 200, 1]))
    assert c.length.tolist() == [0, 70, 192, 0] and c.short.tolist() == [0, 0, 1, 1]
    assert c.ref_count.tolist() == [1] * 5 and (c.page_table[2] >= 0).sum() == 3
    c.dev_err.zero_()
    c.grow(i32([0, 69, 257, 0]))
    assert c.length.tolist() == [0, 70, 192, 0] and c.short.tolist() == [0, 1, 1, 0]
    assert int(c.dev_err) == ops.DEVERR_LEN
    c.free(i32([2]))
    c.dev_err.zero_()
    c.grow(i32([100, 70, 0, 0]))
    c.fork(i32([0, 1]), i32([2, 3]), i32([100, 70]))  # one page for two ends
    assert c.length.tolist() == [100, 70, 100, 64] and c.short.tolist() == [0, 0, 0, 1]
    assert int(c.dev_err) == ops.DEVERR_PAGE and c.ref_count.sum() == (c.page_table >= 0).sum()


def test_a_step_writes_no_token_that_has_no_place():
    """A request whose growth was cut keeps its last position's key and value; the others' tokens are stored."""
    from types import SimpleNamespace

    from two_level_sparse_gb300.paged import sparse_decode_step

    c = make(num_pages=3)
    c.grow(i32([64, 63, 0, 64]))
    c.k.fill_(0x22), c.v.fill_(0x33)
    c.grow(i32([65, 64, 0, 65]))
    pos = torch.zeros(1, 4, 8, dtype=torch.int32, device="cuda")
    step = SimpleNamespace(run=lambda: None, max_len=256, pos=pos)
    x = torch.randn(4, 6, 64, device="cuda").bfloat16()
    ones, cs = torch.ones(64, device="cuda"), torch.ones(256, 64, device="cuda")
    sparse_decode_step(c, step, [x], ones, ones, 1e-6, cs)
    row, page = 128, int(c.page_table[1, 0])
    for pool, byte in ((c.k, 0x22), (c.v, 0x33)):
        new = pool[0, page, 0, 63 * row:].clone()
        assert (new != byte).any()
        pool[0, page, 0, 63 * row:] = byte
        assert (pool == byte).all()

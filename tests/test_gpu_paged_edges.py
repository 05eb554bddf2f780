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

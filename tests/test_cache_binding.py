"""The cache's binding without a GPU: what it hands to the library and which
stream's memory it takes, with the library and the streams replaced."""
import contextlib
import ctypes
import os
from types import SimpleNamespace

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Device(torch.Tensor):
    """A host tensor that says it lives on the GPU."""

    is_cuda = property(lambda self: True)


def dev(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Device)


@pytest.fixture
def cache(monkeypatch):
    from two_level_sparse_gb300 import build

    if not os.path.exists(os.path.join(ROOT, "two_level_sparse_gb300", "libci.so")):
        build.build()
    from two_level_sparse_gb300 import cache as mod

    calls = []

    def entry(name):
        return lambda *a: calls.append((name, a)) or 0

    lib = SimpleNamespace(**{n: entry(n) for n in mod.SIGNATURES if n.startswith(("ci_attn_d", "ci_qk", "ci_pages"))},
                          ci_attn_workspace_bytes=mod.lib.ci_attn_workspace_bytes,
                          ci_cache_page_bytes=mod.lib.ci_cache_page_bytes)
    monkeypatch.setattr(mod, "lib", lib)
    monkeypatch.setattr(mod, "_current_stream", lambda device: 0)
    return SimpleNamespace(mod=mod, calls=calls)


@pytest.fixture
def pools_asked(monkeypatch):
    """(shape, stream) of every torch.empty: the stream whose memory it comes from, None for the current one."""
    asked, on = [], [None]
    empty = torch.empty

    @contextlib.contextmanager
    def stream(s):
        on.append(s)
        yield
        on.pop()

    def recorded(*shape, **kw):
        asked.append((tuple(shape[0]) if len(shape) == 1 and not isinstance(shape[0], int) else shape, on[-1]))
        return empty(*shape, **kw).as_subclass(Device)

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(torch, "empty", recorded)
    return asked


SIDE = SimpleNamespace(cuda_stream=77)


@pytest.mark.parametrize("stream", [None, SIDE])
def test_workspace_comes_from_the_calls_stream(cache, pools_asked, stream):
    q, pool = dev(2, 8, 64, dtype=torch.bfloat16), dev(4, 2, 8192, dtype=torch.uint8)
    cache.mod.ci_attn_decode(q, pool, pool, dev(2, 2), 0, dev(2), 128, 1.0, q, stream=stream)
    n = cache.mod.attn_workspace_bytes(2, 8, 2, 64)
    assert pools_asked == [((n,), stream)]
    assert cache.calls[-1][1][-1] == (77 if stream else 0)


def host_cache(*args):
    """A PagedCache of host tensors that say they live on the GPU."""
    from two_level_sparse_gb300.paged import PagedCache

    c = PagedCache(*args, device="cpu")
    for t in ("k", "v", "page_table", "ref_count", "dev_err"):
        setattr(c, t, getattr(c, t).as_subclass(Device))
    return c


@pytest.mark.parametrize("stream", [None, SIDE])
def test_cache_results_come_from_the_calls_stream(cache, pools_asked, stream):
    c = host_cache(1, 2, 2, 4, 2, 64)
    q, kv = dev(2, 8, 64, dtype=torch.bfloat16), dev(2, 2, 64, dtype=torch.bfloat16)
    pools_asked.clear()
    c.append(0, q, kv, kv, None, None, 1e-6, dev(4, 0, dtype=torch.float32), True, dev(2), 0, stream=stream)
    c.attend(0, q, 0, dev(2), stream=stream)
    assert [name for name, _ in cache.calls] == ["ci_qk_norm_rope_append", "ci_attn_decode"]
    assert len(pools_asked) == 3 and all(on is stream for _, on in pools_asked)


def pool_args(call):
    """Pointers, bytes per page and number of pages that ci_pages_copy was called with."""
    ptrs, sizes, n, pages = call[1][:4]
    return ((ctypes.c_uint64 * n).from_address(ptrs)[:], (ctypes.c_int64 * n).from_address(sizes)[:], pages)


@pytest.mark.parametrize("view", ["whole", "every fourth of four", "one of two", "turned", "expanded", "wide pages"])
def test_copy_takes_pages_as_they_are(cache, view, monkeypatch):
    """A tensor of one pool is contiguous whatever its first stride says."""
    x = {"whole": lambda: dev(4, 3, 64, dtype=torch.uint8),
         "every fourth of four": lambda: dev(4, 3, 64, dtype=torch.uint8)[3::4],
         "one of two": lambda: dev(2, 3, 64, dtype=torch.uint8)[::2],
         "turned": lambda: dev(4, 1, 256, dtype=torch.uint8).transpose(0, 1),
         "expanded": lambda: dev(3, 64, dtype=torch.uint8).as_strided((1, 3, 64), (0, 64, 1)),
         "wide pages": lambda: dev(5, 3, 2, 32, dtype=torch.uint8)}[view]()
    assert x.is_contiguous()
    seen = []
    monkeypatch.setattr(cache.mod.lib, "ci_pages_copy", lambda *a: seen.append(pool_args((None, a))) or 0)
    cache.mod.ci_pages_copy(x, dev(2), dev(2))
    a_pool = x[0].numel()
    cache.mod.ci_pages_copy(list(x), dev(2), dev(2))
    assert seen[0] == ([x.data_ptr() + i * a_pool for i in range(len(x))], [a_pool // x.shape[1]] * len(x), x.shape[1])
    assert seen[1] == seen[0]


def test_workspaces_do_not_grow_with_the_calls(cache, pools_asked):
    """One workspace per stream and number of heads, whatever the rows."""
    c = host_cache(1, 2, 2, 4, 2, 64)

    def taken(rows, heads, stream=None):
        q = dev(rows, heads, 64, dtype=torch.bfloat16)
        pools_asked.clear()
        c.attend(0, q, 1, dev(rows), out=q, stream=stream)
        return len(pools_asked)

    assert taken(2, 8) == 1
    assert [taken(n, 8) for n in (1, 3, 1000, 2)] == [0] * 4
    assert taken(5, 16) == 1 and taken(6, 16) == 0
    assert taken(5, 8, SIDE) == 1 and taken(7, 8, SIDE) == 0
    n = cache.mod.attn_workspace_bytes
    assert all(n(rows, 8, 2, 64) == n(1, 8, 2, 64) for rows in (0, 2, 77, 10 ** 6))


@pytest.mark.parametrize("hkv", [1, 8])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_workspace_goes_by_the_heads(cache, d, hkv):
    """A worker keeps sums and statistics of a unit's heads, padded to 8, 16, 32 or 64, twice: no call needs more."""
    n = {group: cache.mod.attn_workspace_bytes(3, group * hkv, hkv, d) for group in (1, 8, 9, 16, 17, 32, 33, 64, 65, 128)}
    part = 2 * (1 if d == 256 else 2) * (d + 2) * 4  # bytes per SM and head
    sms = n[128] // (64 * part)
    for group, got in n.items():
        heads = next((h for h in (8, 16, 32) if group <= h), 64)
        if d == 128 and 16 < group <= 32:
            heads = 64  # lists of positions take the kernel of many heads
        assert 0 <= got - heads * part * sms <= 32 * sms + 16, group

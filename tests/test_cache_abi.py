"""The cache's part of the C ABI: exported symbols, sizes, and the refusals of
the host-side checks (no GPU needed: they run before any CUDA call)."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "ci_cache.h")
OK, NULL, SHAPE, ALIGN, RANGE, UNSUPPORTED = 0, -1, -2, -3, -4, -5
P = 0x1000  # never dereferenced: the host checks fail first


@pytest.fixture(scope="module")
def cache():
    from two_level_sparse_gb300 import build

    if not os.path.exists(os.path.join(ROOT, "two_level_sparse_gb300", "libci.so")):
        build.build()
    from two_level_sparse_gb300 import cache as mod

    return mod


def test_header_binding_and_library_agree(cache):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = re.findall(r"CI_API\s+\w+\s+(ci_\w+)\s*\(([^;]*)\)\s*;", text)
    assert sorted(n for n, _ in declared) == sorted(cache.SIGNATURES)
    for name, args in declared:
        assert len(args.split(",")) == len(cache.SIGNATURES[name]), name
        assert hasattr(ctypes.CDLL(cache.lib._name), name)


@pytest.mark.parametrize("fmt,d,want", [(0, 64, 8192), (0, 128, 16384), (0, 256, 32768), (1, 64, 4352),
                                        (1, 128, 8448), (1, 256, 16640), (0, 96, UNSUPPORTED), (2, 128, UNSUPPORTED)])
def test_page_bytes(cache, fmt, d, want):
    assert cache.lib.ci_cache_page_bytes(fmt, d) == want


def test_workspace_refusals(cache):
    f = cache.lib.ci_attn_workspace_bytes
    assert f(4, 64, 8, 128) > 0
    assert f(-1, 64, 8, 128) == SHAPE
    assert f(4, 65, 8, 128) == SHAPE
    assert f(4, 129, 1, 128) == RANGE
    assert f(4, 64, 8, 100) == UNSUPPORTED


ATTN = dict(q=P, q_stride=1024, rows=2, hq=8, hkv=2, d=128, scale=1.0, k=P, v=P, pages=4, fmt=0, pt=P, req=2, mp=2,
            layout=0, starts=None, seq=P, max_len=128, pos=None, pos_stride=0, npos=0, out=P, out_stride=1024, lse=None,
            ws=P, ws_bytes=1 << 40, err=None, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(rows=0, q=None, k=None), OK),
    (dict(rows=-1), SHAPE), (dict(max_len=-1), SHAPE),
    (dict(layout=3), UNSUPPORTED), (dict(fmt=2), UNSUPPORTED), (dict(d=32), UNSUPPORTED),
    (dict(hq=7), SHAPE), (dict(hkv=0), SHAPE), (dict(hq=258), RANGE),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(pt=None), NULL), (dict(seq=None), NULL), (dict(ws=None), NULL),
    (dict(req=3), SHAPE), (dict(layout=1), SHAPE), (dict(layout=2), NULL), (dict(layout=2, starts=P, req=5000), RANGE),
    (dict(pages=0), RANGE), (dict(pages=2 ** 25), RANGE),
    (dict(max_len=129), SHAPE), (dict(pos=P, pos_stride=3, npos=4), SHAPE), (dict(pos=P, npos=-1), SHAPE),
    (dict(q_stride=1016), SHAPE), (dict(out_stride=1028), ALIGN), (dict(q=P + 8), ALIGN), (dict(v=P + 4), ALIGN),
    (dict(ws_bytes=0), SHAPE),
])
def test_attn_refusals(cache, change, want):
    assert cache.lib.ci_attn_decode(*dict(ATTN, **change).values()) == want


APPEND = dict(q=P, qs=1024, k=P, ks=256, v=P, vs=256, tokens=2, hq=8, hkv=2, d=128, qn=P, kn=P, eps=1e-6, cs=P,
              max_pos=10, rot=128, neox=1, at=P, cp=None, qo=P, qos=1024, kp=P, vp=P, pages=4, fmt=0, pt=P, req=2,
              mp=2, layout=0, starts=None, err=None, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(tokens=0, q=None), OK), (dict(tokens=-1), SHAPE), (dict(max_pos=-1), SHAPE),
    (dict(rot=8), UNSUPPORTED), (dict(rot=144), UNSUPPORTED), (dict(rot=-16), UNSUPPORTED), (dict(d=80), UNSUPPORTED),
    (dict(fmt=5), UNSUPPORTED), (dict(layout=-1), UNSUPPORTED), (dict(hq=9), SHAPE),
    (dict(q=None), NULL), (dict(v=None), NULL), (dict(at=None), NULL), (dict(cs=None), NULL), (dict(vp=None), NULL),
    (dict(req=1), SHAPE), (dict(ks=248), SHAPE), (dict(qs=1028), ALIGN), (dict(k=P + 2), ALIGN),
    (dict(qn=P + 4), ALIGN), (dict(pages=1 << 31), RANGE),
])
def test_append_refusals(cache, change, want):
    assert cache.lib.ci_qk_norm_rope_append(*dict(APPEND, **change).values()) == want


def test_pages_refusals(cache):
    lib = cache.lib
    assert lib.ci_pages_alloc(None, 0, 0, None, 0, None, None, None, None) == OK
    assert lib.ci_pages_alloc(P, 2, 4, P, 8, None, P, None, None) == NULL
    assert lib.ci_pages_alloc(P, 5000, 4, P, 8, P, P, None, None) == RANGE
    assert lib.ci_pages_alloc(P, 2, 4, P + 4, 8, P, P, None, None) == ALIGN
    assert lib.ci_pages_alloc(P, -1, 4, P, 8, P, P, None, None) == SHAPE
    assert lib.ci_pages_fork(P, 2, 4, P, 8, P, P, P, 0, None, None, None, None) == OK
    assert lib.ci_pages_fork(P, 2, 4, P, 8, P, P, P, 1, None, P, None, None) == NULL
    assert lib.ci_pages_fork(P, 2, 4, P, 8, P, P, P, 4097, P, P, None, None) == RANGE
    assert lib.ci_pages_fork(P, 2, 4, None, 8, P, P, P, 1, P, P, None, None) == NULL
    assert lib.ci_pages_free(P, 2, 4, P, 8, P, 0, None, None) == OK
    assert lib.ci_pages_free(P, 2, 4, P, 8, None, 1, None, None) == NULL
    assert lib.ci_pages_free(P, 2, 4, P, 8, P, -1, None, None) == SHAPE
    assert lib.ci_pages_compact(P, 2, 4, P, 8, P, P, P, None, None, None) == NULL
    assert lib.ci_pages_compact(P, 2, 4, P, 8, None, P, P, P, None, None) == NULL
    assert lib.ci_pages_compact(P, 2, 1 << 30, P, 8, P, P, P, P, None, None) == RANGE
    one, size = (ctypes.c_void_p * 1)(P), lambda n: (ctypes.c_int64 * 1)(n)
    assert lib.ci_pages_copy(one, size(16), 1, 8, P, P, 0, None, None, None) == OK
    assert lib.ci_pages_copy(one, size(16), 0, 8, P, P, 1, None, None, None) == RANGE
    assert lib.ci_pages_copy(one, size(24), 1, 8, P, P, 1, None, None, None) == ALIGN
    assert lib.ci_pages_copy(one, size(0), 1, 8, P, P, 1, None, None, None) == RANGE
    assert lib.ci_pages_copy(one, size(16), 1, 8, None, P, 1, None, None, None) == NULL
    assert lib.ci_pages_copy((ctypes.c_void_p * 1)(P + 8), size(16), 1, 8, P, P, 1, None, None, None) == ALIGN
    assert lib.ci_pages_copy((ctypes.c_void_p * 1)(None), size(16), 1, 8, P, P, 1, None, None, None) == NULL


def test_binding_refuses_what_it_can_see(cache):
    i32 = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):  # not on the GPU
        cache.ci_pages_free(i32.view(2, 2), i32, i32)
    with pytest.raises(TypeError):
        cache.ci_pages_free(i32.view(2, 2).float(), i32, i32)
    with pytest.raises(ValueError):
        cache.ci_pages_copy([], i32, i32)
    with pytest.raises(ValueError):
        cache.cache_format(torch.zeros(2, 1, 100, dtype=torch.uint8), 128)
    with pytest.raises(TypeError):
        cache.ci_attn_decode(torch.zeros(1, 8, 128), None, None, None, 0, None, 0, 1.0, None)
    with pytest.raises(cache.CIError) as e:
        cache.attn_workspace_bytes(1, 7, 2, 128)
    assert e.value.status == SHAPE

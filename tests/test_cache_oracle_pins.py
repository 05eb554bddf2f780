"""Pins of the cache oracle: closed forms, invariants, torch's own decoders."""
import math

import numpy as np
import pytest
import torch

from oracle import cache_oracle as C


def test_decoders_match_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(C.e4m3_values(), want)
    bits = torch.arange(0, 1 << 16, 7, dtype=torch.int32).to(torch.uint16)
    want = bits.view(torch.bfloat16).double().numpy()
    np.testing.assert_array_equal(C.bf16_values(bits.numpy()), want)


def test_page_values_layouts():
    x = torch.randn(3, 2, 64, 128).to(torch.bfloat16)
    pool = x.view(torch.uint8).reshape(3, 2, -1).numpy()
    np.testing.assert_array_equal(C.page_values(pool, 128), x.double().numpy())
    f = torch.randn(3, 2, 64, 128).to(torch.float8_e4m3fn)
    s = torch.rand(3, 2, 64)
    pool = torch.cat([f.view(torch.uint8).reshape(3, 2, -1), s.view(torch.uint8).reshape(3, 2, -1)], -1).numpy()
    np.testing.assert_allclose(C.page_values(pool, 128), f.double().numpy() * s.double().numpy()[..., None])


def test_attention_closed_forms():
    rng = np.random.default_rng(0)
    v = rng.normal(size=(9, 2, 8))
    # equal keys: the mean of the values, and lse = logit + ln n
    k = np.ones((9, 2, 8))
    q = rng.normal(size=(4, 8))
    out, lse, _, size = C.attention(q, k, v, 0.5)
    for h in range(4):
        np.testing.assert_allclose(out[h], v[:, h // 2].mean(0), atol=1e-12)
        np.testing.assert_allclose(lse[h], 0.5 * q[h].sum() + math.log(9))
        np.testing.assert_allclose(size[h], 0.5 * np.abs(q[h]).sum())
    # one key far above the rest: its value
    k[4] = 1000.0
    out, _, _, _ = C.attention(np.ones((4, 8)), k, v, 1.0)
    np.testing.assert_allclose(out[3], v[4, 1])
    out, lse, _, _ = C.attention(q, k[:0], v[:0], 1.0)
    assert (out == 0).all() and (lse == -np.inf).all()


def test_row_positions():
    assert C.row_positions(3, 10) == [0, 1, 2]
    assert C.row_positions(11, 10) == [] and C.row_positions(-1, 10) == []
    assert C.row_positions(5, 10, [0, 4, 4, 5, -1, 2]) == [0, 4, 4, 2]


@pytest.mark.parametrize("neox", [True, False])
def test_norm_rope_is_a_complex_product(neox):
    rng = np.random.default_rng(1)
    x, w, ang = rng.normal(size=16), rng.normal(size=16), rng.normal(size=4)
    got = C.norm_rope(x, w, 1e-3, np.cos(ang), np.sin(ang), neox)
    y = x * w / np.sqrt((x @ x) / 16 + 1e-3)
    z = (y[:4] + 1j * y[4:8] if neox else y[0:8:2] + 1j * y[1:8:2]) * np.exp(1j * ang)
    np.testing.assert_allclose(got[:4] + 1j * got[4:8] if neox else got[0:8:2] + 1j * got[1:8:2], z)
    np.testing.assert_allclose(got[8:], y[8:])
    np.testing.assert_allclose(C.norm_rope(x, None, 1e-3, [], [], neox), x)


def test_pages_keep_every_requests_contents():
    """What a request's positions hold does not change by forking, freeing others and compacting."""
    rng = np.random.default_rng(2)
    table = np.full((6, 4), -1)
    data = rng.integers(0, 1 << 30, size=(2, 20, 64))
    p = C.Pages(table, np.zeros(20, dtype=np.int64), data)
    p.alloc([0, 0, 0, 0, 0, 0], [200, 64, 130, 0, 0, 0])
    assert p.table[0].tolist() == [0, 1, 2, 3] and p.table[1].tolist() == [4, -1, -1, -1]

    def read(r, n):
        return np.concatenate([p.data[:, p.table[r, j]] for j in range(-(-n // 64))], axis=1)[:, :n]

    before = read(0, 200), read(2, 130)
    src, dst = p.fork([0, 0, 2], [3, 4, 5], [200, 64, 130])
    p.copy(src, dst)
    assert dst[1] == -1 and p.ref[0] == 3 and p.ref[3] == 1
    np.testing.assert_array_equal(read(3, 200), before[0])
    np.testing.assert_array_equal(read(4, 64), before[0][:, :64])
    p.free([1, 0])
    movers, holes, _ = p.compact()
    p.copy(movers, holes)
    n = int((p.ref > 0).sum())
    assert (p.ref[:n] > 0).all() and (p.ref[n:] == 0).all()
    np.testing.assert_array_equal(read(3, 200), before[0])
    np.testing.assert_array_equal(read(2, 130), before[1])
    np.testing.assert_array_equal(read(5, 130), before[1])
    np.testing.assert_array_equal(np.bincount(p.table[p.table >= 0], minlength=20), p.ref)

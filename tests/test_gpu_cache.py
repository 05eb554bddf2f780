"""The paged cache's kernels against the float64 oracle.

Tolerances follow from the formats.  bf16 rounds with a relative error of at
most 2^-8, e4m3 of at most 2^-4 (or half its subnormal spacing, 2^-10); fp32
sums of n terms err by at most n 2^-23 of the sum of magnitudes.
"""
import math

import numpy as np
import pytest
import torch

from oracle import cache_oracle as C

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
DEC, PRE, VAR = 0, 1, 2
BF16, FP8 = 0, 1


@pytest.fixture(scope="module")
def cache():
    from two_level_sparse_gb300 import cache as mod

    return mod


def make_pool(gen, pages, hkv, d, fmt):
    x = torch.randn(pages, hkv, 64, d, generator=gen)
    if fmt == BF16:
        return x.to(torch.bfloat16).view(torch.uint8).reshape(pages, hkv, -1)
    s = torch.rand(pages, hkv, 64, generator=gen) * 1.5 + 0.1
    return torch.cat([x.to(torch.float8_e4m3fn).view(torch.uint8).reshape(pages, hkv, -1),
                      s.view(torch.uint8).reshape(pages, hkv, -1)], -1).contiguous()


def make_table(gen, lens, spare=3):
    pages = [-(-max(n, 0) // 64) for n in lens]
    perm = torch.randperm(sum(pages) + spare, generator=gen).to(torch.int32)
    table = torch.full((len(lens), max(max(pages), 1) + 1), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(pages):
        table[r, :n] = perm[at:at + n]
        at += n
    return table, sum(pages) + spare


class Problem:
    def __init__(self, lens, hq, hkv, d, fmt, layout=DEC, rows_per_req=None, pos=None, seed=0, gain=1.5):
        gen = torch.Generator().manual_seed(seed)
        self.d, self.fmt, self.layout, self.hkv = d, fmt, layout, hkv
        self.starts = None
        if layout == DEC:
            self.req, req_len = list(range(len(lens))), list(lens)
        elif layout == PRE:
            self.req, req_len = [0] * len(lens), [max(lens)]
        else:
            self.req = [r for r, n in enumerate(rows_per_req) for _ in range(n)]
            req_len = [max([n for n, q in zip(lens, self.req) if q == r], default=0) for r in range(len(rows_per_req))]
            self.starts = torch.tensor([0] + list(np.cumsum(rows_per_req)), dtype=torch.int32)
        self.lens, self.max_len = list(lens), max(max(lens), 0)
        self.table, pages = make_table(gen, req_len)
        self.k, self.v = make_pool(gen, pages, hkv, d, fmt), make_pool(gen, pages, hkv, d, fmt)
        self.q = (gain * torch.randn(len(lens), hq, d, generator=gen)).to(torch.bfloat16)
        self.pos = None if pos is None else torch.as_tensor(pos, dtype=torch.int32)
        self.scale = 1 / math.sqrt(d)
        self.seq = torch.tensor(self.lens, dtype=torch.int32)

    def run(self, cache, **more):
        g = lambda t: None if t is None else t.cuda()  # noqa: E731
        out = torch.full_like(self.q, math.nan).cuda()
        lse = torch.full(self.q.shape[:2], math.nan, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        args = dict(lse=lse, pos=g(self.pos), dev_err=self.err, req_start=g(self.starts))
        q = more.pop("q", None)
        cache.ci_attn_decode(g(self.q) if q is None else q, g(self.k), g(self.v), g(self.table), self.layout,
                             g(self.seq), self.max_len, self.scale, out, **{**args, **more})
        torch.cuda.synchronize()
        return out, lse

    def check(self, out, lse, err=0):
        assert int(self.err) == err
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        kv, vv = C.page_values(self.k.numpy(), self.d), C.page_values(self.v.numpy(), self.d)
        table = self.table.numpy()
        for t, n in enumerate(self.lens):
            at = C.row_positions(n, self.max_len, None if self.pos is None else self.pos[t].tolist())
            at = [s for s in at if 0 <= table[self.req[t], s // 64] < len(kv)]
            page = table[self.req[t], [s // 64 for s in at]]
            slot = [s % 64 for s in at]
            q = C.bf16_values(self.q[t].view(torch.int16).numpy().view(np.uint16))
            want, z, mag, size = C.attention(q, kv[page, :, slot], vv[page, :, slot], self.scale)
            # the logits' error: D products and the scales, in fp32
            dx = (self.d + 8) * 2.0 ** -23 * size
            soft = 2 * np.expm1(dx) + (len(at) + 64) * 2.0 ** -23  # of every p, and of their sums
            tol = 2.0 ** -8 * (np.abs(want) + mag) * (1 + 2.0 ** -6) + 2 * soft[:, None] * mag + 1e-30
            assert (np.abs(out[t] - want) <= tol).all(), (t, n, np.abs(out[t] - want).max())
            if not at:
                assert (out[t] == 0).all() and (lse[t] == -np.inf).all()
            else:
                ztol = dx + (len(at) + 64) * 2.0 ** -23 + 2.0 ** -21 * (np.abs(z) + 1)
                assert (np.abs(lse[t] - z) <= ztol).all(), (t, n, np.abs(lse[t] - z).max())


LENS = [0, 1, 63, 64, 65, 130, 700]


@pytest.mark.parametrize("fmt", [BF16, FP8])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (4, 4, 64), (7, 1, 256), (28, 4, 128), (16, 1, 128), (64, 1, 128),
                                      (128, 1, 64), (66, 2, 64), (20, 1, 256), (96, 1, 256), (100, 1, 128)])
def test_attention_heads(cache, hq, hkv, d, fmt):
    p = Problem(LENS, hq, hkv, d, fmt, seed=hq + d)
    p.check(*p.run(cache))


@pytest.mark.parametrize("fmt", [BF16, FP8])
@pytest.mark.parametrize("lens", [[1], [5000], [20011], [3, 9000], [0, 0], [64 * 40] * 3, [2000] * 37])
def test_attention_lengths(cache, lens, fmt):
    p = Problem(lens, 8, 2, 128, fmt, seed=len(lens))
    p.check(*p.run(cache))


@pytest.mark.parametrize("fmt", [BF16, FP8])
@pytest.mark.parametrize("hq", [8, 64])
def test_attention_layouts(cache, fmt, hq):
    p = Problem([500 + i for i in range(9)], hq, 1, 128, fmt, layout=PRE, seed=3)
    p.check(*p.run(cache))
    p = Problem([5, 300, 301, 302, 0, 777], hq, 1, 128, fmt, layout=VAR, rows_per_req=[1, 3, 0, 2, 0], seed=4)
    p.check(*p.run(cache))


def picks(rng, lens, k, junk=True):
    """Ascending positions, -1 behind them; with junk, -1 inside and a position twice."""
    pos = np.full((len(lens), k), -1)
    for t, n in enumerate(lens):
        x = np.sort(rng.choice(n, size=min(n, k), replace=False)) if n > 0 else np.empty(0, int)
        pos[t, :len(x)] = x
        if junk and len(x) > 4:
            pos[t, 2], pos[t, 3] = -1, x[1]
    return pos


@pytest.mark.parametrize("fmt", [BF16, FP8])
@pytest.mark.parametrize("hq,hkv,d,k", [(8, 2, 128, 512), (64, 1, 128, 512), (4, 4, 64, 33), (16, 1, 256, 100),
                                        (5, 1, 64, 1), (3, 1, 128, 64)])
def test_attention_over_picked_positions(cache, hq, hkv, d, k, fmt):
    rng = np.random.default_rng(k + d)
    lens = [0, 1, 40, 512, 513, 3000, 2999]
    p = Problem(lens, hq, hkv, d, fmt, pos=picks(rng, lens, k), seed=k)
    p.check(*p.run(cache))
    lens = [900 + i for i in range(21)]
    p = Problem(lens, hq, hkv, d, fmt, layout=PRE, pos=picks(rng, lens, k, False), seed=k)
    p.check(*p.run(cache))


def test_attention_over_no_positions(cache):
    p = Problem([100, 50], 8, 2, 128, BF16, pos=np.full((2, 70), -1))
    p.check(*p.run(cache))
    p = Problem([100, 50], 8, 2, 128, BF16, pos=np.zeros((2, 0)))
    p.check(*p.run(cache))


@pytest.mark.parametrize("fmt", [BF16, FP8])
def test_attention_ignores_what_lies_outside(cache, fmt):
    """NaN and infinities beyond a row's length, in unpicked positions and in the pages of no row."""
    lens = [70, 1, 130, 0]
    for pos in (None, [[0, 69, -1, 3], [0, -1, -1, -1], [129, 64, 63, -1], [-1] * 4]):
        p = Problem(lens, 8, 2, 128, fmt, pos=pos, seed=8)
        clean = p.run(cache)
        for pool in (p.k, p.v):
            used = torch.zeros(pool.shape[0], 64, dtype=torch.bool)
            for t, n in enumerate(lens):
                for s in C.row_positions(n, n, None if pos is None else pos[t]):
                    used[p.table[t, s // 64], s % 64] = True
            row = 128 * (1 if fmt else 2)
            body = pool[:, :, :64 * row].unflatten(-1, (64, row)).transpose(1, 2)
            body[~used] = 0xFF  # NaN in both formats
            if fmt == FP8:
                pool[:, :, 64 * row:].view(torch.float32).transpose(1, 2)[~used] = math.inf
        dirty = p.run(cache)
        assert int(p.err) == 0
        for a, b in zip(clean, dirty):
            assert torch.equal(a, b)


def test_attention_passes_on_what_is_not_finite(cache):
    """A NaN in a position that counts shows in its heads' outputs alone; a value of +inf gives +inf."""
    p = Problem([100, 100], 4, 2, 64, BF16, seed=9)
    k = p.k.view(torch.bfloat16).unflatten(-1, (64, 64))
    v = p.v.view(torch.bfloat16).unflatten(-1, (64, 64))
    k[p.table[0, 1], 1, 7, 3] = math.nan
    v[p.table[1, 0], 0, 9, 5] = math.inf
    out, lse = p.run(cache)
    assert out[0, 2:].isnan().all() and lse[0, 2:].isnan().all()
    assert out[0, :2].isfinite().all() and lse[0, :2].isfinite().all()
    assert (out[1, :2, 5] == math.inf).all() and out[1, :2, :5].isfinite().all() and out[1, 2:].isfinite().all()


def test_attention_large_logits_and_small_scales(cache):
    """Logits in the thousands (one position takes all), and all of them equal."""
    p = Problem([700, 64], 8, 2, 128, BF16, seed=10, gain=400.0)
    p.check(*p.run(cache))
    p.scale = 0.0
    p.check(*p.run(cache))
    p.scale = -0.01
    p.check(*p.run(cache))


def test_attention_strides_stream_and_workspace(cache):
    p = Problem([700, 3, 129], 8, 2, 128, BF16, seed=11)
    want = p.run(cache)
    wide = torch.full((3, 12, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:10] = p.q.cuda()
    res = torch.full((3, 9, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((cache.attn_workspace_bytes(3, 8, 2, 128),), 0xFF, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    lse = torch.empty(3, 8, device="cuda")
    cache.ci_attn_decode(wide[:, 2:10], p.k.cuda(), p.v.cuda(), p.table.cuda(), DEC, p.seq.cuda(), p.max_len, p.scale,
                         res[:, :8], lse=lse, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(res[:, :8], want[0]) and torch.equal(lse, want[1])
    assert (res[:, 8] == 7).all()
    cache.ci_attn_decode(wide[:, 2:10], p.k.cuda(), p.v.cuda(), p.table.cuda(), DEC, p.seq.cuda(), p.max_len, p.scale,
                         res[:, :8])  # no lse, a workspace of the call's own
    torch.cuda.synchronize()
    assert torch.equal(res[:, :8], want[0])


def test_attention_same_bits_every_time(cache):
    p = Problem([9000, 1, 333, 20000], 16, 2, 128, BF16, seed=12)
    a = p.run(cache)
    for _ in range(3):
        b = p.run(cache)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_attention_reports_bad_data(cache):
    p = Problem([100, 200, 300], 8, 2, 128, BF16, seed=13)
    p.max_len, p.lens[1] = 300, 301
    p.seq[1] = 301
    p.check(*p.run(cache), err=cache.DEVERR_LEN)
    p.lens[1] = -5
    p.seq[1] = -5
    p.check(*p.run(cache), err=cache.DEVERR_LEN)
    p = Problem([100, 200, 300], 8, 2, 128, BF16, seed=13)
    p.table[2, 1], p.table[0, 0] = 1000, -1
    p.check(*p.run(cache), err=cache.DEVERR_PAGE)
    p = Problem([100, 200], 8, 2, 128, BF16, pos=[[5, 100, -2, 7], [1, 2, 3, 1 << 30]], seed=13)
    p.check(*p.run(cache), err=cache.DEVERR_POS)


# ------------------------------------------------------------------ append
def cos_sin(n, rot):
    ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1)).float()


def run_append(cache, tokens, hq, hkv, d, rot, neox, fmt, layout, positions, table, pages, seed=0, norms=True,
               starts=None, cache_pos=None, max_pos=None, eps=1e-5):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(tokens, hq + 2 * hkv, d, generator=gen) * torch.rand(tokens, hq + 2 * hkv, 1, generator=gen) * 4)
    x = x.to(torch.bfloat16)
    qn, kn = (1 + 0.3 * torch.randn(d, generator=gen) for _ in range(2)) if norms else (None, None)
    cs = cos_sin(max_pos or max(max(positions) + 1, 1), rot)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    g = lambda t: None if t is None else t.cuda()  # noqa: E731
    pools = [torch.full((pages, hkv, cache.page_bytes(fmt, d)), 0x5A, dtype=torch.uint8, device="cuda")
             for _ in range(2)]
    q_out = torch.full((tokens, hq, d), math.nan, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    xg = x.cuda()
    cache.ci_qk_norm_rope_append(xg[:, :hq], xg[:, hq:hq + hkv], xg[:, hq + hkv:], g(qn), g(kn), eps, cs.cuda(), neox,
                                 i32(positions), q_out, *pools, g(table), layout, dev_err=err,
                                 req_start=None if starts is None else i32(starts),
                                 cache_pos=None if cache_pos is None else i32(cache_pos))
    torch.cuda.synchronize()
    req = (list(range(tokens)) if layout == DEC else [0] * tokens if layout == PRE else
           [r for r in range(len(starts) - 1) for _ in range(starts[r + 1] - starts[r])])
    where = cache_pos if cache_pos is not None else positions
    xs = C.bf16_values(x.view(torch.int16).numpy().view(np.uint16))
    csd = cs.double().numpy()
    raw = [p.cpu().numpy() for p in pools]
    values = [C.page_values(r, d) for r in raw]
    touched = np.zeros((pages, 64), dtype=bool)
    got_q = q_out.double().cpu().numpy()
    for t in range(tokens):
        p, u = positions[t], where[t]
        if not 0 <= p < len(csd):
            assert (got_q[t] == 0).all()
            continue
        c, s = csd[p, :rot // 2], csd[p, rot // 2:]
        page = int(table[req[t], u // 64]) if 0 <= u < 64 * table.shape[1] else -1
        stored = 0 <= page < pages
        if stored:
            touched[page, u % 64] = True
        for h in range(hq + 2 * hkv):
            isq, isk = h < hq, hq <= h < hq + hkv
            w = (qn if isq else kn) if norms and (isq or isk) else None
            w = None if w is None else w.double().numpy()
            want = C.norm_rope(xs[t, h], w, eps, c, s, neox) if isq or isk else xs[t, h]
            # fp32 before the one rounding: the norm's sum and a rotation's two products
            plain = C.norm_rope(xs[t, h], w, eps, [], [], neox) if isq or isk else want
            size = np.abs(plain).max() * 2
            if isq:
                assert (np.abs(got_q[t, h] - want) <= 2.0 ** -8 * np.abs(want) + d * 2.0 ** -23 * size).all()
            elif stored:
                kv, hh = (0, h - hq) if isk else (1, h - hq - hkv)
                got = values[kv][page, hh, u % 64]
                if fmt == BF16:
                    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + d * 2.0 ** -23 * size).all()
                else:
                    scale = max(np.abs(want).max(), 1e-10) / 448
                    gs = raw[kv][page, hh, 64 * d:].view(np.float32)[u % 64]
                    assert abs(gs - scale) <= d * 2.0 ** -23 * size / 448 + 2.0 ** -23 * scale
                    assert (np.abs(got - want) <= (2.0 ** -4 * np.abs(want) + 2.0 ** -10 * scale) * 1.01 +
                            d * 2.0 ** -22 * size).all()
    for kv in range(2):  # nothing else was written
        body = raw[kv][:, :, :64 * d * (1 if fmt else 2)].reshape(pages, hkv, 64, -1)
        assert (body.transpose(0, 2, 1, 3)[~touched] == 0x5A).all()
        if fmt == FP8:
            assert (raw[kv][:, :, 64 * d:].reshape(pages, hkv, 64, 4).transpose(0, 2, 1, 3)[~touched] == 0x5A).all()
    return int(err)


@pytest.mark.parametrize("fmt", [BF16, FP8])
@pytest.mark.parametrize("neox", [True, False])
@pytest.mark.parametrize("hq,hkv,d,rot", [(8, 2, 128, 128), (7, 1, 64, 32), (3, 3, 256, 64), (28, 4, 64, 64),
                                          (5, 1, 128, 0), (2, 1, 256, 256), (40, 8, 128, 48)])
def test_append_heads(cache, hq, hkv, d, rot, neox, fmt):
    gen = torch.Generator().manual_seed(d)
    positions = [0, 63, 64, 1, 200]
    table, pages = make_table(gen, [p + 1 for p in positions])
    assert run_append(cache, 5, hq, hkv, d, rot, neox, fmt, DEC, positions, table, pages, seed=rot + 1) == 0


@pytest.mark.parametrize("fmt", [BF16, FP8])
@pytest.mark.parametrize("norms", [True, False])
def test_append_layouts(cache, fmt, norms):
    gen = torch.Generator().manual_seed(1)
    table, pages = make_table(gen, [300])
    assert run_append(cache, 150, 4, 2, 64, 64, True, fmt, PRE, list(range(100, 250)), table, pages, norms=norms) == 0
    table, pages = make_table(gen, [10, 0, 70, 300])
    at = [9] + list(range(60, 70)) + [299]
    assert run_append(cache, 12, 4, 2, 128, 64, False, fmt, VAR, at, table, pages, starts=[0, 1, 1, 11, 12],
                      norms=norms) == 0


def test_append_many_tokens(cache):
    gen = torch.Generator().manual_seed(2)
    table, pages = make_table(gen, [2000])
    assert run_append(cache, 1500, 1, 1, 64, 16, True, BF16, PRE, list(range(500, 2000)), table, pages) == 0


def test_append_padding_and_bad_positions(cache):
    gen = torch.Generator().manual_seed(3)
    positions = [5, 6, 7, 8, 9]
    table, pages = make_table(gen, [70] * 5)
    args = (cache, 5, 4, 1, 128, 64, True, BF16, DEC)
    assert run_append(*args, positions, table, pages, cache_pos=[0, -1, 69, 3, 4]) == 0
    assert run_append(*args, positions, table, pages, cache_pos=[0, 64 * table.shape[1], 69, 3, 4]) == cache.DEVERR_POS
    assert run_append(*args, [5, -1, 7, 50, 9], table, pages, max_pos=40) == cache.DEVERR_POS
    table[3, 0], table[4, 0] = 10 ** 6, -1
    assert run_append(*args, positions, table, pages) == cache.DEVERR_PAGE


def test_append_zero_and_non_finite_heads(cache):
    """A head of zeros stays zero; a NaN or infinity makes its head non-finite and no other."""
    for fmt in (BF16, FP8):
        x = torch.randn(1, 6, 64).to(torch.bfloat16).cuda()
        x[0, 1], x[0, 3], x[0, 4, 5], x[0, 5, 9] = 0, 0, math.nan, math.inf
        pools = [torch.zeros(1, 2, cache.page_bytes(fmt, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
        q_out = torch.empty(1, 2, 64, dtype=torch.bfloat16, device="cuda")
        ones = torch.ones(64, device="cuda")
        cache.ci_qk_norm_rope_append(x[:, :2], x[:, 2:4], x[:, 4:], ones, ones, 1e-6, cos_sin(4, 64).cuda(), True,
                                     torch.zeros(1, dtype=torch.int32, device="cuda"), q_out, *pools,
                                     torch.zeros(1, 1, dtype=torch.int32, device="cuda"), DEC)
        torch.cuda.synchronize()
        k, v = (C.page_values(p.cpu().numpy(), 64)[0, :, 0] for p in pools)
        assert (q_out[0, 1] == 0).all() and q_out[0, 0].isfinite().all()
        assert np.isfinite(k).all() and (k[1] == 0).all()
        assert not np.isfinite(v[0, 5]) and not np.isfinite(v[1, 9])
        if fmt == BF16:
            assert np.isfinite(v[0, :5]).all()


# ------------------------------------------------------------------ pages
class Table:
    """A cache's pages on the device beside the oracle's."""

    def __init__(self, requests, max_pages, pages, pools=3, page_bytes=176, seed=0):
        rng = np.random.default_rng(seed)
        self.o = C.Pages(np.full((requests, max_pages), -1), np.zeros(pages, dtype=np.int64),
                         rng.integers(0, 256, size=(pools, pages, page_bytes)).astype(np.uint8))
        self.put()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def put(self):
        self.table = torch.from_numpy(self.o.table.astype(np.int32)).cuda()
        self.ref = torch.from_numpy(self.o.ref.astype(np.int32)).cuda()
        self.data = torch.from_numpy(self.o.data).cuda()

    def same(self, err=0):
        np.testing.assert_array_equal(self.table.cpu().numpy(), self.o.table)
        np.testing.assert_array_equal(self.ref.cpu().numpy(), self.o.ref)
        np.testing.assert_array_equal(self.data.cpu().numpy(), self.o.data)
        assert int(self.err) == err


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("requests,max_pages,pages,seed", [(7, 9, 70, 0), (1, 1, 1, 1), (40, 33, 5003, 2),
                                                           (300, 12, 40001, 3)])
def test_pages_life(cache, requests, max_pages, pages, seed):
    """Allocation, forks, releases and compaction in turn, against the bookkeeper."""
    rng = np.random.default_rng(seed)
    t = Table(requests, max_pages, pages, seed=seed)
    half = max(1, requests // 2)
    old = np.zeros(requests, dtype=int)
    for step in range(3):
        room = pages - int((t.o.ref > 0).sum())
        cap = max(1, min(max_pages * 64, room * 64 // (2 * half + 1)))
        new = old.copy()
        new[:half] = np.maximum(old[:half], rng.integers(0, cap + 1, size=half))
        if requests == 1:
            new[0] = 64
        t.o.alloc(old.tolist(), new.tolist())
        cache.ci_pages_alloc(t.table, t.ref, i32(old.tolist()), i32(new.tolist()), dev_err=t.err)
        t.same()
        old = new
        n = min(requests - half, max(0, pages - int((t.o.ref > 0).sum())))
        if n:
            child = rng.choice(np.arange(half, requests), size=n, replace=False).tolist()
            t.o.free(child)
            cache.ci_pages_free(t.table, t.ref, i32(child), dev_err=t.err)
            t.same()
            parent = rng.integers(0, half, size=n).tolist()
            length = [int(rng.integers(0, old[p] + 1)) if step else int(old[p]) for p in parent]
            src, dst = t.o.fork(parent, child, length)
            s, d = i32([0] * n), i32([0] * n)
            cache.ci_pages_fork(t.table, t.ref, i32(parent), i32(child), i32(length), s, d, dev_err=t.err)
            assert s.tolist() == src and d.tolist() == dst
            t.o.copy(src, dst)
            cache.ci_pages_copy(t.data, s, d, dev_err=t.err)
            t.same()
        gone = rng.choice(half, size=max(1, half // 3), replace=False).tolist()
        t.o.free(gone)
        old[gone] = 0
        cache.ci_pages_free(t.table, t.ref, i32(gone), dev_err=t.err)
        t.same()
        movers, holes, remap = t.o.compact()
        m, s, d, c = (torch.full((pages,), 77, dtype=torch.int32, device="cuda") for _ in range(4))
        cache.ci_pages_compact(t.table, t.ref, m, s, d, c, dev_err=t.err)
        k = len(movers)
        assert int(c[0]) == k and s[:k].tolist() == movers and d[:k].tolist() == holes
        assert (s[k:] == -1).all() and (d[k:] == -1).all()
        np.testing.assert_array_equal(m.cpu().numpy(), remap)
        t.o.copy(movers, holes)
        cache.ci_pages_copy(t.data, s, d, count=c, dev_err=t.err)
        t.same()


def test_pages_run_out(cache):
    t = Table(4, 5, 6)
    cache.ci_pages_alloc(t.table, t.ref, i32([0, 0, 0, 0]), i32([150, 64, 200, 1]), dev_err=t.err)
    t.o.alloc([0, 0, 0, 0], [150, 64, 200, 1])
    t.same(err=cache.DEVERR_PAGE)
    assert t.table[2].tolist() == [4, 5, -1, -1, -1] and t.table[3, 0] == -1
    t.err.zero_()
    s, d = i32([9, 9]), i32([9, 9])
    cache.ci_pages_free(t.table, t.ref, i32([2]), dev_err=t.err)
    t.o.free([2])
    cache.ci_pages_alloc(t.table, t.ref, i32([150, 64, 0, 0]), i32([150, 64, 1, 0]), dev_err=t.err)
    t.o.alloc([150, 64, 0, 0], [150, 64, 1, 0])
    t.same()
    cache.ci_pages_fork(t.table, t.ref, i32([0, 2]), i32([3, 1]), i32([150, 1]), s, d, dev_err=t.err)
    assert s.tolist() == [2, -1] and d.tolist() == [5, -1] and int(t.err) == cache.DEVERR_PAGE
    assert t.table[1].tolist() == [-1] * 5 and t.table[3].tolist() == [0, 1, 5, -1, -1]


def test_pages_refuse_bad_requests(cache):
    t = Table(3, 4, 10)
    cache.ci_pages_alloc(t.table, t.ref, i32([0, 100, 0]), i32([130, 50, 300]), dev_err=t.err)
    assert int(t.err) == cache.DEVERR_LEN  # 100 -> 50 shrinks, 300 is past the row
    assert t.table.tolist() == [[0, 1, 2, -1], [-1] * 4, [-1] * 4]
    t.err.zero_()
    s, d = i32([9] * 4), i32([9] * 4)
    cache.ci_pages_fork(t.table, t.ref, i32([0, 0, -1, 0]), i32([3, 0, 1, 2]), i32([130, 130, 130, 70]), s, d,
                        dev_err=t.err)
    assert int(t.err) == cache.DEVERR_REQ
    assert s.tolist() == [-1, -1, -1, 1] and d.tolist() == [-1, -1, -1, 3]
    assert t.table.tolist() == [[0, 1, 2, -1], [-1] * 4, [0, 3, -1, -1]] and t.ref[:5].tolist() == [2, 1, 1, 1, 0]
    t.err.zero_()
    cache.ci_pages_fork(t.table, t.ref, i32([0]), i32([1]), i32([257]), s[:1], d[:1], dev_err=t.err)
    assert int(t.err) == cache.DEVERR_LEN and s[0] == -1
    t.err.zero_()
    cache.ci_pages_free(t.table, t.ref, i32([7]), dev_err=t.err)
    assert int(t.err) == cache.DEVERR_REQ
    t.err.zero_()
    t.table[1, 0], t.table[1, 1] = 8, 99  # a free page, and no page at all
    cache.ci_pages_free(t.table, t.ref, i32([1]), dev_err=t.err)
    assert int(t.err) == cache.DEVERR_PAGE and t.ref.tolist() == [2, 1, 1, 1] + [0] * 6


@pytest.mark.parametrize("sizes", [[16], [16400, 32768, 176], [131072] * 5, [8448 * 3, 16384, 16]])
def test_pages_copy_sizes(cache, sizes):
    gen = torch.Generator(device="cuda").manual_seed(5)
    pools = [torch.randint(0, 256, (40, n), generator=gen, device="cuda", dtype=torch.uint8) for n in sizes]
    want = [p.clone() for p in pools]
    src, dst = [3, -1, 39, 50, 0, 11], [4, -1, 38, 7, 20, -1]
    for w in want:
        for a, b in ((3, 4), (39, 38), (0, 20)):
            w[b] = w[a]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache.ci_pages_copy(pools, i32(src), i32(dst), dev_err=err)
    assert all(torch.equal(a, b) for a, b in zip(pools, want)) and int(err) == cache.DEVERR_PAGE
    cache.ci_pages_copy(pools, i32([8, 9]), i32([30, 31]), count=i32([1]))
    for w in want:
        w[30] = w[8]
    assert all(torch.equal(a, b) for a, b in zip(pools, want))
    cache.ci_pages_copy(pools, i32([8, 9]), i32([33, 34]), count=i32([-4]))
    assert all(torch.equal(a, b) for a, b in zip(pools, want))

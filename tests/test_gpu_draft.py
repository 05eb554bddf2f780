"""Drafted steps over the paged cache against their plain statements.

Tolerances are those of test_gpu_cache.py: bf16 rounds with a relative error of
at most 2^-8, fp32 sums of n terms err by at most n 2^-23 of the sum of
magnitudes.  What is no computed number has to be equal.
"""
import math

import numpy as np
import pytest
import torch

from oracle import cache_oracle as C
from oracle import draft_oracle as D
from test_gpu_cache import BF16, FP8, make_pool, make_table

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
LEN, PAGE_ERR, REQ, POS = 1, 2, 16, 32


@pytest.fixture(scope="module")
def draft():
    from two_level_sparse_gb300 import draft as mod

    return mod


def i32(v):
    return torch.as_tensor(np.asarray(v), dtype=torch.int32).cuda()


def random_trees(rng, nodes, most, wide=8):
    up = np.full((len(nodes), most), -1)
    for r, n in enumerate(nodes):
        for i in range(1, n):
            up[r, i] = rng.integers(max(0, i - wide), i)
    return up


# ------------------------------------------------------------------ attention
class Drafted:
    """Requests with lens positions and nodes[r] drafted rows, whose masks are trees', chains' or any bits."""

    def __init__(self, lens, nodes, hq, hkv, d, fmt, kind="tree", seed=0, gain=1.5, words=None):
        gen, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
        self.lens, self.nodes, self.d, self.hkv = list(lens), list(nodes), d, hkv
        rows = sum(nodes)
        self.starts = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        self.table, pages = make_table(gen, [a + b for a, b in zip(lens, nodes)])
        self.k, self.v = make_pool(gen, pages, hkv, d, fmt), make_pool(gen, pages, hkv, d, fmt)
        self.q = (gain * torch.randn(rows, hq, d, generator=gen)).to(torch.bfloat16)
        self.scale = 1 / math.sqrt(d)
        self.max_rows, self.max_len = max([*nodes, 1]), max(a + b for a, b in zip(lens, nodes))
        self.mask = None
        if kind != "chain":
            words = words or -(-self.max_rows // 32)
            self.mask = np.zeros((rows, words), np.uint32)
            if kind == "any":
                self.mask[:] = rng.integers(0, 2 ** 32, self.mask.shape)
                self.mask[::5] = 0
            else:
                for r, n in enumerate(nodes):
                    up = random_trees(rng, [n], max(n, 1))[0][:n]
                    for i, seen in enumerate(D.ancestors([int(p) for p in up])):
                        for j in seen:
                            self.mask[self.starts[r] + i, j // 32] |= np.uint32(1 << (j % 32))

    def run(self, draft, **more):
        q = more.pop("q", self.q).cuda()
        out, lse = torch.full_like(q, math.nan), torch.full(q.shape[:2], math.nan, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")
        mask = None if self.mask is None else torch.as_tensor(self.mask.view(np.int32)).cuda()
        args = dict(mask=mask, lse=lse, dev_err=self.err, out=out)
        args.update(more)
        out = args.pop("out")
        length = args.pop("length", i32(self.lens))
        starts = args.pop("req_start", i32(self.starts))
        draft.ci_attn_draft(q, self.k.cuda(), self.v.cuda(), self.table.cuda(), starts, length, self.max_len,
                            self.max_rows, self.scale, out, **args)
        torch.cuda.synchronize()
        return out, lse

    def check(self, out, lse, err=0, rows=None, lens=None):
        assert int(self.err) == err
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        kv, vv = C.page_values(self.k.numpy(), self.d), C.page_values(self.v.numpy(), self.d)
        table = self.table.numpy()
        for r, n in enumerate(self.nodes):
            for i in range(n):
                t = self.starts[r] + i
                if rows is not None and t not in rows:
                    continue
                mask = None if self.mask is None else self.mask[t]
                at = np.array(D.sees(self.lens[r], n, i, mask, len(kv), table[r]), dtype=int)
                page, slot = table[r, at // 64], at % 64
                q = C.bf16_values(self.q[t].view(torch.int16).numpy().view(np.uint16))
                want, z, mag, size = C.attention(q, kv[page, :, slot], vv[page, :, slot], self.scale)
                dx = (self.d + 8) * 2.0 ** -23 * size  # the logits' error: D products and the scales, in fp32
                soft = 2 * np.expm1(dx) + (len(at) + 64) * 2.0 ** -23  # of every p, and of their sums
                tol = 2.0 ** -8 * (np.abs(want) + mag) * (1 + 2.0 ** -6) + 2 * soft[:, None] * mag + 1e-30
                assert (np.abs(out[t] - want) <= tol).all(), (r, i, np.abs(out[t] - want).max())
                if not len(at):
                    assert (out[t] == 0).all() and (lse[t] == -np.inf).all(), (r, i)
                else:
                    ztol = dx + (len(at) + 64) * 2.0 ** -23 + 2.0 ** -21 * (np.abs(z) + 1)
                    assert (np.abs(lse[t] - z) <= ztol).all(), (r, i, np.abs(lse[t] - z).max())


LENS, NODES = [0, 1, 63, 64, 65, 130, 127, 700, 128], [3, 1, 2, 0, 33, 5, 1, 17, 4]


@pytest.mark.parametrize("fmt", [BF16, FP8])
@pytest.mark.parametrize("kind", ["tree", "chain", "any"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (4, 4, 64), (7, 1, 256), (28, 4, 128), (64, 1, 128), (128, 1, 64),
                                      (10, 2, 256), (100, 1, 128)])
def test_attention_heads(draft, hq, hkv, d, kind, fmt):
    p = Drafted(LENS, NODES, hq, hkv, d, fmt, kind, seed=hq + d)
    p.check(*p.run(draft))


@pytest.mark.parametrize("fmt", [BF16, FP8])
@pytest.mark.parametrize("kind", ["tree", "chain"])
@pytest.mark.parametrize("lens,nodes", [([0], [1]), ([5000], [1]), ([9000], [20]), ([3, 4001], [64, 2]),
                                        ([0, 0], [1, 128]), ([64 * 20] * 3, [64] * 3), ([300] * 40, [5] * 40),
                                        ([190, 10], [256, 255]), ([0, 500], [0, 9])])
def test_attention_lengths(draft, lens, nodes, kind, fmt):
    p = Drafted(lens, nodes, 8, 2, 128, fmt, kind, seed=len(lens))
    p.check(*p.run(draft))


@pytest.mark.parametrize("fmt", [BF16, FP8])
@pytest.mark.parametrize("nodes", [3, 40])
@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 1), (128, 8, 1), (256, 7, 1)])
def test_attention_many_tiles_per_cta(draft, d, hq, hkv, nodes, fmt):
    """Long units and many of them: whole and split, with logits that grow along the cache; the same bits again."""
    lens = [2000 + 37 * i for i in range(150)]
    p = Drafted(lens, [nodes] * 150, hq, hkv, d, fmt, seed=d + nodes)
    for r in (10, 20):  # keys that outgrow the reference again and again
        for j in range(0, lens[r], 100):
            page, slot = int(p.table[r, j // 64]), j % 64
            t = int(p.starts[r])
            if fmt == BF16:
                k = p.k.view(torch.bfloat16).view(len(p.k), hkv, 64, d)
                k[page, 0, slot] = (p.q[t, 0].float() * (0.3 + j / lens[r])).bfloat16()
            else:
                p.k[..., 64 * d:].view(torch.float32)[page, 0, slot] = 0.1 + 4 * j / lens[r]
    out, lse = p.run(draft)
    rows = {int(p.starts[r]) + i for r in (0, 1, 10, 20, 77, 120, 149) for i in {0, nodes - 1, nodes // 2}}
    p.check(out, lse, rows=rows)
    for _ in range(5):
        again = p.run(draft)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("fmt", [BF16, FP8])
@pytest.mark.parametrize("kind", ["tree", "chain"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("some", [[1, 40, 17, 3], [16, 33], [0, 1, 0, 200]])
def test_attention_blocks_of_one_and_of_two_tiles_of_rows(draft, some, d, kind, fmt):
    """Blocks that weigh unlike in the split over the CTAs, whole ones and such that several share."""
    nodes = some * (96 // len(some))
    lens = [1 + 211 * i % 3001 for i in range(96)]
    p = Drafted(lens, nodes, 8, 1, d, fmt, kind, seed=d + len(some))
    out, lse = p.run(draft)
    rows = {int(p.starts[r]) + i for r in range(0, 96, 5) if nodes[r] for i in {0, nodes[r] // 2, nodes[r] - 1}}
    p.check(out, lse, rows=rows)
    again = p.run(draft)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("fmt", [BF16, FP8])
@pytest.mark.parametrize("d,hq,hkv", [(128, 16, 2), (64, 6, 2), (256, 4, 1)])
def test_attention_long_chain(draft, d, hq, hkv, fmt):
    """A prompt's chunk behind its prefix, and a prompt with none: sampled rows."""
    p = Drafted([1000, 0], [700, 513], hq, hkv, d, fmt, "chain", seed=d)
    rows = {0, 1, 15, 16, 23, 24, 31, 32, 127, 128, 500, 698, 699, 700, 701, 763, 764, 827, 828, 1000, 1212}
    p.check(*p.run(draft), rows=rows)


@pytest.mark.parametrize("fmt", [BF16, FP8])
@pytest.mark.parametrize("kind", ["tree", "chain"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_ignores_what_is_not_seen(draft, d, kind, fmt):
    """NaN and infinities behind the nodes, in other branches, in later nodes and in the pages of no request."""
    p = Drafted([70, 0, 127, 300], [9, 6, 40, 3], 8, 2, d, fmt, kind, seed=8)
    clean = p.run(draft)
    p.check(*clean)
    seen = np.zeros((len(p.k), 64), bool)  # (page, slot) that some row reads
    for r, n in enumerate(p.nodes):
        for s in range(p.lens[r] + n):
            seen[p.table[r, s // 64], s % 64] = True
    for pool in (p.k, p.v):
        if fmt == BF16:
            x = pool.view(torch.bfloat16).view(len(pool), 2, 64, d)
            x.transpose(1, 2)[torch.from_numpy(~seen)] = torch.tensor([math.nan, math.inf, -math.inf]).repeat(d)[:d].bfloat16()
        else:
            x = pool[..., 64 * d:].view(torch.float32)
            x.transpose(1, 2)[torch.from_numpy(~seen)] = math.nan
    again = p.run(draft)
    assert all(torch.equal(a, b) for a, b in zip(clean, again))
    # one node that is not finite: the rows that see it are not either, the others stay as they are
    r, bad = 2, 20
    s = p.lens[r] + bad
    page, slot = int(p.table[r, s // 64]), s % 64
    hit = {p.starts[r] + i for i in range(p.nodes[r])
           if (i >= bad if p.mask is None else (int(p.mask[p.starts[r] + i, bad // 32]) >> (bad % 32)) & 1)}
    assert hit and len(hit) < p.nodes[r]
    for what in (math.nan, math.inf, -math.inf):
        v = p.v.clone()
        if fmt == BF16:
            p.v.view(torch.bfloat16).view(len(p.v), 2, 64, d)[page, :, slot, 5] = what
        else:
            p.v[..., 64 * d:].view(torch.float32)[page, :, slot] = what
        out, lse = p.run(draft)
        for t in range(len(p.q)):
            dims = [5] if fmt == BF16 else list(range(d))
            if t not in hit:
                assert torch.equal(out[t], clean[0][t]), t
            elif fmt == BF16:
                assert (torch.isnan(out[t, :, 5]) if math.isnan(what) else out[t, :, 5] == what).all(), t
                rest = [x for x in range(d) if x not in dims]
                assert torch.equal(out[t][:, rest], clean[0][t][:, rest]), t
            else:
                assert not torch.isfinite(out[t]).any(), t
        assert torch.equal(lse, clean[1])
        p.v = v


@pytest.mark.parametrize("d,nodes", [(128, 2), (128, 7), (128, 16), (128, 40), (64, 3), (256, 3), (256, 20)])
def test_attention_infinite_values_that_all_see(draft, d, nodes):
    """An infinity in the cache gives that dim an infinity in every row, however many there are, and no NaN elsewhere."""
    p = Drafted([700], [nodes], 8, 1, d, BF16, seed=nodes)
    clean, lse = p.run(draft)
    p.v.view(torch.bfloat16).view(len(p.v), 1, 64, d)[int(p.table[0, 4]), 0, 33, 7] = math.inf
    out, again = p.run(draft)
    rest = [x for x in range(d) if x != 7]
    assert torch.isposinf(out[:, :, 7]).all() and torch.equal(out[:, :, rest], clean[:, :, rest])
    assert torch.equal(lse, again)


def test_attention_keys_that_are_not_finite(draft):
    """A NaN in a node's key reaches the rows that see it, and no other."""
    p = Drafted([100], [12], 4, 2, 128, BF16, "tree", seed=1)
    clean, _ = p.run(draft)
    s = 100 + 4
    p.k.view(torch.bfloat16).view(len(p.k), 2, 64, 128)[int(p.table[0, s // 64]), :, s % 64, 3] = math.nan
    out, lse = p.run(draft)
    for t in range(12):
        if (int(p.mask[t, 0]) >> 4) & 1:
            assert torch.isnan(out[t]).all() and torch.isnan(lse[t]).all()
        else:
            assert torch.equal(out[t], clean[t])


@pytest.mark.parametrize("fmt", [BF16, FP8])
def test_attention_strides_and_rows_of_no_request(draft, fmt):
    """Queries and results inside wider rows; rows in front of, between and behind the requests' stay as they are."""
    p = Drafted([77, 200], [5, 6], 8, 2, 128, fmt, seed=2)
    wide = torch.zeros(11, 12, 128, dtype=torch.bfloat16)
    wide[:, 1:9] = p.q
    res = torch.full((11, 20, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    out, lse = p.run(draft, q=wide.cuda()[:, 1:9], out=res[:, 8:16])
    p.check(out, lse)
    assert (res[:, :8] == 7).all() and (res[:, 16:] == 7).all()
    starts = np.array([2, 7, 11], np.int32)  # the second request has 4 rows now, two rows and one are nobody's
    q = torch.cat([torch.full((2, 8, 128), math.nan, dtype=torch.bfloat16), p.q[:5], p.q[5:9],
                   torch.full((1, 8, 128), math.nan, dtype=torch.bfloat16)])
    mask = np.concatenate([np.zeros((2, 1), np.uint32), p.mask[:5], p.mask[5:9], np.zeros((1, 1), np.uint32)])
    out = torch.full((12, 8, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((12, 8), 3.0, device="cuda")
    out, _ = p.run(draft, q=q, out=out, lse=lse, req_start=i32(starts), mask=torch.as_tensor(mask.view(np.int32)).cuda())
    none = [0, 1, 11]
    assert (out[none] == 3).all() and (lse[none] == 3).all() and int(p.err) == 0
    p.nodes, p.starts, p.q, p.mask = [5, 4], starts, q, mask
    p.check(out, lse)


def test_calls_with_no_rows(draft):
    """A step in which nobody drafts: every call runs and changes nothing."""
    p = Drafted([100, 30], [0, 0], 8, 2, 128, BF16)
    p.max_rows = 0
    out, lse = p.run(draft)
    assert out.shape == (0, 8, 128) and int(p.err) == 0
    empty, bits = i32([]), torch.zeros(1, dtype=torch.int32, device="cuda")
    path, kept, after, new = i32([[9, 9]] * 2), i32([9, 9]), i32([9, 9]), i32([9, 9])
    draft.ci_draft_accept(i32([0, 0, 0]), i32([100, 30]), None, empty, empty, path, kept, after, new, dev_err=bits)
    assert path.tolist() == [[-1, -1]] * 2 and kept.tolist() == [0, 0] and after.tolist() == [-1, -1]
    assert new.tolist() == [100, 30]
    pool = p.k.cuda()
    draft.ci_slots_move([pool], 256, 0, p.table.cuda(), i32([100, 30]), path, kept, dev_err=bits)
    assert torch.equal(pool.cpu(), p.k) and int(bits) == 0


@pytest.mark.parametrize("words", [1, 2, 5])
@pytest.mark.parametrize("fmt", [BF16, FP8])
def test_attention_mask_words(draft, words, fmt):
    """Fewer words than a request has nodes (what they do not name is not seen), more, and bits behind its nodes."""
    p = Drafted([200, 33, 0], [40, 7, 70], 8, 2, 128, fmt, "any", seed=words, words=words)
    p.check(*p.run(draft))


def test_attention_reports(draft):
    p = Drafted([100, 200, 50], [4, 5, 3], 4, 2, 128, BF16, seed=5)
    want, wlse = p.run(draft)
    # a length that does not fit: zeros for its rows
    out, lse = p.run(draft, length=i32([100, 1 << 20, 50]))
    assert int(p.err) == LEN and (out[4:9] == 0).all() and torch.isneginf(lse[4:9]).all()
    assert torch.equal(out[:4], want[:4]) and torch.equal(out[9:], want[9:])
    out, lse = p.run(draft, length=i32([-1, 200, 50]))
    assert int(p.err) == LEN and (out[:4] == 0).all() and torch.equal(out[4:], want[4:])
    # more rows than was said
    p.max_rows = 4
    out, lse = p.run(draft)
    assert int(p.err) == LEN and (out[4:9] == 0).all() and torch.equal(out[:4], want[:4]) and torch.equal(out[9:], want[9:])
    p.max_rows = 5
    # starts that descend or leave the rows: none of that request's
    res = torch.full_like(want, 5.0)
    out, _ = p.run(draft, out=res, req_start=i32([0, 4, 99, 12]))
    assert int(p.err) == REQ and torch.equal(out[:4], want[:4]) and (out[4:] == 5).all()
    # pages that are not there
    p.table[1, 1], p.table[0, 0] = 10 ** 6, -1
    p.check(*p.run(draft), err=PAGE_ERR)


def test_attention_far_logits_and_values(draft):
    """Logits far apart and of either sign, scales of either sign, values of 2^80, lengths past many tiles."""
    p = Drafted([1000, 40], [6, 6], 4, 2, 128, BF16, seed=6, gain=40.0)
    p.check(*p.run(draft))
    p.scale = -p.scale
    p.check(*p.run(draft))
    p = Drafted([1000, 40], [6, 6], 4, 2, 128, BF16, seed=6)
    p.v = (p.v.view(torch.bfloat16).clamp(-1, 1) * 2.0 ** 80).view(torch.uint8)
    p.check(*p.run(draft))
    p = Drafted([900, 40], [6, 6], 4, 2, 128, FP8, seed=7)
    scale = p.v[..., 64 * 128:].view(torch.float32)
    scale *= torch.where(torch.rand(scale.shape) < 0.5, 2.0 ** 58, -(2.0 ** -60))
    p.check(*p.run(draft))
    scale = p.k[..., 64 * 128:].view(torch.float32)
    scale *= torch.where(torch.rand(scale.shape) < 0.5, -1.0, 2.0 ** -20)
    p.check(*p.run(draft))


def test_attention_small_codes(draft):
    """e4m3's subnormal codes and its NaN codes (+-480), queries far from 1."""
    for d in (64, 128, 256):
        p = Drafted([150], [5], 4, 1, d, FP8, seed=d)
        for pool in (p.k, p.v):
            codes = pool[..., :64 * d]
            codes.copy_(torch.randint(0, 256, codes.shape, dtype=torch.int32).to(torch.uint8) & 0x87)  # all subnormal
        p.q = (p.q.float() * 100).bfloat16()
        p.check(*p.run(draft))
    p = Drafted([150], [5], 4, 1, 128, FP8, seed=9)
    p.q = (p.q.float() * 2.0 ** torch.randint(-60, 3, p.q.shape)).bfloat16()
    p.check(*p.run(draft))


@pytest.mark.parametrize("fmt", [BF16, FP8])
def test_attention_far_pages(draft, fmt):
    """Pages behind 2^31 bytes and 2^32 bytes of a pool."""
    d, hkv = 128, 2
    bytes_of = 64 * d * 2 if fmt == BF16 else 64 * d + 256
    pages = (2 ** 32 + 2 ** 28) // (hkv * bytes_of)
    p = Drafted([500], [7], 8, hkv, d, fmt, seed=4)
    far = torch.tensor([pages - 1 - i if i % 2 else (2 ** 31) // (hkv * bytes_of) + i for i in range(p.table.shape[1])])
    near, use = p.table[0].clone(), -(-507 // 64)
    k, v = (torch.zeros(pages, hkv, bytes_of, dtype=torch.uint8, device="cuda") for _ in range(2))
    for i in range(use):
        k[far[i]], v[far[i]] = p.k[near[i]].cuda(), p.v[near[i]].cuda()
    small = p.run(draft)
    table = p.table.clone()
    table[0, :use] = far[:use].int()
    out, lse = torch.empty_like(small[0]), torch.empty_like(small[1])
    draft.ci_attn_draft(p.q.cuda(), k, v, table.cuda(), i32(p.starts), i32(p.lens), p.max_len, p.max_rows, p.scale, out,
                        mask=torch.as_tensor(p.mask.view(np.int32)).cuda(), lse=lse)
    assert torch.equal(out, small[0]) and torch.equal(lse, small[1])


# ------------------------------------------------------------------ plan
def run_plan(draft, length, count, parent, token, table, num_pages, rows, most, words, err=0):
    req = len(length)
    full = lambda *s: torch.full(s, 77, dtype=torch.int32, device="cuda")  # noqa: E731
    start, at, slot, tok, mask = full(req + 1), full(rows), full(rows), full(rows), full(rows, words)
    bits = torch.zeros(1, dtype=torch.int32, device="cuda")
    more = {} if token is None else dict(token=i32(token), row_token=tok)
    draft.ci_draft_plan(i32(length), i32(count), None if parent is None else i32(parent), i32(table), num_pages, start,
                        at, slot, mask=mask, max_nodes=most, dev_err=bits, **more)
    want = D.plan(length, count, parent, token, np.asarray(table), num_pages, rows, most, words)
    got = [x.cpu().numpy() for x in (start, at, slot, mask, tok)]
    for name, a, b in zip(("req_start", "positions", "cache_pos", "mask"), got, want):
        np.testing.assert_array_equal(a.view(b.dtype) if name == "mask" else a, b, err_msg=name)
    if token is not None:
        np.testing.assert_array_equal(got[4], want[4])
    assert int(bits) == err
    return got


@pytest.mark.parametrize("req,most,words", [(1, 1, 1), (3, 5, 1), (7, 32, 1), (6, 33, 2), (50, 64, 3), (5, 256, 8),
                                            (4096, 3, 1), (9, 100, 8)])
@pytest.mark.parametrize("tree", [True, False])
def test_plan(draft, req, most, words, tree):
    rng = np.random.default_rng(req + most)
    count = rng.integers(0, most + 1, req)
    count[0] = most
    length = rng.integers(0, 500, req)
    gen = torch.Generator().manual_seed(req)
    table, pages = make_table(gen, [int(a + b) for a, b in zip(length, count)])
    if req > 4:
        table[3, 0], table[4, -2:] = -1, pages + 5
    parent = random_trees(rng, count, most, wide=most) if tree else None
    for rows in (int(count.sum()), int(count.sum()) + 37):
        run_plan(draft, length, count, parent, rng.integers(0, 1000, (req, most)), table, pages, rows, most, words)


def test_plan_reports(draft):
    table = np.arange(12).reshape(3, 4)
    up = [[-1, 0, 1, 1]] * 3
    run_plan(draft, [10, 20, 30], [4, 5, 2], up, None, table, 12, 9, 4, 1, LEN)
    run_plan(draft, [10, 20, 30], [4, -1, 2], up, None, table, 12, 9, 4, 1, LEN)
    run_plan(draft, [10, 254, 30], [4, 3, 2], up, None, table, 12, 9, 4, 1, LEN)
    run_plan(draft, [10, -1, 252], [4, 1, 4], up, None, table, 12, 9, 4, 1, LEN)
    run_plan(draft, [10, 20, 30], [4, 4, 4], up, None, table, 12, 9, 4, 1, LEN)  # more nodes than rows
    run_plan(draft, [10, 20, 30], [4, 4, 4], up, None, table, 12, 0, 4, 1, LEN)
    run_plan(draft, [10, 20, 30], [4, 3, 4], [[-1, 1, 0, 2], [-2, 0, 5, 9], [0, 0, 0, 3]], None, table, 12, 11, 4, 1, POS)


# ------------------------------------------------------------------ accept, move, trim
@pytest.mark.parametrize("req,most", [(1, 1), (5, 7), (40, 33), (3, 64), (6, 100), (4, 256), (4096, 2)])
@pytest.mark.parametrize("tree", [True, False])
def test_accept(draft, req, most, tree):
    rng = np.random.default_rng(req + most)
    count = rng.integers(0, most + 1, req)
    count[0] = most
    start = np.concatenate([[0], np.cumsum(count)])
    parent = random_trees(rng, count, most) if tree else None
    length = rng.integers(0, 1000, req)
    for stored in (None, np.where(rng.random(start[-1]) < 0.95, 5, -1)):
        token, target = rng.integers(0, 3, start[-1] + 4), rng.integers(0, 3, start[-1] + 4)  # ties abound
        path = torch.full((req, most), 9, dtype=torch.int32, device="cuda")
        out = [torch.full((req,), 9, dtype=torch.int32, device="cuda") for _ in range(3)]
        bits = torch.zeros(1, dtype=torch.int32, device="cuda")
        cp = None if stored is None else i32(np.concatenate([stored, [5] * 4]))
        draft.ci_draft_accept(i32(start), i32(length), None if parent is None else i32(parent), i32(token), i32(target),
                              path, *out, cache_pos=cp, dev_err=bits)
        want = D.accept(start, length, parent, token, target, stored, most)
        np.testing.assert_array_equal(path.cpu().numpy(), want[0])
        for a, b in zip(out, want[1:]):
            assert a.tolist() == list(b)
        assert int(bits) == 0


def test_accept_odd_trees_and_reports(draft):
    out = lambda: (torch.full((2, 4), 9, dtype=torch.int32, device="cuda"),  # noqa: E731
                   *(torch.full((2,), 9, dtype=torch.int32, device="cuda") for _ in range(3)))
    tok = i32([1] * 8)
    bits = torch.zeros(1, dtype=torch.int32, device="cuda")
    # parents that are no earlier nodes belong to no path; a second root neither
    o = out()
    draft.ci_draft_accept(i32([0, 4, 8]), i32([5, 6]), i32([[-1, 1, 9, -1], [3, 0, -7, 1]]), tok, tok, *o, dev_err=bits)
    assert o[0].tolist() == [[0, -1, -1, -1], [0, 1, 3, -1]] and o[3].tolist() == [6, 9] and int(bits) == 0
    for starts in ([0, 5, 8], [0, 4, 3], [-1, 2, 4], [0, 4, 9]):
        o = out()
        bits.zero_()
        draft.ci_draft_accept(i32(starts), i32([5, 6]), None, tok, tok, *o, dev_err=bits)
        bad = [not (0 <= a <= b <= 8 and b - a <= 4) for a, b in zip(starts, starts[1:])]
        assert int(bits) == REQ and any(bad)
        for r in range(2):
            n = 0 if bad[r] else starts[r + 1] - starts[r]
            assert int(o[1][r]) == n and int(o[3][r]) == 5 + r + n and int(o[2][r]) == (1 if n else -1)


FORMS = [(2 * 128, 0, 3), (128, 4, 2), (2 * 64, 0, 1), (64, 4, 5), (2 * 256, 0, 2), (256, 4, 1), (16, 4, 1)]


@pytest.mark.parametrize("forms", [FORMS[:1], FORMS[1:2], FORMS])
@pytest.mark.parametrize("req,most", [(1, 1), (3, 6), (30, 40), (2, 256)])
def test_move(draft, req, most, forms):
    rng = np.random.default_rng(req + most)
    gen = torch.Generator().manual_seed(req)
    length = rng.integers(0, 300, req)
    length[0] = 0
    table, pages = make_table(gen, [int(n) + most for n in length])
    count = rng.integers(0, most + 1, req)
    path = np.full((req, most), -1)
    for r, n in enumerate(count):
        path[r, :n] = np.sort(rng.choice(most, n, replace=False))
    if req > 2:
        path[1, :2], count[1] = [0, 1], 2  # nothing moves
        table[2, 0] = -1 if length[2] + most > 64 else table[2, 0]
    pools = [torch.randint(0, 256, (pages, h, 64 * (a + b)), generator=gen, dtype=torch.int32).to(torch.uint8) for a, b, h in forms]
    if len(forms) > 1:
        pools[-1] = pools[-1][:, 0].contiguous()  # as an index pool: no heads
    got = [p.cuda() for p in pools]
    bits = torch.zeros(1, dtype=torch.int32, device="cuda")
    draft.ci_slots_move(got, [f[0] for f in forms], [f[1] for f in forms], i32(table), i32(length), i32(path), i32(count),
                        dev_err=bits)
    for (a, b, _), x, was in zip(forms, got, pools):
        want = D.move(was.reshape(pages, -1, 64 * (a + b)).numpy(), a, b, table.numpy(), length, path, count)
        np.testing.assert_array_equal(x.cpu().numpy().reshape(want.shape), want)
    assert int(bits) in (0, PAGE_ERR)


def test_move_reports(draft):
    gen = torch.Generator().manual_seed(1)
    pool = torch.randint(0, 256, (6, 2, 64 * 20), generator=gen, dtype=torch.int32).to(torch.uint8)
    table = np.arange(6).reshape(3, 2)
    good = [0, 2, 5]
    for length, path, count, err, moved in [
            ([5, 6, 7], [good, [0, 2, 2], good], [3, 3, 3], POS, (0, 2)),
            ([5, 6, 7], [good, [2, 1, 3], good], [3, 3, 3], POS, (0, 2)),
            ([5, 6, 7], [good, [-1, 1, 3], good], [3, 3, 3], POS, (0, 2)),
            ([5, 123, 7], [good, good, good], [3, 3, 3], POS, (0, 2)),
            ([5, -1, 7], [good, good, good], [3, 3, 3], POS, (0, 2)),
            ([5, 6, 7], [good, good, good], [3, 4, -1], POS, (0,)),
            ([5, 6, 7], [good, good, good], [3, 0, 1], 0, (0,))]:
        got, bits = pool.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
        draft.ci_slots_move([got], 16, 4, i32(table), i32(length), i32(path), i32(count), dev_err=bits)
        n = [c if r in moved else 0 for r, c in enumerate(count)]
        np.testing.assert_array_equal(got.cpu().numpy(), D.move(pool.numpy(), 16, 4, table, length, path, n))
        assert int(bits) == err


def test_trim(draft):
    rng = np.random.default_rng(0)
    req, cols = 300, 70
    table = rng.permutation(req * cols).reshape(req, cols)
    table[::7, 20:30] = -1
    ref = np.ones(req * cols, int)
    ref[::3] = 2
    old = rng.integers(0, 64 * cols + 1, req)
    new = (old * rng.random(req)).astype(int)
    new[::4] = old[::4]
    t, f, bits = i32(table), i32(ref), torch.zeros(1, dtype=torch.int32, device="cuda")
    draft.ci_pages_trim(t, f, i32(old), i32(new), dev_err=bits)
    want, want_ref = D.trim(table, ref, old, new)
    np.testing.assert_array_equal(t.cpu().numpy(), want)
    np.testing.assert_array_equal(f.cpu().numpy(), want_ref)
    assert int(bits) == 0
    t, f = i32([[0, 1], [2, 9], [3, 4], [5, 5]]), i32([1, 1, 1, 1, 0, 1])
    draft.ci_pages_trim(t, f, i32([128, 128, 128, 129]), i32([129, 0, 65 - 64, 0]), dev_err=bits)
    assert t.tolist() == [[0, 1], [-1, -1], [3, -1], [5, 5]] and f.tolist() == [1, 1, 0, 1, 0, 1]
    assert int(bits) == LEN | PAGE_ERR


# ------------------------------------------------------------------ together
def test_attention_on_two_streams_and_from_graphs(draft):
    """Calls at the same time on two streams, and replayed graphs, give what calls one after another do."""
    ps = [Drafted([3000 + 50 * i for i in range(20)], [4 + s] * 20, 8, 2, 128, BF16, seed=s) for s in range(2)]
    want = [p.run(draft) for p in ps]
    args, outs = [], []
    for p in ps:
        out, lse = torch.empty_like(want[len(outs)][0]), torch.empty_like(want[len(outs)][1])
        args.append((p.q.cuda(), p.k.cuda(), p.v.cuda(), p.table.cuda(), i32(p.starts), i32(p.lens), p.max_len, p.max_rows,
                     p.scale, out, torch.as_tensor(p.mask.view(np.int32)).cuda(), lse))
        outs.append((out, lse))
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(20):
        for a, stream in zip(args, streams):
            draft.ci_attn_draft(*a[:10], mask=a[10], lse=a[11], stream=stream)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
    graphs = []
    for a, stream in zip(args, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            draft.ci_attn_draft(*a[:10], mask=a[10], lse=a[11])
        graphs.append(graph)
    for out, lse in outs:
        out.zero_(), lse.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


def entries(cache, r, n):
    """A request's first n cached entries, keys and values of all layers, and their scales."""
    at = torch.arange(n, device="cuda")
    page, slot = cache.page_table[r].long()[at // 64], at % 64
    d = cache.head_dim
    width = 2 * d if cache.k.shape[-1] == 64 * 2 * d else d
    got = []
    for pool in (cache.k, cache.v):
        got.append(pool[..., :64 * width].unflatten(-1, (64, width))[:, page, :, slot])
        if width == d:
            got.append(pool[..., 64 * d:].unflatten(-1, (64, 4))[:, page, :, slot])
    return got


@pytest.mark.parametrize("fmt,d,tree,graph", [(BF16, 128, True, False), (FP8, 128, True, False), (BF16, 64, False, False),
                                              (FP8, 256, True, False), (BF16, 128, True, True), (FP8, 64, False, True)])
def test_drafted_steps(fmt, d, tree, graph):
    """Drafted steps leave the cache and give the results that decoding the kept tokens one by one does."""
    from two_level_sparse_gb300.paged import PagedCache, drafted_step

    rng = np.random.default_rng(d + fmt)
    gen = torch.Generator(device="cuda").manual_seed(d)
    hq, hkv, layers, most, steps = 8, 2, 2, 9, 4
    lens = [126, 0, 61, 300]
    caches = [PagedCache(layers, 4, 8, 40, hkv, d, fmt) for _ in range(2)]
    drafted, plain = caches
    companion = torch.randint(0, 256, (40, 8448), dtype=torch.int32, generator=gen, device="cuda").to(torch.uint8)
    drafted.companions.append(companion)
    norm = 1 + 0.1 * torch.randn(d, device="cuda", generator=gen)
    angle = torch.arange(600, device="cuda")[:, None] * 10000.0 ** (-torch.arange(d // 2, device="cuda") / (d // 2))
    cs = torch.cat([angle.cos(), angle.sin()], 1)
    x = torch.randn(sum(lens), hq + 2 * hkv, d, device="cuda", generator=gen).bfloat16()
    starts, at = i32(np.cumsum([0, *lens])), i32([i for n in lens for i in range(n)])
    for c in caches:
        c.grow(i32(lens))
        for j in range(layers):
            c.append(j, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], norm, norm, 1e-6, cs, True, at, 2, req_start=starts)
    buf = dict(count=i32([0] * 4), parent=i32(np.full((4, most), -1)), token=i32(np.zeros((4, most))),
               qkv=torch.zeros(layers, 4 * most, hq + 2 * hkv, d, dtype=torch.bfloat16, device="cuda"),
               target=i32(np.zeros(4 * most)))

    def step():
        dr = drafted.draft(buf["count"], buf["token"], buf["parent"] if tree else None)
        outs = drafted_step(drafted, dr, buf["qkv"], norm, norm, 1e-6, cs)
        return dr, outs, drafted.commit(dr, buf["target"])

    run = step
    if graph:
        step()  # with no tokens
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held = step()

        def run():
            g.replay()
            return held

    for s in range(steps):
        count = [3, most if s else 0, s, 7 - s]
        up = random_trees(rng, count, most, wide=3)
        token, target = rng.integers(0, 2, (4, most)), rng.integers(0, 2, 4 * most)
        buf["count"].copy_(i32(count)), buf["parent"].copy_(i32(up)), buf["token"].copy_(i32(token))
        buf["target"].copy_(i32(target))
        buf["qkv"].copy_(torch.randn(buf["qkv"].shape, device="cuda", generator=gen))
        index_before = companion.clone()
        dr, outs, (path, kept, after) = run()
        drafted.check()
        start = np.concatenate([[0], np.cumsum(count)])
        flat = [int(t) for r in range(4) for t in token[r, :count[r]]]
        want = D.accept(start, lens, up if tree else None, flat, target, None, most)
        np.testing.assert_array_equal(path.cpu().numpy(), want[0])
        assert kept.tolist() == want[1] and after.tolist() == want[2] and drafted.length.tolist() == want[3]
        # the kept tokens, one by one
        for i in range(max(want[1])):
            there = [i < n for n in want[1]]
            pos = [lens[r] + i if there[r] else 0 for r in range(4)]
            plain.grow(i32([lens[r] + min(i + 1, want[1][r]) for r in range(4)]))
            rows = [int(start[r] + want[0][r][i]) if there[r] else 0 for r in range(4)]
            for j in range(layers):
                y = buf["qkv"][j, rows]
                q = plain.append(j, y[:, :hq], y[:, hq:hq + hkv], y[:, hq + hkv:], norm, norm, 1e-6, cs, True, i32(pos), 0,
                                 cache_pos=i32([p if t else -1 for p, t in zip(pos, there)]))
                o = plain.attend(j, q, 0, i32([p + 1 if t else 0 for p, t in zip(pos, there)]))
                for r in range(4):
                    if there[r]:  # each is within its own rounding and its probabilities' of the exact result
                        torch.testing.assert_close(outs[j][rows[r]].float(), o[r].float(), rtol=2 ** -7, atol=2 ** -6)
        lens = want[3]
        for r in range(4):
            for a, b in zip(entries(drafted, r, lens[r]), entries(plain, r, lens[r])):
                assert torch.equal(a, b), r
            pages = -(-lens[r] // 64)
            assert (drafted.page_table[r, :pages] >= 0).all() and (drafted.page_table[r, pages:] == -1).all()
        used = drafted.page_table[drafted.page_table >= 0].long()
        ref = torch.zeros(40, dtype=torch.int32, device="cuda").index_add_(0, used, torch.ones_like(used, dtype=torch.int32))
        assert torch.equal(ref, drafted.ref_count)
        if not graph:  # the index keys moved along (looked at where both pages are still there)
            table = drafted.page_table.cpu().numpy()
            for r in range(4):
                old = lens[r] - want[1][r]
                for i in range(want[1][r]):
                    src, dst = old + int(want[0][r][i]), old + i
                    a, b = table[r, src // 64], table[r, dst // 64]
                    if a >= 0:
                        for row, base in ((128, 0), (4, 64 * 128)):
                            x, y = base + row * (dst % 64), base + row * (src % 64)
                            assert torch.equal(companion[b, x:x + row], index_before[a, y:y + row])


def test_draft_bookkeeping(draft):
    """Drafts that do not fit, pages that run out, an open draft, one that is dropped."""
    from two_level_sparse_gb300.paged import PagedCache

    cache, ones = PagedCache(1, 3, 2, 4, 1, 64), i32(np.ones((3, 9)))
    cache.grow(i32([60, 64, 120]))
    assert (cache.ref_count > 0).all()
    d = cache.draft(i32([3, 2, 4]), ones)  # the second request gets no page
    assert d.cache_pos[:9].tolist() == [60, 61, 62, -1, -1, 120, 121, 122, 123] and int(cache.dev_err) == PAGE_ERR
    for f in (lambda: cache.grow(i32([60, 64, 120])), lambda: cache.free(i32([0])), cache.compact,
              lambda: cache.fork(i32([0]), i32([1]), i32([3])), lambda: cache.draft(i32([1, 1, 1]), ones)):
        with pytest.raises(RuntimeError, match="open"):
            f()
    path, kept, after = cache.commit(d, i32([1] * 27))
    assert kept.tolist() == [3, 0, 4] and after.tolist() == [1, -1, 1] and cache.length.tolist() == [63, 64, 124]
    q = torch.zeros(27, 1, 64, dtype=torch.bfloat16, device="cuda")
    for f in (lambda: cache.commit(d, i32([1] * 27)), lambda: cache.drop(d), lambda: cache.attend_draft(0, q, d)):
        with pytest.raises(RuntimeError, match="not open"):
            f()
    cache.dev_err.zero_()
    d = cache.draft(i32([2, -1, 5]), ones, rows=7)  # 124 + 5 positions do not fit two pages, no page is left for 63 + 2
    assert d.req_start.tolist() == [0, 2, 2, 2] and int(cache.dev_err) == LEN | PAGE_ERR
    assert d.end.tolist() == [65, 64, 124] and d.cache_pos.tolist() == [63, -1, -1, -1, -1, -1, -1]
    cache.commit(d, i32([0] * 7))
    assert cache.length.tolist() == [64, 64, 124]
    cache = PagedCache(1, 2, 4, 8, 1, 64)
    cache.grow(i32([60, 1]))
    before = cache.page_table.clone(), cache.ref_count.clone()
    cache.drop(cache.draft(i32([9, 9]), i32(np.ones((2, 9)))))
    assert torch.equal(cache.page_table, before[0]) and torch.equal(cache.ref_count, before[1])
    assert cache.length.tolist() == [60, 1] and int(cache.dev_err) == 0
    with pytest.raises(ValueError):
        cache.draft(i32([1, 1]), i32(np.ones((2, 257))))
    cache.companions.append(torch.zeros(8, 100, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="companions"):
        cache.draft(i32([1, 1]), i32(np.ones((2, 2))))


@pytest.mark.parametrize("d,lens", [(64, [1000]), (128, [1000]), (256, [1000]), (128, [20000]), (128, [1001] * 160)])
def test_attention_largest_fp8_values(draft, d, lens):
    """The largest code under the largest scale, seen with the same weight by every position: units that several CTAs
    share (one request) and whole ones (a request per CTA and more)."""
    p = Drafted(lens, [1] * len(lens), 2, 1, d, FP8, seed=d)
    p.q.zero_()
    codes, scale = p.v[..., :64 * d].view(len(p.v), 1, 64, d), p.v[..., 64 * d:].view(torch.float32)
    codes.fill_(0x7E)  # 448
    codes[..., d // 2:] |= 0x80
    codes[1::3, :, :, ::8] ^= 0x80  # (dims in which pages cancel)
    scale.fill_(2.0 ** 60)
    out, lse = p.run(draft)
    assert torch.isfinite(out).all()
    p.check(out, lse)


def split_loss(q):
    """What an FP8 call may leave out of a query's elements (float64 [..., d], bf16 values): nothing from 2^-13 of the
    row's largest magnitude on, else at most 2^-21 of it."""
    size = np.abs(q)
    top = size.max(-1, keepdims=True)
    return np.where(size >= 2.0 ** -13 * top, 0, np.minimum(size, 2.0 ** -21 * top))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("far", range(8, 19))
def test_attention_fp8_queries_with_an_outlier(draft, d, far):
    """One dim of the query is 2^far times as large as the others, and 0 in every key: the logits are the others'.  They
    are alike, so that what each of them loses adds up."""
    rng = np.random.default_rng(far)
    p = Drafted([300], [16], 4, 1, d, FP8, seed=far)
    codes = torch.from_numpy(rng.integers(0x30, 0x40, (len(p.k), 1, 64, d)).astype(np.uint8))  # 0.5 .. 1.875
    codes[..., 0] = 0
    p.k[..., :64 * d] = codes.view(len(p.k), 1, 64 * d)
    p.k[..., 64 * d:].view(torch.float32).fill_(1.0)
    small = 1 + torch.from_numpy(rng.integers(0, 128, (16, 4))).double() / 128  # 1 .. 2, exact in bf16
    p.q = small[..., None].expand(16, 4, d).to(torch.bfloat16).contiguous()
    p.q[..., 0] = 2.0 ** far
    p.scale = 8.0 / d
    out, lse = p.run(draft)
    assert int(p.err) == 0
    keys, vals = C.page_values(p.k.numpy(), d)[:, 0], C.page_values(p.v.numpy(), d)[:, 0]
    table = p.table.numpy()
    for i in range(16):
        at = np.array(D.sees(300, 16, i, p.mask[i], len(p.k), table[0]))
        k, v = keys[table[0, at // 64], at % 64], vals[table[0, at // 64], at % 64]
        q = p.q[i].double().numpy()
        x = p.scale * q @ k.T
        # the logits' error: D products and the scales in fp32, and the split
        dx = ((d + 8) * 2.0 ** -23 * p.scale * np.abs(q) @ np.abs(k).T + p.scale * split_loss(q) @ np.abs(k).T).max(-1)
        z = np.log(np.exp(x - x.max(-1, keepdims=True)).sum(-1)) + x.max(-1)
        w = np.exp(x - z[:, None])
        n = len(at)
        ztol = dx + (n + 64) * 2.0 ** -23 + 2.0 ** -21 * (np.abs(z) + 1)
        assert (np.abs(lse[i].double().cpu().numpy() - z) <= ztol).all(), (i, np.abs(lse[i].double().cpu().numpy() - z).max())
        want, mag = w @ v, w @ np.abs(v)
        soft = 2 * np.expm1(dx) + (n + 64) * 2.0 ** -23
        tol = 2.0 ** -8 * (np.abs(want) + mag) * (1 + 2.0 ** -6) + 2 * soft[:, None] * mag + 1e-30
        assert (np.abs(out[i].double().cpu().numpy() - want) <= tol).all(), i


def test_refused_drafts_leave_no_pages(draft):
    """What the plan refuses was allocated already: it goes back, and a draft with what is right finds it."""
    from two_level_sparse_gb300.paged import PagedCache

    cache = PagedCache(1, 3, 4, 8, 1, 64)
    cache.grow(i32([60, 0, 120]))
    before = cache.page_table.clone(), cache.ref_count.clone()
    count, token, parent = i32([9, 9, 9]), i32(np.ones((3, 9))), i32(random_trees(np.random.default_rng(0), [9] * 3, 9))
    for bad in (dict(token=token.long()), dict(token=token.cpu()), dict(token=token.t().contiguous().t()),
                dict(parent=parent.long()), dict(parent=parent[:, :8].contiguous()), dict(parent=parent[:2]),
                dict(count=count.long()), dict(count=count[:1]), dict(rows=-1)):
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            cache.draft(**{**dict(count=count, token=token, parent=parent), **bad})
        assert torch.equal(cache.page_table, before[0]) and torch.equal(cache.ref_count, before[1]), bad
    d = cache.draft(count, token, parent)
    assert (d.cache_pos >= 0).all() and int(cache.dev_err) == 0
    cache.drop(d)
    assert torch.equal(cache.page_table, before[0]) and torch.equal(cache.ref_count, before[1])


@pytest.mark.parametrize("bad", ["none", "source", "behind the pool", "destination", "not moved", "all"])
@pytest.mark.parametrize("req,most", [(1, 70), (5, 64), (30, 200)])
def test_move_reports_pages(draft, req, most, bad):
    """CI_DEVERR_PAGE where a position that moves has no page at one of its ends, and only there; it stays as it is."""
    rng = np.random.default_rng(req + most)
    gen = torch.Generator().manual_seed(req)
    length = rng.integers(0, 200, req)
    length[0] = 60
    table, pages = make_table(gen, [int(n) + most for n in length])
    table = table.numpy().copy()
    count, path = np.zeros(req, int), np.full((req, most), -1)
    for r in range(req):
        path[r, :8] = [0, 1, 4, 5, 9, 30, most - 2, most - 1]
        count[r] = 8
    # of the first request: positions 60, 61 stay; 64, 65, 69, 90, 58 + most, 59 + most go to 62 .. 67
    if bad in ("source", "all"):
        table[0, (60 + most - 1) // 64] = -1
    if bad == "behind the pool":
        table[0, (60 + most - 1) // 64] = pages
    if bad in ("destination", "all"):
        table[0, 0] = -5
    if bad == "not moved":
        table[0, (60 + most - 1) // 64], count[0] = -1, 2  # (the first two stay where they are)
    if bad == "all":
        table[:] = np.where(rng.random(table.shape) < 0.3, pages + 3, table)
    err = 0
    for r in range(req):
        for d in range(count[r]):
            ends = (length[r] + path[r, d], length[r] + d)
            if ends[0] != ends[1] and any(not 0 <= table[r, s // 64] < pages for s in ends):
                err = PAGE_ERR
    assert err == (0 if bad in ("none", "not moved") else PAGE_ERR)
    pool = torch.randint(0, 256, (pages, 2, 64 * 20), generator=gen, dtype=torch.int32).to(torch.uint8)
    got, bits = pool.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    draft.ci_slots_move([got], 16, 4, i32(table), i32(length), i32(path), i32(count), dev_err=bits)
    np.testing.assert_array_equal(got.cpu().numpy(), D.move(pool.numpy(), 16, 4, table, length, path, count))
    assert int(bits) == err


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kind", ["tree", "chain"])
def test_attention_fp8_queries_with_a_large_dim(draft, kind, d):
    """One dim of every query 64 times as large, over keys like any: logits as close as without it."""
    p = Drafted([300, 0, 1, 700], [20, 5, 1, 9], 16, 2, d, FP8, kind, seed=d, gain=0.3)
    p.q[..., 37] *= 64
    p.check(*p.run(draft))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("far", [-110, -118, -119, -121, -126, -130])
def test_attention_fp8_tiny_queries(draft, far, d):
    """Queries of about 2^far under a scale that makes ordinary logits of them: off by what is left out of elements, at
    most 2^-21 of the row's largest or of 2^-119."""
    p = Drafted([200, 3], [6, 2], 4, 1, d, FP8, "chain", seed=-far)
    p.q = (p.q.double() * 2.0 ** far).to(torch.bfloat16)
    p.scale = 2.0 ** (-far - 4) if far > -123 else 2.0 ** 119
    out, lse = p.run(draft)
    assert int(p.err) == 0
    kv, table = C.page_values(p.k.numpy(), d), p.table.numpy()
    for r in range(2):
        for i in range(p.nodes[r]):
            t, at = p.starts[r] + i, np.arange(p.lens[r] + i + 1)
            k = kv[table[r, at // 64], 0, at % 64]
            q = p.q[t].double().numpy()
            x = p.scale * q @ k.T
            size = p.scale * np.abs(q) @ np.abs(k).T
            top = np.maximum(np.abs(q).max(-1, keepdims=True), 2.0 ** -119)
            left = np.where(np.abs(q) >= 2.0 ** -13 * top, 0, 2.0 ** -21 * top)
            dx = ((d + 8) * 2.0 ** -23 * size + p.scale * left @ np.abs(k).T).max(-1)
            z = np.log(np.exp(x - x.max(-1, keepdims=True)).sum(-1)) + x.max(-1)
            ztol = dx + (len(at) + 64) * 2.0 ** -23 + 2.0 ** -21 * (np.abs(z) + 1)
            assert (np.abs(lse[t].double().cpu().numpy() - z) <= ztol).all(), (r, i)

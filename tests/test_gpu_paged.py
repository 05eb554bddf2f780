"""The paged cache's calls together (two_level_sparse_gb300/paged.py), and the
attention where many heads share a key-value head, on many rows, in far pages
and from a graph.  Tolerances as in test_gpu_cache.py, whose helpers are used."""
import math

import numpy as np
import pytest
import torch

from oracle import cache_oracle as C
from test_gpu_cache import BF16, DEC, FP8, PRE, VAR, Problem, cos_sin, i32, picks

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def cache():
    from two_level_sparse_gb300 import cache as mod

    return mod


def check_rows(out, q, k_pool, v_pool, table, positions, d, rows, err=2.0 ** -8):
    """Rows of a device result against the oracle over the pools as they are."""
    kv, vv = (C.page_values(p.cpu().numpy(), d) for p in (k_pool, v_pool))
    table = table.cpu().numpy()
    out = out.double().cpu().numpy()
    q = C.bf16_values(q.cpu().view(torch.int16).numpy().view(np.uint16))
    for t, r in rows:
        at = np.asarray(positions(t), dtype=int)
        page, slot = table[r, at // 64], at % 64
        want, _, mag, size = C.attention(q[t], kv[page, :, slot], vv[page, :, slot], d ** -0.5)
        soft = 2 * np.expm1((d + 8) * 2.0 ** -23 * size) + (len(at) + 64) * 2.0 ** -23
        tol = err * (np.abs(want) + mag) * (1 + 2.0 ** -6) + 2 * soft[:, None] * mag + 1e-30
        assert (np.abs(out[t] - want) <= tol).all(), (t, np.abs(out[t] - want).max())


@pytest.mark.parametrize("fmt", [BF16, FP8])
@pytest.mark.parametrize("hq,hkv", [(16, 4), (64, 1)])
def test_serving(fmt, hq, hkv):
    """Prompts, a fork, decode steps over the indexer's positions, a release and a compaction."""
    from two_level_sparse_gb300 import synth
    from two_level_sparse_gb300.paged import PagedCache, sparse_decode_step
    from two_level_sparse_gb300.step import IndexerStep

    d, layers, steps = 128, 2, 3
    gen = torch.Generator(device="cuda").manual_seed(hq + fmt)
    prompts = [700, 61, 1300]
    end = [n + steps + 1 for n in (700, 61, 1300, 700, 1290)] + [0]
    wl = synth.make_workload("paged", synth.LAYOUT_DECODE, torch.tensor(end), topk_blocks=64, seed=3, layers=layers,
                             device="cuda")
    cache = PagedCache(layers, len(end), wl.page_table.shape[1], wl.num_pages, hkv, d, fmt,
                       companions=[ly.k_pool for ly in wl.layers])
    step = IndexerStep(wl)  # its buffers are for the lengths to come
    wl.page_table, wl.seq_len = cache.page_table, cache.length
    norm = 1 + 0.1 * torch.randn(d, device="cuda", generator=gen)
    cs = cos_sin(max(end), 64).cuda()

    def tokens(n):
        return torch.randn(n, hq + 2 * hkv, d, device="cuda", generator=gen).bfloat16()

    cache.grow(i32(prompts + [0, 0, 0]))
    for r, n in enumerate(prompts):
        at = torch.arange(n, device="cuda", dtype=torch.int32)
        starts = i32([0] * (r + 1) + [n] * (len(end) - r))
        for j in range(layers):
            x = tokens(n)
            q = cache.append(j, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], norm, norm, 1e-6, cs, True, at, VAR,
                             req_start=starts)
            out = cache.attend(j, q, VAR, at + 1, n, req_start=starts)
            check_rows(out, q, cache.k[j], cache.v[j], cache.page_table, lambda t: range(t + 1), d,
                       [(t, r) for t in (0, 1, 60, n - 1)])
    cache.fork(i32([0, 2]), i32([3, 4]), i32([700, 1290]))
    assert cache.page_table[3, :10].tolist() == cache.page_table[0, :10].tolist()
    for s in range(steps):
        cache.grow(torch.where(cache.length > 0, cache.length + 1, 0).to(torch.int32))
        qkv = [tokens(len(end)) for _ in range(layers)]
        outs = sparse_decode_step(cache, step, qkv, norm, norm, 1e-6, cs)
        cache.check()
        for j, x in enumerate(qkv):
            lens = cache.length.tolist()
            assert lens == [n + s + 1 for n in (700, 61, 1300, 700, 1290)] + [0]
            last = (cache.length - 1).clamp(min=0)
            q = torch.empty_like(x[:, :hq])
            kv = [torch.zeros_like(cache.k[j]) for _ in range(2)]
            from two_level_sparse_gb300 import cache as ops
            ops.ci_qk_norm_rope_append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], norm, norm, 1e-6, cs, True, last,
                                       q, *kv, cache.page_table, DEC, cache_pos=cache.length - 1)
            pos = step.pos[j].cpu().numpy()
            assert (pos[5] == -1).all() and (outs[j][5] == 0).all()
            check_rows(outs[j], q, cache.k[j], cache.v[j], cache.page_table, lambda t: pos[t][pos[t] >= 0], d,
                       [(t, t) for t in range(5)])
            for t in range(5):  # the new token's entry is where the row's last position is
                page, slot = int(cache.page_table[t, (lens[t] - 1) // 64]), (lens[t] - 1) % 64
                for got, want in ((cache.k[j], kv[0]), (cache.v[j], kv[1])):
                    w = d * (1 if fmt else 2)
                    assert torch.equal(got[page, :, slot * w:][:, :w], want[page, :, slot * w:][:, :w])
    # the same queries before and after the pages move
    before = [cache.attend(j, q, DEC, cache.length, step.max_len, pos=step.pos[j]) for j in range(layers)]
    cache.free(i32([0, 1]))
    cache.compact()
    cache.check()
    live = int((cache.ref_count > 0).sum())
    assert (cache.ref_count[:live] > 0).all() and live < wl.num_pages
    after = [cache.attend(j, q, DEC, cache.length, step.max_len, pos=step.pos[j]) for j in range(layers)]
    for a, b in zip(before, after):
        assert torch.equal(a[2:], b[2:]) and (b[:2] == 0).all()
    pos = step.pos.clone()
    step.run()  # the indexer's keys moved along
    torch.cuda.synchronize()
    assert torch.equal(step.pos[:, 2:], pos[:, 2:])


def test_example_runs(capsys):
    from two_level_sparse_gb300 import paged

    paged.main()
    assert "lengths [0, 0, 9005, 5004, 9005, 0]" in capsys.readouterr().out


@pytest.mark.parametrize("hq,hkv", [(64, 1), (40, 2)])
def test_many_heads_ignore_what_lies_outside(cache, hq, hkv):
    lens = [70, 1, 130, 0, 256, 300]
    for pos in (None, [[0, 69, -1, 3], [0, -1, -1, -1], [129, 64, 63, -1], [-1] * 4, [255, -1, -1, 0], [5, 6, 7, 8]]):
        p = Problem(lens, hq, hkv, 128, BF16, pos=pos, seed=8)
        clean = p.run(cache)
        p.check(*clean)
        for pool in (p.k, p.v):
            used = torch.zeros(pool.shape[0], 64, dtype=torch.bool)
            for t, n in enumerate(lens):
                for s in C.row_positions(n, n, None if pos is None else pos[t]):
                    used[p.table[t, s // 64], s % 64] = True
            pool.unflatten(-1, (64, 256)).transpose(1, 2)[~used] = 0xFF
        dirty = p.run(cache)
        for a, b in zip(clean, dirty):
            assert torch.equal(a, b)


def test_many_heads_pass_on_what_is_not_finite(cache):
    p = Problem([200, 200, 200], 40, 2, 128, BF16, seed=9)
    k, v = (x.view(torch.bfloat16).unflatten(-1, (64, 128)) for x in (p.k, p.v))
    k[p.table[0, 1], 1, 7, 3] = math.nan
    v[p.table[1, 0], 0, 9, 5] = math.inf
    k[p.table[2, 0], 0, 0] = 0  # the first position's key: its logit is NaN for all heads
    k[p.table[2, 0], 0, 0, 0] = math.nan
    out, lse = p.run(cache)
    assert out[0, 20:].isnan().all() and lse[0, 20:].isnan().all()
    assert out[0, :20].isfinite().all() and lse[0, :20].isfinite().all()
    assert (out[1, :20, 5] == math.inf).all() and out[1, :20, :5].isfinite().all() and out[1, 20:].isfinite().all()
    assert out[2, :20].isnan().all() and out[2, 20:].isfinite().all()


@pytest.mark.parametrize("gain", [60.0, 400.0])
def test_many_heads_large_logits(cache, gain):
    """Logits hundreds to thousands apart: references are passed again and again, in any order of the heads."""
    p = Problem([700, 64, 3000, 1], 64, 1, 128, BF16, seed=10, gain=gain)
    p.check(*p.run(cache))
    rng = np.random.default_rng(1)
    lens = [700, 64, 3000, 1]
    p = Problem(lens, 64, 1, 128, BF16, seed=10, gain=gain, pos=picks(rng, lens, 300))
    p.check(*p.run(cache))
    for p.scale in (0.0, -0.01):
        p.check(*p.run(cache))


@pytest.mark.parametrize("hq,fmt", [(32, BF16), (8, BF16), (8, FP8)])
def test_many_rows(cache, hq, fmt):
    """More rows than workers: many segments for each, whole rows and parts in turn."""
    rng = np.random.default_rng(2)
    lens = [int(n) for n in rng.integers(0, 300, 1300)]
    lens[7], lens[8], lens[1299] = 0, 300, 1
    p = Problem(lens, hq, 1, 128, fmt, layout=PRE, seed=5)
    p.check(*p.run(cache))
    p = Problem(lens, hq, 1, 128, fmt, layout=PRE, seed=5, pos=picks(rng, lens, 140))
    p.check(*p.run(cache))


@pytest.mark.parametrize("hq,d,fmt", [(8, 128, BF16), (64, 128, BF16), (8, 256, FP8)])
def test_far_pages(cache, hq, d, fmt):
    """Pages whose bytes lie beyond 2^32, and a page table of another order, give the same bits."""
    lens = [300, 64, 1]
    for pos in (None, picks(np.random.default_rng(3), lens, 100)):
        p = Problem(lens, hq, 1, d, fmt, seed=6, pos=pos)
        near = p.run(cache)
        nb = p.k.shape[-1]
        pages = 2 ** 32 // nb + 64
        ids = torch.arange(p.k.shape[0]) * 7 + pages - 7 * p.k.shape[0]
        big = [torch.empty(pages, 1, nb, dtype=torch.uint8, device="cuda") for _ in range(2)]
        for b, x in zip(big, (p.k, p.v)):
            b[ids.cuda()] = x.cuda()
        table = torch.where(p.table >= 0, ids[p.table.clamp(min=0).long()].to(torch.int32), -1)
        out, lse = torch.empty_like(near[0]), torch.empty_like(near[1])
        g = None if p.pos is None else p.pos.cuda()
        cache.ci_attn_decode(p.q.cuda(), *big, table.cuda(), DEC, p.seq.cuda(), p.max_len, p.scale, out, lse=lse,
                             pos=g)
        assert torch.equal(out, near[0]) and torch.equal(lse, near[1])
        x = torch.randn(3, hq + 2, d, device="cuda").bfloat16()
        q_out = torch.empty(3, hq, d, dtype=torch.bfloat16, device="cuda")
        one = [torch.zeros_like(p.k, device="cuda") for _ in range(2)]
        for pools, tab in ((one, p.table), (big, table)):
            cache.ci_qk_norm_rope_append(x[:, :hq], x[:, hq:hq + 1], x[:, hq + 1:], None, None, 1e-6,
                                         cos_sin(300, 64).cuda(), True, i32([299, 63, 0]), q_out, *pools, tab.cuda(),
                                         DEC)
        row = d * (1 if fmt else 2)
        for a, b in zip(one, big):
            for t, s in enumerate((299, 63, 0)):
                at = int(p.table[t, s // 64])
                s = s % 64 * row
                assert torch.equal(a[at, 0, s:s + row], b[int(ids[at]), 0, s:s + row])
        cache.ci_pages_copy(big, i32([int(ids[0])]), i32([pages - 1]))
        assert all(torch.equal(b[pages - 1], b[int(ids[0])]) for b in big)


@pytest.mark.parametrize("hq", [8, 64])
def test_from_a_graph(cache, hq):
    """Append and attention captured once, replayed over other lengths and tokens."""
    p = Problem([400, 30, 129], hq, 1, 128, BF16, seed=14)
    g = {n: getattr(p, n).cuda() for n in ("k", "v", "table", "seq")}
    x = torch.randn(3, hq + 2, 128, device="cuda").bfloat16()
    norm, cs = torch.ones(128, device="cuda"), cos_sin(400, 128).cuda()
    q, out = (torch.empty(3, hq, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.empty(cache.attn_workspace_bytes(3, hq, 1, 128), dtype=torch.uint8, device="cuda")

    last = torch.empty_like(g["seq"])

    def work():
        torch.sub(g["seq"], 1, out=last)
        cache.ci_qk_norm_rope_append(x[:, :hq], x[:, hq:hq + 1], x[:, hq + 1:], norm, norm, 1e-6, cs, True, last, q,
                                     g["k"], g["v"], g["table"], DEC)
        cache.ci_attn_decode(q, g["k"], g["v"], g["table"], DEC, g["seq"], 400, p.scale, out, workspace=ws)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        work()
    for n in ([400, 30, 129], [1, 2, 64], [333, 5, 128]):
        g["seq"].copy_(i32(n))
        x.copy_(torch.randn(3, hq + 2, 128, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        work()
        torch.cuda.synchronize()
        assert torch.equal(got, out)
        check_rows(got, q, g["k"], g["v"], g["table"], lambda t: range(n[t]), 128, [(t, t) for t in range(3)])


@pytest.mark.parametrize("fmt", [BF16, FP8])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("hq", [8, 80])
def test_nan_reaches_the_reader(cache, hq, what, fmt):
    """A NaN in a new token's key or value shows in its heads' attention, whatever the format, and in no other's."""
    d, n = 128, 3
    x = torch.randn(n, hq + 4, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    x[1, hq + (0 if what == "k" else 2), 5] = math.nan
    pools = [torch.zeros(1, 2, cache.page_bytes(fmt, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    q, out = (torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table, at = i32([[0]]), i32([0, 1, 2])
    cache.ci_qk_norm_rope_append(x[:, :hq], x[:, hq:hq + 2], x[:, hq + 2:], None, None, 1e-6, cos_sin(4, 0).cuda(), True,
                                 at, q, *pools, table, PRE)
    cache.ci_attn_decode(q, *pools, table, PRE, at + 1, 64, d ** -0.5, out)
    assert out[0].isfinite().all() and out[1:, hq // 2:].isfinite().all()
    if what == "k" or fmt == FP8:
        assert out[1:, :hq // 2].isnan().all()
    else:
        assert out[1:, :hq // 2, 5].isnan().all()

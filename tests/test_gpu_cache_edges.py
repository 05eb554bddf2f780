"""The paged cache's kernels at the edges of what they promise: other work on
the card, values and logits near the ends of their ranges, non-finite heads.
Helpers and tolerances as in test_gpu_cache.py."""
import numpy as np
import pytest
import torch

from test_gpu_cache import BF16, FP8, PRE, Problem, cos_sin, picks

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.fixture(scope="module")
def cache():
    from two_level_sparse_gb300 import cache as mod

    return mod


@pytest.mark.parametrize("listed", [False, True])
@pytest.mark.parametrize("hq", [64, 8])
def test_attention_beside_other_work(cache, hq, listed):
    """More units than workers while another stream's products hold some of the SMs, so that CTAs start at
    different times: every row is written, with the bits of a quiet run."""
    rng = np.random.default_rng(7)
    lens = [int(n) for n in rng.integers(0, 500, 1300)]
    p = Problem(lens, hq, 1, 128, BF16, layout=PRE, seed=15, pos=picks(rng, lens, 300) if listed else None)
    out, lse = p.run(cache)
    p.check(out, lse)
    g = {n: getattr(p, n).cuda() for n in ("q", "k", "v", "table", "seq")}
    pos = p.pos.cuda() if listed else None
    res = [(torch.full_like(out, float("nan")), torch.full_like(lse, float("nan"))) for _ in range(12)]
    ws = torch.full((cache.attn_workspace_bytes(1300, hq, 1, 128),), 0xFF, dtype=torch.uint8, device="cuda")
    a = torch.randn(4096, 4096, device="cuda").bfloat16()
    b, side = torch.empty_like(a), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(40):
            torch.matmul(a, a, out=b)
    for o, z in res:
        cache.ci_attn_decode(g["q"], g["k"], g["v"], g["table"], PRE, g["seq"], p.max_len, p.scale, o, lse=z, pos=pos,
                             workspace=ws)
    torch.cuda.synchronize()
    for o, z in res:
        assert torch.equal(o, out) and torch.equal(z, lse)


@pytest.mark.parametrize("hq", [64, 8])
def test_attention_on_another_stream(cache, hq):
    """A call on a stream that is not the current one, with no workspace given, while the current stream
    allocates and writes the same amounts of memory."""
    from two_level_sparse_gb300.paged import PagedCache

    p = Problem([20000, 1, 9000, 0], hq, 1, 128, BF16, seed=21)
    out, lse = p.run(cache)
    p.check(out, lse)
    g = [getattr(p, n).cuda() for n in ("q", "k", "v", "table", "seq")]
    c = PagedCache(1, 4, g[3].shape[1], g[1].shape[0], 1, 128)
    c.k[0].copy_(g[1]), c.v[0].copy_(g[2]), c.page_table.copy_(g[3])
    n, side = cache.attn_workspace_bytes(4, hq, 1, 128), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        o = torch.empty_like(out)
        side.wait_stream(torch.cuda.current_stream())
        cache.ci_attn_decode(*g[:4], 0, g[4], p.max_len, p.scale, o, stream=side)
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF)
        got += [o, c.attend(0, g[0], 0, g[4], p.max_len, p.scale, stream=side)]
        torch.empty(out.numel(), dtype=torch.bfloat16, device="cuda").fill_(7)
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in got)


@pytest.mark.parametrize("hq", [64, 8])
@pytest.mark.parametrize("logit", [11.0, 16.5, 27.0, 28.0])
def test_attention_largest_values(cache, hq, logit):
    """Values of 2^80, the most that is promised, under hundreds of equal logits far above the first one's."""
    n = 700
    p = Problem([n] * 700, hq, 1, 128, BF16, layout=PRE, seed=17)
    p.scale = 1.0
    p.q.zero_()
    p.q[:, :, 0] = 1.0
    k = p.k.view(torch.bfloat16).unflatten(-1, (64, 128))
    k.zero_()
    k[..., 0] = logit
    k[p.table[0, 0], 0, 0, 0] = 0
    p.v.view(torch.bfloat16).fill_(2.0 ** 80)
    out, lse = p.run(cache)
    assert ((out.double() / 2.0 ** 80 - 1).abs() <= 2.0 ** -8).all()
    want = np.log(1 + (n - 1) * np.exp(logit))
    assert ((lse.double() - want).abs() <= (n + 64) * 2.0 ** -23 + 2.0 ** -21 * (want + 1) + 136 * 2.0 ** -23 * logit).all()


@pytest.mark.parametrize("hq", [64, 8])
def test_attention_rising_logits(cache, hq):
    """Logits that rise through a row in steps of every size: each passes what the ones before were kept against."""
    rng = np.random.default_rng(18)
    lens = [3000, 700, 129, 64]
    for step in (0.01, 0.1, 1.0, 20.0):
        p = Problem(lens, hq, 1, 128, BF16, seed=18)
        p.scale = 1.0
        k = p.k.view(torch.bfloat16).unflatten(-1, (64, 128))
        p.q.normal_(generator=torch.Generator().manual_seed(2))
        k.mul_(0.05)
        p.q[:, :, 0] = torch.from_numpy(rng.choice([1.0, -1.0, 2.0], size=(4, hq))).to(torch.bfloat16)
        for t, n in enumerate(lens):
            s = torch.arange(n)
            k[p.table[t, s // 64].long(), 0, s % 64, 0] = (step * s).bfloat16()
        p.check(*p.run(cache))


@pytest.mark.parametrize("hq", [64, 8])
@pytest.mark.parametrize("power", [40, 60, 80, 100, 110])
@pytest.mark.parametrize("sign", [1, -1])
def test_attention_huge_logits(cache, hq, power, sign):
    """Logits of whole numbers times 2^power, both signs, one position ahead of all others: the result is its
    value, to the bit, and lse its logit."""
    d, lens, group = 128, [1, 64, 700, 3000, 129], hq
    p = Problem(lens, hq, 1, d, BF16, seed=16)
    p.scale = 0.75
    p.q.zero_()
    p.q[:, :, 0] = 2.0 ** (power // 2)
    k = p.k.view(torch.bfloat16).unflatten(-1, (64, d))
    v = p.v.view(torch.bfloat16).unflatten(-1, (64, d))
    k.zero_()
    rng = np.random.default_rng(power)
    best = []
    for t, n in enumerate(lens):
        best.append(int(rng.integers(0, n)))
        s = np.arange(n)
        size = torch.from_numpy(rng.integers(2, 100, n).astype(np.float32))
        size[best[t]] = 1 if sign < 0 else 101
        k[p.table[t, s // 64].long(), 0, torch.from_numpy(s % 64), 0] = (sign * size * 2.0 ** (power - power // 2)).bfloat16()
    out, lse = p.run(cache)
    out, lse = out.cpu(), lse.double().cpu()
    for t, s in enumerate(best):
        want = v[p.table[t, s // 64], 0, s % 64]
        z = p.scale * sign * (1 if sign < 0 else 101) * 2.0 ** power
        assert torch.equal(out[t], want.expand(group, d)), (t, s)
        assert ((lse[t] - z).abs() <= 2.0 ** -20 * abs(z)).all()


def codes_of(x):
    """e4m3 codes and scales of bf16 heads [..., d], by fp32 division."""
    x = x.float().numpy()
    scale = np.maximum(np.abs(x).max(-1), np.float32(1e-10)) / np.float32(448)
    with np.errstate(invalid="ignore"):
        y = torch.from_numpy(x / scale[..., None])
    return y.to(torch.float8_e4m3fn).view(torch.uint8).numpy(), scale


def append_raw(cache, x, d):
    """Keys and values x [tokens, 2, d] as they are into FP8 pages: the codes and scales of both."""
    n = x.shape[0]
    pools = [torch.zeros(-(-n // 64), 1, cache.page_bytes(FP8, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    g, table = x.cuda(), torch.arange(-(-n // 64), dtype=torch.int32, device="cuda")[None]
    cache.ci_qk_norm_rope_append(g[:, :1], g[:, :1], g[:, 1:], None, None, 1e-6, cos_sin(n, 0).cuda(), True,
                                 torch.arange(n, dtype=torch.int32, device="cuda"), torch.empty_like(g[:, :1]), *pools,
                                 table, PRE)
    body = [p[:, 0, :64 * d].reshape(-1, d)[:n].cpu().numpy() for p in pools]
    scale = [p[:, 0, 64 * d:].contiguous().view(torch.float32).reshape(-1)[:n].cpu().numpy() for p in pools]
    return body, scale


def test_append_codes_are_a_divisions(cache):
    """The codes that a reciprocal and its correction give are those of an IEEE division, over all sizes of heads."""
    gen = torch.Generator().manual_seed(19)
    x = torch.randn(20000, 2, 128, generator=gen)
    x *= 2.0 ** (torch.rand(20000, 2, 1, generator=gen) * 200 - 90)
    x[:300] = torch.randint(-448, 449, (300, 2, 128), generator=gen).float()  # many exact ties
    x = x.bfloat16()
    body, scale = append_raw(cache, x, 128)
    for i in range(2):
        want, z = codes_of(x[:, i])
        assert np.array_equal(scale[i], z)
        assert np.array_equal(body[i], want)


def test_append_infinite_heads(cache):
    """FP8: x / scale with an infinite scale is 0 where x is finite, NaN where it is not."""
    x = torch.randn(6, 2, 64, generator=torch.Generator().manual_seed(20)).bfloat16()
    x[1, 0, 5] = x[2, 1, 9] = x[3, :, 0] = float("inf")
    x[4, :, 63] = -float("inf")
    x[4, :, 7] = float("nan")
    body, scale = append_raw(cache, x, 64)
    for i in range(2):
        for t in range(6):
            head = x[t, i].float()
            codes = body[i][t] & 0x7F
            if head.isnan().any():
                assert np.isnan(scale[i][t])
            elif head.isinf().any():
                assert np.isposinf(scale[i][t])
                assert np.array_equal(codes == 0x7F, head.isinf().numpy()) and (codes[head.isfinite().numpy()] == 0).all()
            else:
                want, z = codes_of(x[t, i])
                assert np.array_equal(body[i][t], want) and scale[i][t] == z


@pytest.mark.parametrize("fmt", [BF16, FP8])
@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 128), (12, 1, 64), (17, 1, 128), (64, 2, 128), (40, 1, 128), (128, 1, 128),
                                      (8, 1, 256), (60, 2, 256), (33, 1, 64)])
def test_attention_keeps_to_its_workspace(cache, hq, hkv, d, fmt):
    """The bytes that are asked for, between bytes that stay as they are."""
    rng = np.random.default_rng(22)
    lens = [int(n) for n in rng.integers(1, 700, 40)]
    n, guard = cache.attn_workspace_bytes(40, hq, hkv, d), 64 << 20
    ws = torch.full((n + 2 * guard,), 0x5A, dtype=torch.uint8, device="cuda")
    for pos in (None, picks(rng, lens, 200)):
        p = Problem(lens, hq, hkv, d, fmt, seed=22, pos=pos)
        p.check(*p.run(cache, workspace=ws[guard:guard + n]))
    assert (ws[:guard] == 0x5A).all() and (ws[guard + n:] == 0x5A).all()


@pytest.mark.parametrize("hq", [64, 8])
def test_attention_on_two_streams_at_once(cache, hq):
    """Calls that overlap, from two threads, each with its own workspace: the bits of calls one after another."""
    import threading

    problems = [Problem([30000 + n, 1, 5000], hq, 1, 128, BF16, seed=23 + n) for n in (0, 1)]
    want = [p.run(cache) for p in problems]
    got, sides = [[], []], [torch.cuda.Stream() for _ in problems]
    args = [[getattr(p, n).cuda() for n in ("q", "k", "v", "table", "seq")] for p in problems]
    torch.cuda.synchronize()

    def work(i):
        with torch.cuda.stream(sides[i]):
            for _ in range(30):
                o, z = torch.empty_like(want[i][0]), torch.empty_like(want[i][1])
                cache.ci_attn_decode(*args[i][:4], 0, args[i][4], problems[i].max_len, problems[i].scale, o, lse=z)
                got[i].append((o, z))

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i in (0, 1):
        assert len(got[i]) == 30
        assert all(torch.equal(o, want[i][0]) and torch.equal(z, want[i][1]) for o, z in got[i])


@pytest.mark.parametrize("fmt", [BF16, FP8])
def test_views_of_larger_tensors(cache, fmt):
    """Pools, tables and lists that are slices of larger tensors, as layers of one allocation are."""
    rng = np.random.default_rng(24)
    lens = [700, 3, 129]
    p = Problem(lens, 8, 2, 128, fmt, seed=24, pos=picks(rng, lens, 100))
    want = p.run(cache)

    def inside(t):
        x = torch.full((3, *t.shape), 0x55, dtype=t.dtype, device="cuda")
        x[1] = t.cuda()
        return x[1]

    out = torch.empty_like(want[0])
    cache.ci_attn_decode(inside(p.q), inside(p.k), inside(p.v), inside(p.table), 0, inside(p.seq), p.max_len, p.scale, out,
                         pos=inside(p.pos))
    torch.cuda.synchronize()
    assert torch.equal(out, want[0])
    pools = torch.randint(0, 256, (4, 5, 64), dtype=torch.uint8, device="cuda")
    before = pools.clone()
    one = lambda v: torch.tensor([v], dtype=torch.int32, device="cuda")  # noqa: E731
    cache.ci_pages_copy(pools[1::4], one(0), one(4))
    before[1, 4] = before[1, 0]
    assert torch.equal(pools, before)

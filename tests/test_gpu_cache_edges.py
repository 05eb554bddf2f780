"""The paged cache's kernels at the edges of what they promise: other work on
the card, values and logits near the ends of their ranges, non-finite heads.
Helpers and tolerances as in test_gpu_cache.py."""
import numpy as np
import pytest
import torch

from test_gpu_cache import BF16, PRE, Problem, picks

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

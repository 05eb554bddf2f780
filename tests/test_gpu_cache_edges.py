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

"""A served model's paged cache: the entry points of ``cache`` put together.

``PagedCache`` owns what several of the calls share -- every layer's key and
value pool, the page table, the reference counts, the lengths, the attention's
workspace -- and strings the calls together: a fork is the release of what the
child held, the shared pages and the copy of the partly filled ones; a
compaction is the moves and their copies.  Pools of the same page ids that
others fill (the indexer's keys) are copied along as ``companions``.

``sparse_decode_step`` is one decode step of the layers behind the indexer:
the new tokens' keys and values into every layer's pages, the indexer's
positions (``step.IndexerStep``), every layer's attention over its positions.

``python -m two_level_sparse_gb300.paged`` serves a few synthetic requests:
prompts, a fork, decode steps, a release and a compaction.

As in ``step``, this module allocates buffers and marshals arguments; the
computation runs in libci.so.
"""
from __future__ import annotations

import torch

from . import cache as ops

_I32 = torch.int32


class PagedCache:
    """``layers`` attention layers' keys and values for ``requests`` requests
    of up to ``64 * max_pages`` positions, in ``num_pages`` pages (every
    layer's pools use the same ids).  All lengths and ids that the methods take
    are int32 tensors on the cache's device; nothing but ``check`` waits.
    ``length`` [requests] is what every request holds; ``short`` is 1 where its
    last growth or fork got less than it asked for.
    ``append`` and ``attend`` run on ``stream`` (None: the current one), whose
    memory their results are."""

    def __init__(self, layers: int, requests: int, max_pages: int, num_pages: int, kv_heads: int, head_dim: int,
                 cache_format: int = ops.CACHE_BF16, companions=(), device="cuda"):
        shape = (layers, num_pages, kv_heads, ops.page_bytes(cache_format, head_dim))
        self.head_dim = head_dim
        self.k = torch.zeros(shape, dtype=torch.uint8, device=device)
        self.v = torch.zeros(shape, dtype=torch.uint8, device=device)
        self.companions = list(companions)
        self.page_table = torch.full((requests, max_pages), -1, dtype=_I32, device=device)
        self.ref_count = torch.zeros(num_pages, dtype=_I32, device=device)
        # one column more than there are requests, for what is said of others
        self._state = torch.zeros(2, requests + 1, dtype=_I32, device=device)
        self.length, self.short = self._state[:, :requests]
        self._column = torch.arange(max_pages, dtype=_I32, device=device)
        self.dev_err = torch.zeros(1, dtype=_I32, device=device)
        self._pairs = torch.empty(3, num_pages, dtype=_I32, device=device)  # remap, copy_src, copy_dst
        self._count = torch.empty(1, dtype=_I32, device=device)
        self._workspace = {}

    def _copy(self, src, dst, count=None):
        pools = [*self.k, *self.v, *self.companions]
        for at in range(0, len(pools), ops.MAX_POOLS):
            ops.ci_pages_copy(pools[at:at + ops.MAX_POOLS], src, dst, count=count, dev_err=self.dev_err)

    def _limit(self):
        return ops.PAGE * self.page_table.shape[1]

    def _room(self, rows):
        """The positions for which rows of the page table have pages, from the first on."""
        return ops.PAGE * torch.where(rows < 0, self._column, self._column.shape[0]).amin(1)

    def grow(self, new_len):
        """Pages up to ``new_len`` [requests] positions; a request that is not to grow has its present length.
        Where the pages run out the length goes as far as they do, where the call refuses (fewer positions than
        there are, or more than a row has) it stays; either is ``short`` then, and in ``dev_err``."""
        ops.ci_pages_alloc(self.page_table, self.ref_count, self.length, new_len, dev_err=self.dev_err)
        asked = torch.where(new_len <= self._limit(), new_len, 0)
        torch.maximum(self.length, torch.minimum(asked, self._room(self.page_table)), out=self.length)
        self.short.copy_(self.length != new_len)

    def _known(self, req):
        return (req >= 0) & (req < self.length.shape[0])

    def _at(self, req, known):
        """Where ``_state`` has the requests; its last column where they are not known."""
        return torch.where(known, req, self.length.shape[0]).long()

    def fork(self, parent, child, length):
        """``child[i]`` becomes the first ``length[i]`` positions of ``parent[i]``; what it held is released.
        A fork that the call refuses (its bits are in ``dev_err``) leaves both as they are; a child without a page
        for its end is ``short`` of it."""
        done = self._known(parent) & self._known(child) & (parent != child)
        done &= (length >= 0) & (length <= self._limit())
        child_done = torch.where(done, child, -1)
        bits = torch.zeros_like(self.dev_err)
        ops.ci_pages_free(self.page_table, self.ref_count, child_done, dev_err=bits)
        self.dev_err |= bits & ~ops.DEVERR_REQ  # (the fork itself says which requests are bad)
        src, dst = torch.empty_like(parent), torch.empty_like(parent)
        ops.ci_pages_fork(self.page_table, self.ref_count, parent, child, length, src, dst, dev_err=self.dev_err)
        self._copy(src, dst)
        at = self._at(child, done)
        got = torch.minimum(length, self._room(self.page_table[at.clamp(max=self.length.shape[0] - 1)]))
        self._state.index_copy_(1, at, torch.stack([got, (got != length).to(_I32)]))

    def free(self, req):
        ops.ci_pages_free(self.page_table, self.ref_count, req, dev_err=self.dev_err)
        self._state.index_fill_(1, self._at(req, self._known(req)), 0)

    def compact(self):
        """Every live page into the lowest ids."""
        remap, src, dst = self._pairs
        ops.ci_pages_compact(self.page_table, self.ref_count, remap, src, dst, self._count, dev_err=self.dev_err)
        self._copy(src, dst, self._count)

    def append(self, layer, q, k, v, q_norm, k_norm, eps, cos_sin, is_neox, positions, layout, q_out=None, stream=None,
               **kw):
        """The new tokens' keys and values into their pages; returns the normed and rotated queries."""
        q_out = ops.empty_on(stream, q.shape, q.dtype, q.device) if q_out is None else q_out
        ops.ci_qk_norm_rope_append(q, k, v, q_norm, k_norm, eps, cos_sin, is_neox, positions, q_out, self.k[layer],
                                   self.v[layer], self.page_table, layout, dev_err=self.dev_err, stream=stream, **kw)
        return q_out

    def attend(self, layer, q, layout, seq_len, max_len=None, scale=None, pos=None, out=None, stream=None, **kw):
        """Attention of q [rows, heads, head_dim] over the cache or over ``pos``."""
        rows, heads, d = q.shape
        out = ops.empty_on(stream, q.shape, q.dtype, q.device) if out is None else out
        on = stream if stream is not None else torch.cuda.current_stream(q.device)
        key = (heads, on.cuda_stream)  # calls on two streams may overlap; the rows do not change the size
        if key not in self._workspace:
            n = ops.attn_workspace_bytes(rows, heads, self.k.shape[2], d)
            self._workspace[key] = ops.empty_on(stream, (n,), torch.uint8, q.device)
        max_len = ops.PAGE * self.page_table.shape[1] if max_len is None else max_len
        ops.ci_attn_decode(q, self.k[layer], self.v[layer], self.page_table, layout, seq_len, max_len,
                           d ** -0.5 if scale is None else scale, out, pos=pos, workspace=self._workspace[key],
                           dev_err=self.dev_err, stream=stream, **kw)
        return out

    def check(self):
        """Waits for the device; raises if any call so far met bad data."""
        bits = int(self.dev_err)
        if bits:
            raise RuntimeError(f"device error bits {bits}")


def sparse_decode_step(cache: PagedCache, step, qkv, q_norm, k_norm, eps, cos_sin, is_neox=True):
    """One decode step of every layer of ``step`` (an IndexerStep over
    ``cache.page_table``): one new token per request, at its last position.
    It puts the calls together where every layer's inputs are at hand, as
    ``step`` has every layer's index queries, under one pair of norms; a model
    whose layers follow from one another makes the same two calls, ``append``
    and ``attend``, layer by layer.
    ``qkv[layer]``: bf16 [requests, q_heads + 2 kv_heads, head_dim].  Returns
    the layers' attention outputs; a request of length 0 gets zeros.  Where a
    request is ``short`` its last position is an older token's and nothing is
    stored: its output does not count."""
    hkv = cache.k.shape[2]
    hq = qkv[0].shape[1] - 2 * hkv
    last = cache.length - 1
    where = last.clamp(min=0)  # a request of length 0: any row of cos_sin, and nothing is stored (-1)
    last = torch.where(cache.short != 0, -1, last)
    queries = [cache.append(j, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], q_norm, k_norm, eps, cos_sin, is_neox,
                            where, ops.LAYOUT_DECODE, cache_pos=last) for j, x in enumerate(qkv)]
    step.run()
    return [cache.attend(j, q, ops.LAYOUT_DECODE, cache.length, step.max_len, pos=step.pos[j])
            for j, q in enumerate(queries)]


def main():
    from . import synth
    from .step import IndexerStep

    dev, layers, hq, hkv, d, steps = "cuda", 5, 64, 8, 128, 4
    gen = torch.Generator(device=dev).manual_seed(0)
    ints = lambda *v: torch.tensor(v, dtype=_I32, device=dev)  # noqa: E731
    prompts = [5000, 130, 9001]
    end = [n + steps for n in prompts + [prompts[0], prompts[2], 0]]  # the two forks, and a request that stays empty
    end[5] = 0
    wl = synth.make_workload("paged", synth.LAYOUT_DECODE, torch.tensor(end), topk_blocks=2048, seed=0, layers=layers,
                             device=dev)
    cache = PagedCache(layers, len(end), wl.page_table.shape[1], wl.num_pages, hkv, d, ops.CACHE_FP8,
                       companions=[ly.k_pool for ly in wl.layers])
    step = IndexerStep(wl)  # its buffers are for the lengths to come
    wl.page_table, wl.seq_len = cache.page_table, cache.length
    norm = torch.ones(d, device=dev)
    angle = torch.arange(max(end), device=dev)[:, None] * 10000.0 ** (-torch.arange(d // 2, device=dev) / (d // 2))
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1)
    tokens = lambda n: torch.randn(n, hq + 2 * hkv, d, device=dev, generator=gen).bfloat16()  # noqa: E731

    cache.grow(ints(*prompts, 0, 0, 0))
    for r, n in enumerate(prompts):  # every prompt is one chunk of its request
        at = torch.arange(n, device=dev, dtype=_I32)
        starts = ints(*[0] * (r + 1), *[n] * (len(end) - r))
        for j in range(layers):
            x = tokens(n)
            q = cache.append(j, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], norm, norm, 1e-6, cos_sin, True, at,
                             ops.LAYOUT_VARLEN, req_start=starts)
            cache.attend(j, q, ops.LAYOUT_VARLEN, at + 1, n, req_start=starts)
    cache.fork(ints(0, 2), ints(3, 4), ints(prompts[0], prompts[2]))
    for _ in range(steps):
        cache.grow(torch.where(cache.length > 0, cache.length + 1, 0).to(_I32))
        sparse_decode_step(cache, step, [tokens(len(end)) for _ in range(layers)], norm, norm, 1e-6, cos_sin)
    used = int((cache.ref_count > 0).sum())
    cache.free(ints(0, 1))
    cache.compact()
    left = int((cache.ref_count > 0).sum())
    outs = sparse_decode_step(cache, step, [tokens(len(end)) for _ in range(layers)], norm, norm, 1e-6, cos_sin)
    cache.check()
    print(f"lengths {cache.length.tolist()}, {used} pages in use, {left} after the release; largest output "
          f"{max(float(o.abs().max()) for o in outs):.3f}")


if __name__ == "__main__":
    main()

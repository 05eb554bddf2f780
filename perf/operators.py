"""The paged-cache operators as they are measured: attention of new tokens over
a paged key-value cache, the norm + rotation + append that fills it, and the
management of its pages.

Each case runs in the plain form (elementary torch operations in 32 bits) or,
with ``own`` set, through the library's entry points
(``two_level_sparse_gb300.cache``).

A cache pool is uint8 [num_pages, kv_heads, bytes]; one (page, head) holds 64
positions: 64 x D bf16, or 64 x D e4m3 followed by 64 fp32 scales.
"""
import math
import random

import torch

own = False

PAGE = 64
EPS = 1e-6
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a handful of requests in the middle of a chat: latency of one decode step's attention
        dict(name="attn_4rows_1k-4k", op="attn", rows=4, min_len=1024, max_len=4096, hq=64, hkv=8, d=128, fp8=False,
             topk=0, shared=False),
        # a full decode batch over long contexts, FP8 cache: the bandwidth case
        dict(name="attn_64rows_16k-64k_fp8", op="attn", rows=64, min_len=16384, max_len=65536, hq=64, hkv=8, d=128,
             fp8=True, topk=0, shared=False),
        # one user with a very long document: only the split over the length fills the card
        dict(name="attn_1row_256k", op="attn", rows=1, min_len=262144, max_len=262144, hq=28, hkv=4, d=128, fp8=False,
             topk=0, shared=False),
        # one key-value head for all query heads, ragged lengths from an empty request on
        dict(name="attn_mqa_17rows_0-100k", op="attn", rows=17, min_len=0, max_len=100003, hq=64, hkv=1, d=128,
             fp8=False, topk=0, shared=False),
        # a decode batch that reads the indexer's 512 positions of each row only
        dict(name="attn_sel512_64rows", op="attn", rows=64, min_len=16384, max_len=65536, hq=64, hkv=8, d=128,
             fp8=False, topk=512, shared=False),
        # a prefill chunk's rows, each over its own 512 positions of the request's one cache
        dict(name="attn_sel512_chunk4096", op="attn", rows=4096, min_len=15360, max_len=16384, hq=64, hkv=1, d=128,
             fp8=False, topk=512, shared=True),
        # the new tokens of a small decode batch: launch latency
        dict(name="append_8tokens", op="append", tokens=8, hq=64, hkv=8, d=128, rot=128, neox=True, fp8=False,
             prefix=4000, shared=False),
        # a prefill chunk into an FP8 cache
        dict(name="append_chunk16384_fp8", op="append", tokens=16384, hq=64, hkv=8, d=128, rot=128, neox=True,
             fp8=True, prefix=245760, shared=True),
        # an odd chunk, narrow heads, interleaved pairs over half of the head
        dict(name="append_chunk1001_d64", op="append", tokens=1001, hq=28, hkv=4, d=64, rot=32, neox=False, fp8=False,
             prefix=777, shared=True),
        # parallel sampling of short prompts: drop the old children, fork anew, copy their last pages
        dict(name="fork_4x2_1k-4k", op="fork", parents=4, children=2, min_len=1000, max_len=4097, pools=2,
             page_bytes=34816, spare=64),
        # beams over a long decode batch, every layer's pools
        dict(name="fork_64x4_16k-64k", op="fork", parents=64, children=4, min_len=16384, max_len=65536, pools=10,
             page_bytes=16384, spare=600),
        # a fragmented pool after many requests have left
        dict(name="compact_6000pages", op="compact", requests=48, min_len=64, max_len=10000, pools=8,
             page_bytes=131072, pages=6000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["attn", "attn", "sel", "append", "append", "fork", "compact"])
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 3, 4, 5, 7, 8, 8, 12, 16])
    if hkv == 1 and rng.random() < 0.4:
        hq = 64
    if hq == 24 or hq * d == 12 * 256:
        hq = 6 * hkv
    fp8 = rng.random() < 0.5
    if op in ("attn", "sel"):
        shared = op == "sel" and rng.random() < 0.5
        rows = _log(rng, 8, 4096) if shared else _log(rng, 1, 128)
        most = 2 ** 27 // (hkv * d) if shared else 2 ** 31 // (rows * hkv * d)  # elements of the padded cache
        hi = _log(rng, 16, min(200000, most))
        lo = max(hi - rows, hi // 2) if shared else rng.choice([0, 1, hi // 4, hi // 2, hi])
        topk = 0
        if op == "sel":
            topk = rng.choice([33, 128, 256, 512, 512, 512, 1000])
            while rows * topk * hkv * d > 2 ** 29:
                rows = rows // 2
        return dict(op="attn", rows=rows, min_len=lo, max_len=hi, hq=hq, hkv=hkv, d=d, fp8=fp8, topk=topk,
                    shared=shared)
    if op == "append":
        shared = rng.random() < 0.6
        tokens = _log(rng, 16, 16384 * 128 // d) if shared else _log(rng, 1, 256)
        while tokens * (hq + 2 * hkv) * d > 16384 * 80 * 128:
            tokens //= 2
        return dict(op="append", tokens=tokens, hq=hq, hkv=hkv, d=d, rot=rng.choice([d, d, d // 2, d // 4]),
                    neox=rng.random() < 0.6, fp8=fp8, prefix=_log(rng, 1, 100000 if shared else 4000), shared=shared)
    page_bytes = hkv * (PAGE * d + 256 if fp8 else PAGE * d * 2)
    pools = 2 * rng.choice([1, 2, 4, 5])
    if op == "fork":
        parents, children = _log(rng, 1, 64), rng.choice([1, 2, 3, 4])
        hi = _log(rng, 70, 65536)
        while parents * (hi // PAGE + 1 + children) * pools * page_bytes > 2 ** 32:
            hi = hi // 2 + 1
        return dict(op="fork", parents=parents, children=children, min_len=hi // 3, max_len=hi, pools=pools,
                    page_bytes=page_bytes, spare=parents * children + rng.randrange(200))
    requests = _log(rng, 2, 128)
    hi = _log(rng, 70, 20000)
    while requests * (hi // PAGE + 1) * pools * page_bytes > 2 ** 32:
        hi = hi // 2 + 1
    pages = int(requests * (hi * 0.75 // PAGE + 2) * rng.uniform(1.05, 2.0)) + 3
    return dict(op="compact", requests=requests, min_len=hi // 2, max_len=hi, pools=pools, page_bytes=page_bytes,
                pages=pages)


# ------------------------------------------------------------------ sizes
def _lengths(lo, hi, n):
    """n lengths spread evenly from lo to hi (hi alone for n = 1)."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _page_bytes(d, fp8):
    return PAGE * d + 4 * PAGE if fp8 else PAGE * d * 2


def work(case):
    c = case
    if c["op"] == "attn":
        L = _lengths(c["min_len"], c["max_len"], c["rows"])
        used = [min(n, c["topk"]) if c["topk"] else n for n in L]
        pos_bytes = 2 * c["hkv"] * (c["d"] + 4 if c["fp8"] else 2 * c["d"])
        total = sum(used)
        cache = (min(total, max(L)) if c["shared"] else total) * pos_bytes
        io = c["rows"] * c["hq"] * (4 * c["d"] + 4) + 4 * c["rows"]
        table = 4 * (_pages(max(L)) if c["shared"] else sum(map(_pages, L))) if not c["topk"] else 8 * total
        return {"bytes": cache + io + table, "flops": 4 * total * c["hq"] * c["d"]}
    if c["op"] == "append":
        t, pos = c["tokens"], (c["d"] + 4 if c["fp8"] else 2 * c["d"])
        return {"bytes": t * (2 * (2 * c["hq"] + 2 * c["hkv"]) * c["d"] + 2 * c["hkv"] * pos + 8 + 4 * c["rot"]),
                "flops": t * (c["hq"] + c["hkv"]) * c["d"] * 8}
    if c["op"] == "fork":
        L = _lengths(c["min_len"], c["max_len"], c["parents"])
        n = c["children"]
        entries = n * sum(map(_pages, L))
        copies = n * sum(x % PAGE != 0 for x in L)
        spare = c["spare"] + sum(map(_pages, L))
        return {"bytes": 4 * (3 * entries + spare) + 2 * copies * c["pools"] * c["page_bytes"], "flops": 0}
    live = sum(map(_pages, _lengths(c["min_len"], c["max_len"], c["requests"])))
    moves = live * (c["pages"] - live) / c["pages"]
    return {"bytes": 4 * (3 * c["pages"] + 2 * live) + 2 * moves * c["pools"] * c["page_bytes"], "flops": 0}


# ------------------------------------------------------------------ inputs
def _fill(pool, d, fp8, gen):
    """Normally distributed values; FP8 with scales in [0.5, 2) / 1.5."""
    step = max(1, 2 ** 27 // (pool.shape[1] * PAGE * d))
    for p in range(0, pool.shape[0], step):
        part = pool[p:p + step]
        x = torch.randn(*part.shape[:2], PAGE * d, generator=gen, device=DEV, dtype=torch.bfloat16)
        if fp8:
            part[..., :PAGE * d] = x.to(torch.float8_e4m3fn).view(torch.uint8)
            scale = torch.rand(*part.shape[:2], PAGE, generator=gen, device=DEV) + 1 / 3
            part[..., PAGE * d:] = scale.view(torch.uint8)
        else:
            part.copy_(x.view(torch.uint8))
    return pool


def _tables(pages, spare, cpu_gen):
    """Page tables of requests with so many pages each, in a random physical order, and the pages in all."""
    total = sum(pages) + spare
    perm = torch.randperm(max(total, 1), generator=cpu_gen).to(torch.int32)
    width = max(max(pages), 1)
    table = torch.full((len(pages), width), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(pages):
        table[r, :n] = perm[at:at + n]
        at += n
    return table, max(total, 1)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    s = {"case": c}
    if c["op"] == "attn":
        rows, hq, hkv, d = c["rows"], c["hq"], c["hkv"], c["d"]
        L = torch.tensor(_lengths(c["min_len"], c["max_len"], rows), dtype=torch.int32)
        if not c["shared"]:
            L = L[torch.randperm(rows, generator=cpu)]
        s["max_len"] = int(L.max())
        table, total = _tables([_pages(s["max_len"])] if c["shared"] else [_pages(n) for n in L.tolist()], 0, cpu)
        s["k_pool"], s["v_pool"] = (
            _fill(torch.empty(total, hkv, _page_bytes(d, c["fp8"]), dtype=torch.uint8, device=DEV), d, c["fp8"], gen)
            for _ in range(2))
        s["page_table"], s["seq_len"] = table.to(DEV), L.to(DEV)
        # logits of standard deviation 2: a few positions of a long cache carry most of a row
        s["q"] = (2 * torch.randn(rows, hq, d, generator=gen, device=DEV)).to(torch.bfloat16)
        s["scale"] = 1 / math.sqrt(d)
        s["pos"] = None
        if c["topk"]:
            k = c["topk"]
            # a row's positions: distinct, ascending, -1 behind them where the row is shorter
            s["pos"] = torch.empty(rows, k, dtype=torch.int32, device=DEV)
            width = max(s["max_len"], k)
            step = max(1, 2 ** 27 // width)
            for r in range(0, rows, step):
                n = s["seq_len"][r:r + step, None]
                at = torch.arange(width, device=DEV)[None]
                x = torch.rand(n.shape[0], width, generator=gen, device=DEV).masked_fill_(at >= n, -1.0)
                score, p = x.topk(k, dim=1)
                p = torch.where(score < 0, 2 ** 31 - 1, p).sort(dim=1).values
                s["pos"][r:r + step] = torch.where(p == 2 ** 31 - 1, -1, p).to(torch.int32)
        s["out"] = torch.empty(rows, hq, d, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(rows, hq, dtype=torch.float32, device=DEV)
        if own:
            from two_level_sparse_gb300 import cache
            s["ws"] = torch.empty(cache.attn_workspace_bytes(rows, hq, hkv, d), dtype=torch.uint8, device=DEV)
    elif c["op"] == "append":
        t, hq, hkv, d = c["tokens"], c["hq"], c["hkv"], c["d"]
        if c["shared"]:
            at = torch.arange(c["prefix"], c["prefix"] + t, dtype=torch.int32)
            pages = [_pages(c["prefix"] + t)]
        else:
            at = torch.tensor(_lengths(c["prefix"] // 4, c["prefix"], t), dtype=torch.int32)
            at = at[torch.randperm(t, generator=cpu)]
            pages = [_pages(n + 1) for n in at.tolist()]
        first = c["prefix"] // PAGE if c["shared"] else 0  # a chunk's pool holds the chunk's own pages
        table, total = _tables([n - first for n in pages], 0, cpu)
        table = torch.cat([torch.full((table.shape[0], first), -1, dtype=torch.int32), table], dim=1)
        s["k_pool"], s["v_pool"] = (
            torch.zeros(total, hkv, _page_bytes(d, c["fp8"]), dtype=torch.uint8, device=DEV) for _ in range(2))
        s["page_table"], s["positions"] = table.to(DEV).contiguous(), at.to(DEV)
        x = torch.randn(t, hq + 2 * hkv, d, generator=gen, device=DEV)
        x *= torch.exp(torch.randn(t, hq + 2 * hkv, 1, generator=gen, device=DEV))  # heads differ in size
        x = x.to(torch.bfloat16)
        s["q"], s["k"], s["v"] = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        s["q_norm"], s["k_norm"] = (1 + 0.2 * torch.randn(d, generator=gen, device=DEV) for _ in range(2))
        half = c["rot"] // 2
        freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
        ang = torch.arange(int(at.max()) + 1, dtype=torch.float64)[:, None] * freq[None]
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], dim=1).float().to(DEV).contiguous()
        s["q_out"] = torch.empty(t, hq, d, dtype=torch.bfloat16, device=DEV)
    elif c["op"] == "fork":
        L = _lengths(c["min_len"], c["max_len"], c["parents"])
        L = [L[i] for i in torch.randperm(len(L), generator=cpu).tolist()]
        n = len(L) * c["children"]
        table, total = _tables([_pages(x) for x in L], c["spare"], cpu)
        ref = torch.zeros(total, dtype=torch.int32)
        ref[table[table >= 0].long()] = 1
        parent = torch.arange(len(L)).repeat_interleave(c["children"])
        length = torch.tensor(L)[parent]
        # every child is there already, from the step before: it shares all its parent's pages
        ref.index_add_(0, table[parent][table[parent] >= 0].long(), torch.ones((), dtype=torch.int32).expand(
            int((table[parent] >= 0).sum())))
        s["page_table"] = torch.cat([table, table[parent]]).to(DEV)
        s["ref"] = ref.to(DEV)
        s["parent"], s["length"] = parent.to(DEV, torch.int32), length.to(DEV, torch.int32)
        s["child"] = torch.arange(len(L), len(L) + n, dtype=torch.int32, device=DEV)
        s["src"], s["dst"] = (torch.empty(n, dtype=torch.int32, device=DEV) for _ in range(2))
        s["pools"] = torch.randint(0, 256, (c["pools"], total, c["page_bytes"]), generator=gen, device=DEV,
                                   dtype=torch.uint8)
    else:
        L = _lengths(c["min_len"], c["max_len"], c["requests"])
        table, total = _tables([_pages(x) for x in L], c["pages"] - sum(map(_pages, L)), cpu)
        ref = torch.zeros(total, dtype=torch.int32)
        ref[table[table >= 0].long()] = 1
        s["table0"], s["ref0"] = table.to(DEV), ref.to(DEV)  # the tables as the scheduler hands them over
        s["page_table"], s["ref"] = torch.empty_like(s["table0"]), torch.empty_like(s["ref0"])
        s["remap"], s["src"], s["dst"] = (torch.empty(total, dtype=torch.int32, device=DEV) for _ in range(3))
        s["count"] = torch.empty(1, dtype=torch.int32, device=DEV)
        s["pools"] = torch.randint(0, 256, (c["pools"], total, c["page_bytes"]), generator=gen, device=DEV,
                                   dtype=torch.uint8)
    s["dev_err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


# ------------------------------------------------------------------ runs
def _decoded(rows, d, fp8, scales):
    """The fp32 values of raw rows [..., bytes], with their scales [...]."""
    if fp8:
        return rows.view(torch.float8_e4m3fn).float() * scales[..., None]
    return rows.view(torch.bfloat16).float()


def _gathered(s, pool):
    """fp32 [rows, kv_heads, positions, d] of what the rows read."""
    c, table = s["case"], s["page_table"].long().clamp(min=0)
    d, fp8, width = c["d"], c["fp8"], c["d"] * (1 if c["fp8"] else 2)
    values = pool[..., :PAGE * width].unflatten(-1, (PAGE, width))
    scales = pool[..., PAGE * width:].view(torch.float32) if fp8 else None
    if c["topk"]:
        at = s["pos"].long().clamp(min=0)
        page = (table.expand(c["rows"], -1) if c["shared"] else table).gather(1, at // PAGE)
        x = _decoded(values[page, :, at % PAGE], d, fp8, scales[page, :, at % PAGE] if fp8 else None)
        return x.transpose(1, 2)
    x = _decoded(values[table], d, fp8, scales[table] if fp8 else None)  # [rows, pages, heads, 64, d]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attn(s):
    c = s["case"]
    k = _gathered(s, s["k_pool"])
    q = s["q"].float().unflatten(1, (c["hkv"], c["hq"] // c["hkv"]))
    logit = torch.matmul(q, k.transpose(2, 3)) * s["scale"]  # [rows, kv_heads, group, positions]
    del k
    if c["topk"]:
        valid = s["pos"] >= 0
    else:
        valid = torch.arange(logit.shape[-1], device=DEV)[None] < s["seq_len"][:, None]
    logit = torch.where(valid[:, None, None], logit, -math.inf)
    top = logit.amax(-1, keepdim=True)
    p = torch.exp(logit - torch.where(top == -math.inf, 0.0, top))
    del logit
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, _gathered(s, s["v_pool"])) / torch.where(total == 0, 1.0, total)
    lse = top + torch.log(total)
    return out.flatten(1, 2).to(torch.bfloat16), lse.flatten(1)


def _plain_norm_rope(x, w, cs, rot, neox):
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * w
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    a, b = (y[..., :rot // 2], y[..., rot // 2:rot]) if neox else (y[..., :rot:2], y[..., 1:rot:2])
    a, b = a * c - b * s, b * c + a * s
    ab = torch.cat([a, b], -1) if neox else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([ab, y[..., rot:]], -1)


def _plain_store(pool, x, page, slot, d, fp8):
    if fp8:
        scale = x.abs().amax(-1).clamp(min=1e-10) / 448
        pool[..., :PAGE * d].unflatten(-1, (PAGE, d))[page, :, slot] = (
            (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8))
        pool[..., PAGE * d:].view(torch.float32)[page, :, slot] = scale
    else:
        pool.view(torch.bfloat16).unflatten(-1, (PAGE, d))[page, :, slot] = x.to(torch.bfloat16)


def _plain_append(s):
    c = s["case"]
    at = s["positions"].long()
    cs = s["cos_sin"][at]
    q = _plain_norm_rope(s["q"], s["q_norm"], cs, c["rot"], c["neox"]).to(torch.bfloat16)
    k = _plain_norm_rope(s["k"], s["k_norm"], cs, c["rot"], c["neox"])
    table = s["page_table"].long()
    page = (table.expand(c["tokens"], -1) if c["shared"] else table).gather(1, at[:, None] // PAGE)[:, 0]
    _plain_store(s["k_pool"], k, page, at % PAGE, c["d"], c["fp8"])
    _plain_store(s["v_pool"], s["v"].float(), page, at % PAGE, c["d"], c["fp8"])
    return q


def _plain_lowest(free, n):
    """The n lowest ids where `free`."""
    rank = torch.where(free, torch.cumsum(free, 0) - 1, n).clamp(max=n)
    ids = torch.empty(n + 1, dtype=torch.int64, device=DEV)
    ids.scatter_(0, rank, torch.arange(free.shape[0], device=DEV))
    return ids[:n]


def _plain_copy(s):
    ok = s["dst"] >= 0
    src, dst = s["src"][ok].long(), s["dst"][ok].long()
    s["pools"][:, dst] = s["pools"][:, src]


def _plain_fork(s):
    table, ref, child, parent = s["page_table"], s["ref"], s["child"].long(), s["parent"].long()
    old = table[child].flatten()
    ref.index_add_(0, old.clamp(min=0).long(), -(old >= 0).int())
    table[child] = -1
    full, part = s["length"] // PAGE, s["length"] % PAGE != 0
    col = torch.arange(table.shape[1], device=DEV)[None]
    shared = torch.where(col < full[:, None], table[parent], -1)
    ids = _plain_lowest(ref == 0, child.shape[0])
    new = torch.where(part, ids[(torch.cumsum(part, 0) - 1).clamp(min=0)], -1).int()
    last = table[parent].gather(1, full[:, None].long().clamp(max=table.shape[1] - 1))[:, 0]
    s["src"].copy_(torch.where(part, last, -1))
    s["dst"].copy_(new)
    rows = torch.where((col == full[:, None]) & part[:, None], new[:, None], shared)
    table[child] = rows
    ref.index_add_(0, rows.flatten().clamp(min=0).long(), (rows.flatten() >= 0).int())
    _plain_copy(s)


def _plain_compact(s):
    table, ref = s["page_table"], s["ref"]
    live = ref > 0
    n, ids = live.sum(), torch.arange(ref.shape[0], device=DEV, dtype=torch.int32)
    hole, mover = ~live & (ids < n), live & (ids >= n)
    s["count"].copy_(mover.sum()[None])
    s["src"].fill_(-1)
    s["dst"].fill_(-1)
    s["src"][:int(s["count"])] = ids[mover]
    s["dst"][:int(s["count"])] = ids[hole]
    s["remap"].copy_(torch.where(live, ids, -1))
    s["remap"][ids[mover].long()] = ids[hole]
    ref[ids[hole].long()] = ref[ids[mover].long()]
    ref[ids[mover].long()] = 0
    table.copy_(torch.where(table >= 0, s["remap"][table.clamp(min=0).long()], -1))
    _plain_copy(s)


def _cache_values(s):
    """The cache as the values that it holds: bf16, or e4m3 and its scales."""
    c = s["case"]
    if not c["fp8"]:
        return {"k": s["k_pool"].view(torch.bfloat16), "v": s["v_pool"].view(torch.bfloat16)}
    n = PAGE * c["d"]
    return {"k": s["k_pool"][..., :n].view(torch.float8_e4m3fn), "k_scale": s["k_pool"][..., n:].view(torch.float32),
            "v": s["v_pool"][..., :n].view(torch.float8_e4m3fn), "v_scale": s["v_pool"][..., n:].view(torch.float32)}


def run(state):
    s = state
    c = s["case"]
    if own:
        from two_level_sparse_gb300 import cache
    if c["op"] == "attn":
        if own:
            cache.ci_attn_decode(s["q"], s["k_pool"], s["v_pool"], s["page_table"],
                                 cache.LAYOUT_PREFILL if c["shared"] else cache.LAYOUT_DECODE, s["seq_len"],
                                 s["max_len"], s["scale"], s["out"], lse=s["lse"], pos=s["pos"], workspace=s["ws"],
                                 dev_err=s["dev_err"])
            return {"out": s["out"], "lse": s["lse"]}
        out, lse = _plain_attn(s)
        return {"out": out, "lse": lse}
    if c["op"] == "append":
        if own:
            cache.ci_qk_norm_rope_append(s["q"], s["k"], s["v"], s["q_norm"], s["k_norm"], EPS, s["cos_sin"],
                                         c["neox"], s["positions"], s["q_out"], s["k_pool"], s["v_pool"],
                                         s["page_table"], cache.LAYOUT_PREFILL if c["shared"] else cache.LAYOUT_DECODE,
                                         dev_err=s["dev_err"])
            return {"q": s["q_out"], **_cache_values(s)}
        q = _plain_append(s)
        return {"q": q, **_cache_values(s)}
    if c["op"] == "fork":
        if own:
            cache.ci_pages_free(s["page_table"], s["ref"], s["child"], dev_err=s["dev_err"])
            cache.ci_pages_fork(s["page_table"], s["ref"], s["parent"], s["child"], s["length"], s["src"], s["dst"],
                                dev_err=s["dev_err"])
            cache.ci_pages_copy(s["pools"], s["src"], s["dst"], dev_err=s["dev_err"])
        else:
            _plain_fork(s)
        return {"page_table": s["page_table"], "ref": s["ref"], "src": s["src"], "dst": s["dst"], "pools": s["pools"]}
    s["page_table"].copy_(s["table0"])
    s["ref"].copy_(s["ref0"])
    if own:
        cache.ci_pages_compact(s["page_table"], s["ref"], s["remap"], s["src"], s["dst"], s["count"],
                               dev_err=s["dev_err"])
        cache.ci_pages_copy(s["pools"], s["src"], s["dst"], count=s["count"], dev_err=s["dev_err"])
    else:
        _plain_compact(s)
    return {"page_table": s["page_table"], "ref": s["ref"], "remap": s["remap"], "src": s["src"], "dst": s["dst"],
            "count": s["count"], "pools": s["pools"]}


# ------------------------------------------------------------------ 64 bits
def _e4m3_table():
    """The 256 e4m3 values, from their bit fields."""
    v = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = math.nan if (b & 127) == 127 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v.append(-x if b >> 7 else x)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _read64(pool, page, slot, d, fp8):
    """[n, kv_heads, d] of positions (page, slot)."""
    if fp8:
        at = slot[:, None] * d + torch.arange(d, device=DEV)
        byte = pool[page[:, None], :, at].permute(0, 2, 1)
        at = PAGE * d + 4 * slot[:, None] + torch.arange(4, device=DEV)
        scale = pool[page[:, None], :, at].permute(0, 2, 1).reshape(-1).view(torch.float32).double()
        return _e4m3_table()[byte.long()] * scale.reshape(*byte.shape[:2], 1)
    at = 2 * slot[:, None] * d + torch.arange(2 * d, device=DEV)
    rows = pool[page[:, None], :, at].permute(0, 2, 1)
    return rows.reshape(-1).view(torch.bfloat16).double().reshape(-1, pool.shape[1], d)


def _exact_attn(s):
    c = s["case"]
    out = torch.zeros(c["rows"], c["hq"], c["d"], dtype=torch.float64, device=DEV)
    lse = torch.full((c["rows"], c["hq"]), -math.inf, dtype=torch.float64, device=DEV)
    g = c["hq"] // c["hkv"]
    lens = s["seq_len"].tolist()
    for t, n in enumerate(lens):
        at = torch.arange(n, device=DEV)
        if c["topk"]:
            at = s["pos"][t].long()
            at = at[at >= 0]
        if at.numel() == 0:
            continue
        page = s["page_table"][0 if c["shared"] else t].long()[at // PAGE]
        k = _read64(s["k_pool"], page, at % PAGE, c["d"], c["fp8"])
        x = torch.einsum("hgd,nhd->hgn", s["q"][t].double().reshape(c["hkv"], g, c["d"]), k) * s["scale"]
        z = torch.logsumexp(x, -1)
        v = _read64(s["v_pool"], page, at % PAGE, c["d"], c["fp8"])
        out[t] = torch.einsum("hgn,nhd->hgd", torch.exp(x - z[..., None]), v).reshape(c["hq"], c["d"])
        lse[t] = z.reshape(-1)
    return {"out": out, "lse": lse}


def _exact_append(s):
    c = s["case"]
    t, d, half, fp8 = c["tokens"], c["d"], c["rot"] // 2, c["fp8"]
    # the rotation as a product of complex numbers
    w = torch.complex(s["cos_sin"][:, :half].double(), s["cos_sin"][:, half:].double())[s["positions"].long()][:, None]

    def turned(x, gain):
        y = x.double()
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / d + EPS) * gain.double()
        first = torch.arange(half, device=DEV) * (1 if c["neox"] else 2)
        second = first + (half if c["neox"] else 1)
        z = torch.complex(y[..., first], y[..., second]) * w
        y[..., first], y[..., second] = z.real, z.imag
        return y

    at = s["positions"].long()
    page = s["page_table"].long()[torch.zeros_like(at) if c["shared"] else torch.arange(t, device=DEV), at // PAGE]

    def stored(x):
        shape = (s["k_pool"].shape[0], c["hkv"], PAGE)
        values = torch.zeros(*shape, d, dtype=torch.float64, device=DEV)
        scales = torch.zeros(shape, dtype=torch.float64, device=DEV)
        if fp8:
            z = x.abs().amax(-1).clamp(min=1e-10) / 448
            scales[page, :, at % PAGE] = z
            x = x / z[..., None]
        values[page, :, at % PAGE] = x
        return values.flatten(2), scales

    q = turned(s["q"], s["q_norm"])
    k, k_scale = stored(turned(s["k"], s["k_norm"]))
    v, v_scale = stored(s["v"].double())
    return {"q": q, "k": k, "v": v, **({"k_scale": k_scale, "v_scale": v_scale} if fp8 else {})}


def exact(case, seed):
    if case["op"] not in ("attn", "append"):
        return None  # ids, counts and copied bytes: no rounding anywhere
    s = prepare(case, seed)
    return _exact_attn(s) if case["op"] == "attn" else _exact_append(s)

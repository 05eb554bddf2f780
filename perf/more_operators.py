"""The drafted step's operators as they are measured: a tree of drafted tokens
per request is laid out behind the request's cache, attends to the cache and to
its own ancestors, and what the model agrees with becomes part of the cache.

- plan: pages for the drafts, and the rows, positions, slots and masks that the
  other calls take, from the requests' lengths and trees;
- attn: attention of all drafted rows;
- commit: the accepted path of every tree, its keys and values moved to where
  the cache goes on, the pages behind them released.

Each case runs in the plain form (elementary torch operations in 32 bits) or,
with ``own`` set, through the library's entry points
(``two_level_sparse_gb300.cache`` and ``two_level_sparse_gb300.draft``).

A cache pool is uint8 [num_pages, kv_heads, bytes]; one (page, head) holds 64
positions: 64 x D bf16, or 64 x D e4m3 followed by 64 fp32 scales.  Node i of a
request's tree is kept at position length + i; its parent is an earlier node, or
-1; node 0 is the token that the request goes on with.
"""
import math
import random

import torch

own = False

PAGE = 64
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a small chat batch drafts a few tokens per request: launch latency
        dict(name="plan_8req_16nodes", op="plan", requests=8, min_nodes=16, max_nodes=16, min_len=1000, max_len=4000,
             spare=64, tree=True),
        # a full batch with ragged trees, some requests without any
        dict(name="plan_200req_0-64nodes", op="plan", requests=200, min_nodes=0, max_nodes=64, min_len=100,
             max_len=65000, spare=1000, tree=True),
        # the small chat batch's attention: latency
        dict(name="attn_4req_16nodes_1k-4k", op="attn", requests=4, min_nodes=16, max_nodes=16, min_len=1024,
             max_len=4096, hq=64, hkv=8, d=128, fp8=False, tree=True),
        # a decode batch over long contexts, FP8 cache, short chains of drafts: the bandwidth case
        dict(name="attn_64req_chain4_16k-64k_fp8", op="attn", requests=64, min_nodes=4, max_nodes=4, min_len=16384,
             max_len=65536, hq=64, hkv=8, d=128, fp8=True, tree=False),
        # wide trees on many requests: products and bandwidth both count
        dict(name="attn_64req_64nodes_4k-16k", op="attn", requests=64, min_nodes=64, max_nodes=64, min_len=4096,
             max_len=16384, hq=64, hkv=8, d=128, fp8=False, tree=True),
        # one user with a very long document: only the split over the length fills the card
        dict(name="attn_1req_60nodes_256k", op="attn", requests=1, min_nodes=60, max_nodes=60, min_len=262144,
             max_len=262144, hq=28, hkv=4, d=128, fp8=False, tree=True),
        # one key-value head for all query heads, ragged trees and lengths from an empty request on
        dict(name="attn_mqa_17req_1-20nodes_0-100k", op="attn", requests=17, min_nodes=1, max_nodes=20, min_len=0,
             max_len=100003, hq=64, hkv=1, d=128, fp8=False, tree=True),
        # wide heads in FP8, odd sizes
        dict(name="attn_9req_33nodes_d256_fp8", op="attn", requests=9, min_nodes=5, max_nodes=33, min_len=777,
             max_len=30011, hq=14, hkv=2, d=256, fp8=True, tree=True),
        # a prompt's chunk behind its cached prefix: a chain of many tokens, bound by the products
        dict(name="attn_chunk2048_16k", op="attn", requests=1, min_nodes=2048, max_nodes=2048, min_len=16384,
             max_len=16384, hq=64, hkv=8, d=128, fp8=False, tree=False),
        # the small chat batch, one layer's pools: launch latency
        dict(name="commit_8req_16nodes", op="commit", requests=8, min_nodes=16, max_nodes=16, min_len=1000,
             max_len=4000, hkv=8, d=128, fp8=False, pools=2, tree=True),
        # a full batch of ragged trees, the pools of twenty layers
        dict(name="commit_200req_0-64nodes_40pools", op="commit", requests=200, min_nodes=0, max_nodes=64, min_len=100,
             max_len=1500, hkv=8, d=128, fp8=True, pools=40, tree=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["plan", "attn", "attn", "attn", "chunk", "commit"])
    tree = rng.random() < 0.75
    if op == "plan":
        most = _log(rng, 1, 256)
        return dict(op="plan", requests=_log(rng, 1, 400), min_nodes=rng.choice([0, 1, most // 2, most]),
                    max_nodes=most, min_len=rng.choice([0, 50, 1000]), max_len=_log(rng, 1000, 100000),
                    spare=rng.randrange(64, 2000), tree=tree)
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    fp8 = rng.random() < 0.5
    if op == "commit":
        most = _log(rng, 1, 128)
        requests, pools = _log(rng, 1, 200), 2 * rng.choice([1, 2, 5, 12])
        hi = _log(rng, 64, 5000)
        while requests * (hi // PAGE + 3) * PAGE * hkv * d * pools > 2 ** 31:
            hi = hi // 2 + 1
            pools = max(2, pools // 2)
        return dict(op="commit", requests=requests, min_nodes=rng.choice([0, 1, most]), max_nodes=most,
                    min_len=hi // 4, max_len=hi, hkv=hkv, d=d, fp8=fp8, pools=pools, tree=tree)
    hq = hkv * rng.choice([1, 3, 4, 5, 7, 8, 8, 12, 16])
    if hkv == 1 and rng.random() < 0.4:
        hq = 64
    if op == "chunk":
        requests, nodes, tree = rng.choice([1, 1, 2, 3]), _log(rng, 65, 2048), False
        hi = _log(rng, 16, 16384)
    else:
        requests, nodes = _log(rng, 1, 96), _log(rng, 1, 100)
        hi = _log(rng, 16, 200000)
    most = min(2 ** 30 // (requests * hkv * d), 2 ** 40 // (4 * requests * nodes * hq * d))
    hi = max(1, min(hi, most - nodes))
    return dict(op="attn", requests=requests, min_nodes=rng.choice([0, 1, nodes // 2, nodes, nodes]), max_nodes=nodes,
                min_len=rng.choice([0, 1, hi // 4, hi // 2, hi]), max_len=hi, hq=hq, hkv=hkv, d=d, fp8=fp8, tree=tree)


# ------------------------------------------------------------------ sizes
def _spread(lo, hi, n):
    """n whole numbers spread evenly from lo to hi (hi alone for n = 1)."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _sizes(c):
    """Lengths and node counts: short requests may have large trees."""
    n = c["requests"]
    nodes = _spread(c["min_nodes"], c["max_nodes"], n)
    return _spread(c["min_len"], c["max_len"], n), [nodes[(7 * i + 3) % n] for i in range(n)]


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _words(nodes):
    return (nodes + 31) // 32


def _page_bytes(d, fp8):
    return PAGE * d + 4 * PAGE if fp8 else PAGE * d * 2


def work(case):
    c = case
    lens, nodes = _sizes(c)
    if c["op"] == "plan":
        rows = sum(nodes)
        new = sum(_pages(a + b) - _pages(a) for a, b in zip(lens, nodes))
        return {"bytes": 4 * (4 * c["requests"] + 2 * rows + rows * (3 + _words(c["max_nodes"])) + 3 * new),
                "flops": 0}
    if c["op"] == "attn":
        keys = sum((a + b) for a, b in zip(lens, nodes) if b)
        entry = 2 * c["hkv"] * (c["d"] + 4 if c["fp8"] else 2 * c["d"])
        # a row reads its request's cache and its ancestors (of a chain: half of the nodes on average; of a tree: few)
        pairs = sum(b * (a + ((b + 1) / 2 if not c["tree"] else min(b, 8))) for a, b in zip(lens, nodes))
        return {"bytes": keys * entry + sum(nodes) * c["hq"] * (4 * c["d"] + 4), "flops": 4 * pairs * c["hq"] * c["d"]}
    entry = c["hkv"] * (c["d"] + 4 if c["fp8"] else 2 * c["d"])
    moved = sum(min(b, 4) for b in nodes)  # about four tokens of a tree are accepted
    return {"bytes": 2 * moved * c["pools"] * entry + 4 * (4 * sum(nodes) + 8 * c["requests"]), "flops": 0}


# ------------------------------------------------------------------ inputs
def _fill(pool, d, fp8, gen):
    """Normally distributed values; FP8 with scales in [1 / 3, 4 / 3)."""
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


def _tables(pages, spare, width, cpu_gen):
    """Page tables of requests with so many pages each, in a random physical order, and the pages in all."""
    total = max(sum(pages) + spare, 1)
    perm = torch.randperm(total, generator=cpu_gen).to(torch.int32)
    table = torch.full((len(pages), max(width, 1)), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(pages):
        table[r, :n] = perm[at:at + n]
        at += n
    return table, total


def _trees(c, nodes, cpu_gen):
    """Parents [requests, max_nodes], -1 behind the last node: every node hangs on one of the eight before it."""
    n = max(c["max_nodes"], 1)
    i = torch.arange(n)
    reach = torch.clamp(i, max=8)
    back = 1 + (torch.rand(len(nodes), n, generator=cpu_gen) * reach).long().clamp(max=(reach - 1).clamp(min=0))
    parent = torch.where(i > 0, i - back, -1) if c["tree"] else (i - 1).expand(len(nodes), n)
    return torch.where(i < torch.tensor(nodes)[:, None], parent, -1).to(torch.int32).contiguous()


def _ancestors(parent):
    """bool [requests, n, n]: whether node j is i or one of its ancestors."""
    r, n = parent.shape
    up = torch.eye(n, device=parent.device).repeat(r, 1, 1)
    has = parent >= 0
    up.scatter_add_(2, parent.clamp(min=0).long()[..., None], has[..., None].float())
    for _ in range(max(1, (n - 1).bit_length())):
        up = (torch.matmul(up, up) > 0).float()
    return up > 0


def _packed(bits, words):
    """Bits [..., n] as int32 [..., words], bit j of word w for entry 32 w + j."""
    n = bits.shape[-1]
    x = torch.zeros(*bits.shape[:-1], 32 * words, dtype=torch.int64, device=bits.device)
    x[..., :n] = bits
    v = (x.unflatten(-1, (words, 32)) << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(v >= 2 ** 31, v - 2 ** 32, v).to(torch.int32)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    lens, nodes = _sizes(c)
    order = torch.randperm(len(lens), generator=cpu).tolist()
    lens, nodes = [lens[i] for i in order], [nodes[i] for i in order]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    s = {"case": c, "lens": lens, "nodes": nodes, "length": ints(lens), "count": ints(nodes)}
    ends = [a + b for a, b in zip(lens, nodes)]
    width = _pages(max(ends))
    starts = [0]
    for n in nodes:
        starts.append(starts[-1] + n)
    s["starts"], s["req_start"] = starts, ints(starts)
    rows = starts[-1]
    parent = _trees(c, nodes, cpu)
    s["parent"] = parent.to(DEV)
    n = parent.shape[1]
    there = torch.arange(n) < torch.tensor(nodes)[:, None]
    if c["op"] == "plan":
        held = [_pages(a) for a in lens]
        new = sum(map(_pages, ends)) - sum(held)
        table, total = _tables(held, new + c["spare"], width, cpu)
        ref = torch.zeros(total, dtype=torch.int32)
        ref[table[table >= 0].long()] = 1
        s["table0"], s["ref0"] = table.to(DEV), ref.to(DEV)  # the tables as the step before left them
        s["page_table"], s["ref"] = torch.empty_like(s["table0"]), torch.empty_like(s["ref0"])
        s["end"] = ints(ends)
        s["token"] = torch.randint(0, 100000, parent.shape, generator=cpu).to(DEV, torch.int32)
        cap = c["requests"] * n  # a captured step's rows are as many as there can be
        for name, shape in dict(req_start=(c["requests"] + 1,), positions=(cap,), cache_pos=(cap,), row_token=(cap,),
                                mask=(cap, _words(n))).items():
            s[name] = torch.empty(shape, dtype=torch.int32, device=DEV)
    elif c["op"] == "attn":
        hq, hkv, d = c["hq"], c["hkv"], c["d"]
        table, total = _tables([_pages(e) for e in ends], 0, width, cpu)
        s["page_table"] = table.to(DEV)
        s["max_len"], s["max_rows"] = max(ends), max(nodes)
        s["k_pool"], s["v_pool"] = (
            _fill(torch.empty(total, hkv, _page_bytes(d, c["fp8"]), dtype=torch.uint8, device=DEV), d, c["fp8"], gen)
            for _ in range(2))
        # logits of standard deviation 2: a few positions of a long cache carry most of a row
        s["q"] = (2 * torch.randn(rows, hq, d, generator=gen, device=DEV)).to(torch.bfloat16)
        s["scale"] = 1 / math.sqrt(d)
        s["mask"] = None
        if c["tree"]:
            s["mask"] = _packed(_ancestors(parent).to(DEV)[there.to(DEV)], _words(n)).contiguous()
        s["out"] = torch.empty(rows, hq, d, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(rows, hq, dtype=torch.float32, device=DEV)
        if own:
            from two_level_sparse_gb300 import draft
            s["ws"] = torch.empty(draft.attn_draft_workspace_bytes(s["max_rows"], hq, hkv, d), dtype=torch.uint8,
                                  device=DEV)
    else:
        row = c["d"] if c["fp8"] else 2 * c["d"]
        table, total = _tables([_pages(e) for e in ends], 3, width, cpu)
        ref = torch.zeros(total, dtype=torch.int32)
        ref[table[table >= 0].long()] = 1
        s["table0"], s["ref0"] = table.to(DEV), ref.to(DEV)
        s["page_table"], s["ref"] = torch.empty_like(s["table0"]), torch.empty_like(s["ref0"])
        s["end"] = ints(ends)
        s["row_bytes"], s["scale_bytes"] = row, 4 if c["fp8"] else 0
        s["pools"] = torch.randint(0, 256, (c["pools"], total, c["hkv"], _page_bytes(c["d"], c["fp8"])), generator=gen,
                                   device=DEV, dtype=torch.uint8)
        # drafted tokens, and what the model says behind each: a child's token four times out of five
        token = torch.randint(0, 100000, parent.shape, generator=cpu)
        target = torch.randint(0, 100000, parent.shape, generator=cpu)
        says = torch.rand(parent.shape, generator=cpu) < 0.8
        for i in range(n - 1, 0, -1):  # (an earlier child overrules a later one)
            up = parent[:, i].clamp(min=0).long()[:, None]
            use = (parent[:, i:i + 1] >= 0) & says.gather(1, up)
            target.scatter_(1, up, torch.where(use, token[:, i:i + 1], target.gather(1, up)))
        s["row_token"], s["target"] = (x[there].to(DEV, torch.int32) for x in (token, target))
        at = torch.tensor(lens)[:, None] + torch.arange(n)
        s["cache_pos"] = at[there].to(DEV, torch.int32)
        s["path"] = torch.empty(c["requests"], n, dtype=torch.int32, device=DEV)
        s["accepted"], s["next"], s["new_len"] = (torch.empty(c["requests"], dtype=torch.int32, device=DEV)
                                                  for _ in range(3))
    s["dev_err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
    return s


# ------------------------------------------------------------------ plain forms
def _plain_plan(s):
    table, ref, length, count = s["page_table"], s["ref"], s["length"], s["count"]
    # the lowest free pages, in order of the requests
    first, last = (length + PAGE - 1) // PAGE, (s["end"] + PAGE - 1) // PAGE
    need = (last - first).long()
    before = torch.cumsum(need, 0) - need
    col = torch.arange(table.shape[1], device=DEV)[None]
    new = (col >= first[:, None]) & (col < last[:, None])
    free = ref == 0
    rank = torch.where(free, torch.cumsum(free, 0) - 1, ref.shape[0])
    ids = torch.empty(ref.shape[0] + 1, dtype=torch.int64, device=DEV)
    ids.scatter_(0, rank, torch.arange(ref.shape[0], device=DEV))
    page = ids[torch.where(new, before[:, None] + col - first[:, None], 0)]
    table.copy_(torch.where(new, page, table))
    ref.copy_(torch.where(free & (rank < need.sum()), 1, ref))
    # rows
    r, n = s["parent"].shape
    rows = s["positions"].shape[0]
    s["req_start"].zero_()
    s["req_start"][1:] = torch.cumsum(count, 0)
    node = torch.arange(n, device=DEV)[None]
    there = node < count[:, None]
    up = _ancestors(s["parent"])
    at = torch.where(there, s["req_start"][:-1, None] + node, rows).flatten()  # where no row is: one behind the last

    def spread(x, empty):
        out = torch.full((rows + 1, *x.shape[2:]), empty, dtype=torch.int32, device=DEV)
        return out.index_copy_(0, at, x.flatten(0, 1).to(torch.int32))[:rows]

    s["positions"].copy_(spread(length[:, None] + up.sum(-1) - 1, 0))
    s["cache_pos"].copy_(spread(length[:, None] + node, -1))
    s["row_token"].copy_(spread(s["token"], 0))
    s["mask"].copy_(spread(_packed(up, s["mask"].shape[1]), 0))


def _decoded(rows, fp8, scales):
    """The fp32 values of raw rows [..., bytes], with their scales [...]."""
    if fp8:
        return rows.view(torch.float8_e4m3fn).float() * scales[..., None]
    return rows.view(torch.bfloat16).float()


def _gathered(s, pool, request, positions):
    """fp32 [kv_heads, positions, d] of a request's first positions."""
    c = s["case"]
    d, fp8, width = c["d"], c["fp8"], c["d"] * (1 if c["fp8"] else 2)
    page = s["page_table"][request, :_pages(positions)].long()
    x = pool[page]  # [pages, heads, bytes]
    values = x[..., :PAGE * width].unflatten(-1, (PAGE, width))
    scales = x[..., PAGE * width:].contiguous().view(torch.float32) if fp8 else None
    return _decoded(values.contiguous(), fp8, scales).transpose(0, 1).flatten(1, 2)[:, :positions]


def _plain_attn(s):
    c = s["case"]
    group = c["hq"] // c["hkv"]
    for r, (length, n) in enumerate(zip(s["lens"], s["nodes"])):
        if n == 0:
            continue
        t0 = s["starts"][r]
        k, v = (_gathered(s, s[p], r, length + n) for p in ("k_pool", "v_pool"))
        node = torch.arange(n, device=DEV)
        if s["mask"] is None:
            sees = node[None] <= node[:, None]
        else:
            word = s["mask"][t0:t0 + n].long()
            sees = (word[:, node // 32] >> (node % 32)) & 1 == 1
        q = s["q"][t0:t0 + n].float().unflatten(1, (c["hkv"], group)).permute(1, 2, 0, 3)  # [hkv, group, n, d]
        step = max(1, 2 ** 31 // (group * n * (length + n)))  # heads at a time
        for h in range(0, c["hkv"], step):
            logit = torch.matmul(q[h:h + step].flatten(1, 2), k[h:h + step].transpose(1, 2)) * s["scale"]
            logit = logit.unflatten(1, (group, n))
            logit[..., length:] = torch.where(sees, logit[..., length:], -math.inf)
            top = logit.amax(-1, keepdim=True)
            p = torch.exp(logit - torch.where(top == -math.inf, 0.0, top))
            total = p.sum(-1, keepdim=True)
            out = torch.matmul(p.flatten(1, 2), v[h:h + step]).unflatten(1, (group, n))
            out = out / torch.where(total == 0, 1.0, total)
            heads = slice(h * group, (h + out.shape[0]) * group)
            s["out"][t0:t0 + n, heads] = out.flatten(0, 1).transpose(0, 1).to(torch.bfloat16)
            s["lse"][t0:t0 + n, heads] = (top + torch.log(total))[..., 0].flatten(0, 1).transpose(0, 1)


def _plain_commit(s):
    c = s["case"]
    r, n = s["parent"].shape
    node = torch.arange(n, device=DEV)[None]
    there = node < s["count"][:, None]
    row = torch.where(there, s["req_start"][:-1, None] + node, 0).long()
    token = s["row_token"][row] if s["row_token"].numel() else torch.zeros_like(s["parent"])
    target = s["target"][row] if s["target"].numel() else torch.zeros_like(s["parent"])
    path, accepted = s["path"], s["accepted"]
    path.fill_(-1)
    accepted.zero_()
    s["next"].fill_(-1)
    at = torch.zeros(r, dtype=torch.int64, device=DEV)
    alive = s["count"] > 0
    for step in range(n):
        path[:, step] = torch.where(alive, at, -1)
        accepted += alive
        says = target.gather(1, at[:, None])
        s["next"].copy_(torch.where(alive, says[:, 0], s["next"]))
        fits = (s["parent"] == at[:, None]) & (token == says) & there & (node > 0)
        alive = alive & fits.any(1)
        at = torch.where(alive, fits.int().argmax(1), at)
    torch.add(s["length"], accepted, out=s["new_len"])
    # the accepted entries to where the cache goes on
    take = (path >= 0) & (path != node)
    req = torch.arange(r, device=DEV)[:, None].expand(r, n)[take]
    src, dst = ((s["length"][:, None] + x)[take].long() for x in (path, node))
    table = s["page_table"].long()
    a, b, x, y = table[req, src // PAGE], table[req, dst // PAGE], src % PAGE, dst % PAGE
    values = s["pools"][..., :PAGE * s["row_bytes"]].unflatten(-1, (PAGE, s["row_bytes"]))
    values[:, b, :, y] = values[:, a, :, x]
    if s["scale_bytes"]:
        scales = s["pools"][..., PAGE * s["row_bytes"]:].unflatten(-1, (PAGE, s["scale_bytes"]))
        scales[:, b, :, y] = scales[:, a, :, x]
    # the pages that nothing is in any more
    col = torch.arange(s["page_table"].shape[1], device=DEV)[None]
    gone = (col >= _pages(s["new_len"])[:, None]) & (col < _pages(s["end"])[:, None])
    ids = torch.where(gone, s["page_table"], -1).flatten()
    s["ref"].index_add_(0, ids.clamp(min=0).long(), -(ids >= 0).int())
    s["page_table"].masked_fill_(gone, -1)


def run(state):
    s = state
    c = s["case"]
    if own:
        from two_level_sparse_gb300 import cache, draft
    if c["op"] == "attn":
        if own:
            draft.ci_attn_draft(s["q"], s["k_pool"], s["v_pool"], s["page_table"], s["req_start"], s["length"],
                                s["max_len"], s["max_rows"], s["scale"], s["out"], mask=s["mask"], lse=s["lse"],
                                workspace=s["ws"], dev_err=s["dev_err"])
        else:
            _plain_attn(s)
        return {"out": s["out"], "lse": s["lse"]}
    s["page_table"].copy_(s["table0"])
    s["ref"].copy_(s["ref0"])
    if c["op"] == "plan":
        if own:
            cache.ci_pages_alloc(s["page_table"], s["ref"], s["length"], s["end"], dev_err=s["dev_err"])
            draft.ci_draft_plan(s["length"], s["count"], s["parent"], s["page_table"], s["ref"].shape[0],
                                s["req_start"], s["positions"], s["cache_pos"], mask=s["mask"], token=s["token"],
                                row_token=s["row_token"], dev_err=s["dev_err"])
        else:
            _plain_plan(s)
        return {k: s[k] for k in ("page_table", "ref", "req_start", "positions", "cache_pos", "mask", "row_token")}
    if own:
        draft.ci_draft_accept(s["req_start"], s["length"], s["parent"], s["row_token"], s["target"], s["path"],
                              s["accepted"], s["next"], s["new_len"], cache_pos=s["cache_pos"], dev_err=s["dev_err"])
        draft.ci_slots_move(s["pools"], s["row_bytes"], s["scale_bytes"], s["page_table"], s["length"], s["path"],
                            s["accepted"], dev_err=s["dev_err"])
        draft.ci_pages_trim(s["page_table"], s["ref"], s["end"], s["new_len"], dev_err=s["dev_err"])
    else:
        _plain_commit(s)
    return {k: s[k] for k in ("path", "accepted", "next", "new_len", "pools", "page_table", "ref")}


# ------------------------------------------------------------------ 64 bits
def _e4m3_table():
    """The 256 e4m3 values, from their bit fields."""
    v = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = math.nan if (b & 127) == 127 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        v.append(-x if b >> 7 else x)
    return torch.tensor(v, dtype=torch.float64, device=DEV)


def _read64(pool, head, page, slot, d, fp8):
    """[n, d] of a head's positions (page, slot)."""
    part = pool[:, head]
    if fp8:
        byte = part[page[:, None], slot[:, None] * d + torch.arange(d, device=DEV)]
        scale = part[page[:, None], PAGE * d + 4 * slot[:, None] + torch.arange(4, device=DEV)]
        return _e4m3_table()[byte.long()] * scale.reshape(-1).view(torch.float32).double()[:, None]
    rows = part[page[:, None], 2 * slot[:, None] * d + torch.arange(2 * d, device=DEV)]
    return rows.reshape(-1).view(torch.bfloat16).double().reshape(-1, d)


def exact(case, seed):
    if case["op"] != "attn":
        return None  # ids, counts and copied bytes: no rounding anywhere
    s = prepare(case, seed)
    c = case
    rows, group = s["starts"][-1], c["hq"] // c["hkv"]
    out = torch.zeros(rows, c["hq"], c["d"], dtype=torch.float64, device=DEV)
    lse = torch.full((rows, c["hq"]), -math.inf, dtype=torch.float64, device=DEV)
    parent = s["parent"].tolist()
    for r, (length, n) in enumerate(zip(s["lens"], s["nodes"])):
        if n == 0:
            continue
        # node by node: its parent's row of ancestors, and itself
        sees = torch.zeros(n, length + n, dtype=torch.bool)
        sees[:, :length] = True
        for i in range(n):
            if parent[r][i] >= 0:
                sees[i] |= sees[parent[r][i]]
            sees[i, length + i] = True
        sees = sees.to(DEV)
        at = torch.arange(length + n, device=DEV)
        page, slot = s["page_table"][r].long()[at // PAGE], at % PAGE
        rows_of = slice(s["starts"][r], s["starts"][r] + n)
        for h in range(c["hkv"]):
            k = _read64(s["k_pool"], h, page, slot, c["d"], c["fp8"])
            v = _read64(s["v_pool"], h, page, slot, c["d"], c["fp8"])
            for g in range(h * group, (h + 1) * group):
                x = s["q"][rows_of, g].double() @ k.T * s["scale"]
                x = x.masked_fill(~sees, -math.inf)
                z = torch.logsumexp(x, -1)
                out[rows_of, g] = torch.exp(x - z[:, None]) @ v
                lse[rows_of, g] = z
    return {"out": out, "lse": lse}

"""PagedCache's drafted steps without a GPU: the calls are replaced by plain
statements of their contract over host tensors."""
import numpy as np
import pytest
import torch

from oracle import draft_oracle as D
from test_paged_host import i32, make  # noqa: F401  (the fixture replaces the page calls)


@pytest.fixture
def cache(make, monkeypatch):  # noqa: F811
    from two_level_sparse_gb300 import paged

    drafts = paged.drafts

    def put(to, value):
        to.copy_(torch.from_numpy(np.asarray(value).astype(np.int64)).to(torch.int32))

    def plan(length, count, parent, table, num_pages, start, positions, cache_pos, mask, token, row_token, dev_err):
        words = mask.shape[1] if mask is not None else 8
        got = D.plan(length.tolist(), count.tolist(), None if parent is None else parent.tolist(), token.tolist(),
                     table.numpy(), num_pages, len(positions), token.shape[1], words)
        for to, value in zip((start, positions, cache_pos, mask, row_token), got):
            if to is not None:
                put(to, value.astype(np.uint32).view(np.int32) if to is mask else value)

    def accept(start, length, parent, row_token, target, path, kept, after, new_len, cache_pos, dev_err):
        got = D.accept(start.tolist(), length.tolist(), None if parent is None else parent.tolist(), row_token.tolist(),
                       target.tolist(), cache_pos.tolist(), path.shape[1])
        for to, value in zip((path, kept, after, new_len), got):
            put(to, value)

    def move(pools, rows, scales, table, length, path, kept, dev_err):
        for p, row, scale in zip(pools, rows, scales, strict=True):
            q = D.move(p.numpy().reshape(len(p), -1, p.shape[-1]), row, scale, table.numpy(), length.tolist(),
                       path.tolist(), kept.tolist())
            p.copy_(torch.from_numpy(q.reshape(p.shape)))

    def trim(table, ref, old, new, dev_err):
        t, f = D.trim(table.numpy(), ref.numpy(), old.tolist(), new.tolist())
        put(table, t), put(ref, f)

    monkeypatch.setattr(drafts, "ci_draft_plan", plan)
    monkeypatch.setattr(drafts, "ci_draft_accept", accept)
    monkeypatch.setattr(drafts, "ci_slots_move", move)
    monkeypatch.setattr(drafts, "ci_pages_trim", trim)
    return make


def write(c, draft, names):
    """Every stored row's key gets its name (its first byte)."""
    for t, (r, at) in enumerate(names):
        if at >= 0 and draft.cache_pos[t] >= 0:
            page = int(c.page_table[r, int(draft.cache_pos[t]) // 64])
            c.k[0, page, 0, 128 * (int(draft.cache_pos[t]) % 64)] = at


def held(c, r):
    return [int(c.k[0, int(c.page_table[r, s // 64]), 0, 128 * (s % 64)]) for s in range(int(c.length[r]))]


def consistent(c):
    table, ref = c.page_table.numpy(), np.zeros(len(c.ref_count), int)
    for r, n in enumerate(c.length.tolist()):
        pages = -(-n // 64)
        assert (table[r, :pages] >= 0).all() and (table[r, pages:] == -1).all()
        np.add.at(ref, table[r, :pages], 1)
    np.testing.assert_array_equal(ref, c.ref_count.numpy())


@pytest.mark.parametrize("tree", [True, False])
def test_steps_keep_what_was_accepted(cache, tree):
    rng = np.random.default_rng(tree)
    c = cache(requests=3, max_pages=3, num_pages=8)
    c.grow(i32(60, 0, 5))
    want = [[0] * 60, [], [0] * 5]
    name = 0
    for step in range(12):
        count = rng.integers(0, 8, 3)
        parent = np.full((3, 7), -1)
        for r in range(3):
            for i in range(1, count[r]):
                parent[r, i] = rng.integers(0, i)
        token, target = rng.integers(0, 2, (3, 7)), rng.integers(0, 2, 21)
        c.dev_err.zero_()
        d = c.draft(i32(*count.tolist()), torch.tensor(token, dtype=torch.int32),
                    torch.tensor(parent, dtype=torch.int32) if tree else None)
        starts, names = d.req_start.tolist(), []
        for r in range(3):
            for _ in range(starts[r + 1] - starts[r]):
                name = (name + 1) % 256
                names.append((r, name))
        write(c, d, names)
        if step % 4 == 3:
            c.drop(d)
        else:
            path, kept, after = c.commit(d, torch.tensor(target, dtype=torch.int32))
            for r in range(3):
                want[r] += [names[starts[r] + i][1] for i in path[r, :int(kept[r])].tolist()]
        consistent(c)
        assert [held(c, r) for r in range(3)] == want


def test_nothing_else_changes_the_requests_meanwhile(cache):
    c = cache()
    c.grow(i32(60, 64, 0, 5))
    tokens = torch.ones(4, 3, dtype=torch.int32)
    d = c.draft(i32(3, 0, 1, 2), tokens)
    for f in (lambda: c.grow(c.length), lambda: c.free(i32(0)), c.compact, lambda: c.fork(i32(0), i32(1), i32(3)),
              lambda: c.draft(i32(0, 0, 0, 0), tokens)):
        with pytest.raises(RuntimeError, match="open"):
            f()
    c.drop(d)
    consistent(c)
    with pytest.raises(RuntimeError, match="not open"):
        c.drop(d)
    c.grow(c.length + 1)
    consistent(c)


def test_drafts_that_do_not_fit(cache):
    c = cache(requests=2, max_pages=2, num_pages=3)
    c.grow(i32(128, 60))
    ones = torch.ones(2, 5, dtype=torch.int32)
    d = c.draft(i32(1, -1), ones)
    assert d.req_start.tolist() == [0, 0, 0] and d.end.tolist() == [128, 60]
    assert c.commit(d, torch.ones(10, dtype=torch.int32))[1].tolist() == [0, 0]
    c.ref_count[c.ref_count == 0] = 1  # no page is free
    d = c.draft(i32(0, 5), ones)
    assert d.cache_pos[:5].tolist() == [60, 61, 62, 63, -1]
    path, kept, after = c.commit(d, torch.ones(10, dtype=torch.int32))
    assert kept.tolist() == [0, 4] and after.tolist() == [-1, 1] and c.length.tolist() == [128, 64]


def test_a_refused_draft_leaves_no_pages(cache, monkeypatch):
    from two_level_sparse_gb300 import paged

    c = cache(requests=3, max_pages=4, num_pages=6)
    c.grow(i32(60, 0, 128))
    before = c.page_table.clone(), c.ref_count.clone()
    plan = paged.drafts.ci_draft_plan

    def refuses(*args, **kw):
        raise TypeError("token must be torch.int32, got torch.int64")

    tokens = torch.ones(3, 9, dtype=torch.int32)
    monkeypatch.setattr(paged.drafts, "ci_draft_plan", refuses)
    for _ in range(3):  # (each would take four of the last three pages)
        with pytest.raises(TypeError, match="token"):
            c.draft(i32(9, 9, 9), tokens.long())
        assert torch.equal(c.page_table, before[0]) and torch.equal(c.ref_count, before[1])
    monkeypatch.setattr(paged.drafts, "ci_draft_plan", plan)
    with pytest.raises(RuntimeError):  # no tensor has so many rows
        c.draft(i32(9, 9, 9), tokens, rows=-1)
    assert torch.equal(c.page_table, before[0]) and torch.equal(c.ref_count, before[1])
    c.drop(c.draft(i32(9, 9, 9), tokens))
    assert torch.equal(c.page_table, before[0]) and torch.equal(c.ref_count, before[1])


def test_companions_that_layers_share_are_moved_once(cache):
    c = cache(requests=1, max_pages=2, num_pages=2)
    shared = torch.randint(0, 256, (2, 8448), dtype=torch.int32).to(torch.uint8)
    c.companions += [shared, torch.zeros(2, 4352, dtype=torch.uint8), shared[:, None], shared]
    c.grow(i32(10))
    parent = i32(-1, 0, 0, 1, 2, 4).view(1, 6)
    d = c.draft(i32(6), i32(0, 1, 2, 3, 4, 5).view(1, 6), parent)
    was = shared.clone()
    path, kept, _ = c.commit(d, i32(2, 0, 4, 0, 5, 0))
    assert path[0, :int(kept)].tolist() == [0, 2, 4, 5]
    page, row = int(c.page_table[0, 0]), lambda t, at: t[page, 128 * at:128 * at + 128]
    for at, node in enumerate([0, 2, 4, 5]):
        assert torch.equal(row(shared, 10 + at), row(was, 10 + node))


@pytest.mark.parametrize("bad", [torch.zeros(2, 8448, dtype=torch.uint8), torch.zeros(4, 8448, dtype=torch.uint8),
                                 torch.zeros(3, 8448), torch.zeros(3, 8448, dtype=torch.uint8, device="meta"),
                                 torch.zeros(8448, 3, dtype=torch.uint8).t(), torch.zeros(3, 8192, dtype=torch.uint8)])
def test_companions_are_looked_at_before_anything_happens(cache, bad):
    c = cache(requests=1, max_pages=3, num_pages=3)
    c.grow(i32(64))
    before = c.page_table.clone(), c.ref_count.clone()
    tokens = torch.ones(1, 3, dtype=torch.int32)
    c.companions.append(bad)
    with pytest.raises(ValueError, match="companions"):
        c.draft(i32(3), tokens)
    assert torch.equal(c.page_table, before[0]) and torch.equal(c.ref_count, before[1])
    c.companions.pop()
    d = c.draft(i32(3), tokens)
    c.companions.append(bad)
    keys = c.k.clone()
    with pytest.raises(ValueError, match="companions"):  # the draft stays open, nothing has moved
        c.commit(d, torch.ones(3, dtype=torch.int32))
    assert torch.equal(c.k, keys) and c.length.tolist() == [64]
    c.companions.pop()
    assert c.commit(d, torch.ones(3, dtype=torch.int32))[1].tolist() == [3] and c.length.tolist() == [67]
    consistent(c)

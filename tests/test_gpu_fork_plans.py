"""kv4_fork where its plan has more to do than a decode step leaves it: many part pages in calls
whose workgroups each plan by themselves. Rules and inputs are those of test_gpu_continuations."""
import numpy as np
import pytest

from test_gpu_continuations import fork_check, fork_reference, fork_run, vbq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("olds,news", [(1, 64), (3, 64), (64, 64), (9, 33), (3, 65), (40, 1100)])
def test_part_pages_of_many_pieces(vbq, olds, news):  # noqa: F811
    """Pages that take many pieces to copy, of other lengths each, for most sequences of the call: a copy that workgroups
    count in another place would be made twice, or by none."""
    page, heads, dim, W = 512, 4, 128, 3
    rng = np.random.default_rng(olds + news)
    lens = rng.integers(page + 1, 2 * page, olds).astype(np.int32)
    lens[0] = page + 500
    used = 2 * olds
    n_pages = used + news + 5
    table = np.full((olds, W), -1, np.int32)
    table[:, :2] = rng.permutation(n_pages)[:used].reshape(olds, 2)
    refs = np.bincount(table[table >= 0], minlength=n_pages).astype(np.int32)
    parents = rng.integers(-1, olds, news).astype(np.int32)
    parents[:olds] = rng.permutation(olds)[:news]
    reserve = rng.integers(0, 30, news).astype(np.int32)
    reserve[parents < 0] = 0
    want = fork_reference(page, n_pages, table, lens, refs, parents, reserve)
    assert want[4] & 8 or len(want[3]) >= (parents >= 0).sum() - olds
    for _ in range(3):
        run = fork_run(vbq, page, heads, dim, n_pages, table, lens, refs, parents, reserve)
        fork_check(*run, want, page, heads, dim)


LONG = [
    # old sequences, new ones, width, most entries in reserve, pages to spare
    (1, 8, 64, 50, 400), (2, 3, 1200, 1100, 3500), (64, 64, 64, 60, 5000), (20, 64, 60, 40, 40), (63, 64, 63, 9, 300),
    (64, 300, 130, 120, 40000), (700, 900, 40, 30, 30000), (1100, 2100, 20, 18, 30000), (5, 70, 3000, 2900, 250000),
    (4200, 3000, 12, 10, 30000),
]


@pytest.mark.parametrize("case", range(len(LONG)))
def test_many_entries_in_reserve(vbq, case):  # noqa: F811
    """Rows of the table that name pages far beyond their tokens, with gaps, pages that another row names too and numbers
    outside the cache among them: the first continuation keeps those that are its own, others are taken."""
    olds, news, W, most, spare = LONG[case]
    page = 32
    rng = np.random.default_rng(case)
    table = np.full((olds, W), -1, np.int32)
    lens = rng.integers(0, (W - most) * page + 1, olds).astype(np.int32)
    used = 0
    for b in range(olds):
        n = -(-int(lens[b]) // page) + int(rng.choice([0, 1, 5, 8, 9, most], p=[0.1, 0.1, 0.1, 0.1, 0.1, 0.5]))
        n = min(n, W)
        table[b, :n] = np.arange(used, used + n)
        used += n
    n_pages = used + spare
    number = rng.permutation(n_pages).astype(np.int32)
    table = np.where(table >= 0, number[np.maximum(table, 0)], -1).astype(np.int32)
    held = np.arange(W)[None] >= -(-lens[:, None] // page)
    gaps = held & (rng.random((olds, W)) < 0.1)
    table[gaps] = -1
    again = held & (table >= 0) & (rng.random((olds, W)) < 0.05)       # named by another row too
    table[again] = rng.choice(table[table >= 0], int(again.sum())) if again.any() else table[again]
    if case % 3 == 1:
        table[held & (rng.random((olds, W)) < 0.02)] = n_pages + 7
    there = (table >= 0) & (table < n_pages)
    refs = np.bincount(table[there], minlength=n_pages).astype(np.int32)
    parents = rng.integers(-1, olds, news).astype(np.int32)
    reserve = np.minimum(rng.choice([0, 1, 9 * page, most * page, (most + 3) * page], news), W * page).astype(np.int32)
    want = fork_reference(page, n_pages, table, lens, refs, parents, reserve)
    run = fork_run(vbq, page, 1, 64, n_pages, table, lens, refs, parents, reserve)
    fork_check(*run, want, page, 1, 64)


@pytest.mark.parametrize("olds,news", [(5, 30), (90, 200)])
def test_a_stack_of_layers(vbq, olds, news):  # noqa: F811
    """A cache a layer, one table: a call for each with the same inputs gives the same numbers, into the same outputs."""
    import torch

    from test_gpu_continuations import fork_case
    page, W = 64, 6
    rng = np.random.default_rng(olds)
    n_pages, table, lens, refs, parents, more = fork_case(rng, olds, news, W, page, 2000, reserve=90)
    want = fork_reference(page, n_pages, table, lens, refs, parents, more)
    shapes = [(2, 64), (1, 128), (3, 64)]
    caches = [vbq.Kv4Cache(n_pages, page, heads, dim) for heads, dim in shapes]
    before = []
    for c in caches:
        c.data.copy_(torch.randint(0, 256, (c.nbytes,), dtype=torch.uint8))
        before.append(c.data.clone())
    t = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (refs, table, lens, parents)]
    more = torch.from_numpy(more).cuda()
    out, ws = None, vbq.kv4_fork_workspace(caches[0], news, W, olds)
    for c in caches:
        out = vbq.kv4_fork(c, *t, reserve=more, out=out, workspace=ws)
    torch.cuda.synchronize()
    for c, b, (heads, dim) in zip(caches, before, shapes):
        fork_check(c, b, [o.cpu().numpy() for o in out], want, page, heads, dim)

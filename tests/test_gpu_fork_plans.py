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

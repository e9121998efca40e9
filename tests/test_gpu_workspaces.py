"""One workspace for the calls of a serving step one after the other: attention of each sequence by itself and attention
with shared tokens keep counters in it between calls, and neither may leave numbers in the other's."""
import numpy as np
import pytest

from test_gpu_continuations import vbq  # noqa: F401
from test_gpu_shared import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,ratio,dim,count", [(2, 1, 64, 8), (2, 4, 128, 6), (1, 2, 256, 8), (2, 4, 128, 40)])
@pytest.mark.parametrize("source", ["shared", "attention"])
def test_attention_of_both_kinds_on_one_workspace(vbq, heads, ratio, dim, count, source):  # noqa: F811
    """Few rows (8 to 32 a group) and many, cut into parts that are joined by the last."""
    import torch
    rng = np.random.default_rng(dim + count)
    case = Case(rng, heads, ratio, dim, 64, [(4000, [(int(n), 1) for n in rng.integers(1, 90, count)])])
    args = case.args(vbq, far=True)
    one = dict(args, max_shared=4000)
    table = torch.from_numpy(np.ascontiguousarray(case.full)).cuda()   # (every sequence's own row for its shared tokens too)
    apart = vbq.Kv4Cache(case.n_pages, 64, heads, dim, data=torch.from_numpy(case.data).cuda())
    plain = (apart, args["q"], table, args["kv_lens"], args["cu_q"], 1, max(case.lens))
    want_plain, want_far, want_one = vbq.kv4_attention(*plain), vbq.kv4_attention_shared(**args), vbq.kv4_attention_shared(**one)
    H, group = heads * ratio, (1, len(case.q), heads * ratio, 1)
    sizes = [vbq.kv4_attention_shared_workspace(args["cache"], count, *group, m, args["max_own"]) for m in (1 << 22, 4000)]
    sizes.append(vbq.kv4_attention_workspace(apart, count, len(case.q), H, 1, max(case.lens)))
    most = max(w.numel() for w in sizes)
    assert sizes[2].numel() > 8 * vbq.KV4_COUNTERS
    first = sizes[0] if source == "shared" else sizes[2]
    ws = torch.full((most,), 0xFF, dtype=torch.uint8, device="cuda")
    counters = 8 * vbq.KV4_COUNTERS
    ws[:counters] = first[:counters]
    for _ in range(3):
        for call, want in ((lambda: vbq.kv4_attention(*plain, workspace=ws), want_plain),
                           (lambda: vbq.kv4_attention_shared(**args, workspace=ws), want_far),
                           (lambda: vbq.kv4_attention_shared(**one, workspace=ws), want_one)):
            assert torch.equal(call(), want)
            assert not ws[:counters].any()

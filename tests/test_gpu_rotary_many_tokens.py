"""head_norm_rotary on more tokens than one dimension of a launch holds."""
import pytest

from test_gpu_continuations import vbq  # noqa: F401

pytestmark = pytest.mark.gpu


def test_more_tokens_than_a_launch_is_wide(vbq):  # noqa: F811
    """One head of 64 in place (8.6 GB): every token holds the same numbers, at position 0 but for a few, so what each
    has to give is known from a short call."""
    import torch
    T = (1 << 26) + 5
    plan = vbq.HeadRotary(64, torch.linspace(1, 0.01, 32, device="cuda"), q_weight=torch.full((64,), 0.75, device="cuda"))
    row = torch.randn(64, generator=torch.Generator().manual_seed(0)).bfloat16().cuda()
    q = row.expand(T, 1, 64).contiguous()
    at = torch.zeros(T, dtype=torch.int32, device="cuda")
    special = [1, (1 << 25) - 1, 1 << 25, 1 << 25 | 3, (1 << 26) - 1, 1 << 26, T - 1]
    at[special] = torch.arange(1, len(special) + 1, dtype=torch.int32, device="cuda")
    few = torch.arange(len(special) + 1, dtype=torch.int32, device="cuda")
    want = vbq.head_norm_rotary(plan, row.expand(len(few), 1, 64).contiguous(), None, few)[0]
    assert not torch.equal(want[0], row.view(1, 64)) and len({tuple(w.view(-1).tolist()) for w in want}) == len(few)
    vbq.head_norm_rotary(plan, q, None, at, q_out=q)
    for i in range(0, T, 1 << 23):
        part = q[i:i + (1 << 23)]
        assert torch.equal(part, want[at[i:i + (1 << 23)].long()]), i

"""token_logprobs on finite logits of every size (masks with large negative numbers, rows
around the sizes at which exponents are worked out in another way), against the formula in
64 bits; the reference and the bounds are those of test_gpu_continuations."""
import numpy as np
import pytest

from test_gpu_continuations import dtype_of, logprob_bounds, logprob_reference, vbq  # noqa: F401

pytestmark = pytest.mark.gpu

FILLS = [-1e9, -3e9, -1e10, -3e10, -1e12, -1e20, -1e30, -3e38]


def hold(vbq, x, top, seed=0):  # noqa: F811
    """x: CPU rows; every output against the formula, of tokens at random and of the largest logit."""
    import torch
    M, V = x.shape
    tokens = np.random.default_rng(seed).integers(0, V, M)
    tokens[1::2] = x.float().argmax(1).numpy()[1::2]
    r = vbq.token_logprobs(x.cuda(), torch.from_numpy(tokens).cuda(), top=top)
    x = x.double().numpy()
    lse, entropy, logp, rank, top_logp, top_index = logprob_reference(x, tokens, top)
    b_lse, b_ent, b_top = logprob_bounds(x, lse, entropy, V, np.concatenate([logp[:, None], top_logp], 1))
    with np.errstate(over="ignore"):       # differences that fp32 does not hold are -infinity
        logp, top_logp = (np.where(np.isneginf(a.astype(np.float32)), -np.inf, a) for a in (logp, top_logp))
    assert np.array_equal(r.rank.cpu().numpy(), rank)
    assert np.array_equal(r.top_index.cpu().numpy(), top_index)
    for got, ref, bound, what in ((r.lse, lse, b_lse, "lse"), (r.entropy, entropy, b_ent, "entropy"),
                                  (r.logprob, logp, b_top[:, 0], "logprob"), (r.top_logprob, top_logp, b_top[:, 1:], "top")):
        got = got.double().cpu().numpy()
        assert np.array_equal(np.isneginf(got), np.isneginf(ref)) and not np.isnan(got).any(), f"{what}: {got}"
        fine = np.isfinite(ref)
        off = np.abs(np.where(fine, got - np.where(fine, ref, 0), 0)) - np.where(fine, bound, 0)
        assert off.max() <= 0, f"{what}: {off.max()} beyond the bound"


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,vocab", [(5, 128256), (5, 1500), (600, 5003)])       # shared out, of a wavefront, of a workgroup
@pytest.mark.parametrize("fill", FILLS)
def test_masks_of_large_negative_numbers(vbq, dtype, rows, vocab, fill):  # noqa: F811
    import torch
    x = torch.randn(rows, vocab, generator=torch.Generator().manual_seed(vocab)) * 3
    few = vocab // 40
    x[0::5, :-few] = fill                              # ordinary logits behind,
    x[1::5, few:] = fill                               # in front,
    x[2::5, :vocab // 2] = fill                        # in the middle,
    x[2::5, vocab // 2 + few:] = fill
    x[3::5, torch.arange(vocab) % 997 != 5] = fill     # here and there
    x[4::5] = fill                                     # nowhere
    hold(vbq, x.to(dtype_of(dtype)), 20)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,vocab", [(4, 50001), (4, 2047), (515, 4097)])
@pytest.mark.parametrize("size", [1e6, 4e6, 5e6, 1e9, 2e9, 1e10, 1e20, 1e30, 3e38])
def test_rows_of_large_numbers(vbq, dtype, rows, vocab, size):  # noqa: F811
    import torch
    g = torch.Generator().manual_seed(vocab)
    x = torch.randn(rows, vocab, generator=g)
    x[0::4] += size
    x[1::4] = x[1::4].clamp(-1, 1) * size
    x[2::4] -= size
    x[3::4] = torch.where(torch.rand(vocab, generator=g) < 0.5, size, -size)
    hold(vbq, x.to(dtype_of(dtype)), 32)


@pytest.mark.parametrize("rows,vocab", [(9, 40003), (9, 1999), (540, 6007)])
@pytest.mark.parametrize("edge", [2.0 ** 21, 2.0 ** 22, 2.0 ** 23, 2.0 ** 29, 2.0 ** 30, 2.0 ** 31, 2.0 ** 100])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_maxima_on_both_sides(vbq, rows, vocab, edge, sign):  # noqa: F811
    """Stretches of a row whose maxima are of either kind, as near to each other as fp32 has numbers, and further away."""
    step = edge * 2.0 ** -23
    g = np.random.default_rng(int(np.log2(edge)))
    x = np.empty((rows, vocab))
    for r in range(rows):
        reach = (2, 5, 0.1 * edge / step)[r % 3]
        near = edge + step * np.round(g.uniform(-reach, reach, vocab))
        if r % 9 < 3:            # rising stretches
            near = np.sort(near)
        elif r % 9 < 6:          # falling ones
            near = np.sort(near)[::-1]
        x[r] = sign * near
    import torch
    hold(vbq, torch.from_numpy(x.astype(np.float32)), 32)

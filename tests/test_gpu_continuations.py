"""The operators for several continuations of one prompt on the GPU, each against its
formula in 64 bits: head_norm_rotary, kv4_fork, token_logprobs."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

HALF_STEP = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8, "float32": 2.0 ** -24}
TINY = {"float16": 2.0 ** -25, "bfloat16": 0.0, "float32": 0.0}   # half a step of the type's smallest numbers


@pytest.fixture(scope="module")
def vbq():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import packed_decode_gemv_amd as vbq
    return vbq


def dtype_of(name):
    import torch
    return getattr(torch, name)


# ---- head_norm_rotary --------------------------------------------------------------
def rotary_reference(x, pos, inv_freq, axis, interleaved, weight, eps):
    """x float64 [T][H][D], pos int [axes][T]: the formula in 64 bits, and the size of the numbers that enter
    each output's sum."""
    D, half = x.shape[2], len(inv_freq)
    n = x if weight is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    out, size = n.copy(), np.abs(n)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        phi = pos[axis[i]].astype(np.float64) * np.float64(inv_freq[i])
        c, s = np.cos(phi)[:, None], np.sin(phi)[:, None]
        out[..., a] = n[..., a] * c - n[..., b] * s
        out[..., b] = n[..., b] * c + n[..., a] * s
        size[..., a] = size[..., b] = np.abs(n[..., a]) + np.abs(n[..., b])
    return out, size


def rotary_bound(ref, size, out_dtype, far, normed):
    """Each output is a c - b s in binary32 with n of relative error: norm: the sum of D <= 256 squares (16 in a
    chain, then 4 exchanges: 20 roundings, halved by the root: 10), the mean's and eps's (1), the root (2), two
    products (2): 15. cos and sin: 2 steps each and the angle's: turns to binary32 2^-25 of a turn at most half a
    turn, 2 pi times: 2^-22.3, so 4 steps of 2^-24 and the binary64 error of positions beyond 2^20 (2^-52 of the
    turns, 2 pi times). Two products and a sum: 2. Then one rounding to the output's type."""
    u = 2.0 ** -24
    rel = ((15 if normed else 0) + 2 + 4 + 2) * u + 2.0 ** -52 * 4 * (far + 1)
    return rel * size + HALF_STEP[out_dtype] * (np.abs(ref) + rel * size) + TINY[out_dtype]


ROTARY = [
    # in, out, tokens, heads, kv heads, dim, rotary, axes, interleaved, norm, far
    ("float32", "float16", 1, 12, 12, 64, 64, 1, False, True, 4000),
    ("float32", "float32", 3, 5, 1, 64, 64, 1, True, False, 1 << 31),
    ("float16", "float16", 5, 8, 2, 128, 128, 1, False, True, 1 << 20),
    ("bfloat16", "bfloat16", 70, 32, 8, 128, 64, 3, False, True, 100000),
    ("bfloat16", "float32", 2, 7, 3, 192, 192, 2, True, True, 5000),
    ("float16", "bfloat16", 9, 6, 2, 192, 96, 1, False, True, 5000),
    ("float32", "bfloat16", 130, 16, 4, 256, 128, 3, True, True, 1200),
    ("float32", "float16", 4, 5, 1, 256, 256, 1, False, False, 1200),
    ("bfloat16", "float16", 6, 17, 3, 128, 16, 2, True, False, 1200),
    ("float16", "float32", 2, 3, 1, 128, 0, 1, False, True, 1),
]


def rotary_inputs(case, seed=0):
    import torch
    din, dout, T, H, K, D, R, axes, inter, norm, far = case
    rng = np.random.default_rng(seed + T + D + R)
    x = [torch.from_numpy(rng.normal(0, 3, (T, n, D)).astype(np.float32)).to(dtype_of(din)) for n in (H, K)]
    pos = rng.integers(-far if far < 1 << 31 else -(1 << 31), far, (axes, T)).astype(np.int32)
    inv = (10000.0 ** (-np.arange(R // 2) / max(1, R // 2))).astype(np.float32)
    axis = rng.integers(0, axes, R // 2).astype(np.uint8)
    w = [rng.normal(1, 0.3, D).astype(np.float32) if norm else None for _ in range(2)]
    return x, pos, inv, axis, w


def rotary_plan(vbq, case, inv, axis, w, eps=1e-5):
    import torch
    axes, inter, D = case[7], case[8], case[5]
    return vbq.HeadRotary(D, torch.from_numpy(inv).cuda() if len(inv) else None,
                          axis=torch.from_numpy(axis).cuda() if axes > 1 else None, axes=axes, interleaved=inter,
                          q_weight=None if w[0] is None else torch.from_numpy(w[0]).cuda(),
                          k_weight=None if w[1] is None else torch.from_numpy(w[1]).cuda(), eps=eps)


def close(got, ref, bound, what=""):
    got = got.detach().double().cpu().numpy()
    off = np.abs(got - ref) - bound
    assert got.shape == ref.shape and (off <= 0).all(), f"{what}: {off.max()} beyond the bound at {np.unravel_index(off.argmax(), off.shape)}"


@pytest.mark.parametrize("case", range(len(ROTARY)))
@pytest.mark.parametrize("layout", ["apart", "slices", "in place"])
def test_rotary_against_the_formula(vbq, case, layout):
    import torch
    case = ROTARY[case]
    din, dout, T, H, K, D, R, axes, inter, norm, far = case
    x, pos, inv, axis, w = rotary_inputs(case)
    plan = rotary_plan(vbq, case, inv, axis, w)
    q, k = (t.cuda() for t in x)
    dpos = torch.from_numpy(pos if axes > 1 else pos[0]).cuda()
    out = dtype_of(dout)
    if layout == "slices":
        both = torch.cat([q.flatten(1), k.flatten(1), torch.zeros(T, 64, dtype=q.dtype, device="cuda")], 1)
        q, k = both[:, :H * D].unflatten(1, (H, D)), both[:, H * D:(H + K) * D].unflatten(1, (K, D))
    if layout == "in place":
        dout, out = din, dtype_of(din)
        gq, gk = vbq.head_norm_rotary(plan, q, k, dpos, q_out=q, k_out=k)
        assert gq is q and gk is k
    else:
        before = q.clone()
        gq, gk = vbq.head_norm_rotary(plan, q, k, dpos, q_dtype=out, k_dtype=out)
        assert torch.equal(q, before)
    for got, t, weight in ((gq, x[0], w[0]), (gk, x[1], w[1])):
        assert got.dtype is out
        ref, size = rotary_reference(t.double().numpy(), pos, inv, axis, inter, weight, 1e-5)
        close(got, ref, rotary_bound(ref, size, dout, far, norm))


def test_rotary_one_tensor_and_one_norm(vbq):
    import torch
    case = ROTARY[2]
    x, pos, inv, axis, w = rotary_inputs(case)
    plan = rotary_plan(vbq, case, inv, axis, (w[0], None))
    q, k, p = x[0].cuda(), x[1].cuda(), torch.from_numpy(pos[0]).cuda()
    both = vbq.head_norm_rotary(plan, q, k, p)
    only_q, none = vbq.head_norm_rotary(plan, q, None, p)
    none2, only_k = vbq.head_norm_rotary(plan, None, k, p)
    assert none is None and none2 is None
    assert torch.equal(both[0], only_q) and torch.equal(both[1], only_k)
    ref, size = rotary_reference(x[1].double().numpy(), pos, inv, axis, False, None, 0)
    close(only_k, ref, rotary_bound(ref, size, "float16", case[10], False))


def test_rotary_of_no_tokens_and_special_numbers(vbq):
    import torch
    case = ROTARY[2]
    x, pos, inv, axis, w = rotary_inputs(case)
    plan = rotary_plan(vbq, case, inv, axis, w)
    p = torch.from_numpy(pos[0]).cuda()
    q, k = vbq.head_norm_rotary(plan, x[0][:0].cuda(), x[1][:0].cuda(), p[:0])
    assert q.shape == (0, 8, 128) and k.shape == (0, 2, 128)
    a, b = x[0].clone(), x[1].clone()
    a[1, 2, 5] = float("nan")
    a[3, 0, 7] = float("inf")
    b[2] = 0.0
    clean = vbq.head_norm_rotary(plan, x[0].cuda(), x[1].cuda(), p)
    got = vbq.head_norm_rotary(plan, a.cuda(), b.cuda(), p)
    touched = torch.zeros(5, 8, dtype=torch.bool)
    touched[1, 2] = touched[3, 0] = True
    assert got[0][touched.cuda()].isnan().any(-1).all()
    assert torch.equal(got[0][~touched.cuda()], clean[0][~touched.cuda()])    # a head keeps its numbers to itself
    assert (got[1][2] == 0).all()                                            # eps keeps zeros


def test_rotary_stream_and_graph(vbq):
    import torch
    case = ROTARY[3]
    x, pos, inv, axis, w = rotary_inputs(case)
    plan = rotary_plan(vbq, case, inv, axis, w)
    q, k, p = x[0].cuda(), x[1].cuda(), torch.from_numpy(pos).cuda()
    want = vbq.head_norm_rotary(plan, q, k, p)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = vbq.head_norm_rotary(plan, q, k, p, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = [torch.zeros_like(t) for t in want]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        vbq.head_norm_rotary(plan, q, k, p, q_out=out[0], k_out=out[1])
    for shift in (0, 7, 1000):
        p.copy_(torch.from_numpy(pos + shift))
        g.replay()
        want = vbq.head_norm_rotary(plan, q, k, p)
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_rotary_refusals(vbq):
    import torch
    inv = torch.ones(32, device="cuda")
    plan = vbq.HeadRotary(64, inv)
    q = torch.zeros(3, 2, 64, device="cuda")
    p = torch.zeros(3, dtype=torch.int32, device="cuda")
    for bad in (dict(inv_freq=inv[:4]), dict(inv_freq=torch.ones(40, device="cuda")), dict(inv_freq=inv.double()),
                dict(inv_freq=None), dict(inv_freq=inv, axes=2), dict(inv_freq=inv, eps=-1.0),
                dict(inv_freq=inv, q_weight=torch.ones(32, device="cuda")), dict(inv_freq=inv.cpu()),
                dict(inv_freq=inv, axis=torch.full((32,), 2, dtype=torch.uint8, device="cuda"), axes=2),
                dict(inv_freq=inv, k_weight=torch.ones(65, device="cuda")[1:])):
        with pytest.raises(ValueError):
            vbq.HeadRotary(64, **bad)
    with pytest.raises(ValueError):
        vbq.HeadRotary(96, inv)
    for args in ((q.double(), None, p), (q[:, :, :32], None, p), (q, q[:2], p), (q, q.half(), p), (q, None, p[:2]),
                 (q, None, p.long()), (None, None, p), (q.cpu(), None, p), (q.transpose(1, 2), None, p), (q[0], None, p)):
        with pytest.raises(ValueError):
            vbq.head_norm_rotary(plan, *args)
    with pytest.raises(ValueError):
        vbq.head_norm_rotary(plan, q, None, p, q_out=torch.zeros(2, 2, 64, device="cuda"))
    with pytest.raises(ValueError):
        vbq.head_norm_rotary(plan, q, None, p, q_out=q, q_dtype=torch.float16)
    with pytest.raises(ValueError):
        vbq.head_norm_rotary(plan, torch.zeros(3 * 128 + 1, device="cuda")[1:].view(3, 2, 64), None, p)


# ---- token_logprobs ----------------------------------------------------------------
def logprob_reference(x, tokens, top):
    """x float64 [M][V]: lse, entropy, the tokens' log probabilities and ranks, and the most likely ones."""
    with np.errstate(invalid="ignore", divide="ignore"):
        m = x.max(1, keepdims=True)
        safe = np.where(np.isfinite(m), m, 0.0)
        log_s = np.log(np.exp(x - safe).sum(1, keepdims=True))
        lse = (safe + log_s)[:, 0]
        logp = (x - safe) - log_s
        logp[np.isneginf(x)] = -np.inf
        p = np.exp(logp)
        entropy = -np.where(p > 0, p * logp, 0.0).sum(1)
    order = np.argsort(-x, axis=1, kind="stable")
    place = np.empty_like(order)
    np.put_along_axis(place, order, np.arange(x.shape[1])[None], 1)
    rows = np.arange(len(x))
    return lse, entropy, logp[rows, tokens], place[rows, tokens], np.take_along_axis(logp, order[:, :top], 1), order[:, :top]


def logprob_bounds(x, lse, entropy, vocab, logp):
    """s and t are sums of up to `vocab` terms: a lane adds a 256th or more of them in a chain (with a row over one
    workgroup, vocab / 256 + 64 numbers), then 6 + 2 + 6 joins, each with a factor: n roundings, and each term e has
    3 steps (difference relative to itself, product, exp2: the exponent's error is |d| log2(e) 2^-23, and e d is
    below 2^-1.4 in size). lse = m + log s: log's error is s's relative one and 2 steps of itself."""
    u = 2.0 ** -24
    n = vocab / 256 + 64 + 40
    finite = np.isfinite(lse)
    top = np.where(finite, np.where(np.isfinite(x), x, -np.inf).max(1), 0.0)
    log_s = np.where(finite, lse - top, 0.0)
    rel = (n + 24) * u                    # of s (a term of weight e has |d| e <= 0.53 s, 16 steps of it)
    b_log = rel + 4 * u * np.abs(log_s)
    b_lse = b_log + 4 * u * (np.abs(top) + np.abs(log_s))
    b_ent = b_log + (2 * rel + 8 * u) * (entropy + log_s + 1)
    b_logp = b_log[:, None] + 4 * u * (np.abs(np.where(np.isfinite(logp), logp, 0)) + np.abs(log_s)[:, None])
    return b_lse, b_ent, b_logp


LOGPROBS = [
    # dtype, rows, vocab, top, kind
    ("float32", 1, 1, 1, "plain"), ("float32", 3, 2, 2, "plain"), ("float16", 5, 7, 5, "ties"),
    ("float32", 2, 300, 32, "plain"), ("bfloat16", 9, 1001, 16, "ties"), ("float32", 1, 2048, 20, "plain"),
    ("float32", 2, 2051, 32, "masked"), ("float16", 4, 4097, 32, "masked"), ("bfloat16", 3, 8191, 32, "ties"),
    ("float32", 1, 32001, 20, "plain"), ("bfloat16", 70, 32001, 16, "masked"), ("float16", 2, 50001, 8, "ascending"),
    ("float32", 2, 128256, 32, "ascending"), ("float32", 3, 128256, 32, "equal"), ("bfloat16", 2, 128256, 32, "equal"),
    ("float32", 2, 128256, 20, "few"), ("float32", 1100, 5003, 5, "plain"), ("float32", 5, 9999, 0, "plain"),
    ("float32", 2, 262147, 32, "far"), ("float32", 4, 3001, 7, "lowest"), ("float32", 1, 700001, 32, "descending"),
]


def logits_of(dtype, M, V, kind, seed):
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, V, generator=g) * 3
    if kind == "ties":
        x = (x * 2).round() / 2
    if kind == "masked":
        x[:, torch.randperm(V, generator=g)[:V - V // 50]] = -math.inf
    if kind == "ascending":
        x = torch.sort(x, 1).values
    if kind == "descending":
        x = torch.sort(x, 1, descending=True).values
    if kind == "equal":
        x = torch.full((M, V), -0.0)
        x[:, ::2] = 0.0
    if kind == "few":
        x[:] = -math.inf
        x[0, 77::9999] = 1.0
        x[1, V - 1] = -5.0
    if kind == "far":
        x += 3000.0
    if kind == "lowest":
        x[1] = torch.finfo(torch.float32).min
        x[2, 5:] = torch.finfo(torch.float32).min
        x[3] = -math.inf
    return x.to(dtype_of(dtype))


@pytest.mark.parametrize("case", range(len(LOGPROBS)))
@pytest.mark.parametrize("strided", [False, True])
def test_logprobs_against_the_formula(vbq, case, strided):
    import torch
    dtype, M, V, top, kind = LOGPROBS[case]
    x = logits_of(dtype, M, V, kind, case)
    rng = np.random.default_rng(case)
    tokens = rng.integers(0, V, M)
    if kind in ("masked", "few"):      # a token that is not masked, where there is one
        for r in range(0, M, 2):
            there = torch.isfinite(x[r].float()).nonzero()
            tokens[r] = int(there[int(rng.integers(len(there)))]) if len(there) else tokens[r]
    d = x.cuda()
    if strided:                         # rows at odd places
        wide = torch.full((M, V + 5), 99.0, dtype=d.dtype, device="cuda")
        wide[:, 3:3 + V] = d
        d = wide[:, 3:3 + V]
    r = vbq.token_logprobs(d, torch.from_numpy(tokens).cuda(), top=top)
    x = x.double().numpy()
    lse, entropy, logp, rank, top_logp, top_index = logprob_reference(x, tokens, top)
    b_lse, b_ent, b_top = logprob_bounds(x, lse, entropy, V, np.concatenate([logp[:, None], top_logp], 1))
    for got, ref, bound, what in ((r.lse, lse, b_lse, "lse"), (r.entropy, entropy, b_ent, "entropy"),
                                  (r.logprob, logp, b_top[:, 0], "logprob"),
                                  (r.top_logprob, top_logp, b_top[:, 1:], "top")):
        if got is None:
            assert top == 0
            continue
        got = got.double().cpu().numpy()
        assert np.array_equal(np.isneginf(got), np.isneginf(ref)) and not np.isnan(got).any(), what
        fine = np.isfinite(ref)
        off = (np.abs(np.where(fine, got - np.where(fine, ref, 0), 0)) - bound).max()
        assert off <= 0, f"{what}: {off} beyond the bound"
    assert np.array_equal(r.rank.cpu().numpy(), rank)
    if top:
        assert np.array_equal(r.top_index.cpu().numpy(), top_index)


def test_logprobs_rows_with_nan_or_infinity_and_tokens_outside(vbq):
    import torch
    x = torch.randn(6, 9001, device="cuda")
    clean = vbq.token_logprobs(x, torch.arange(6, device="cuda"), top=4)
    bad = x.clone()
    bad[1, 8000] = float("nan")
    bad[4, 3] = float("inf")
    tokens = torch.tensor([0, 1, -1, 9001, 4, 5], device="cuda")
    for t in (tokens, tokens.int()):
        r = vbq.token_logprobs(bad, t, top=4)
        for row in range(6):
            hurt = row in (1, 4)
            for got, want in ((r.lse, clean.lse), (r.entropy, clean.entropy), (r.top_logprob, clean.top_logprob)):
                assert got[row].isnan().all() if hurt else torch.equal(got[row], want[row])
            assert (r.top_index[row] == -1).all() if hurt else torch.equal(r.top_index[row], clean.top_index[row])
            if hurt or row in (2, 3):
                assert r.logprob[row].isnan() and int(r.rank[row]) == -1
            else:
                assert torch.equal(r.logprob[row], clean.logprob[row]) and int(r.rank[row]) == int(clean.rank[row])


def test_logprobs_without_tokens_or_rows(vbq):
    import torch
    x = torch.randn(3, 40000, device="cuda")
    a = vbq.token_logprobs(x, top=3)
    b = vbq.token_logprobs(x, torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert a.logprob is None and a.rank is None and b.top_index is None
    assert torch.equal(a.lse, b.lse) and torch.equal(a.entropy, b.entropy)
    e = vbq.token_logprobs(x[:0], torch.zeros(0, dtype=torch.int64, device="cuda"), top=2)
    assert e.logprob.shape == (0,) and e.top_index.shape == (0, 2)


def test_logprobs_graph_streams_and_one_workspace_for_other_sizes(vbq):
    import torch
    x = torch.randn(2, 128256, device="cuda")
    t = torch.tensor([5, 128255], device="cuda")
    w = vbq.token_logprobs_workspace(8, 128256, 20)
    w1 = vbq.token_logprobs_workspace(2, 128256, 20)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = vbq.token_logprobs(x, t, top=20, workspace=w1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        vbq.token_logprobs(x, t, top=20, out=out, workspace=w1)
    for i in range(4):
        x.copy_(torch.randn(2, 128256, device="cuda"))
        g.replay()
        want = vbq.token_logprobs(x, t, top=20, workspace=w)
        many = vbq.token_logprobs(x[:1].expand(8, -1), t[:1].expand(8).contiguous(), top=3, workspace=w)
        torch.cuda.synchronize()
        for u, v in zip(out, want):
            assert torch.equal(u, v)
        assert torch.equal(many.top_index, want.top_index[:1, :3].expand(8, -1))
    got = vbq.token_logprobs(x, t, top=20, stream=side)
    side.synchronize()
    for u, v in zip(got, out):
        assert torch.equal(u, v)


def test_logprobs_refusals(vbq):
    import torch
    x = torch.zeros(2, 100, device="cuda")
    t = torch.zeros(2, dtype=torch.int64, device="cuda")
    for bad in (dict(logits=x[0]), dict(logits=x.double()), dict(logits=x.cpu()), dict(logits=x.t()), dict(top=33),
                dict(top=-1), dict(logits=x[:, :3], top=4), dict(tokens=t[:1]), dict(tokens=t.float()),
                dict(tokens=t.cpu()), dict(workspace=torch.zeros(9, device="cuda"))):
        with pytest.raises(ValueError):
            vbq.token_logprobs(**{**dict(logits=x, tokens=t), **bad})
    r = vbq.token_logprobs(x, t, top=2)
    with pytest.raises(ValueError):
        vbq.token_logprobs(x, t, top=2, out=r._replace(rank=r.rank.long()))
    with pytest.raises(ValueError):
        vbq.token_logprobs(x, t, top=2, out=r._replace(top_index=None))
    with pytest.raises(vbq.VbqError):   # a workspace that is too small
        big = torch.zeros(1, 128256, device="cuda")
        vbq.token_logprobs(big, top=2, workspace=vbq.token_logprobs_workspace(1, 100, 2))


# ---- kv4_fork ------------------------------------------------------------------------
def fork_reference(page, n_pages, table, lens, refs, parents, reserve):
    """The rules one by one: new table, lengths, counts, copies (source page, destination page, blocks), and flags."""
    B, W = table.shape
    out = np.full((len(parents), W), -1, np.int32)
    new_lens = np.zeros(len(parents), np.int32)
    free = [p for p in range(n_pages) if refs[p] == 0]
    seen, copies, flags = set(), [], 0
    new_refs = refs.copy()
    for row in table:
        for e in row:
            if 0 <= e < n_pages:
                new_refs[e] -= 1
            elif e != -1:
                flags |= 1
    for b, p in enumerate(parents):
        more = int(reserve[b])
        if more < 0:
            more, flags = 0, flags | 2
        if p >= B:
            p, flags = -1, flags | 2
        L = 0
        if p >= 0:
            if 0 <= lens[p] <= W * page:
                L = int(lens[p])
            else:
                p, flags = -1, flags | 2
        first = p >= 0 and p not in seen
        seen.add(p)
        new_lens[b] = L
        need = -(-(L + more) // page)
        if need > W:
            need, flags = W, flags | 2
        for j in range(need):
            e = int(table[p, j]) if p >= 0 else -1
            valid = 0 <= e < n_pages
            if j * page < L and not valid:
                flags |= 1
            if j < L // page:
                out[b, j] = e if valid else -1
                continue
            if first and valid and refs[e] == 1:
                out[b, j] = e
                continue
            if not free:
                flags |= 8
                continue
            out[b, j] = free.pop(0)
            if j == L // page and L % page and valid:
                copies.append((e, out[b, j], -(-(L % page) // 32)))
    for row in out:
        for e in row:
            if e >= 0:
                new_refs[e] += 1
    return out, new_lens, new_refs, copies, flags


def fork_case(rng, B, N, W, page, spare, shared=True, reserve=0):
    """Sequences of a cache of which some share whole pages; parents of N new ones at random."""
    table = np.full((B, W), -1, np.int32)
    lens = rng.integers(0, W * page + 1, B).astype(np.int32)
    used = 0
    for b in range(B):
        have, whole = -(-int(lens[b]) // page), int(lens[b]) // page
        common = int(rng.integers(0, min(whole, lens[b - 1] // page) + 1)) if shared and b and rng.random() < 0.5 else 0
        table[b, :common] = table[b - 1, :common]
        more = have - common + (1 if rng.random() < 0.3 and have < W else 0)    # at times a page in reserve
        table[b, common:common + more] = np.arange(used, used + more)
        used += more
    n_pages = used + spare
    number = rng.permutation(n_pages).astype(np.int32)
    table = np.where(table >= 0, number[np.maximum(table, 0)], -1).astype(np.int32)
    refs = np.bincount(table[table >= 0], minlength=n_pages).astype(np.int32)
    parents = rng.integers(-1, B, N).astype(np.int32)
    more = rng.integers(0, reserve + 1, N).astype(np.int32)
    return n_pages, table, lens, refs, parents, more


def fork_run(vbq, page, heads, dim, n_pages, table, lens, refs, parents, reserve, **kw):
    import torch
    gen = torch.Generator().manual_seed(len(parents))
    cache = vbq.Kv4Cache(n_pages, page, heads, dim)
    cache.data.copy_(torch.randint(0, 256, (cache.nbytes,), generator=gen, dtype=torch.uint8))
    before = cache.data.clone()
    t = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (refs, table, lens, parents)]
    kept = [u.clone() for u in t]
    r = None if reserve is None else torch.from_numpy(reserve).cuda()
    got = vbq.kv4_fork(cache, *t, reserve=r, **kw)
    torch.cuda.synchronize()
    for u, v in zip(t, kept):
        assert torch.equal(u, v)
    return cache, before, [g.cpu().numpy() for g in got]


def fork_check(cache, before, got, want, page, heads, dim):
    import torch
    table, lens, refs, copies, flags = want
    assert np.array_equal(got[0], table) and np.array_equal(got[1], lens) and np.array_equal(got[2], refs)
    data = before.view(-1, heads, page // 32, 36 * dim).clone()
    for src, dst, blocks in copies:
        data[dst, :, :blocks] = data[src, :, :blocks]
    assert torch.equal(cache.data, data.view(-1))
    assert int(cache.flags.item()) == flags


FORK = [
    # before, after, width, page, spare pages, heads, dim, reserve
    (1, 1, 1, 32, 2, 1, 64, 0), (1, 8, 5, 32, 60, 2, 64, 40), (4, 20, 7, 64, 200, 3, 128, 100),
    (30, 30, 9, 128, 300, 1, 192, 1), (3, 5, 3, 256, 20, 2, 256, 300), (100, 700, 6, 32, 5000, 1, 64, 33),
    (1500, 1300, 4, 32, 20000, 1, 64, 5), (5000, 4200, 3, 32, 30000, 1, 64, 1), (2, 3, 300, 32, 700, 1, 64, 9000),
    (2, 2, 3, 2048, 9, 2, 64, 10), (7, 40, 4, 64, 3, 2, 64, 70),
    # many pages beside few sequences, and the sizes at which calls stop being small
    (5, 9, 6, 32, 4090, 1, 64, 40), (64, 64, 64, 32, 20000, 1, 64, 70), (64, 65, 8, 32, 900, 1, 64, 33),
    (65, 3, 8, 32, 900, 1, 64, 33), (64, 64, 65, 32, 5000, 1, 64, 70), (3, 4, 5, 32, 65520, 1, 64, 40),
    (3, 4, 5, 32, 65560, 1, 64, 40), (64, 20, 3, 512, 40, 3, 256, 600), (9, 64, 4, 1024, 200, 2, 128, 5),
]


@pytest.mark.parametrize("case", range(len(FORK)))
@pytest.mark.parametrize("kept", [False, True])
def test_fork_against_the_rules(vbq, case, kept):
    import torch
    B, N, W, page, spare, heads, dim, reserve = FORK[case]
    rng = np.random.default_rng(case)
    n_pages, table, lens, refs, parents, more = fork_case(rng, B, N, W, page, spare, reserve=reserve)
    kw = {}
    if kept:
        kw["out"] = tuple(torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((N, W), (N,), (n_pages,)))
        c = vbq.Kv4Cache(n_pages, page, heads, dim)
        kw["workspace"] = vbq.kv4_fork_workspace(c, N, W, B).fill_(0x5A)
    run = fork_run(vbq, page, heads, dim, n_pages, table, lens, refs, parents, more, **kw)
    fork_check(*run, fork_reference(page, n_pages, table, lens, refs, parents, more), page, heads, dim)


def test_fork_shapes_of_use(vbq):
    """One prompt continued eight times, then beams reordered, then all but one ended; pages held elsewhere stay."""
    page, heads, dim, W = 32, 2, 64, 6
    n_pages = 40
    table, lens = np.full((1, W), -1, np.int32), np.array([77], np.int32)
    table[0, :3] = (5, 9, 2)
    refs = np.zeros(n_pages, np.int32)
    refs[[5, 9, 2]] = 1
    refs[0] = 4
    for parents in ([0] * 8, [3, 3, 3, 0, 7, 7, 1, 3], [-1, -1, 4, -1], [-1, 2], [1, 1]):
        parents = np.array(parents, np.int32)
        more = np.full(len(parents), 1, np.int32)
        run = fork_run(vbq, page, heads, dim, n_pages, table, lens, refs, parents, more)
        want = fork_reference(page, n_pages, table, lens, refs, parents, more)
        fork_check(*run, want, page, heads, dim)
        table, lens, refs = want[:3]
        lens = lens + (lens > 0)          # a token each
        assert refs[0] == 4 and want[4] == 0
        held = np.bincount(table[table >= 0], minlength=n_pages)
        held[0] += 4
        assert np.array_equal(held, refs)


def test_fork_reports_what_does_not_fit(vbq):
    page, heads, dim, W = 32, 1, 64, 4
    table = np.array([[0, 1, 2, -1], [3, 99, 4, -1], [5, -1, -1, -1], [6, -2, 7, -1]], np.int32)
    for lens, parents, more in (([70, 70, 32, 65], [0, 4, 0, -1], [0, 0, 0, 0]),      # a parent beyond the sequences
                                ([70, 70, 32, 65], [1, 1, 0], [0, 0, 0]),              # an entry beyond the cache
                                ([70, 70, 129, 65], [2, 0], [0, 0]),                   # a length beyond the table
                                ([70, 70, -1, 65], [2, 0], [40, 0]),
                                ([70, 70, 64, 65], [2, 2], [0, 0]),                    # a page that is not there
                                ([70, 70, 63, 65], [2, 2, 3], [0, 0, 0]),
                                ([70, 70, 32, 65], [0, 0], [60, 500]),                 # a reserve beyond the table
                                ([70, 70, 32, 65], [0, 0], [-5, 2 ** 31 - 1]),
                                ([70, 70, 32, 65], [0] * 12, [33] * 12)):              # too few free pages
        lens, parents, more = (np.array(v, np.int32) for v in (lens, parents, more))
        refs = np.bincount(table[(table >= 0) & (table < 20)], minlength=20).astype(np.int32)
        run = fork_run(vbq, page, heads, dim, 20, table, lens, refs, parents, more)
        want = fork_reference(page, 20, table, lens, refs, parents, more)
        assert want[4]
        fork_check(*run, want, page, heads, dim)
        with pytest.raises(vbq.VbqError):
            run[0].check()


def test_fork_in_a_graph(vbq):
    import torch
    rng = np.random.default_rng(5)
    n_pages, table, lens, refs, parents, more = fork_case(rng, 12, 16, 5, 64, 80, reserve=3)
    cache = vbq.Kv4Cache(n_pages, 64, 2, 128)
    cache.data.copy_(torch.randint(0, 256, (cache.nbytes,), dtype=torch.uint8))
    dev = [torch.from_numpy(a).cuda() for a in (refs, table, lens, parents, more)]
    w = vbq.kv4_fork_workspace(cache, 16, 5, 12)
    out = vbq.kv4_fork(cache, *dev[:4], reserve=dev[4], workspace=w)
    torch.cuda.synchronize()
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        vbq.kv4_fork(cache, *dev[:4], reserve=dev[4], out=out, workspace=w)
    for _ in range(4):
        parents = rng.integers(-1, 12, 16).astype(np.int32)
        dev[3].copy_(torch.from_numpy(parents))
        before = cache.data.clone()
        g.replay()
        torch.cuda.synchronize()
        want = fork_reference(64, n_pages, table, lens, refs, parents, more)
        fork_check(cache, before, [o.cpu().numpy() for o in out], want, 64, 2, 128)


def test_fork_refusals(vbq):
    import torch
    cache = vbq.Kv4Cache(10, 32, 1, 64)
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lens, refs, parents = (torch.zeros(s, **i32) for s in ((2, 3), (2,), (10,), (4,)))
    for bad in (dict(refs=refs[:9]), dict(block_table=table[0]), dict(block_table=table.t()), dict(lens=lens.long()),
                dict(lens=lens[:1]), dict(parents=parents.cpu()), dict(parents=parents[:0]), dict(reserve=lens),
                dict(out=(table, lens, refs)), dict(workspace=torch.zeros(100, device="cuda"))):
        with pytest.raises(ValueError):
            vbq.kv4_fork(**{**dict(cache=cache, refs=refs, block_table=table, lens=lens, parents=parents), **bad})
    for out in ((torch.zeros(2, 3, **i32), torch.zeros(2, **i32), refs), (table, torch.zeros(2, **i32), torch.zeros(10, **i32))):
        with pytest.raises(vbq.VbqError):    # an output that is an input
            vbq.kv4_fork(cache, refs, table, lens, torch.zeros(2, **i32), out=out)
    with pytest.raises(vbq.VbqError):        # a workspace that is too small
        vbq.kv4_fork(cache, refs, table, lens, parents, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))


# ---- together ------------------------------------------------------------------------
@pytest.mark.parametrize("beams,prompt,steps", [(1, 5, 3), (4, 70, 6), (8, 200, 5), (3, 64, 9)])
def test_the_beam_search_example(vbq, beams, prompt, steps):
    """All operators as they are used together: scores of beams that share a prompt's pages are those of every
    sequence decoded by itself. A log probability differs by the rounding of fp16 activations that two kernels leave
    apart (2^-11 of the logits' size, logits of standard deviation 4 and 4 sigma, a few times a step)."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import continuations
    model = continuations.Model(hidden=256, heads=8, kv_heads=2, dim=64, vocab=997)
    r = continuations.run(beams, prompt, steps, model=model)
    assert all(a >= b for a, b in zip(r["scores"], r["scores"][1:]))
    assert all(np.isfinite(r["scores"]))
    for a, b in zip(r["scores"], r["alone"]):
        assert abs(a - b) <= steps * 8 * 2.0 ** -11 * 16
    assert r["pages"] <= r["apart"]

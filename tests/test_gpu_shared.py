"""kv4_attention_shared on the GPU against softmax attention in 64 bits over the cache's
bytes; the reader, the reference and the bounds are those of kv4_attention's tests."""
import numpy as np
import pytest

from test_gpu_kv4 import Layout, check, cum, gpu, random_cache, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def vbq():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import packed_decode_gemv_amd as vbq
    return vbq


class Case:
    """groups: (shared tokens, [(own tokens, queries)]) each; alone: sequences before and behind the groups that share
    nothing. Entries that are not to be read are -1, blocks that are not to be read hold NaN and infinity."""

    def __init__(self, rng, heads, ratio, dim, page, groups, dtype="float16", alone=((), ()), gain=1.0):
        import torch
        self.page, self.heads, self.ratio, self.dim, self.dtype = page, heads, ratio, dim, dtype
        seqs = [(0, o, n) for o, n in alone[0]]
        cu_groups, self.shared = [len(seqs)], []
        for s, members in groups:
            seqs += [(s, o, n) for o, n in members]
            cu_groups.append(len(seqs))
            self.shared.append(s)
        seqs += [(0, o, n) for o, n in alone[1]]
        self.cu_groups = np.array(cu_groups, np.int32)
        self.lens = [s + o for s, o, n in seqs]
        self.news = [n for s, o, n in seqs]
        self.own = max(o for s, o, n in seqs)
        B = len(seqs)
        width = max(1, -(-max(self.lens) // page))
        self.table = np.full((B, width), -1, np.int32)
        first = {}
        for g in range(len(groups)):
            for b in range(cu_groups[g], cu_groups[g + 1]):
                first[b] = cu_groups[g]
        used, copies = 0, []
        for b, (s, o, n) in enumerate(seqs):
            whole = s // 32 * 32
            skip = 0 if first.get(b, b) == b else whole // page     # entries that only the first row needs
            need = -(-self.lens[b] // page)
            self.table[b, skip:need] = np.arange(used, used + max(0, need - skip))
            used += max(0, need - skip)
            if skip < need and first.get(b, b) != b:
                copies.append((b, first[b], whole))
        self.n_pages = used + 2
        number = rng.permutation(self.n_pages).astype(np.int32)
        self.table = np.where(self.table >= 0, number[np.maximum(self.table, 0)], -1).astype(np.int32)
        data = random_cache(rng, self.n_pages, page, heads, dim)
        blocks = data.reshape(self.n_pages, heads, page // 32, -1)
        held = blocks.copy()
        self.full = self.table.copy()
        for b, f, whole in copies:             # what the formula sees, and what lies there
            j, n = whole // page, whole % page // 32
            self.full[b, :j] = self.table[f, :j]
            if n:
                blocks[self.table[b, j], :, :n] = held[self.table[f, j], :, :n]
                held[self.table[b, j], :, :n] = 0x7E
        for b in range(B):
            if first.get(b, b) != b:
                self.full[b, :seqs[b][0] // 32 * 32 // page] = self.table[first[b], :seqs[b][0] // 32 * 32 // page]
        self.data = data
        self.cache_data = held.reshape(-1)
        T = sum(self.news)
        self.q = torch.from_numpy(rng.normal(0, gain, (T, heads * ratio, dim)).astype(np.float32)).to(getattr(torch, dtype))
        self.group_q = max([0] + [sum(n for _, n in m) for _, m in groups])

    def args(self, vbq, far=False):
        """far: a bound on the shared tokens that makes the rows of a group take them together."""
        cache = vbq.Kv4Cache(self.n_pages, self.page, self.heads, self.dim, data=gpu(self.cache_data))
        return dict(cache=cache, q=self.q.cuda(), block_table=gpu(self.table), kv_lens=gpu(np.array(self.lens, np.int32)),
                    cu_q=gpu(cum(self.news)), cu_groups=gpu(self.cu_groups), shared=gpu(np.array(self.shared, np.int32)),
                    max_q=max(self.news), max_shared=1 << 22 if far else max(self.shared), max_own=self.own, max_group_q=self.group_q)

    def want(self, scale=None, causal=True):
        return reference(Layout(self.page, self.heads, self.dim), self.data, self.full, self.lens, self.news,
                         self.q.double().numpy(), self.dim ** -0.5 if scale is None else scale, causal, 0, 0)


def attend(vbq, case, scale=None, causal=True):
    """Both ways to take the shared tokens, against the reference."""
    import torch
    want = case.want(scale, causal)
    for far in (False, True):
        args = case.args(vbq, far)
        lse = torch.full(case.q.shape[:2], float("nan"), device="cuda")
        out = vbq.kv4_attention_shared(**args, scale=scale, causal=causal, lse=lse)
        assert args["cache"].check() is False
        check(out.double().cpu().numpy(), want[0], want[2], want[3], case.dtype, case.dim)
        tol = (case.dim + 40) * 2.0 ** -24 * (want[3] + np.abs(want[1]) + 30)
        assert (np.abs(lse.cpu().numpy() - want[1]) <= tol).all()
    return args, out, lse


ONE = [(1, 1), (5, 1), (33, 1), (64, 1), (70, 1)]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("heads,ratio,dim,page", [(2, 4, 128, 64), (3, 1, 64, 32), (1, 7, 128, 32), (2, 2, 192, 32),
                                                  (1, 4, 256, 128), (1, 20, 64, 32), (1, 1, 256, 32), (1, 8, 192, 64)])
@pytest.mark.parametrize("shared", [1, 31, 32, 33, 64, 200])
def test_one_token_each(vbq, dtype, heads, ratio, dim, page, shared):
    rng = np.random.default_rng(dim + ratio + shared)
    attend(vbq, Case(rng, heads, ratio, dim, page, [(shared, ONE)], dtype))


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
def test_groups_of_all_kinds(vbq, dtype, dim):
    """Groups of one and of many, without shared tokens, without queries, and sequences of no group around them."""
    rng = np.random.default_rng(dim)
    groups = [(100, ONE), (0, ONE[:2]), (7, [(40, 1)]), (350, [(2, 1)] * 12), (64, []), (96, [(30, 0), (9, 1), (8, 0)]),
              (160, [(12, 0), (3, 0)])]
    attend(vbq, Case(rng, 1, 4, dim, 32, groups, dtype, alone=([(50, 1), (0, 0)], [(1, 1), (80, 1)])))


@pytest.mark.parametrize("heads,ratio,dim,page,groups", [
    (2, 4, 128, 64, [(170, [(9, 3), (40, 5), (5, 5)])]),
    (1, 4, 64, 32, [(70, [(30, 30), (60, 1)]), (40, [(64, 64)])]),             # many rows of a sequence's own
    (1, 3, 256, 64, [(129, [(50, 20), (41, 41)])]),
    (1, 8, 128, 128, [(600, [(5, 5)] * 9), (31, [(5, 5)] * 2)]),
    (1, 1, 192, 32, [(96, [(130, 128)]), (96, [(129, 129)])]),
])
@pytest.mark.parametrize("causal", [True, False])
def test_several_tokens_each(vbq, heads, ratio, dim, page, groups, causal):
    rng = np.random.default_rng(dim + ratio)
    for dtype in ("float16", "bfloat16"):
        attend(vbq, Case(rng, heads, ratio, dim, page, groups, dtype), causal=causal, scale=0.2)


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("count,ratio", [(2, 2), (3, 2), (4, 4), (8, 4), (40, 4)])      # 4, 8, 16, 32 and more rows a group
def test_long_shared_and_own_tokens_are_cut(vbq, dim, count, ratio):
    rng = np.random.default_rng(dim + count)
    attend(vbq, Case(rng, 1, ratio, dim, 32, [(1500, [(1100, 1)] + [(7, 1)] * (count - 1)), (900, [(30, 1)])]))


@pytest.mark.parametrize("dim,new", [(256, 1), (256, 4), (128, 1)])
def test_more_tiles_of_own_tokens_than_units(vbq, dim, new):
    """Many tiles of own tokens, short and long, behind tiles of many rows over shared ones."""
    rng = np.random.default_rng(dim + new)
    groups = [(70, [(5, new)] * 30), (320, [(int(rng.integers(new, 90)), new) for _ in range(37)])]
    attend(vbq, Case(rng, 4, 4, dim, 32, groups, "bfloat16"))


@pytest.mark.parametrize("dim,new", [(64, 1), (128, 3), (192, 1), (256, 9)])
def test_less_than_a_block_in_common_and_far_bounds_of_own_tokens(vbq, dim, new):
    """Nothing is taken together, and the sequences' bound is too large to take them as small."""
    import torch
    rng = np.random.default_rng(dim + new)
    case = Case(rng, 2, 4, dim, 32, [(31, [(new, new), (700, new)]), (0, [(50, new)]), (1, [(32, new)] * 3)], "bfloat16")
    want = case.want()
    args = {**case.args(vbq), "max_own": 1 << 22}
    lse = torch.full(case.q.shape[:2], float("nan"), device="cuda")
    out = vbq.kv4_attention_shared(**args, lse=lse)
    assert args["max_shared"] == 31 and args["cache"].check() is False
    check(out.double().cpu().numpy(), want[0], want[2], want[3], case.dtype, case.dim)
    tol = (case.dim + 40) * 2.0 ** -24 * (want[3] + np.abs(want[1]) + 30)
    assert (np.abs(lse.cpu().numpy() - want[1]) <= tol).all()


def test_more_sequences_and_groups_than_lanes(vbq):
    rng = np.random.default_rng(4)
    groups = [(int(rng.integers(0, 90)), [(int(rng.integers(1, 50)), 1) for _ in range(int(rng.integers(0, 4)))])
              for _ in range(150)]
    groups[70] = (1200, [(5, 1)] * 100)
    groups[149] = (700, [(900, 1)])
    attend(vbq, Case(rng, 1, 2, 64, 32, groups, "bfloat16"))


def test_results_repeat_and_strides_and_workspaces_change_nothing(vbq):
    import torch
    rng = np.random.default_rng(5)
    for groups in ([(1500, [(40, 1)] * 6)], [(900, [(40, 5)] * 10), (64, [(33, 2)])]):
        case = Case(rng, 2, 4, 128, 64, groups)
        _, out, lse = attend(vbq, case)
        args = case.args(vbq, True)
        n = len(case.lens)
        ws = vbq.kv4_attention_shared_workspace(args["cache"], n, len(groups), len(case.q), 8, args["max_q"],
                                                args["max_shared"], args["max_own"], args["max_group_q"])
        ws[8 * vbq.KV4_COUNTERS:] = 255
        wide = torch.zeros(len(case.q), 11, 128, dtype=torch.float16, device="cuda")
        wide[:, 2:10] = args["q"]
        args["q"] = wide[:, 2:10]
        near = dict(args, max_shared=max(case.shared))        # the other way, with the same workspace
        alone = vbq.kv4_attention_shared(**near)
        for _ in range(3):
            assert torch.equal(vbq.kv4_attention_shared(**args, workspace=ws), out)
            assert torch.equal(vbq.kv4_attention_shared(**near, workspace=ws), alone)


def test_scores_far_out_and_special_queries(vbq):
    import torch
    rng = np.random.default_rng(6)
    for count in (4, 40):
        case = Case(rng, 1, 4, 64, 32, [(200, [(9, 1)] * count)], "bfloat16", gain=20.0)
        attend(vbq, case)
        for far in (False, True):
            args = case.args(vbq, far)
            clean = vbq.kv4_attention_shared(**args)
            args["q"][1, 2] = float("nan")
            args["q"][3, 0, 5] = float("inf")
            got = vbq.kv4_attention_shared(**args)
            hurt = torch.zeros(got.shape[:2], dtype=torch.bool, device="cuda")
            hurt[1, 2] = hurt[3, 0] = True
            assert not got[hurt].isfinite().any() and torch.equal(got[~hurt], clean[~hurt])


def test_shared_pages_that_are_missing_count_as_hidden(vbq):
    import torch
    rng = np.random.default_rng(7)
    for count, far in ((3, False), (3, True), (40, True), (40, False)):
        case = Case(rng, 1, 4, 64, 32, [(2300, [(5, 1)] * count)])
        args = case.args(vbq, far)
        holed = case.table.copy()
        lost = [0, 1, 7, 62, 63, 64, 65, 70]
        holed[0, lost] = [-1, case.n_pages, 2 ** 31 - 1, -5, case.n_pages + 7, -1, -2 ** 31, case.n_pages]
        args["block_table"] = gpu(holed)
        got = vbq.kv4_attention_shared(**args)
        with pytest.raises(vbq.VbqError, match="block-table"):
            args["cache"].check()
        # the same tokens by a table without the holes
        keep = [j for j in range(2300 // 32) if j not in lost]
        args = case.args(vbq, far)
        tight = np.full_like(case.table, -1)
        moved = len(lost)
        tight[0, :len(keep)] = case.table[0, keep]
        tight[:, 71 - moved:72 - moved + 1] = case.table[:, 71:73]
        args["block_table"] = gpu(tight)
        args["kv_lens"] = args["kv_lens"] - 32 * moved
        args["shared"] = args["shared"] - 32 * moved
        want = vbq.kv4_attention_shared(**args)
        assert args["cache"].check() is False
        off = (got.double() - want.double()).abs().max()
        assert float(off) < 2 ** -9 * float(want.double().abs().max())       # two outputs in fp16, each within its bound


def test_what_does_not_fit_is_left_out(vbq):
    import torch
    rng = np.random.default_rng(8)
    for page, ratio, far in ((32, 2, False), (32, 2, True), (64, 16, True), (64, 16, False), (64, 40, True)):
        case = Case(rng, 1, ratio, 64, page, [(100, [(9, 1), (12, 2), (5, 1)]), (40, [(20, 1)] * 3), (64, [(5, 1)])],
                    alone=([(9, 1)], []))
        clean = vbq.kv4_attention_shared(**case.args(vbq, far))
        rows = cum(case.news)
        for key, at, value, gone in (("shared", 0, 105 if far else 101, (3,) if far else (1, 2, 3)),
                                     ("shared", 0, -1, (1, 2, 3)), ("shared", 1, 61, (4, 5, 6)),
                                     ("kv_lens", 2, 101, (2,)), ("kv_lens", 2, -1, (2,)), ("kv_lens", 4, 10 ** 6, (4,)),
                                     ("kv_lens", 7, 64 + 60, (7,)), ("cu_groups", 3, 9, (7,)),
                                     ("cu_groups", 2, -3, (4, 5, 6, 7)), ("cu_groups", 0, -1, (1, 2, 3, 0))):
            args = case.args(vbq, far)
            args[key][at] = value
            out = torch.full_like(clean, 7.0)
            vbq.kv4_attention_shared(**args, out=out)
            torch.cuda.synchronize()
            assert int(args["cache"].flags.item()) & 2, (key, at, value)
            for b in range(len(case.lens)):
                mine = slice(int(rows[b]), int(rows[b + 1]))
                if b in gone:
                    assert (out[mine] == 7.0).all(), (key, at, value, b)
                elif key != "cu_groups" and not (key == "shared" and far and b in (1, 2)):
                    assert torch.equal(out[mine], clean[mine]), (key, at, value, b)
        args = case.args(vbq, far)
        args["max_group_q"] = 3                # the first group has 4
        out = vbq.kv4_attention_shared(**args, out=torch.full_like(clean, 7.0))
        assert (out[1:5] == 7.0).all() and int(args["cache"].flags.item()) == 2
        assert torch.allclose(out[5:].float(), clean[5:].float(), atol=2e-3)


def test_in_a_graph_while_sequences_grow(vbq):
    import torch
    rng = np.random.default_rng(9)
    for count, heads, dim, far in ((6, 2, 128, False), (6, 2, 128, True), (40, 1, 64, True)):
        case = Case(rng, heads, 4, dim, 64, [(700, [(120, 1)] * count)])
        args = case.args(vbq, far)
        ws = vbq.kv4_attention_shared_workspace(args["cache"], count, 1, count, 4 * heads, 1, args["max_shared"], 120, count)
        out = torch.zeros_like(args["q"])
        lens = args["kv_lens"]
        lens -= 100
        vbq.kv4_attention_shared(**args, out=out, workspace=ws)
        torch.cuda.synchronize()
        g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(g, stream=side):
            vbq.kv4_attention_shared(**args, out=out, workspace=ws)
        for step in range(4):
            lens += 23
            args["q"].copy_(torch.randn(args["q"].shape, device="cuda"))
            g.replay()
            want = vbq.kv4_attention_shared(**args)
            torch.cuda.synchronize()
            assert torch.equal(out, want), step
        on_side = vbq.kv4_attention_shared(**args, stream=side)
        side.synchronize()
        assert torch.equal(on_side, want)
        assert args["cache"].check() is False


def test_agrees_with_attention_of_every_sequence_by_itself(vbq):
    """Larger than the reference reads: against kv4_attention over the same pages, each within half a step of its
    output type and 2^-10 of the values' size of the exact result."""
    import torch
    rng = np.random.default_rng(10)
    for heads, ratio, dim, shared, count, new in ((8, 4, 128, 9000, 33, 1), (4, 1, 64, 20000, 5, 2), (2, 2, 256, 4000, 30, 1)):
        page = 64
        case = Case(rng, heads, ratio, dim, page, [(shared // page * page, [(int(n), new) for n in rng.integers(new, 500, count)])])
        args = case.args(vbq, True)
        got = vbq.kv4_attention_shared(**args)
        want = vbq.kv4_attention(args["cache"], args["q"], gpu(case.full), args["kv_lens"], args["cu_q"], new,
                                 max(case.lens))
        assert args["cache"].check() is False
        off = (got.double() - want.double()).abs() - 2.0 ** -10 * want.double().abs()
        assert float(off.max()) <= 2.0 ** -9 * 6.0          # values are below 6 here


def test_refusals(vbq):
    import torch
    rng = np.random.default_rng(11)
    args = Case(rng, 1, 2, 64, 32, [(40, [(5, 1)] * 2)]).args(vbq)
    for bad in (dict(q=args["q"][0]), dict(q=args["q"].float()), dict(shared=args["shared"].long()), dict(shared=args["shared"][:0]),
                dict(cu_groups=args["cu_groups"][:1]), dict(kv_lens=args["kv_lens"][:1]), dict(max_q=-1), dict(max_own=-1),
                dict(max_shared=-1), dict(max_group_q=-1), dict(max_own=2 ** 31 - 40), dict(max_shared=2 ** 31),
                dict(out=args["q"].float()), dict(lse=torch.zeros(2, 2, device="cuda").half()),
                dict(workspace=torch.zeros(4, device="cuda"))):
        with pytest.raises(ValueError):
            vbq.kv4_attention_shared(**{**args, **bad})
    for bad in (dict(scale=0.0), dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(vbq.VbqError):
            vbq.kv4_attention_shared(**{**args, **bad})
    empty = dict(args, q=args["q"][:0], cu_q=torch.zeros_like(args["cu_q"]))
    assert vbq.kv4_attention_shared(**empty).shape == (0, 2, 64)


def test_rows_behind_the_last_sequence_stay(vbq):
    import torch
    rng = np.random.default_rng(12)
    for count, far in ((5, False), (5, True), (40, True)):
        case = Case(rng, 1, 4, 64, 32, [(100, [(9, 1)] * count)])
        args = case.args(vbq, far)
        want = vbq.kv4_attention_shared(**args)
        args["q"] = torch.cat([args["q"], torch.full_like(args["q"][:3], float("nan"))])
        out = torch.full((count + 3, 4, 64), 7.0, dtype=torch.float16, device="cuda")
        vbq.kv4_attention_shared(**args, out=out)
        assert torch.equal(out[:count], want) and (out[count:] == 7.0).all()
        assert args["cache"].check() is False


def test_calls_on_two_streams_at_once(vbq):
    """Each with a workspace of its own; a captured graph replays beside eager calls of another size."""
    import torch
    rng = np.random.default_rng(13)
    case = Case(rng, 2, 4, 128, 64, [(1500, [(60, 1)] * 6)])
    big = Case(rng, 1, 4, 64, 32, [(900, [(30, 2)] * 40)])
    a, b = case.args(vbq, True), big.args(vbq, True)
    want = [vbq.kv4_attention_shared(**a), vbq.kv4_attention_shared(**b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, (args, s) in enumerate(zip((a, b), streams)):
            got[i].append(vbq.kv4_attention_shared(**args, stream=s))
    torch.cuda.synchronize()
    for outs, w in zip(got, want):
        assert all(torch.equal(o, w) for o in outs)


def test_far_pages_of_a_large_cache(vbq):
    """Pages beyond 4 GiB: attention reads them, a fork copies them."""
    import torch
    heads, dim, page = 1, 64, 1024
    n_pages = (5 << 30) // (1024 * 72)
    cache = vbq.Kv4Cache(n_pages, page, heads, dim)
    rng = np.random.default_rng(14)
    case = Case(rng, heads, 2, dim, page, [(1500, [(40, 1)] * 3)])
    args = case.args(vbq, True)
    near = dict(args, max_shared=1500)
    want, want_near = vbq.kv4_attention_shared(**args), vbq.kv4_attention_shared(**near)
    far = n_pages - case.n_pages
    cache.data[far * cache.page_bytes:] = args["cache"].data
    args["cache"] = cache
    args["block_table"] = torch.where(args["block_table"] >= 0, args["block_table"] + far, args["block_table"])
    assert torch.equal(vbq.kv4_attention_shared(**args), want)
    assert torch.equal(vbq.kv4_attention_shared(**dict(args, max_shared=1500)), want_near)
    # a fork of the first sequence, where only the last pages are free
    i32 = dict(dtype=torch.int32, device="cuda")
    refs = torch.ones(n_pages, **i32)
    src = int(args["block_table"][0, 1])
    dst = far + case.n_pages - 1 if src != far + case.n_pages - 1 else far + case.n_pages - 2
    refs[dst] = 0
    table, lens, counts = vbq.kv4_fork(cache, refs, args["block_table"][:1].contiguous(), args["kv_lens"][:1].contiguous(),
                                       torch.zeros(2, **i32))
    assert table[1, 1] == dst and table[0, 1] == src and table[1, 0] == table[0, 0]
    assert counts[dst] == 1 and counts[int(table[0, 0])] == 2
    blocks = -(-(1540 - 1024) // 32) * 2304
    pages = cache.data.view(n_pages, -1)
    assert torch.equal(pages[dst, :blocks], pages[src, :blocks])
    assert cache.check() is False

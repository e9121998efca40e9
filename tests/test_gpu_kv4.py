"""The 4-bit key/value cache on the GPU: kv4_append and kv4_read bit for bit
against a plain numpy writer and reader of the layout that include/vbq.h
states, kv4_attention against softmax attention in 64 bits."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

BLOCK = 32
CLAMP = np.float32(61440.0)


@pytest.fixture(scope="module")
def vbq():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import packed_decode_gemv_amd as vbq
    return vbq


# ---- plain quantiser and layout -----------------------------------------------------
def quantise(x):
    """Codes, scale and offset (float16) of groups on the last axis (64 long), in binary32."""
    x = np.asarray(x, np.float32)
    x = np.where(np.isnan(x), np.float32(0), np.clip(x, -CLAMP, CLAMP)).astype(np.float32)
    lo, hi = x.min(-1), x.max(-1)
    s = ((hi - lo).astype(np.float32) * (np.float32(1) / np.float32(15))).astype(np.float16)
    o = lo.astype(np.float16)
    sf, of = s.astype(np.float32)[..., None], o.astype(np.float32)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(sf == 0, np.float32(0), np.clip(np.rint((x - of) / sf), 0, 15))
    return q.astype(np.uint32), s, o


def value_of(q, s, o):
    return (s.astype(np.float32)[..., None] * q.astype(np.float32) + o.astype(np.float32)[..., None]).astype(np.float32)


class Layout:
    """Addresses of one cache's codes, scales and offsets, from the header's text."""

    def __init__(self, page, heads, dim):
        self.page, self.heads, self.dim, self.G = page, heads, dim, dim // 64

    def block(self, page, head, tok_in_page):
        return ((page * self.heads + head) * (self.page // BLOCK) + tok_in_page // BLOCK) * 2304 * self.G

    def key_word(self, t, c):       # byte offset of the word in the group's codes, and the code's first bit
        return 4 * (4 * (16 * (c % 32 // 8) + 4 * (t // 8) + t % 4) + 2 * (t % 8 // 4) + c // 32), 4 * (c % 8)

    def value_word(self, t, c):
        return 4 * (64 * (t // 8) + c), 4 * (t % 8)

    def places(self, base, t, kv):
        """Byte offsets of the scale and the offset per group."""
        first = base + 2048 * self.G + (128 * self.G if kv else 0)
        e = 8 * (t // 8) + 2 * (t % 4) + t % 8 // 4 if kv else t
        return [(first + 128 * g + 2 * e, first + 128 * g + 64 + 2 * e) for g in range(self.G)]

    def write(self, data, base, t, kv, q, s, o):
        """data: uint8; q [G][64], s, o [G]: one token of one head."""
        for g in range(self.G):
            for c in range(64):
                off, bit = (self.value_word if kv else self.key_word)(t, c)
                w = data[base + 1024 * (self.G * kv + g) + off:][:4].view(np.uint32)
                w[0] = (int(w[0]) & ~(15 << bit) & 0xFFFFFFFF) | (int(q[g, c]) << bit)
        for g, (a, b) in enumerate(self.places(base, t, kv)):
            data[a:a + 2].view(np.float16)[0] = s[g]
            data[b:b + 2].view(np.float16)[0] = o[g]

    def read(self, data, base, t, kv):
        """float32 [dim] of one token of one head."""
        out = np.empty((self.G, 64), np.float32)
        c = np.arange(64)
        off, bit = (self.value_word if kv else self.key_word)(t, c)
        for g, (a, b) in enumerate(self.places(base, t, kv)):
            w = data.view(np.uint32)[(base + 1024 * (self.G * kv + g) + off) // 4]
            s, o = data[a:a + 2].view(np.float16), data[b:b + 2].view(np.float16)
            out[g] = value_of((w >> np.asarray(bit).astype(np.uint32)) & 15, s, o)[0]
        return out.reshape(-1)


def random_cache(rng, n_pages, page, heads, dim):
    """Bytes of a cache whose every place holds finite values: codes at random, scales and offsets of
    ordinary size, as uint8."""
    G = dim // 64
    blocks = n_pages * heads * (page // BLOCK)
    data = rng.integers(0, 256, (blocks, 2304 * G), dtype=np.uint8)
    so = np.empty((blocks, 2, G, 2, 32), np.float16)
    so[:, :, :, 0] = rng.uniform(0.02, 0.4, so[:, :, :, 0].shape)
    so[:, :, :, 1] = rng.normal(-1.5, 0.7, so[:, :, :, 1].shape)
    data[:, 2048 * G:] = so.reshape(blocks, -1).view(np.uint8)
    return data.reshape(-1)


def table_for(rng, lens, page, spare=1):
    """A block table of distinct pages in random order, -1 where a sequence has none."""
    need = [-(-n // page) for n in lens]
    width = max(1, max(need))
    perm = rng.permutation(sum(need) + spare).astype(np.int32)
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, len(perm)


def gpu(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def cum(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


# ---- append and read ---------------------------------------------------------------
APPEND = [
    # dtype, heads, dim, page, [(start, new)]
    ("float16", 3, 64, 32, [(0, 1)]),
    ("float16", 2, 128, 64, [(0, 8), (5, 3), (31, 2), (63, 1)]),
    ("bfloat16", 1, 128, 32, [(7, 1), (8, 1), (30, 70), (0, 0), (3, 33)]),
    ("float32", 2, 192, 64, [(60, 9), (1, 7), (0, 65)]),
    ("float32", 1, 256, 128, [(100, 60), (0, 17)]),
    ("bfloat16", 5, 64, 256, [(250, 9), (13, 3)]),
]


@pytest.mark.parametrize("case", range(len(APPEND)))
@pytest.mark.parametrize("strided", [False, True])
def test_append_writes_the_stated_bytes_and_no_others(vbq, case, strided):
    import torch
    dtype, heads, dim, page, seqs = APPEND[case]
    rng = np.random.default_rng(case)
    lens = [s + n for s, n in seqs]
    table, n_pages = table_for(rng, lens, page)
    data = random_cache(rng, n_pages, page, heads, dim)
    T = sum(n for _, n in seqs)
    x = rng.normal(0, 1, (2, T, heads, dim)).astype(np.float32)
    x[:, :, :, ::13] *= 6
    x[0, T // 2] = 0.25                      # a constant group: scale 0
    x[1, T - 1, :, 5] = 3e38                 # clamped
    x[0, 0, 0, 9] = -np.inf
    xt = torch.from_numpy(x).to(getattr(torch, dtype))
    if dtype == "float16":
        xt = torch.nan_to_num(xt, posinf=float("inf"), neginf=float("-inf"))
    if strided:   # keys and values are slices of one projection, heads interleaved with others
        both = torch.zeros(T, 2, heads + 2, dim, dtype=xt.dtype)
        both[:, 0, 1:heads + 1], both[:, 1, 1:heads + 1] = xt[0], xt[1]
        both = both.cuda()
        k, v = both[:, 0, 1:heads + 1], both[:, 1, 1:heads + 1]
    else:
        k, v = xt[0].contiguous().cuda(), xt[1].contiguous().cuda()
    cache = vbq.Kv4Cache(n_pages, page, heads, dim, data=gpu(data.copy()))
    start = np.array([s for s, _ in seqs], np.int32)
    cu = cum([n for _, n in seqs])
    vbq.kv4_append(cache, k, v, gpu(table), gpu(start), gpu(cu), max_tokens=max(n for _, n in seqs))
    assert cache.check() is False
    lay = Layout(page, heads, dim)
    xf = xt.float().numpy()
    want = data.copy()
    for b, (s, n) in enumerate(seqs):
        for i in range(n):
            p = s + i
            for h in range(heads):
                base = lay.block(int(table[b, p // page]), h, p % page)
                for kv in range(2):
                    lay.write(want, base, p % 32, kv, *quantise(xf[kv, cu[b] + i, h].reshape(-1, 64)))
    got = cache.data.cpu().numpy()
    assert np.array_equal(got, want), np.flatnonzero(got != want)[:8]


def test_the_scale_is_rounded_to_binary32_and_then_to_binary16(vbq):
    """Ranges whose product with f32(1/15) is halfway between two fp16 numbers in binary32 though the exact product
    is not: rounding once would give the neighbour."""
    import torch
    ranges = [float.fromhex(h) for h in ("0x1.5779fe0p+4", "0x1.4cb1fe0p+3", "0x1.a189fe0p+3",
                                         "0x1.0da6000p+3", "0x1.60d9fe0p+3")]
    x = np.zeros((len(ranges), 1, 64), np.float32)
    x[:, 0, 17] = ranges
    x[:, 0, 40] = np.float32(ranges) / 3
    want = quantise(x.astype(np.float64))[1]
    once = (np.float32(ranges).astype(np.float64) * np.float64(np.float32(1 / 15))).astype(np.float16)
    assert (once != want.reshape(-1)).all()      # numpy rounds float64 to float16 once
    cache = vbq.Kv4Cache(1, 32, 1, 64)
    i32 = dict(dtype=torch.int32, device="cuda")
    vbq.kv4_append(cache, gpu(x), gpu(x), torch.zeros(1, 1, **i32), torch.zeros(1, **i32),
                   torch.tensor([0, len(ranges)], **i32))
    data, lay = cache.data.cpu().numpy(), Layout(32, 1, 64)
    for t in range(len(ranges)):
        for kv in range(2):
            a, _ = lay.places(lay.block(0, 0, t), t, kv)[0]
            assert data[a:a + 2].view(np.float16)[0] == want.reshape(-1)[t]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("heads,dim,page,seqs", [
    (1, 64, 32, [(0, 1)]),
    (2, 128, 64, [(3, 70), (0, 0), (62, 5), (0, 64)]),
    (3, 192, 32, [(31, 2), (8, 40)]),
    (1, 256, 256, [(255, 9)]),
])
def test_read_returns_the_values_held(vbq, dtype, heads, dim, page, seqs):
    import torch
    rng = np.random.default_rng(dim + len(seqs))
    lens = [s + n for s, n in seqs]
    table, n_pages = table_for(rng, lens, page)
    data = random_cache(rng, n_pages, page, heads, dim)
    cache = vbq.Kv4Cache(n_pages, page, heads, dim, data=gpu(data))
    start, cu = np.array([s for s, _ in seqs], np.int32), cum([n for _, n in seqs])
    dt = getattr(torch, dtype)
    k, v = vbq.kv4_read(cache, gpu(table), gpu(start), gpu(cu), int(cu[-1]), dt, max_tokens=max(n for _, n in seqs))
    lay = Layout(page, heads, dim)
    want = np.empty((2, int(cu[-1]), heads, dim), np.float32)
    for b, (s, n) in enumerate(seqs):
        for i in range(n):
            p = s + i
            for h in range(heads):
                base = lay.block(int(table[b, p // page]), h, p % page)
                for kv in range(2):
                    want[kv, cu[b] + i, h] = lay.read(data, base, p % 32, kv)
    w = torch.from_numpy(want).to(dt)
    assert torch.equal(k.cpu(), w[0]) and torch.equal(v.cpu(), w[1])
    assert cache.check() is False


def test_tokens_one_at_a_time_equal_all_at_once(vbq):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(3)
    heads, dim, page, n = 4, 128, 64, 77
    k = torch.randn(n, heads, dim, generator=gen, device="cuda").half()
    v = torch.randn(n, heads, dim, generator=gen, device="cuda").half()
    table = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    one, all_ = (vbq.Kv4Cache(3, page, heads, dim) for _ in range(2))
    i32 = dict(dtype=torch.int32, device="cuda")
    vbq.kv4_append(all_, k, v, table, torch.zeros(1, **i32), torch.tensor([0, n], **i32))
    cu = torch.tensor([0, 1], **i32)
    for i in range(n):
        vbq.kv4_append(one, k[i:i + 1], v[i:i + 1], table, torch.tensor([i], **i32), cu)
    assert torch.equal(one.data, all_.data)


def test_nan_is_stored_as_zero_and_reported(vbq):
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    k = torch.ones(2, 1, 64, device="cuda")
    v = torch.full((2, 1, 64), 2.0, device="cuda")
    k[1, 0, 7] = float("nan")
    v[0, 0, 1] = float("inf")
    v[0, 0, 2] = -float("inf")
    cache = vbq.Kv4Cache(1, 32, 1, 64)
    args = (torch.zeros(1, 1, **i32), torch.zeros(1, **i32), torch.tensor([0, 2], **i32))
    vbq.kv4_append(cache, k, v, *args)
    assert cache.check() is True and cache.check() is False
    rk, rv = vbq.kv4_read(cache, *args, 2, torch.float32)
    assert rk[1, 0, 7] == 0 and torch.isfinite(rk).all()
    assert rv[0, 0, 1] == 61440 and rv[0, 0, 2] == -61440
    assert torch.isfinite(vbq.kv4_read(cache, *args, 2, torch.float16)[1]).all()


# ---- attention ---------------------------------------------------------------------
def reference(lay, data, table, lens, news, q, scale, causal, window, sinks):
    """Outputs, lse, sum of p |v| and a bound of the scores' magnitudes per row, in 64 bits.
    q: float64 [T][H][D]."""
    T, H, D = q.shape
    R = H // lay.heads
    out, mass = np.zeros((T, H, D)), np.zeros((T, H, D))
    lse, size = np.full((T, H), -np.inf), np.zeros((T, H))
    at = 0
    for b, (L, n) in enumerate(zip(lens, news)):
        for h in range(lay.heads):
            K, V = np.zeros((L, D)), np.zeros((L, D))
            for t in range(L):
                base = lay.block(int(table[b, t // lay.page]), h, t % lay.page)
                K[t], V[t] = lay.read(data, base, t % 32, 0), lay.read(data, base, t % 32, 1)
            # the score is formed from codes and offsets apart: their magnitudes bound its rounding
            Kabs = np.abs(K) + 2 * np.abs(K).max() if L else K
            for i in range(n):
                p = L - n + i
                j = np.arange(L)
                see = j <= p if causal else j < L
                if window:
                    see &= (j > p - window) | (j < sinks)
                if not see.any():
                    continue
                for r in range(h * R, h * R + R):
                    s = scale * (K[see] @ q[at + i, r])
                    e = np.exp(s - s.max())
                    w = e / e.sum()
                    out[at + i, r] = w @ V[see]
                    mass[at + i, r] = w @ np.abs(V[see])
                    lse[at + i, r] = s.max() + math.log(e.sum())
                    size[at + i, r] = scale * (Kabs[see] @ np.abs(q[at + i, r])).max()
        at += n
    return out, lse, mass, size


def check(got, want, mass, size, dtype, D):
    """Rounding bound of one output, u = 2^-24 and h = 2^-11 the half ulps of fp32 and fp16.
    A score of magnitude at most S takes at most D + 16 roundings in fp32 (products are exact) and its
    exponential's argument and value two more each: its probability is off by (D + 24) u S + 8 u at most,
    numerator and denominator alike. Probabilities and values are rounded to fp16 once each (h; absolute
    2^-25 below fp16's normal range, where probabilities carry 2^15), sums of up to 2^17 terms in blocks of 32
    lose under 2^13 u. The output is rounded once."""
    u, h = 2.0 ** -24, 2.0 ** -11
    out_h = h if dtype == "float16" else 2.0 ** -8
    rel = 2 * ((D + 24) * u * size + 8 * u) + 2.1 * h + 2 ** 13 * u
    bound = rel[..., None] * mass + out_h * np.abs(want) + 2.0 ** -24
    err = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (err <= bound).all(), (float((err / bound).max()), np.argwhere(err > bound)[:4])


def attend(vbq, rng, heads, ratio, dim, page, lens, news, dtype="float16", causal=True, window=0, sinks=0,
           scale=None, spoil=True, max_kv=None, gain=1.0):
    """Runs kv4_attention on a random cache and returns everything a check needs."""
    import torch
    table, n_pages = table_for(rng, lens, page)
    data = random_cache(rng, n_pages, page, heads, dim)
    lay = Layout(page, heads, dim)
    if spoil:   # places past a sequence's end hold NaN and infinity scales
        for b, L in enumerate(lens):
            for t in range(L, -(-L // page) * page):
                for h in range(heads):
                    base = lay.block(int(table[b, t // page]), h, t % page)
                    for kv in range(2):
                        for a, o in lay.places(base, t % 32, kv):
                            data[a:a + 2].view(np.uint16)[0] = 0x7E00 if t % 2 else 0x7C00
                            data[o:o + 2].view(np.uint16)[0] = 0xFC00
    cache = vbq.Kv4Cache(n_pages, page, heads, dim, data=gpu(data))
    T = sum(news)
    q = torch.from_numpy(rng.normal(0, gain, (T, heads * ratio, dim)).astype(np.float32)).to(getattr(torch, dtype))
    qd = q.cuda()
    lse = torch.full((T, heads * ratio), float("nan"), device="cuda")
    kw = dict(scale=scale, causal=causal, window=window, sinks=sinks)
    args = (cache, qd, gpu(table), gpu(np.array(lens, np.int32)), gpu(cum(news)), max(news),
            max(lens) if max_kv is None else max_kv)
    out = vbq.kv4_attention(*args, lse=lse, **kw)
    assert cache.check() is False
    sc = dim ** -0.5 if scale is None else scale
    want = reference(lay, data, table, lens, news, q.double().numpy(), sc, causal, window, sinks)
    check(out.double().cpu().numpy(), want[0], want[2], want[3], dtype, dim)
    gl, wl = lse.cpu().numpy().astype(np.float64), want[1]
    seen = np.isfinite(wl)
    assert np.array_equal(np.isneginf(gl), ~seen)
    tol = (dim + 40) * 2.0 ** -24 * (want[3] + np.abs(np.where(seen, wl, 0)) + 30)
    assert (np.abs(gl[seen] - wl[seen]) <= tol[seen]).all()
    return args, kw, out


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("heads,ratio,dim,page", [
    (2, 4, 128, 64), (3, 1, 64, 32), (1, 7, 128, 32), (1, 16, 64, 64), (2, 2, 192, 32), (1, 4, 256, 128),
    (1, 20, 128, 32),
])
def test_attention_of_single_tokens(vbq, dtype, heads, ratio, dim, page):
    rng = np.random.default_rng(dim + ratio)
    lens = [1, 31, 32, 33, 150, 0, 257, 64]
    attend(vbq, rng, heads, ratio, dim, page, lens, [1] * len(lens), dtype)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("heads,ratio,dim,page,lens,news", [
    (2, 4, 128, 32, [40, 33, 5, 300], [5, 1, 5, 3]),
    (1, 1, 64, 64, [100, 70], [100, 33]),
    (1, 5, 128, 32, [64, 31, 97], [64, 0, 50]),
    (1, 3, 256, 64, [90], [41]),
    (2, 2, 192, 32, [65, 50], [20, 50]),
    (1, 4, 64, 32, [3, 20], [7, 20]),       # more queries than tokens: the first rows see nothing
])
def test_attention_of_several_tokens(vbq, dtype, heads, ratio, dim, page, lens, news):
    rng = np.random.default_rng(sum(lens) + dim)
    attend(vbq, rng, heads, ratio, dim, page, lens, news, dtype)
    attend(vbq, rng, heads, ratio, dim, page, lens, news, dtype, causal=False, scale=0.3)


@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 1), (32, 4), (50, 33), (64, 200), (1000, 4), (33, 64)])
@pytest.mark.parametrize("lens,news", [([200, 1, 37, 99], [1, 1, 1, 1]), ([210, 70], [9, 70]), ([33, 160], [20, 64])])
def test_attention_under_a_window(vbq, window, sinks, lens, news):
    rng = np.random.default_rng(window + sinks + lens[0])
    attend(vbq, rng, 2, 2, 64, 32, lens, news, window=window, sinks=sinks)
    attend(vbq, rng, 1, 5, 128, 64, lens, news, "bfloat16", window=window, sinks=sinks)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 40, 600])
def test_attention_of_more_queries_than_tokens(vbq, window):
    """Queries before position 0 see nothing, and do not disturb the others, whatever the window."""
    rng = np.random.default_rng(8)
    for ratio, lens, news in ((4, [3, 500, 0], [5, 8, 2]), (4, [50, 700], [60, 90])):
        attend(vbq, rng, 1, ratio, 64, 32, lens, news, window=window, sinks=2)


def test_attention_in_pieces_and_whole(vbq):
    """A long sequence is split over workgroups, beside short ones that are not."""
    rng = np.random.default_rng(5)
    attend(vbq, rng, 1, 4, 128, 64, [4200, 3, 600, 0], [1, 1, 1, 1], max_kv=6000)
    attend(vbq, rng, 1, 8, 64, 128, [3000, 700], [4, 2], "bfloat16")
    attend(vbq, rng, 1, 4, 256, 64, [1500], [9], window=900, sinks=5)


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("ratio,new", [(3, 1), (5, 1), (4, 3), (8, 4)])      # 4, 8, 16 and 32 rows a tile
def test_attention_in_parts_for_every_tile(vbq, dim, ratio, new):
    """Tiles cut into parts, for every head size and number of rows: lengths of one block and of many, and a
    sequence that sees nothing beside them."""
    rng = np.random.default_rng(dim + ratio)
    attend(vbq, rng, 1, ratio, dim, 32, [1100, 0, 37], [new, 1, min(new, 2)], max_kv=1200)


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_attention_of_many_rows_in_parts(vbq, dim, dtype):
    """More than 32 rows a head over caches long enough to be cut, and joined by a launch of its own: sequences that
    are not cut, see nothing, or have no query beside one that is; windows; all tokens visible."""
    rng = np.random.default_rng(dim)
    attend(vbq, rng, 1, 4, dim, 32, [1500, 0, 90, 400], [12, 9, 0, 1], dtype)
    attend(vbq, rng, 1, 40, dim, 64, [900], [1], dtype, causal=False)
    attend(vbq, rng, 1, 3, dim, 64, [1100, 700], [90, 20], dtype, window=450, sinks=40)


def test_attention_of_many_rows_in_parts_repeats(vbq):
    import torch
    rng = np.random.default_rng(3)
    args, kw, out = attend(vbq, rng, 1, 8, 128, 64, [2000, 300], [8, 6], "bfloat16")
    ws = vbq.kv4_attention_workspace(args[0], 2, 14, 8, 8, 2000)
    assert ws.numel() > 0
    ws[4 * vbq.KV4_COUNTERS:] = 255           # only the counters are zero before the first call
    for _ in range(3):
        assert torch.equal(vbq.kv4_attention(*args, workspace=ws, **kw), out)


def test_attention_of_more_sequences_than_lanes(vbq):
    """Parts of tiles are found by scanning the sequences 64 at a time."""
    rng = np.random.default_rng(11)
    lens = [int(n) for n in rng.integers(0, 90, 150)]
    lens[3], lens[70], lens[149] = 1500, 0, 900
    attend(vbq, rng, 1, 2, 64, 32, lens, [1] * 150)
    lens[149] = 0
    attend(vbq, rng, 1, 4, 64, 64, lens, [0 if n % 7 == 0 else 1 for n in range(150)], window=300, sinks=3)


def test_attention_parts_where_pages_are_missing(vbq):
    """A page that is not in the cache counts as tokens that nobody sees, wherever it lies."""
    import torch
    rng = np.random.default_rng(12)
    for ratio, new in ((4, 1), (4, 40)):
        page, dim, L = 32, 64, 2300            # more than 64 blocks: addresses are looked up 64 at a time
        lens, news = [L], [new]
        table, n_pages = table_for(rng, lens, page)
        data = random_cache(rng, n_pages, page, 1, dim)
        cache = vbq.Kv4Cache(n_pages, page, 1, dim, data=gpu(data))
        q = torch.from_numpy(rng.normal(0, 1, (new, ratio, dim)).astype(np.float32)).half()
        lost = [0, 1, 7, 62, 63, 64, 65, 70]
        holed = table.copy()
        holed[0, lost] = [-1, n_pages, 2 ** 31 - 1, -5, n_pages + 7, -1, -2 ** 31, n_pages]
        args = (gpu(np.array(lens, np.int32)), gpu(cum(news)), new, L)
        got = vbq.kv4_attention(cache, q.cuda(), gpu(holed), *args)
        with pytest.raises(vbq.VbqError, match="block-table"):
            cache.check()
        lay = Layout(page, 1, dim)
        hide = np.zeros(L, bool)
        for e in lost:
            hide[e * page:(e + 1) * page] = True
        K = np.stack([lay.read(data, lay.block(int(table[0, t // page]), 0, t % page), t % 32, 0) for t in range(L)])
        V = np.stack([lay.read(data, lay.block(int(table[0, t // page]), 0, t % page), t % 32, 1) for t in range(L)])
        K, V = K.astype(np.float64), V.astype(np.float64)
        want, mass, size = (np.zeros((new, ratio, n)) for n in (dim, dim, 1))
        for i in range(new):
            see = ~hide & (np.arange(L) <= L - new + i)
            for r in range(ratio):
                qv = q[i, r].double().numpy()
                s = K[see] @ qv * dim ** -0.5
                w = np.exp(s - s.max())
                w /= w.sum()
                want[i, r], mass[i, r] = w @ V[see], w @ np.abs(V[see])
                size[i, r] = ((np.abs(K) + 2 * np.abs(K).max()) @ np.abs(qv)).max() * dim ** -0.5
        check(got.double().cpu().numpy(), want, mass, size[..., 0], "float16", dim)


def test_attention_of_more_tiles_than_counters(vbq):
    """Beyond 2048 tiles none is cut; a workspace is not needed."""
    import torch
    rng = np.random.default_rng(13)
    B = 300
    table = torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1)
    data = random_cache(rng, B, 1024, 8, 64)
    cache = vbq.Kv4Cache(B, 1024, 8, 64, data=gpu(data))
    q = torch.randn(B, 8, 64, device="cuda").half()
    lens = torch.full((B,), 1000, dtype=torch.int32, device="cuda")
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    assert vbq.kv4_attention_workspace(cache, B, B, 8, 1, 1000).numel() == 0
    out = vbq.kv4_attention(cache, q, table, lens, cu, 1, 1000)
    few = vbq.kv4_attention(cache, q[7:9], table[7:9].contiguous(), lens[:2], cu[:3], 1, 1000)
    err = (out[7:9].double() - few.double()).abs().max()
    assert float(err) <= 2.0 ** -10 * float(few.abs().max())
    assert cache.check() is False


def test_attention_of_values_of_any_size(vbq):
    """The product of probability and scale is held around the largest scale a row has met: scales from fp16's
    smallest to the clamp's, growing and shrinking along the sequence."""
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(5)
    L, dim = 700, 64
    k = torch.randn(L, 1, dim, generator=gen, device="cuda")
    table = torch.arange(32, device="cuda").int().view(1, 32)
    cu, lens = torch.tensor([0, L], **i32), torch.tensor([L], **i32)
    size = torch.linspace(-18, 15, L, device="cuda")
    for exps in (size, size.flip(0), torch.full_like(size, -20.0), torch.full_like(size, 15.5)):
        v = torch.randn(L, 1, dim, generator=gen, device="cuda") * torch.exp2(exps)[:, None, None]
        cache = vbq.Kv4Cache(32, 32, 1, dim)
        vbq.kv4_append(cache, k, v, table, torch.zeros(1, **i32), cu)
        rk, rv = (x.double().cpu().numpy()[:, 0] for x in vbq.kv4_read(cache, table, torch.zeros(1, **i32), cu, L,
                                                                       torch.float32))
        for rows in (1, 50):
            q = torch.randn(rows, 4, dim, generator=gen, device="cuda").half()
            got = vbq.kv4_attention(cache, q, table, lens, torch.tensor([0, rows], **i32), rows, L)
            for i in (0, rows - 1):
                p = L - rows + i + 1
                for r in range(4):
                    s = rk[:p] @ q[i, r].double().cpu().numpy() * dim ** -0.5
                    w = np.exp(s - s.max())
                    w /= w.sum()
                    want, mass = w @ rv[:p], w @ np.abs(rv[:p])
                    # as in check(), with scores of up to 64 in magnitude, and fp16's subnormal outputs and values
                    bound = (2 * (88 * 2.0 ** -24 * 64 + 2.0 ** -21) + 2.1 * 2.0 ** -11 + 2.0 ** -11) * mass + 2.0 ** -23
                    assert (np.abs(got[i, r].double().cpu().numpy() - want) <= bound).all(), (i, r)


def test_attention_of_peaked_and_flat_scores(vbq):
    rng = np.random.default_rng(6)
    attend(vbq, rng, 1, 4, 128, 64, [700], [1], gain=12.0)
    attend(vbq, rng, 1, 4, 128, 64, [700], [1], gain=1e-4)
    attend(vbq, rng, 1, 4, 128, 64, [300], [20], gain=12.0)


@pytest.mark.parametrize("dtype,gain", [("float16", 6e4), ("bfloat16", 1e5), ("bfloat16", 1e28)])
@pytest.mark.parametrize("dim,ratio,new", [(64, 4, 1), (128, 7, 4), (64, 4, 30), (256, 2, 40)])
def test_attention_of_scores_far_out(vbq, dtype, gain, dim, ratio, new):
    """Queries and keys at the end of their ranges: the largest score takes the row, as long as fp32 holds it.
    A score is off by (D + 16) u times the sum of its terms' magnitudes at most (u = 2^-24, one more rounding by
    to_log2): rows whose two largest scores are nearer than 8 times that say nothing and are left out."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(dim + new)
    i32 = dict(dtype=torch.int32, device="cuda")
    L = 1500 if new < 10 else 200
    k = ((torch.rand(L, 1, dim, generator=gen, device="cuda") - 0.5) * 122880).float()
    v = torch.randn(L, 1, dim, generator=gen, device="cuda")
    q = ((torch.rand(new, ratio, dim, generator=gen, device="cuda") - 0.5) * 2 * gain).to(getattr(torch, dtype))
    cache = vbq.Kv4Cache(64, 32, 1, dim)
    table, cu = torch.arange(64, **i32).view(1, 64), torch.tensor([0, L], **i32)
    vbq.kv4_append(cache, k, v, table, torch.zeros(1, **i32), cu)
    rk, rv = (x.double()[:, 0] for x in vbq.kv4_read(cache, table, torch.zeros(1, **i32), cu, L, torch.float32))
    lse = torch.empty(new, ratio, device="cuda")
    got = vbq.kv4_attention(cache, q, table, torch.tensor([L], **i32), torch.tensor([0, new], **i32), new, L, lse=lse)
    assert torch.isfinite(got).all() and torch.isfinite(lse).all()
    out_h = 2.0 ** -11 if dtype == "float16" else 2.0 ** -8
    used = 0
    for i in range(new):
        for r in range(ratio):
            p = L - new + i + 1
            qd = q[i, r].double()
            s = rk[:p] @ qd * dim ** -0.5
            # keys are s c + o with |o| and |s c| up to twice the key's range
            off = (dim + 17) * 2.0 ** -24 * float(qd.abs().sum() * 4 * rk.abs().max()) * dim ** -0.5
            top = torch.topk(s, 2).values
            assert abs(float(lse[i, r]) - float(top[0])) <= off + 2.0 ** -22 * abs(float(top[0]))
            if float(top[0] - top[1]) < 8 * off + 40:
                continue
            used += 1
            want = rv[int(s.argmax())]
            assert ((got[i, r].double() - want).abs() <= (out_h + 2.1 * 2.0 ** -11) * want.abs() + 2.0 ** -24).all()
    assert used * 2 >= new * ratio


def test_attention_repeats_and_strided_queries_agree(vbq):
    import torch
    rng = np.random.default_rng(7)
    args, kw, out = attend(vbq, rng, 2, 4, 128, 64, [900, 2000], [3, 1])
    ws = vbq.kv4_attention_workspace(args[0], 2, 4, 8, 3, 2000)
    for _ in range(4):
        again = vbq.kv4_attention(*args, workspace=ws, **kw)
        assert torch.equal(again, out)
    q = args[1]
    wide = torch.randn(q.shape[0], 3, 12, 128, device="cuda").half()
    wide[:, 1, 2:10] = q
    assert torch.equal(vbq.kv4_attention(args[0], wide[:, 1, 2:10], *args[2:], **kw), out)
    turned = q.transpose(0, 1).contiguous().transpose(0, 1)     # heads first in memory
    assert torch.equal(vbq.kv4_attention(args[0], turned, *args[2:], **kw), out)


def test_a_hidden_token_cannot_reach_an_output(vbq):
    """Appending infinities and NaN after a query's position leaves its output as it was."""
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn(40, 1, 64, generator=gen, device="cuda")
    v = torch.randn(40, 1, 64, generator=gen, device="cuda")
    q = torch.randn(40, 4, 64, generator=gen, device="cuda").half()
    outs = []
    for bad in (False, True):
        if bad:
            k[20:, :, 3], v[20:, :, 5], v[25] = float("nan"), float("-inf"), float("inf")
        cache = vbq.Kv4Cache(2, 32, 1, 64)
        table, z, cu = torch.tensor([[1, 0]], **i32), torch.zeros(1, **i32), torch.tensor([0, 40], **i32)
        vbq.kv4_append(cache, k, v, table, z, cu)
        outs.append(vbq.kv4_attention(cache, q, table, torch.tensor([40], **i32), cu, 40, 40))
    assert torch.equal(outs[0][:20], outs[1][:20])
    assert torch.isfinite(outs[1]).all()


def test_a_nan_query_spoils_its_own_rows_only(vbq):
    import torch
    rng = np.random.default_rng(8)
    args, kw, out = attend(vbq, rng, 2, 4, 64, 32, [90, 50], [6, 1])
    q = args[1].clone()
    q[2, 5, 11] = float("nan")
    got = vbq.kv4_attention(args[0], q, *args[2:], **kw)
    assert torch.isnan(got[2, 5]).all()
    got[2, 5] = out[2, 5]
    assert torch.equal(got, out)


def test_cache_calls_on_another_stream_and_in_a_graph(vbq):
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(2)
    heads, dim, B, n = 2, 128, 3, 200
    cache = vbq.Kv4Cache(B * 4, 64, heads, dim)
    table = torch.randperm(B * 4, generator=gen, device="cuda").int().view(B, 4)
    kv = torch.randn(2, B * n, heads, dim, generator=gen, device="cuda").half()
    vbq.kv4_append(cache, kv[0], kv[1], table, torch.zeros(B, **i32), torch.arange(0, B * n + 1, n, **i32))
    k1, v1 = torch.randn(2, B, heads, dim, generator=gen, device="cuda").half()
    q = torch.randn(B, 8, dim, generator=gen, device="cuda").half()
    start, lens = torch.full((B,), n, **i32), torch.full((B,), n + 1, **i32)
    cu = torch.arange(B + 1, **i32)
    ws = vbq.kv4_attention_workspace(cache, B, B, 8, 1, 256)
    out = torch.empty_like(q)

    def step():
        vbq.kv4_append(cache, k1, v1, table, start, cu, max_tokens=1)
        vbq.kv4_attention(cache, q, table, lens, cu, 1, 256, out=out, workspace=ws)

    step()
    eager = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = vbq.kv4_attention(cache, q, table, lens, cu, 1, 256, stream=side)
    side.synchronize()
    assert torch.equal(got, eager)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        k1.copy_(torch.randn(k1.shape, generator=gen, device="cuda"))
        q.copy_(torch.randn(q.shape, generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        replayed = out.clone()
        step()
        assert torch.equal(out, replayed)


def test_far_pages_of_a_large_cache(vbq):
    """Byte offsets past 4 GiB."""
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    heads, dim, page = 8, 128, 1024
    n_pages = 4 * 2 ** 30 // vbq.lib.kv4_page_bytes(page, heads, dim) + 20
    cache = vbq.Kv4Cache(n_pages, page, heads, dim)
    small = vbq.Kv4Cache(2, page, heads, dim)
    gen = torch.Generator(device="cuda").manual_seed(4)
    kv = torch.randn(2, 1100, heads, dim, generator=gen, device="cuda").bfloat16()
    q = torch.randn(3, 32, dim, generator=gen, device="cuda").bfloat16()
    outs = []
    for c, table in ((cache, [[n_pages - 1, n_pages - 2]]), (small, [[0, 1]])):
        t = torch.tensor(table, **i32)
        cu = torch.tensor([0, 1100], **i32)
        vbq.kv4_append(c, kv[0], kv[1], t, torch.zeros(1, **i32), cu)
        outs.append((vbq.kv4_attention(c, q, t, torch.tensor([1100], **i32), torch.tensor([0, 3], **i32), 3, 1100),
                     *vbq.kv4_read(c, t, torch.zeros(1, **i32), cu, 1100, torch.float16)))
        assert c.check() is False
    for x, y in zip(*outs):
        assert torch.equal(x, y)


# ---- what does not fit ---------------------------------------------------------------
def test_wrong_tables_and_lengths_are_reported_and_touch_nothing(vbq):
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = vbq.Kv4Cache(3, 32, 1, 64)
    k = torch.randn(4, 1, 64, device="cuda")
    cu = torch.tensor([0, 1, 4], **i32)
    good = torch.tensor([[0, 1], [2, 1]], **i32)
    cases = [
        (torch.tensor([[3, 1], [-1, 1]], **i32), torch.zeros(2, **i32), cu, 3, "block-table"),
        (good, torch.tensor([-1, 64], **i32), cu, 3, "lengths"),
        (good, torch.zeros(2, **i32), torch.tensor([0, 3, 1], **i32), 2, "lengths"),
        (good, torch.zeros(2, **i32), torch.tensor([0, 0, 5], **i32), 9, "lengths"),
    ]
    for table, start, c, most, what in cases:
        before = cache.data.clone()
        vbq.kv4_append(cache, k, k, table, start, c, max_tokens=most)
        with pytest.raises(vbq.VbqError, match=what):
            cache.check()
        assert torch.equal(cache.data, before)
        assert cache.check() is False
    q = torch.randn(2, 2, 64, device="cuda").half()
    cu2 = torch.tensor([0, 1, 2], **i32)
    for table, lens, c, max_q, max_kv, what in [
        (torch.tensor([[0, 7], [2, 1]], **i32), [40, 40], cu2, 1, 64, "block-table"),
        (good, [65, 3], cu2, 1, 100, "lengths"),
        (good, [33, 3], cu2, 1, 32, "lengths"),
        (good, [-1, 3], cu2, 1, 64, "lengths"),
        (good, [3, 3], torch.tensor([0, 1, 9], **i32), 1, 64, "lengths"),
    ]:
        vbq.kv4_attention(cache, q, table, torch.tensor(lens, **i32), c, max_q, max_kv)
        with pytest.raises(vbq.VbqError, match=what):
            cache.check()
    # a page that is not there counts as no tokens; reading it gives zeros
    table = torch.tensor([[5, 1]], **i32)
    rk, rv = vbq.kv4_read(cache, table, torch.zeros(1, **i32), torch.tensor([0, 4], **i32), 4, torch.float32)
    assert not rk.any() and not rv.any()
    with pytest.raises(vbq.VbqError):
        cache.check()


def test_the_binding_refuses_what_does_not_fit(vbq):
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = vbq.Kv4Cache(2, 32, 2, 64)
    table, lens, cu = torch.zeros(1, 2, **i32), torch.tensor([3], **i32), torch.tensor([0, 1], **i32)
    q = torch.zeros(1, 4, 64, device="cuda").half()
    k = torch.zeros(1, 2, 64, device="cuda").half()
    with pytest.raises(ValueError, match="dtype"):
        vbq.kv4_attention(cache, q.float(), table, lens, cu, 1, 3)
    with pytest.raises(ValueError, match="shape"):
        vbq.kv4_attention(cache, q[:, :3], table, lens, cu, 1, 3)
    with pytest.raises(ValueError, match="lengths: dtype"):
        vbq.kv4_attention(cache, q, table, lens.long(), cu, 1, 3)
    with pytest.raises(ValueError, match="window"):
        vbq.kv4_attention(cache, q, table, lens, cu, 1, 3, causal=False, window=4)
    with pytest.raises(ValueError, match="aligned"):
        vbq.kv4_attention(cache, torch.zeros(1 * 4 * 64 + 1, device="cuda").half()[1:].view(1, 4, 64), table, lens, cu, 1, 3)
    with pytest.raises(ValueError, match="channels"):
        vbq.kv4_append(cache, k.transpose(1, 2).contiguous().transpose(1, 2), k, table, lens, cu)
    with pytest.raises(ValueError, match="v:"):
        vbq.kv4_append(cache, k, k.bfloat16(), table, lens, cu)
    with pytest.raises(ValueError, match="on cpu"):
        vbq.kv4_append(cache, k.cpu(), k, table, lens, cu)
    with pytest.raises(ValueError, match="out k"):
        vbq.kv4_read(cache, table, lens, cu, 1, torch.float16, out=(k.float(), k.float()))
    with pytest.raises(vbq.VbqError, match="layout does not match"):
        vbq.kv4_attention(cache, q, table, lens, cu, 1, 4096, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(vbq.VbqError, match="invalid argument"):
        vbq.kv4_attention(cache, q, table, lens, cu, 1, 3, scale=-1.0)
    with pytest.raises(ValueError, match="refused"):
        vbq.kv4_attention(cache, q, table, lens, cu, 1, -3)


# ---- the layer that runs them together ------------------------------------------------
@pytest.mark.parametrize("batch,prompt,steps,window", [(3, 70, 5, 0), (1, 200, 4, 60)])
def test_the_decode_example(vbq, batch, prompt, steps, window):
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import attention_decode as ex
    layer = ex.AttentionLayer(hidden=256, heads=8, kv_heads=2, dim=64)
    r = ex.run(batch, prompt, steps, window, layer=layer)
    assert r["tokens"] == prompt + steps + 1
    # probabilities, their product with a scale and the output are rounded to fp16 or better
    assert r["rel_l2"] <= 3 * 2.0 ** -11
    assert r["cache_bytes"] * 32 == r["bf16_bytes"] * 9


# ---- every output is written -----------------------------------------------------------
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("ratio,new", [(4, 1), (5, 1), (2, 3), (7, 1), (2, 4), (8, 1), (3, 3), (16, 1), (5, 4), (8, 4)])
def test_a_join_of_parts_writes_every_row(vbq, dim, ratio, new):
    """Every row count at which a tile's outputs take another turn of the joining workgroup, up to the full 4, 8, 16 and
    32 rows: what was in `out` and `lse` before the call is gone."""
    import torch
    rng = np.random.default_rng(100 * dim + 10 * ratio + new)
    lens, news = [1100, 37], [new, 1]
    args, kw, out = attend(vbq, rng, 1, ratio, dim, 32, lens, news, max_kv=1200)
    assert dim == 256 and ratio * new > 16 or \
        vbq.kv4_attention_workspace(args[0], 2, sum(news), ratio, new, 1200).numel() > 0     # (cut into parts)
    filled = torch.full_like(out, float("nan"))
    lse = torch.full(out.shape[:2], float("nan"), device="cuda")
    vbq.kv4_attention(*args, out=filled, lse=lse, **kw)
    assert torch.equal(filled, out) and torch.isfinite(lse).all()


# ---- sequences without new tokens --------------------------------------------------------
@pytest.mark.parametrize("start", [0, 3, 35, 63, 4000])
@pytest.mark.parametrize("dtype", ["float16", "float32"])
def test_an_append_of_no_tokens_looks_at_nothing(vbq, start, dtype):
    """A sequence that adds nothing neither needs pages nor rewrites them: its row of the table may be stale, -1, or name
    a page that another sequence of the call writes."""
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(start)
    k, v = torch.randn(2, 20, 2, 64, generator=gen, device="cuda").to(getattr(torch, dtype))
    data = random_cache(np.random.default_rng(start), 4, 32, 2, 64)
    alone, beside = (vbq.Kv4Cache(4, 32, 2, 64, data=gpu(data.copy())) for _ in range(2))
    vbq.kv4_append(alone, k, v, torch.tensor([[1, 2]], **i32), torch.tensor([30], **i32), torch.tensor([0, 20], **i32))
    for idle in ([-1, -1], [9, 9], [1, 2], [2, 1]):
        beside.data.copy_(gpu(data))
        vbq.kv4_append(beside, k, v, torch.tensor([idle, [1, 2], idle], **i32),
                       torch.tensor([start, 30, start], **i32), torch.tensor([0, 0, 20, 20], **i32), max_tokens=20)
        assert torch.equal(beside.data, alone.data)
        assert beside.check() is False
    assert alone.check() is False


# ---- queries near the end of bfloat16's range ---------------------------------------------
@pytest.mark.parametrize("dim,ratio,new", [(64, 4, 1), (128, 7, 4), (192, 2, 4), (64, 4, 30), (256, 2, 40)])
def test_attention_of_the_largest_queries(vbq, dim, ratio, new):
    """Queries of up to 2^119 on keys of ordinary size: scores are numbers that fp32 holds, and the largest takes its row.
    Rows whose two largest scores are nearer than 8 times their rounding (see the scores far out) are left out."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(dim + new)
    i32 = dict(dtype=torch.int32, device="cuda")
    L = 300
    k, v = torch.randn(2, L, 1, dim, generator=gen, device="cuda")
    q = ((torch.rand(new, ratio, dim, generator=gen, device="cuda") - 0.5) * 2.0 ** 120).bfloat16()
    cache = vbq.Kv4Cache(16, 32, 1, dim)
    table, cu = torch.arange(16, **i32).view(1, 16), torch.tensor([0, L], **i32)
    vbq.kv4_append(cache, k, v, table, torch.zeros(1, **i32), cu)
    rk, rv = (x.double()[:, 0] for x in vbq.kv4_read(cache, table, torch.zeros(1, **i32), cu, L, torch.float32))
    lse = torch.empty(new, ratio, device="cuda")
    got = vbq.kv4_attention(cache, q, table, torch.tensor([L], **i32), torch.tensor([0, new], **i32), new, L, lse=lse)
    assert torch.isfinite(got).all() and torch.isfinite(lse).all()
    used = 0
    for i in range(new):
        for r in range(ratio):
            qd = q[i, r].double()
            s = rk[:L - new + i + 1] @ qd * dim ** -0.5
            off = (dim + 17) * 2.0 ** -24 * float(qd.abs().sum() * 4 * rk.abs().max()) * dim ** -0.5
            top = torch.topk(s, 2).values
            assert abs(float(lse[i, r]) - float(top[0])) <= off + 2.0 ** -22 * abs(float(top[0]))
            if float(top[0] - top[1]) < 8 * off + 40:
                continue
            used += 1
            want = rv[int(s.argmax())]
            assert ((got[i, r].double() - want).abs() <= (2.0 ** -8 + 2.1 * 2.0 ** -11) * want.abs() + 2.0 ** -24).all()
    assert used * 2 >= new * ratio


# ---- products of codes lose nothing that binary32 holds -------------------------------------
def blank_cache(n_pages, heads, dim):
    return np.zeros(n_pages * heads * 2304 * (dim // 64), np.uint8), Layout(32, heads, dim)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("ratio,new", [(4, 1), (8, 1), (8, 2), (8, 4), (8, 5)])      # every tile
def test_scores_that_binary32_holds_are_exact(vbq, dtype, dim, ratio, new):
    """Sequences of one token, so lse is the score. One channel of the query is 2^8 times the others, scales are 1 and
    offsets -8: every sum of products is a whole multiple of 2^-18 below 2^5 in magnitude, in any order, which
    binary32 holds exactly. What is left are roundings of the score on its way to lse, u = 2^-24: scale * log2(e), two
    products and a difference, one u each of the score, and exponential and logarithm of a number of magnitude up
    to 16, a last place each, and its own rounding: below 8 u |score| + 2^-18."""
    import torch
    rng = np.random.default_rng(dim + new + ratio)
    B, G = 6, dim // 64
    data, lay = blank_cache(B, 1, dim)
    codes = rng.integers(0, 16, (B, G, 64)).astype(np.uint32)
    one, off, zero = np.ones(G, np.float16), np.full(G, -8, np.float16), np.zeros(G, np.float16)
    for b in range(B):
        lay.write(data, lay.block(b, 0, 0), 0, 0, codes[b], one, off)
        lay.write(data, lay.block(b, 0, 0), 0, 1, codes[b], one, zero)
    T, steps = B * new, 1024 if dtype == "float16" else 128
    q = (1 + rng.integers(0, steps, (T, ratio, dim)) / steps) * rng.choice([-1, 1], (T, ratio, dim)) * 2.0 ** -8
    big = rng.integers(0, 64, (T, ratio))
    np.put_along_axis(q, big[..., None], np.take_along_axis(q, big[..., None], -1) * 2.0 ** 8, -1)
    qt = torch.from_numpy(q).to(getattr(torch, dtype))
    assert np.array_equal(qt.double().numpy(), q)
    cache = vbq.Kv4Cache(B, 32, 1, dim, data=gpu(data))
    lse = torch.full((T, ratio), float("nan"), device="cuda")
    vbq.kv4_attention(cache, qt.cuda(), torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1),
                      gpu(np.ones(B, np.int32)), gpu(cum([new] * B)), new, 1, scale=8.0, causal=False, lse=lse)
    K = codes.reshape(B, dim).astype(np.float64) - 8
    want = 8 * np.einsum("trd,td->tr", q, np.repeat(K, new, 0))
    err = np.abs(lse.cpu().numpy().astype(np.float64) - want)
    bound = 8 * 2.0 ** -24 * np.abs(want) + 2.0 ** -18
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("dim,ratio,new", [(d, r, n) for d in (64, 128, 192, 256)      # every tile of the few-row kernel
                                           for r, n in ((4, 1), (8, 1), (8, 2), (8, 4)) if d < 256 or r * n <= 16])
def test_sums_of_values_that_binary32_holds_are_exact(vbq, dim, ratio, new):
    """Sixteen tokens of equal probability (queries of 0), two with scales 2^8 times the others', offsets about -7.5
    scales: sums of s c are whole multiples of 2^-18 below 2^6 and those of offsets too, in any order, so binary32 holds
    them and their difference, and the output is the exact mean, rounded once."""
    import torch
    rng = np.random.default_rng(dim + new + ratio)
    G, n = dim // 64, 16
    data, lay = blank_cache(1, 1, dim)
    want = np.zeros(dim)
    for t in range(n):
        codes = rng.integers(0, 16, (G, 64)).astype(np.uint32)
        s = ((1 + rng.integers(0, 1024, G) / 1024) * (1.0 if t in (5, 8) else 2.0 ** -8)).astype(np.float16)
        o = (-7.5 * s.astype(np.float64)).astype(np.float16)
        lay.write(data, lay.block(0, 0, t), t, 0, codes, s, o)
        lay.write(data, lay.block(0, 0, t), t, 1, codes, s, o)
        want += (codes * s.astype(np.float64)[:, None] + o.astype(np.float64)[:, None]).reshape(-1)
    cache = vbq.Kv4Cache(1, 32, 1, dim, data=gpu(data))
    i32 = dict(dtype=torch.int32, device="cuda")
    got = vbq.kv4_attention(cache, torch.zeros(new, ratio, dim, device="cuda").half(), torch.zeros(1, 1, **i32),
                            torch.tensor([n], **i32), torch.tensor([0, new], **i32), new, n, causal=False)
    want = (want / n).astype(np.float16)
    assert (got.cpu().numpy() == want).all()


@pytest.mark.parametrize("batch,heads,ratio,dim,kv", [(8, 4, 4, 128, 1500), (6, 4, 1, 64, 5000), (4, 4, 2, 192, 1700),
                                                      (6, 2, 6, 128, 2500), (5, 2, 20, 64, 1500), (4, 2, 8, 256, 1500)])
def test_few_rows_are_as_near_as_the_output_type_allows(vbq, batch, heads, ratio, dim, kv):
    """Keys with strong channels over many tokens, fp16 outputs: the root mean square error exceeds that of the exact
    outputs' own rounding by what binary32 scores leave. A score's terms have magnitudes that add up to
    S = scale sum |q| (|s c| + |o|), up to 250 here; its sums take four roundings of such a size (two products a
    group, scale, offset): 4 u S = 6e-5 of a probability."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(dim + kv)
    i32 = dict(dtype=torch.int32, device="cuda")
    pages = -(-kv // 256)
    cache = vbq.Kv4Cache(batch * pages, 256, heads, dim)
    table = torch.randperm(batch * pages, generator=gen, device="cuda").int().view(batch, pages)
    gain = torch.ones(dim, device="cuda")
    gain[::17] = 4.0
    k, v = torch.randn(2, batch * kv, heads, dim, generator=gen, device="cuda")
    k = k * gain + torch.randn(heads, dim, generator=gen, device="cuda")
    start, cu = torch.zeros(batch, **i32), torch.arange(0, batch * kv + 1, kv, **i32)
    vbq.kv4_append(cache, k, v, table, start, cu, max_tokens=kv)
    k, v = (x.double().view(batch, kv, heads, dim) for x in
            vbq.kv4_read(cache, table, start, cu, batch * kv, torch.float32, max_tokens=kv))
    q = (torch.randn(batch, heads * ratio, dim, generator=gen, device="cuda") * 1.5).half()
    got = vbq.kv4_attention(cache, q, table, torch.full((batch,), kv, **i32), torch.arange(batch + 1, **i32), 1, kv)
    want = torch.empty(batch, heads * ratio, dim, dtype=torch.float64, device="cuda")
    for b in range(batch):
        for h in range(heads):
            rows = slice(h * ratio, (h + 1) * ratio)
            p = torch.softmax(q[b, rows].double() @ k[b, :, h].T.contiguous() * dim ** -0.5, -1)
            want[b, rows] = p @ v[b, :, h].contiguous()
    rms = lambda x: float(x.square().mean().sqrt())
    more = rms(got.double() - want) ** 2 - rms(want.half().double() - want) ** 2
    assert max(more, 0.0) ** 0.5 <= 6e-5 * rms(want), (max(more, 0.0) ** 0.5 / rms(want))


@pytest.mark.parametrize("dim", [64, 128, 192, 256])
@pytest.mark.parametrize("ratio,new", [(4, 1), (8, 2), (8, 4), (8, 5), (2, 40)])
@pytest.mark.parametrize("exp", [-14, -12, -9, -4, 0, 15])
def test_key_offsets_of_any_size_enter_scores_in_binary32(vbq, dim, ratio, new, exp):
    """Sequences of one token whose keys are constant groups (scale 0, offset o of about 2^exp), so lse is scale * sum of
    o sum(q). Queries of one binade: their sums are exact in binary32. Products with offsets and their sum over groups,
    all of one sign, take below 8 u; with the roundings of test_scores_that_binary32_holds_are_exact below
    16 u |score| + 2^-18."""
    import torch
    rng = np.random.default_rng(dim + new + ratio + 50 + exp)
    B, G = 4, dim // 64
    data, lay = blank_cache(B, 1, dim)
    off = ((1 + rng.integers(0, 1024, (B, G)) / 1024) * 2.0 ** exp).astype(np.float16)
    off = np.minimum(off, np.float16(61440))
    for b in range(B):
        zero = np.zeros(G, np.float16)
        lay.write(data, lay.block(b, 0, 0), 0, 0, rng.integers(0, 16, (G, 64)).astype(np.uint32), zero, off[b])
        lay.write(data, lay.block(b, 0, 0), 0, 1, np.zeros((G, 64), np.uint32), zero, zero)
    T = B * new
    q = 1 + rng.integers(0, 1024, (T, ratio, dim)) / 1024
    scale = 2.0 ** (-2 - exp)
    cache = vbq.Kv4Cache(B, 32, 1, dim, data=gpu(data))
    lse = torch.full((T, ratio), float("nan"), device="cuda")
    vbq.kv4_attention(cache, torch.from_numpy(q).half().cuda(),
                      torch.arange(B, dtype=torch.int32, device="cuda").view(B, 1), gpu(np.ones(B, np.int32)),
                      gpu(cum([new] * B)), new, 1, scale=scale, causal=False, lse=lse)
    sums = q.reshape(T, ratio, G, 64).sum(-1)
    want = scale * np.einsum("trg,tg->tr", sums, np.repeat(off.astype(np.float64), new, 0))
    err = np.abs(lse.cpu().numpy().astype(np.float64) - want)
    bound = 16 * 2.0 ** -24 * np.abs(want) + 2.0 ** -18
    assert (err <= bound).all(), float((err / bound).max())


def test_check_waits_for_calls_on_other_streams(vbq):
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = vbq.Kv4Cache(2, 32, 1, 64)
    k = torch.zeros(1, 1, 64, device="cuda")
    args = (torch.tensor([[7]], **i32), torch.zeros(1, **i32), torch.tensor([0, 1], **i32))      # page 7 of 2
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)        # work ahead of the call on its stream
    vbq.kv4_append(cache, k, k, *args, stream=side)
    with pytest.raises(vbq.VbqError, match="block-table"):
        cache.check()
    assert cache.check() is False


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32 + 1, 2 ** 40, -2 ** 31 - 1])
def test_the_binding_refuses_numbers_beyond_an_int(vbq, big):
    """As a ValueError, whichever argument it is; a workspace is not sized for what is left of such a number."""
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = vbq.Kv4Cache(2, 32, 2, 64)
    table, lens, cu = torch.zeros(1, 2, **i32), torch.tensor([3], **i32), torch.tensor([0, 1], **i32)
    q = torch.zeros(1, 4, 64, device="cuda").half()
    k = torch.zeros(1, 2, 64, device="cuda").half()
    ws = vbq.kv4_attention_workspace(cache, 1, 1, 4, 1, 4096)
    for kw in (dict(max_q=big), dict(max_kv=big), dict(window=big), dict(sinks=big, window=4)):
        args = dict(dict(max_q=1, max_kv=3), **kw)
        with pytest.raises(ValueError, match="kv4_attention"):
            vbq.kv4_attention(cache, q, table, lens, cu, workspace=ws, **args)
        with pytest.raises(ValueError, match="kv4_attention"):
            vbq.kv4_attention(cache, q, table, lens, cu, **args)
    for sizes in ((big, 1, 4, 1, 9), (1, big, 4, 1, 9), (1, 1, 2 * big, 1, 9), (1, 1, 4, big, 9), (1, 1, 4, 1, big)):
        with pytest.raises(ValueError, match="kv4_attention"):
            vbq.kv4_attention_workspace(cache, *sizes)
    with pytest.raises(ValueError, match="kv4_append"):
        vbq.kv4_append(cache, k, k, table, lens, cu, max_tokens=big)
    with pytest.raises(ValueError, match="kv4_read"):
        vbq.kv4_read(cache, table, lens, cu, 1, torch.float16, max_tokens=big)
    assert cache.check() is False


# ---- maxima that say nothing -----------------------------------------------------------------
@pytest.mark.parametrize("most", [2 ** 24, 2 ** 29 + 500, 2 ** 30, 2 ** 31 - 1])
@pytest.mark.parametrize("heads", [1, 8])
def test_a_maximum_far_beyond_the_lengths_changes_nothing(vbq, most, heads):
    """max_tokens and max_q may be any number that no sequence passes."""
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(heads)
    k, v = torch.randn(2, 700, heads, 64, generator=gen, device="cuda").half()
    table, start = torch.arange(8, **i32).view(2, 4), torch.tensor([5, 100], **i32)
    cu = torch.tensor([0, 300, 700], **i32)
    a, b = (vbq.Kv4Cache(8, 128, heads, 64) for _ in range(2))
    vbq.kv4_append(a, k, v, table, start, cu, max_tokens=400)
    vbq.kv4_append(b, k, v, table, start, cu, max_tokens=most)
    assert torch.equal(a.data, b.data) and a.data.any()
    out = torch.full((2, 700, heads, 64), 9.0, device="cuda").half()
    vbq.kv4_read(a, table, start, cu, 700, torch.float16, max_tokens=most, out=(out[0], out[1]))
    for x, y in zip(out, vbq.kv4_read(a, table, start, cu, 700, torch.float16, max_tokens=400)):
        assert torch.equal(x, y)
    most = min(most, 2 ** 31 - 1 - 128)
    q = torch.randn(700, heads, 64, generator=gen, device="cuda").half()
    args = (a, q, table, start + torch.tensor([300, 400], **i32), cu)
    ws = vbq.kv4_attention_workspace(a, 2, 700, heads, most, 128)      # too short to be cut, whatever max_q
    want = vbq.kv4_attention(*args, 400, 512)
    got = torch.full_like(want, float("nan"))
    vbq.kv4_attention(*args, most, 512, out=got)
    # the same kernel; with the smaller maximum it may have cut the tiles, which sums in another order
    assert float((got.double() - want.double()).abs().max()) <= 2.0 ** -9 * float(want.abs().max())
    assert ws.numel() == 0 and a.check() is False and b.check() is False


@pytest.mark.parametrize("dtype,size", [("float16", 2.0 ** -12), ("bfloat16", 2.0 ** -12), ("bfloat16", 2.0 ** -120)])
@pytest.mark.parametrize("scale", [1e-45, 1e-41, 1e-30, 1e-3])
@pytest.mark.parametrize("dim,ratio,new", [(64, 4, 1), (128, 4, 3), (64, 4, 30), (256, 2, 40)])
def test_attention_of_vanishing_scores(vbq, dtype, size, scale, dim, ratio, new):
    """However small scale and queries are, tokens that are seen weigh the same and hidden ones nothing: scores are below
    2^-8 in magnitude, so probabilities are off by 2^-7 of themselves at most, and the rest is as in check()."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(dim + new)
    i32 = dict(dtype=torch.int32, device="cuda")
    L = 70
    k, v = torch.randn(2, L, 1, dim, generator=gen, device="cuda")
    q = ((torch.rand(new, ratio, dim, generator=gen, device="cuda") - 0.5) * 2 * size).to(getattr(torch, dtype))
    cache = vbq.Kv4Cache(4, 32, 1, dim)
    table, cu = torch.arange(4, **i32).view(1, 4), torch.tensor([0, L], **i32)
    vbq.kv4_append(cache, k, v, table, torch.zeros(1, **i32), cu)
    rv = vbq.kv4_read(cache, table, torch.zeros(1, **i32), cu, L, torch.float32)[1].double()[:, 0]
    lse = torch.empty(new, ratio, device="cuda")
    got = vbq.kv4_attention(cache, q, table, torch.tensor([L], **i32), torch.tensor([0, new], **i32), new, L,
                            scale=scale, window=40, sinks=2, lse=lse)
    for i in range(new):
        p = L - new + i
        see = [j for j in range(p + 1) if j > p - 40 or j < 2]
        want, mass = rv[see].mean(0), rv[see].abs().mean(0)
        bound = (2.0 ** -7 + 2.1 * 2.0 ** -11) * mass + 2.0 ** -8 * want.abs() + 2.0 ** -24
        assert ((got[i].double() - want).abs() <= bound).all()
        assert ((lse[i].double() - math.log(len(see))).abs() <= 2.0 ** -7).all()

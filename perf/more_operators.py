"""Operators for several continuations of one prompt, as they are measured.

Four operators around the packed projections and the 4-bit key/value cache
(its layout is stated in include/vbq.h, "4-bit key/value cache"):

- rotary: queries and keys of every head are normed and rotated by their
  positions (one axis, or several for images and video) in one pass;
- fork: sequences of the cache become continuations of others; whole pages are
  shared, part pages copied, pages that nobody names any more are free again;
- shared: attention of sequences that have their first tokens in common, group
  by group;
- logprobs: log probabilities of given tokens, their ranks, entropies and the
  most likely tokens, from rows of logits.

``own`` selects the framework's kernels; otherwise ``run`` computes the same
results with elementary torch operations in 32 bits (angles in 64).
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}
EPS = 1e-6


# ---- cases -----------------------------------------------------------------------
def _rotary(dtype, out, tokens, heads, kv_heads, dim, rotary, axes=1, interleaved=False, norm=True, far=4096):
    """Queries and keys of `dtype` to `out`; positions up to `far`."""
    return dict(op="rotary", dtype=dtype, out=out, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim,
                rotary=rotary, axes=axes, interleaved=interleaved, norm=norm, far=far)


def _fork(prompts, beams, kv_heads, dim, page, tokens, reserve, pattern, ragged=0):
    """prompts * beams sequences after the call. pattern "first": each prompt's beams all go on from its one
    sequence; "beams": from its beams at random; "some": so too, and one in five ends."""
    return dict(op="fork", prompts=prompts, beams=beams, kv_heads=kv_heads, dim=dim, page=page, tokens=tokens,
                reserve=reserve, pattern=pattern, ragged=ragged)


def _shared(dtype, groups, per, heads, kv_heads, dim, page, shared, mine, new, ragged=0):
    """`per` sequences a group; `shared` tokens in common, then up to `mine` of their own, the `new` last ones queried."""
    return dict(op="shared", dtype=dtype, groups=groups, per=per, heads=heads, kv_heads=kv_heads, dim=dim, page=page,
                shared=shared, mine=mine, new=new, ragged=ragged)


def _logprobs(dtype, rows, vocab, top, masked=False):
    return dict(op="logprobs", dtype=dtype, rows=rows, vocab=vocab, top=top, masked=masked)


def listed():
    cases = []

    def add(name, case):
        cases.append(dict(name=name, **case))

    # one decode step of one conversation, 131M-class model (hidden 768: 12 heads of 64), from the packed GEMV
    add("rotary_one", _rotary("f32", "f16", 1, 12, 12, 64, 64))
    # prompts of odd lengths in all, 9B-class model with normed queries and keys
    add("rotary_prompts", _rotary("bf16", "bf16", 25763, 32, 8, 128, 128, far=131072))
    # images and text of odd number: time, height and width, neighbouring channels paired, half of a head turned
    add("rotary_images", _rotary("f32", "f16", 7001, 16, 4, 256, 128, axes=3, interleaved=True, far=1200))
    # a prompt is about to be continued eight times, 131M-class model
    add("fork_one", _fork(1, 8, 12, 64, 32, 577, 1, "first"))
    # a step of beam search: 64 prompts with eight beams each, 9B-class model
    add("fork_beams", _fork(64, 8, 8, 128, 256, 4001, 1, "beams", ragged=1))
    # eight continuations of a short prompt, 131M-class model
    add("shared_few", _shared("f16", 1, 8, 12, 12, 64, 32, 545, 33, 1, ragged=2))
    # a decode step of 32 continuations of one long prompt, 9B-class model
    add("shared_step", _shared("f16", 1, 32, 32, 8, 128, 64, 8192, 512, 1, ragged=3))
    # six prompts of odd lengths, 16 continuations each, three drafted tokens of each are checked
    add("shared_groups", _shared("bf16", 6, 16, 32, 8, 128, 128, 4097, 301, 3, ragged=4))
    # 64 questions about one book
    add("shared_long", _shared("bf16", 1, 64, 32, 8, 128, 256, 65000, 257, 1, ragged=5))
    # the next token's alternatives of one conversation, the LM head of the 9B-class stack
    add("logprobs_one", _logprobs("f32", 1, 128256, 20))
    # a step of beam search over a vocabulary of odd size of which a grammar masks a part
    add("logprobs_beams", _logprobs("bf16", 64, 32001, 16, masked=True))
    # the tokens of a long prompt are scored
    add("logprobs_prompt", _logprobs("f32", 2047, 128256, 5))
    return cases


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(12, 1, 64), (8, 4, 128), (16, 1, 128), (4, 4, 256), (8, 4, 64), (2, 7, 128), (4, 8, 128), (8, 2, 192)]


def draw(rng):
    op = rng.choice(["rotary", "fork", "shared", "shared", "logprobs"])
    kv_heads, group, dim = rng.choice(HEADS)
    page, ragged = rng.choice([32, 64, 128, 256]), rng.randrange(1, 1 << 20)
    if op == "rotary":
        axes = rng.choice([1, 1, 2, 3])
        tokens = min(_log(rng, 1, 25763), 25763 * 40 * 128 // (kv_heads * (1 + group) * dim))
        dtype = rng.choice(["f16", "bf16", "f32"])
        tokens = tokens if dtype != "f32" else max(1, tokens // 2)
        return _rotary(dtype, rng.choice(["f16", "bf16"]), tokens, kv_heads * group, kv_heads, dim,
                       rng.choice([dim, dim, dim // 2, 32]), axes, rng.random() < 0.4, rng.random() < 0.7,
                       _log(rng, 100, 1 << 20))
    if op == "fork":
        prompts, beams = _log(rng, 1, 64), rng.choice([1, 2, 3, 4, 5, 8])
        most = 64 * 4001 * 1024 // (kv_heads * dim * prompts)
        return _fork(prompts, beams, kv_heads, dim, page, max(1, min(_log(rng, 1, 9000), most)),
                     rng.choice([0, 1, 1, 5]), rng.choice(["first", "beams", "beams", "some"]), ragged)
    if op == "shared":
        dtype = rng.choice(["f16", "bf16"])
        groups, per = rng.choice([1, 1, _log(rng, 2, 12)]), _log(rng, 2, 64)
        new = rng.choice([1, 1, 1, rng.randrange(2, 6)])
        shared = _log(rng, 32, 65000)
        mine = new + _log(rng, 1, 600)
        pairs = 6 * 10 ** 10 // (kv_heads * group * dim)     # (row, token) pairs a head
        shared = max(1, min(shared, pairs // (4 * groups * per * new), 65000 * 1024 // (kv_heads * dim * groups)))
        return _shared(dtype, groups, per, kv_heads * group, kv_heads, dim, page, shared, mine, new, ragged)
    vocab = rng.choice([128256, 32001, 1000, _log(rng, 300, 160001)])
    dtype = rng.choice(["f32", "f32", "bf16", "f16"])
    rows = max(1, min(_log(rng, 1, 4000), 2047 * 128256 // vocab))
    return _logprobs(dtype, rows, vocab, rng.choice([0, 1, 5, 8, 20, 32]), rng.random() < 0.3)


def _lengths(case):
    """Shared tokens of every group, and tokens of every sequence."""
    rng = random.Random(case["ragged"])
    shared = [case["shared"]] + [rng.randint(case["shared"] // 2, case["shared"]) for _ in range(case["groups"] - 1)]
    lens = []
    for g in shared:
        for _ in range(case["per"]):
            lens.append(g + rng.randint(case["new"], case["mine"]))
    lens[0] = shared[0] + case["mine"]
    return shared, lens


def _sequences(case):
    """A cache's sequences before a fork: pages [B][W] (numbers in order of use, -1: none), lengths, parents of the
    sequences after it, and how many pages are in use."""
    rng = random.Random(case["ragged"])
    page, width = case["page"], -(-(case["tokens"] + case["reserve"] + 3) // case["page"])
    rows, lens, parents, used = [], [], [], 0
    before = 1 if case["pattern"] == "first" else case["beams"]
    for p in range(case["prompts"]):
        n = case["tokens"] if p == 0 else rng.randint(1 + case["tokens"] // 2, case["tokens"])
        # the beams had the first `common` pages together and a page or more of their own since
        common = n // page if before == 1 else rng.randint(0, n // page)
        shared = list(range(used, used + common))
        used += common
        for b in range(before):
            more = -(-n // page) - common
            rows.append(shared + list(range(used, used + more)) + [-1] * (width - common - more))
            used += more
            lens.append(n)
        for b in range(case["beams"]):
            parent = p * before + (0 if before == 1 else rng.randrange(before))
            parents.append(-1 if case["pattern"] == "some" and rng.random() < 0.2 else parent)
    return rows, lens, parents, used, width


def work(case):
    if case["op"] == "rotary":
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        return dict(bytes=n * (BYTES[case["dtype"]] + BYTES[case["out"]]) + 4 * case["tokens"] * case["axes"], flops=8 * n)
    if case["op"] == "fork":
        rows, lens, parents, used, width = _sequences(case)
        block = case["kv_heads"] * case["dim"] // 64 * 2304
        seen, copied = set(), 0
        for p in parents:
            if p >= 0 and p in seen:
                copied += -(-(lens[p] % case["page"]) // 32) * block
            seen.add(p)
        pages = _pool(case, used)
        return dict(bytes=2 * copied + 4 * (width * (len(rows) + len(parents)) + 2 * pages + len(rows) + 3 * len(parents)),
                    flops=0)
    if case["op"] == "shared":
        shared, lens = _lengths(case)
        held = case["kv_heads"] * case["dim"] * 9 // 8       # bytes of a token's keys and values
        own_tokens = sum(n - shared[b // case["per"]] for b, n in enumerate(lens))
        pairs = sum(sum(range(n - case["new"] + 1, n + 1)) for n in lens)
        io = 2 * len(lens) * case["new"] * case["heads"] * case["dim"] * 2
        return dict(bytes=(sum(shared) + own_tokens) * held + io + 4 * len(lens), flops=4 * case["dim"] * case["heads"] * pairs)
    n = case["rows"] * case["vocab"]
    return dict(bytes=n * BYTES[case["dtype"]] + case["rows"] * (20 + 8 * case["top"]), flops=6 * n)


# ---- inputs ----------------------------------------------------------------------
def _pool(case, used):
    """Pages of a fork's cache."""
    return used + case["prompts"] * case["beams"] * (2 + case["reserve"] // case["page"]) + 8


def _prepare_rotary(case, gen):
    T, H, K, D = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    dt = DTYPES[case["dtype"]]
    if case["dtype"] == "f32":   # outputs of two packed projections
        q = torch.randn(T, H, D, generator=gen, device="cuda") * 2.0
        k = torch.randn(T, K, D, generator=gen, device="cuda") * 2.0
        q[..., ::13] *= 5.0
        k[..., ::17] *= 5.0
    else:                        # slices of one projection's output
        both = torch.randn(T, (H + 2 * K) * D, generator=gen, device="cuda", dtype=dt) * 2.0
        both[:, ::13] *= 5.0
        q, k = both[:, :H * D].unflatten(-1, (H, D)), both[:, H * D:(H + K) * D].unflatten(-1, (K, D))
    pos = torch.randint(0, case["far"], (case["axes"], T), generator=gen, device="cuda", dtype=torch.int32)
    half = case["rotary"] // 2
    inv_freq = (10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()
    axis = (torch.arange(half) % case["axes"]).to(torch.uint8).cuda()
    st = dict(case=case, q=q, k=k, pos=pos if case["axes"] > 1 else pos[0], inv_freq=inv_freq, axis=axis, qw=None, kw=None)
    if case["norm"]:
        st["qw"] = 1.0 + 0.2 * torch.randn(D, generator=gen, device="cuda")
        st["kw"] = 1.0 + 0.2 * torch.randn(D, generator=gen, device="cuda")
    if own:
        import packed_decode_gemv_amd as vbq
        st["plan"] = vbq.HeadRotary(D, inv_freq, axis=axis if case["axes"] > 1 else None, axes=case["axes"],
                                    interleaved=case["interleaved"], q_weight=st["qw"], k_weight=st["kw"], eps=EPS)
    return st


def _prepare_fork(case, gen):
    rows, lens, parents, used, width = _sequences(case)
    n_pages = _pool(case, used)
    words = case["page"] // 32 * case["kv_heads"] * case["dim"] // 64 * 576
    number = torch.randperm(n_pages, generator=gen, device="cuda").int()
    table = torch.tensor(rows, dtype=torch.int32).cuda()
    table = torch.where(table >= 0, number[table.clamp(min=0).long()], table).contiguous()
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs.index_add_(0, table.flatten().clamp(min=0).long(), (table.flatten() >= 0).int())
    refs[number[-2:].long()] = 1                            # pages that something else holds
    data = torch.randint(-2 ** 31, 2 ** 31 - 1, (n_pages, words), generator=gen, device="cuda", dtype=torch.int32)
    st = dict(case=case, table=table, refs=refs, data=data, lens=torch.tensor(lens, dtype=torch.int32).cuda(),
              parents=torch.tensor(parents, dtype=torch.int32).cuda(),
              reserve=torch.full((len(parents),), case["reserve"], dtype=torch.int32, device="cuda"))
    if own:
        import packed_decode_gemv_amd as vbq
        st["cache"] = vbq.Kv4Cache(n_pages, case["page"], case["kv_heads"], case["dim"],
                                   data=data.view(torch.uint8).view(-1))
        st["workspace"] = vbq.kv4_fork_workspace(st["cache"], len(parents), width)
    return st


def _quantise(x):
    """Codes (int32), scale and offset (float16) of groups of 64 values on the last axis, in 32 bits."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s, o = ((hi - lo) / 15.0).half(), lo.half()
    sf = s.float()
    q = torch.where(sf == 0, torch.zeros_like(x), ((x - o.float()) / sf).round().clamp(0, 15))
    return q.int(), s.squeeze(-1), o.squeeze(-1)


def _nibbles(q):
    """int32 words of eight 4-bit codes on the last axis, the first lowest."""
    return (q << torch.arange(0, 32, 4, device=q.device, dtype=torch.int32)).sum(-1, dtype=torch.int32)


def _blocks(kq, ks, ko, vq, vs, vo):
    """Cache blocks (int32 words) of 32 tokens: codes [*, 32, G, 64], scales and offsets [*, 32, G]."""
    lead, G = kq.shape[:-3], kq.shape[-2]
    n = len(lead)
    keep = list(range(n))
    kw = kq.reshape(*lead, 4, 2, 4, G, 2, 4, 8).permute(*keep, n + 3, n + 5, n, n + 2, n + 1, n + 4, n + 6)
    vw = vq.reshape(*lead, 4, 8, G, 64).permute(*keep, n + 2, n, n + 3, n + 1)

    def so(s, o, order):
        t = torch.stack([s, o], -1).reshape(*lead, 4, 8, G, 2)[..., order, :, :]
        return t.permute(*keep, n + 2, n + 3, n, n + 1).reshape(*lead, -1).contiguous().view(torch.int32)

    return torch.cat([_nibbles(kw).reshape(*lead, -1), _nibbles(vw).reshape(*lead, -1), so(ks, ko, list(range(8))),
                      so(vs, vo, [0, 4, 1, 5, 2, 6, 3, 7])], -1)


def _prepare_shared(case, gen):
    shared, lens = _lengths(case)
    G, per, page, H, D = case["groups"], case["per"], case["page"], case["kv_heads"], case["dim"]
    B, T = G * per, G * per * case["new"]
    width = -(-max(lens) // page)
    rows, used = [], 0
    for g in range(G):
        whole = shared[g] // page
        first = list(range(used, used + whole))
        used += whole
        for b in range(g * per, g * per + per):
            n = -(-lens[b] // page) - whole
            rows.append(first + list(range(used, used + n)) + [0] * (width - whole - n))
            used += n
    n_pages = used + 3
    number = torch.randperm(n_pages, generator=gen, device="cuda").int()
    table = number[torch.tensor(rows).cuda()].contiguous()
    words, blocks = D // 64 * 576, page // 32
    data = torch.empty(n_pages, H, blocks, words, dtype=torch.int32, device="cuda")
    gain = torch.ones(H, 1, 1, D, device="cuda")
    gain[..., ::17] = 4.0
    shift = torch.randn(H, 1, 1, D, generator=gen, device="cuda")
    step = max(1, (1 << 25) // (H * blocks * 32 * D))
    for p in range(0, n_pages, step):
        m = min(step, n_pages - p)
        k = torch.randn(m, H, blocks, 32, D, generator=gen, device="cuda") * gain + shift
        v = torch.randn(m, H, blocks, 32, D, generator=gen, device="cuda")
        data[p:p + m] = _blocks(*_quantise(k.unflatten(-1, (-1, 64))), *_quantise(v.unflatten(-1, (-1, 64))))
    # a part page in common is a copy of its own in every sequence, as a fork leaves it
    for g in range(G):
        if shared[g] % page:
            at = table[g * per:g * per + per, shared[g] // page].long()
            n = -(-(shared[g] % page) // 32)
            data[at, :, :n] = data[at[0], :, :n].clone()
    st = dict(case=case, table=table, data=data, lens=torch.tensor(lens, dtype=torch.int32).cuda(),
              shared=torch.tensor(shared, dtype=torch.int32).cuda(),
              cu=(torch.arange(B + 1, device="cuda") * case["new"]).int(),
              cu_groups=(torch.arange(G + 1, device="cuda") * per).int(),
              q=(torch.randn(T, case["heads"], D, generator=gen, device="cuda") * 1.5).to(DTYPES[case["dtype"]]))
    if own:
        import packed_decode_gemv_amd as vbq
        st["cache"] = vbq.Kv4Cache(n_pages, page, H, D, data=data.view(torch.uint8).view(-1))
        st["workspace"] = vbq.kv4_attention_shared_workspace(st["cache"], B, G, T, case["heads"], max_q=case["new"],
                                                             max_shared=case["shared"], max_own=case["mine"],
                                                             max_group_q=per * case["new"])
    return st


def _prepare_logprobs(case, gen):
    M, V = case["rows"], case["vocab"]
    sharp = torch.rand(M, 1, generator=gen, device="cuda") * 2.5 + 1.0
    x = torch.randn(M, V, generator=gen, device="cuda")
    x *= sharp
    tokens = torch.randint(0, V, (M,), generator=gen, device="cuda")
    likely = torch.randint(0, V, (M, 4), generator=gen, device="cuda")
    x.scatter_add_(1, likely, torch.rand(M, 4, generator=gen, device="cuda") * 14.0)
    tokens[::2] = likely[::2, 0]                           # half of the tokens are likely ones
    if case["masked"]:                                      # a grammar leaves every third token, of some rows only a few
        x[:, 1::3] = -math.inf
        x[:, 2::3] = -math.inf
        x[::5, 30:] = -math.inf
        tokens = (tokens - tokens % 3)
        tokens[::5] %= 30
        tokens -= tokens % 3
    st = dict(case=case, logits=x.to(DTYPES[case["dtype"]]), tokens=tokens)
    if own:
        import packed_decode_gemv_amd as vbq
        st["workspace"] = vbq.token_logprobs_workspace(M, V, case["top"], device="cuda")
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"rotary": _prepare_rotary, "fork": _prepare_fork, "shared": _prepare_shared,
            "logprobs": _prepare_logprobs}[case["op"]](case, gen)


# ---- plain forms -----------------------------------------------------------------
def _plain_rotary(st):
    case, half = st["case"], st["case"]["rotary"] // 2
    pos = st["pos"].reshape(case["axes"], -1)[st["axis"].long()].T.double()      # [T][pairs]
    angle = pos * st["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    out = []
    for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
        if case["interleaved"]:
            a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:2 * half]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        out.append(torch.cat([turned, x[..., 2 * half:]], -1).to(DTYPES[case["out"]]))
    return out


def _plain_fork(st):
    page, table, refs, parents = st["case"]["page"], st["table"], st["refs"], st["parents"]
    n_pages, W = refs.numel(), table.shape[1]
    goes_on = parents >= 0
    p = parents.clamp(min=0).long()
    lens = torch.where(goes_on, st["lens"][p], 0)
    rows = table[p]
    j = torch.arange(W, device="cuda")
    whole, have, need = lens // page, (lens + page - 1) // page, (lens + st["reserve"] + page - 1) // page
    need = torch.minimum(need, torch.full_like(need, W))
    index = torch.arange(len(parents), device="cuda")
    same = (parents[:, None] == parents[None, :]) & goes_on[:, None] & (index[None, :] < index[:, None])
    first = goes_on & ~same.any(1)
    mine = first[:, None] & (rows >= 0) & (refs[rows.clamp(min=0).long()] == 1)
    share = goes_on[:, None] & (j < whole[:, None])
    keep = share | (mine & (j >= whole[:, None]) & (j < need[:, None]))
    fresh = ~keep & (j >= whole[:, None]) & (j < need[:, None])
    free = (refs == 0).nonzero().squeeze(-1)
    order = (torch.cumsum(fresh.flatten().int(), 0) - 1).view_as(fresh)
    taken = free[order.clamp(min=0)].int()
    new_table = torch.where(keep, rows, torch.where(fresh, taken, torch.full_like(rows, -1)))
    new_refs = refs.clone()
    for t, sign in ((table, -1), (new_table, 1)):
        t = t.flatten()
        new_refs.index_add_(0, t.clamp(min=0).long(), (t >= 0).int() * sign)
    # the part pages of the sequences that got one of their own
    at = (fresh & (j == whole[:, None]) & (j < have[:, None])).nonzero()
    blocks = (lens[at[:, 0]] % page + 31) // 32
    data = st["data"].view(n_pages, st["case"]["kv_heads"], page // 32, -1)
    src, dst = rows[at[:, 0], at[:, 1]].long(), new_table[at[:, 0], at[:, 1]].long()
    i, blk = (torch.arange(page // 32, device="cuda") < blocks[:, None]).nonzero().unbind(1)
    data[dst[i], :, blk] = data[src[i], :, blk]
    return [new_table, lens, new_refs, st["data"]]


def _plain_unpack(blocks, G):
    """Keys and values [*, 32, G * 64] in 32 bits of cache blocks [*, words]."""
    lead = blocks.shape[:-1]
    n = len(lead)
    keep = list(range(n))
    shift = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)

    def codes(w):
        return (w.unsqueeze(-1) >> shift) & 15

    kq = codes(blocks[..., :256 * G]).reshape(*lead, G, 4, 4, 4, 2, 2, 8)
    kq = kq.permute(*keep, n + 2, n + 4, n + 3, n, n + 5, n + 1, n + 6).reshape(*lead, 32, G, 64)
    vq = codes(blocks[..., 256 * G:512 * G]).reshape(*lead, G, 4, 64, 8)
    vq = vq.permute(*keep, n + 1, n + 3, n, n + 2).reshape(*lead, 32, G, 64)

    def so(w, order):
        t = w.contiguous().view(torch.float16).reshape(*lead, G, 2, 4, 8)[..., order]
        return t.permute(*keep, n + 1, n + 2, n + 3, n).reshape(*lead, 2, 32, G, 1).float().unbind(n)

    ks, ko = so(blocks[..., 512 * G:544 * G], list(range(8)))
    vs, vo = so(blocks[..., 544 * G:], [0, 2, 4, 6, 1, 3, 5, 7])
    return (ks * kq + ko).flatten(-2), (vs * vq + vo).flatten(-2)


def _plain_gather(st, table, first, count):
    """Keys and values [B][H][count * 32][D] of `count` blocks of every row of `table` from block `first` [B] on."""
    page = st["case"]["page"]
    j = first[:, None] + torch.arange(count, device="cuda")
    at = j.clamp(max=table.shape[1] * page // 32 - 1)
    pages = torch.gather(table, 1, at * 32 // page).long()
    blocks = st["data"].transpose(1, 2)[pages, at % (page // 32)].transpose(1, 2)
    k, v = _plain_unpack(blocks, st["case"]["dim"] // 64)
    return k.flatten(2, 3), v.flatten(2, 3), (j[:, :, None] * 32 + torch.arange(32, device="cuda")).flatten(1)


def _plain_shared(st):
    case = st["case"]
    G, per, N, H, D = case["groups"], case["per"], case["new"], case["kv_heads"], case["dim"]
    B, R = G * per, case["heads"] // H
    # the shared tokens once a group (whole blocks of them), the others of every sequence
    k0, v0, key0 = _plain_gather(st, st["table"][::per], torch.zeros_like(st["shared"]), -(-case["shared"] // 32))
    first = (st["shared"] // 32).repeat_interleave(per)
    k1, v1, key1 = _plain_gather(st, st["table"], first, (case["mine"] + 31) // 32 + 1)
    q = st["q"].float().view(B, N, H, R, D).permute(0, 2, 1, 3, 4) * (1.0 / math.sqrt(D))     # [B][H][N][R][D]
    qg = q.reshape(G, per, H, N * R, D).transpose(1, 2).reshape(G, H, per * N * R, D)
    s0 = torch.matmul(qg, k0.transpose(-1, -2).contiguous())
    s0 = s0.masked_fill(key0[:, None, None] >= (st["shared"] // 32 * 32)[:, None, None, None], -math.inf)
    s1 = torch.matmul(q.reshape(B, H, N * R, D), k1.transpose(-1, -2).contiguous())
    p = st["lens"][:, None] - N + torch.arange(N, device="cuda")                                # [B][N]
    s1 = s1.unflatten(2, (N, R)).masked_fill((key1[:, None, :] > p[:, :, None])[:, None, :, None], -math.inf).flatten(2, 3)
    m0 = s0.amax(-1, keepdim=True).view(G, H, per, N * R, 1).transpose(1, 2).reshape(B, H, N * R, 1)
    m = torch.maximum(m0, s1.amax(-1, keepdim=True))
    mg = m.view(G, per, H, N * R, 1).transpose(1, 2).reshape(G, H, per * N * R, 1)
    s0, s1 = torch.exp(s0 - mg), torch.exp(s1 - m)

    def rows(t):
        return t.view(G, H, per, N * R, -1).transpose(1, 2).reshape(B, H, N * R, -1)

    total = rows(s0.sum(-1, keepdim=True)) + s1.sum(-1, keepdim=True)
    o = (rows(torch.matmul(s0, v0)) + torch.matmul(s1, v1)) / total
    return o.view(B, H, N, R, D).permute(0, 2, 1, 3, 4).reshape(B * N, H * R, D).to(DTYPES[case["dtype"]])


def _plain_logprobs(st):
    case = st["case"]
    x = st["logits"].float()
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    given = x.gather(1, st["tokens"][:, None])
    index = torch.arange(case["vocab"], device="cuda")
    rank = ((x > given) | ((x == given) & (index < st["tokens"][:, None]))).sum(1, dtype=torch.int32)
    e = torch.where(e > 0, e * (x - top), e)
    entropy = log_total.squeeze(1) - e.sum(1) / total.squeeze(1)
    out = [(given - top - log_total).squeeze(1), rank, entropy, (top + log_total).squeeze(1)]
    if case["top"]:
        # numbers in the order of their values, then the lowest index: keys of 64 bits that never tie
        bits = (x + 0.0).view(torch.int32)
        key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * (1 << 32) + (0xFFFFFFFF - index)
        best = 0xFFFFFFFF - (torch.topk(key, min(case["top"], case["vocab"]), 1).values & 0xFFFFFFFF)
        out += [x.gather(1, best) - top - log_total, best.int()]
    return out


def run(state):
    case = state["case"]
    if not own:
        return {"rotary": _plain_rotary, "fork": _plain_fork, "shared": _plain_shared,
                "logprobs": _plain_logprobs}[case["op"]](state)
    import packed_decode_gemv_amd as vbq
    if case["op"] == "rotary":
        out = DTYPES[case["out"]]
        return list(vbq.head_norm_rotary(state["plan"], state["q"], state["k"], state["pos"], q_dtype=out, k_dtype=out))
    if case["op"] == "fork":
        table, lens, refs = vbq.kv4_fork(state["cache"], state["refs"], state["table"], state["lens"], state["parents"],
                                         reserve=state["reserve"], workspace=state["workspace"])
        return [table, lens, refs, state["data"]]
    if case["op"] == "shared":
        return vbq.kv4_attention_shared(state["cache"], state["q"], state["table"], state["lens"], state["cu"],
                                        state["cu_groups"], state["shared"], max_q=case["new"],
                                        max_shared=case["shared"], max_own=case["mine"],
                                        max_group_q=case["per"] * case["new"], workspace=state["workspace"])
    r = vbq.token_logprobs(state["logits"], state["tokens"], top=case["top"], workspace=state["workspace"])
    out = [r.logprob, r.rank, r.entropy, r.lse]
    return out + [r.top_logprob, r.top_index] if case["top"] else out


# ---- the definition in 64 bits -----------------------------------------------------
def _exact_values(data, case, pages, pos, head):
    """Keys and values [n, D] of the tokens at positions `pos` of `pages`, each nibble found by its address."""
    page, H, D = case["page"], case["kv_heads"], case["dim"]
    t, c = (pos % 32)[:, None], torch.arange(D, device="cuda")[None, :]
    g, r, G = c // 64, c % 64, D // 64
    base = (((pages * H + head) * (page // 32) + pos % page // 32) * (576 * G))[:, None]
    kw = base + 256 * g + 4 * (16 * (r % 32 // 8) + 4 * (t // 8) + t % 4) + 2 * (t % 8 // 4) + r // 32
    vw = base + 256 * (G + g) + 64 * (t // 8) + r
    words, halves = data.view(-1), data.view(torch.float16).view(-1)
    kc = ((words[kw] >> (4 * (r % 8))) & 15).double()
    vc = ((words[vw] >> (4 * (t % 8))) & 15).double()
    ks = 2 * (base + 512 * G + 32 * g) + t
    vs = 2 * (base + 544 * G + 32 * g) + 8 * (t // 8) + 2 * (t % 4) + t % 8 // 4
    return (halves[ks].double() * kc + halves[ks + 32].double(), halves[vs].double() * vc + halves[vs + 32].double())


def _exact_shared(case, st):
    shared, lens = _lengths(case)
    per, N, R, page = case["per"], case["new"], case["heads"] // case["kv_heads"], case["page"]
    out = torch.empty(len(lens) * N, case["heads"], case["dim"], dtype=torch.float64, device="cuda")
    for h in range(case["kv_heads"]):
        for g, cut in enumerate(shared):
            for b in range(g * per, g * per + per):
                n = lens[b]
                pos = torch.arange(cut, n, device="cuda")
                if b == g * per:
                    common = torch.arange(cut, device="cuda")
                    k0, v0 = _exact_values(st["data"], case, st["table"][b].long()[common // page], common, h)
                k1, v1 = _exact_values(st["data"], case, st["table"][b].long()[pos // page], pos, h)
                q = st["q"][b * N:b * N + N, h * R:h * R + R].double().reshape(N * R, -1)
                s = torch.cat([q @ k0.T, q @ k1.T], 1).view(N, R, n) / math.sqrt(case["dim"])
                late = torch.arange(n, device="cuda") > torch.arange(n - N, n, device="cuda")[:, None]
                p = torch.softmax(s.masked_fill(late[:, None], -math.inf), -1).view(N * R, n)
                o = p[:, :cut] @ v0 + p[:, cut:] @ v1
                out[b * N:b * N + N, h * R:h * R + R] = o.view(N, R, -1)
    return out


def exact(case, seed):
    if case["op"] == "fork":
        return None                                         # whole numbers only
    st = prepare(case, seed)
    if case["op"] == "shared":
        return _exact_shared(case, st)
    if case["op"] == "rotary":
        out, R = [], case["rotary"]
        c = torch.arange(case["dim"], device="cuda")
        pair = (c // 2 if case["interleaved"] else c % (R // 2)).clamp(max=R // 2 - 1)
        second = (c % 2 if case["interleaved"] else c // (R // 2)) == 1
        other = torch.where(second, c - 1, c + 1) if case["interleaved"] else torch.where(second, c - R // 2, c + R // 2)
        turned = c < R
        other = torch.where(turned, other, c)
        angle = st["pos"].view(case["axes"], -1).double()[st["axis"].long()[pair]] * st["inv_freq"].double()[pair][:, None]
        angle = torch.where(turned[:, None], angle, torch.zeros_like(angle)).T[:, None]
        for x, w in ((st["q"], st["qw"]), (st["k"], st["kw"])):
            x = x.double()
            if w is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / case["dim"] + EPS) * w.double()
            sign = torch.where(turned, torch.where(second, 1.0, -1.0), 0.0).double()
            out.append(x * torch.cos(angle) + x[..., other] * sign * torch.sin(angle))
        return out
    parts = []
    step = max(1, (1 << 27) // case["vocab"])
    for at in range(0, case["rows"], step):
        x, t = st["logits"][at:at + step].double(), st["tokens"][at:at + step]
        lse = torch.logsumexp(x, 1)
        logp = x - lse[:, None]
        entropy = -torch.where(logp > -math.inf, logp.exp() * logp, torch.zeros_like(logp)).sum(1)
        part = [logp.gather(1, t[:, None]).squeeze(1), entropy, lse]
        if case["top"]:
            part.append(torch.sort(logp, 1, descending=True).values[:, :case["top"]])
        parts.append(part)
    cols = [torch.cat(c) for c in zip(*parts)]
    out = [cols[0], None, cols[1], cols[2]]
    return out + [cols[3], None] if case["top"] else out

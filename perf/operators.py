"""The operators of the 4-bit key/value cache, as they are measured.

Three operators over one cache format (the layout is stated in include/vbq.h,
"4-bit key/value cache"):

- append: keys and values of new tokens are quantised as they are written to
  the cache, and the values now held there are read back;
- read: a range of every sequence's cached tokens, dequantised;
- attend: softmax attention of new query tokens over the cached tokens,
  causal, with an optional sliding window and first tokens that stay visible.

``own`` selects the framework's kernels; otherwise ``run`` computes the same
results with elementary torch operations in 32 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}
CLAMP = 61440.0


# ---- cases -----------------------------------------------------------------------
def _case(op, dtype, batch, heads, kv_heads, dim, page, kv, new, ragged=0, window=0, sinks=0):
    """kv: tokens of the longest sequence, the `new` last ones included; ragged: 0 for
    sequences of equal length, otherwise the seed of their lengths."""
    return dict(op=op, dtype=dtype, batch=batch, heads=heads, kv_heads=kv_heads, dim=dim, page=page, kv=kv,
                new=new, ragged=ragged, window=window, sinks=sinks)


def listed():
    cases = []

    def add(name, *a, **k):
        cases.append(dict(name=name, **_case(*a, **k)))

    # one decode step of one conversation, 131M-class model (hidden 768: 12 heads of 64)
    add("append_one", "append", "f16", 1, 12, 12, 64, 64, 577, 1)
    # a decode step of 64 conversations, 9B-class model; k and v come from the packed GEMV in float32
    add("append_step", "append", "f32", 64, 32, 8, 128, 64, 4000, 1, ragged=1)
    # five prompts of odd lengths enter the cache, 9B-class model
    add("append_prompts", "append", "bf16", 5, 32, 8, 128, 128, 8191, 8191, ragged=2)
    # a short shared prefix is read back, 131M-class model
    add("read_prefix", "read", "f16", 3, 12, 12, 64, 32, 333, 333, ragged=3)
    # whole conversations are read back (for another kernel, or to move them), 9B-class model
    add("read_long", "read", "bf16", 8, 32, 8, 128, 256, 16384, 16384, ragged=4)
    # attention of one decode step of one conversation, 131M-class model
    add("attend_one", "attend", "f16", 1, 12, 12, 64, 64, 577, 1)
    # attention of a decode step of 32 conversations, 9B-class model
    add("attend_step", "attend", "f16", 32, 32, 8, 128, 64, 8192, 1, ragged=5)
    # one conversation of 128K tokens: the token axis has to be split
    add("attend_long", "attend", "bf16", 1, 32, 8, 128, 256, 131072, 1)
    # long conversations of the 1.0B-class model (16 heads of 128) under a window with first tokens kept
    add("attend_window", "attend", "f16", 16, 16, 16, 128, 64, 32768, 1, ragged=6, window=1024, sinks=4)
    # a few drafted tokens per conversation are checked at once
    add("attend_draft", "attend", "bf16", 8, 32, 8, 128, 32, 4097, 5, ragged=7)
    # a chunk of a long prompt attends to itself and to what the cache already holds
    add("attend_chunk", "attend", "bf16", 1, 32, 8, 128, 128, 10240, 2048)
    # three prompts of odd lengths under a window, heads of 256
    add("attend_prompts_window", "attend", "f16", 3, 16, 4, 256, 64, 2600, 2500, ragged=8, window=500, sinks=4)
    return cases


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "attend"])
    dtype = rng.choice(["f16", "bf16", "f32"] if op != "attend" else ["f16", "bf16"])
    kv_heads, group, dim = rng.choice([(12, 1, 64), (8, 4, 128), (16, 1, 128), (4, 4, 256), (8, 4, 64), (2, 7, 128),
                                       (4, 8, 128), (8, 2, 192), (1, 16, 64)])
    page = rng.choice([32, 64, 128, 256])
    ragged = rng.choice([0, rng.randrange(1, 1 << 20)])
    window = sinks = 0
    if op != "attend":
        new = 1 if rng.random() < 0.3 else _log(rng, 2, 8191)
        most = (60000 if op == "read" else 20000) * 1024
        new = min(new, most // (kv_heads * dim))
        batch = max(1, min(_log(rng, 1, 64), most // (new * kv_heads * dim)))
        kv = new + (0 if op == "read" else _log(rng, 1, 4000))
    else:
        kind = rng.choice(["step", "step", "draft", "chunk"])
        kv = _log(rng, 17, 131072 if kind != "chunk" else 8192)
        new = 1 if kind == "step" else min(kv, rng.randrange(2, 9) if kind == "draft" else _log(rng, 16, 2048))
        most = 130000 * 1024 // (kv_heads * dim)
        kv = min(kv, most)
        new = min(new, kv)
        batch = max(1, min(_log(rng, 1, 64), most // kv))
        if kind == "chunk":
            pairs = 8 * 10 ** 10 // (kv_heads * group * dim)
            new = max(1, min(new, pairs // kv))
            batch = max(1, min(batch, pairs // (kv * new)))
        if rng.random() < 0.35:
            window, sinks = _log(rng, 8, 4096), rng.choice([0, 1, 4, 16])
    return _case(op, dtype, batch, kv_heads * group, kv_heads, dim, page, kv, new, ragged, window, sinks)


def _lengths(case):
    """(tokens, new tokens) of every sequence; the longest comes first."""
    kv, new = [case["kv"]], [case["new"]]
    rng = random.Random(case["ragged"])
    for _ in range(case["batch"] - 1):
        if case["ragged"]:
            n = case["new"] if case["new"] < 16 else rng.randint(1, case["new"])
            past = case["kv"] - case["new"]
            kv.append(n + rng.randint(past // 4, past))
            new.append(n)
        else:
            kv.append(case["kv"])
            new.append(case["new"])
    return kv, new


def _pairs(p_first, n, window, sinks):
    """Visible (query, key) pairs of n queries at positions p_first..., and the keys that any of them sees."""
    if not window:
        return sum(range(p_first + 1, p_first + n + 1)), p_first + n
    pairs = 0
    for p in range(p_first, p_first + n):
        lo = max(0, p - window + 1)
        pairs += p + 1 - lo + min(sinks, lo)
    lo = max(0, p_first - window + 1)
    return pairs, p_first + n - lo + min(sinks, lo)


def work(case):
    kv, new = _lengths(case)
    H, D = case["kv_heads"], case["dim"]
    held = H * D * 9 // 8          # bytes of a token's keys and values in the cache: 72 per 64 + 64 values
    table = 4 * sum(-(-n // case["page"]) for n in kv)
    if case["op"] != "attend":
        values = sum(new) * H * D * 2
        return dict(bytes=values * BYTES[case["dtype"]] + sum(new) * held + table, flops=values * 4)
    pairs = keys = 0
    for n, m in zip(kv, new):
        p, k = _pairs(n - m, m, case["window"], case["sinks"])
        pairs, keys = pairs + p, keys + k
    io = 2 * sum(new) * case["heads"] * D * BYTES[case["dtype"]]
    return dict(bytes=keys * held + io + table, flops=4 * D * case["heads"] * pairs)


# ---- inputs ----------------------------------------------------------------------
def _quantise(x):
    """Codes (int32), scale and offset (float16) of groups of 64 values on the last axis, in 32 bits."""
    x = torch.nan_to_num(x.float(), nan=0.0, posinf=CLAMP, neginf=-CLAMP).clamp(-CLAMP, CLAMP)
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s, o = ((hi - lo) / 15.0).half(), lo.half()
    sf = s.float()
    q = torch.where(sf == 0, torch.zeros_like(x), ((x - o.float()) / sf).round().clamp(0, 15))
    return q.int(), s.squeeze(-1), o.squeeze(-1)


def _nibbles(q):
    """int32 words of eight 4-bit codes on the last axis, the first lowest."""
    w = q[..., 0].clone()
    for n in range(1, 8):
        w |= q[..., n] << (4 * n)
    return w


def _blocks(kq, ks, ko, vq, vs, vo):
    """Cache blocks (int32 words) of 32 tokens: codes [*, 32, G, 64], scales and offsets [*, 32, G]."""
    lead, G = kq.shape[:-3], kq.shape[-2]
    n = len(lead)
    perm = list(range(n))
    # tokens 32 = (4 octets, 2 halves, 4), channels 64 = (2 steps, 4 quarters, 8)
    kw = kq.reshape(*lead, 4, 2, 4, G, 2, 4, 8).permute(*perm, n + 3, n + 5, n, n + 2, n + 1, n + 4, n + 6)
    vw = vq.reshape(*lead, 4, 8, G, 64).permute(*perm, n + 2, n, n + 3, n + 1)
    order = [0, 4, 1, 5, 2, 6, 3, 7]

    def so(s, o, swap):
        t = torch.stack([s, o], -1).reshape(*lead, 4, 8, G, 2)
        t = t[..., order, :, :] if swap else t
        return t.permute(*perm, n + 2, n + 3, n, n + 1).reshape(*lead, -1).contiguous().view(torch.int32)

    return torch.cat([_nibbles(kw).reshape(*lead, -1), _nibbles(vw).reshape(*lead, -1),
                      so(ks, ko, False), so(vs, vo, True)], -1)


def _block_words(case):
    return case["dim"] // 64 * 576


def _filled_cache(case, n_pages, gen):
    """A cache whose pages all hold quantised tokens: keys with a few strong channels, values without."""
    H, D, per = case["kv_heads"], case["dim"], case["page"] // 32
    data = torch.empty(n_pages, H, per, _block_words(case), dtype=torch.int32, device="cuda")
    gain = torch.ones(H, 1, 1, D, device="cuda")
    gain[..., ::17] = 4.0
    shift = torch.randn(H, 1, 1, D, generator=gen, device="cuda")
    step = max(1, (1 << 24) // (H * per * 32 * D))
    for p in range(0, n_pages, step):
        m = min(step, n_pages - p)
        k = torch.randn(m, H, per, 32, D, generator=gen, device="cuda") * gain + shift
        v = torch.randn(m, H, per, 32, D, generator=gen, device="cuda")
        data[p:p + m] = _blocks(*_quantise(k.unflatten(-1, (-1, 64))), *_quantise(v.unflatten(-1, (-1, 64))))
    return data


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kv, new = _lengths(case)
    B, page, H, D = case["batch"], case["page"], case["kv_heads"], case["dim"]
    width = -(-max(kv) // page)
    n_pages = sum(-(-n // page) for n in kv) + 3
    perm = torch.randperm(n_pages, generator=gen, device="cuda").int()
    table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(kv):
        m = -(-n // page)
        table[b, :m] = perm[at:at + m]
        at += m
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    state = dict(case=case, table=table, total=cu[-1],
                 data=_filled_cache(case, n_pages, gen),
                 cu=torch.tensor(cu, dtype=torch.int32).cuda(),
                 start=torch.tensor([n - m for n, m in zip(kv, new)], dtype=torch.int32).cuda(),
                 lens=torch.tensor(kv, dtype=torch.int32).cuda())
    dt = DTYPES[case["dtype"]]
    if case["op"] == "append":
        # the projections' common output: keys and values are slices of one tensor
        both = torch.randn(cu[-1], 2 * H * D, generator=gen, device="cuda")
        both[:, ::29] *= 5.0
        both = both.to(dt)
        state["k"] = both[:, :H * D].unflatten(-1, (H, D))
        state["v"] = both[:, H * D:].unflatten(-1, (H, D))
    elif case["op"] == "attend":
        state["q"] = (torch.randn(cu[-1], case["heads"], D, generator=gen, device="cuda") * 1.5).to(dt)
    if own:
        import packed_decode_gemv_amd as vbq
        state["cache"] = vbq.Kv4Cache(n_pages, page, H, D, data=state["data"].view(torch.uint8).view(-1))
        if case["op"] == "attend":
            state["workspace"] = vbq.kv4_attention_workspace(state["cache"], B, cu[-1], case["heads"], case["new"],
                                                             case["kv"], window=case["window"],
                                                             sinks=case["sinks"])
    return state


# ---- plain forms -----------------------------------------------------------------
def _plain_positions(st):
    """Sequence and position of every new token."""
    t = torch.arange(st["total"], device="cuda")
    b = torch.searchsorted(st["cu"][1:].long(), t, right=True)
    return b, st["start"][b] + t - st["cu"][b]


def _plain_unpack(blocks, G):
    """Keys and values [*, 32, G * 64] in 32 bits of cache blocks [*, words]."""
    lead = blocks.shape[:-1]
    n = len(lead)
    perm = list(range(n))
    shift = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)

    def codes(w):
        return (w.unsqueeze(-1) >> shift) & 15

    kw = codes(blocks[..., :256 * G]).reshape(*lead, G, 4, 4, 4, 2, 2, 8)
    kq = kw.permute(*perm, n + 2, n + 4, n + 3, n, n + 5, n + 1, n + 6).reshape(*lead, 32, G, 64)
    vw = codes(blocks[..., 256 * G:512 * G]).reshape(*lead, G, 4, 64, 8)
    vq = vw.permute(*perm, n + 1, n + 3, n, n + 2).reshape(*lead, 32, G, 64)

    def so(w, swap):
        t = w.contiguous().view(torch.float16).reshape(*lead, G, 2, 4, 8)
        t = t[..., [0, 2, 4, 6, 1, 3, 5, 7]] if swap else t
        return t.permute(*perm, n + 1, n + 2, n + 3, n).reshape(*lead, 2, 32, G, 1).float().unbind(n)

    ks, ko = so(blocks[..., 512 * G:544 * G], False)
    vs, vo = so(blocks[..., 544 * G:], True)
    return (ks * kq + ko).flatten(-2), (vs * vq + vo).flatten(-2)


def _plain_read(st):
    case = st["case"]
    G, page = case["dim"] // 64, case["page"]
    b, pos = _plain_positions(st)
    # each touched block once: blocks of a sequence are numbered from its first touched one
    first = st["start"] // 32
    counts = (st["start"] + st["cu"][1:] - st["cu"][:-1] - 1) // 32 - first + 1
    base = torch.cumsum(counts, 0) - counts
    nblk = st["total"] // 32 + 2 * case["batch"]
    at = torch.arange(nblk, device="cuda")
    seq = torch.searchsorted(torch.cumsum(counts, 0), at, right=True).clamp(max=case["batch"] - 1)
    j = torch.minimum(first[seq] + at - base[seq], (st["lens"][seq] - 1) // 32)
    pages = st["table"][seq, j * 32 // page].long()
    blocks = st["data"].transpose(1, 2)[pages, j % (page // 32)]                # [nblk, H, words]
    slot = base[b] + pos // 32 - first[b]
    dt = DTYPES[case["dtype"]]
    out = []
    for x in _plain_unpack(blocks, G):
        out.append(x.transpose(1, 2)[slot, pos % 32].to(dt))                    # [total, H, D]
    return out


def _plain_append(st):
    case = st["case"]
    G, page, H = case["dim"] // 64, case["page"], case["kv_heads"]
    b, pos = _plain_positions(st)
    words = _block_words(case)
    pages = st["table"][b, pos // page].long()
    heads = torch.arange(H, device="cuda")
    base = ((pages[:, None] * H + heads) * (page // 32) + (pos % page // 32)[:, None]) * words     # [T, H]
    flat, half = st["data"].view(-1), st["data"].view(torch.float16).view(-1)
    tok = pos % 32
    grp = torch.arange(G, device="cuda")
    kq, ks, ko = _quantise(st["k"].unflatten(-1, (G, 64)))
    vq, vs, vo = _quantise(st["v"].unflatten(-1, (G, 64)))
    # keys: eight channels of one token are one word
    quarter, step = torch.arange(4, device="cuda"), torch.arange(2, device="cuda")
    m = tok // 8 * 4 + tok % 4
    idx = (16 * quarter[None, None, :] + m[:, None, None]) * 4 + 2 * (tok // 4 % 2)[:, None, None] + step[None, :, None]
    idx = base[:, :, None, None, None] + 256 * grp[None, None, :, None, None] + idx[:, None, None]
    flat[idx] = _nibbles(kq.reshape(*kq.shape[:-1], 2, 4, 8))
    # values: eight tokens of one channel are one word; the tokens of one place in the eight at a time
    idx = base[:, :, None, None] + 256 * (G + grp)[:, None] + (64 * (tok // 8))[:, None, None, None] \
        + torch.arange(64, device="cuda")
    for n in range(8):
        here = (tok % 8 == n).nonzero().squeeze(-1)
        i = idx[here]
        flat[i] = (flat[i] & ~(15 << (4 * n) if n < 7 else -(1 << 28))) | (vq[here] << (4 * n))
    swap = tok // 8 * 8 + 2 * (tok % 4) + tok % 8 // 4
    for first, s, o, place in ((512, ks, ko, tok), (544, vs, vo, swap)):
        i = 2 * (base[:, :, None] + first * G + 32 * grp) + place[:, None, None]
        half[i] = s
        half[i + 32] = o
    return _plain_read(st)


def _plain_attend(st):
    case = st["case"]
    B, H, D, page, L, N = case["batch"], case["kv_heads"], case["dim"], case["page"], case["kv"], case["new"]
    R = case["heads"] // H
    # blocks to look at: all, or the first tokens' and those from the window of the first query on
    keep = -(-case["sinks"] // 32) if case["window"] else 0
    look = -(-L // 32)
    j = torch.arange(look, device="cuda").expand(B, -1)
    if case["window"] and look > keep + -(-(case["window"] + N) // 32) + 1:
        look = -(-(case["window"] + N) // 32) + 1
        near = ((st["start"] - case["window"] + 1).clamp(min=0) // 32).clamp(min=keep)
        j = torch.cat([torch.arange(keep, device="cuda").expand(B, -1),
                       near[:, None] + torch.arange(look, device="cuda")], 1)
    at = torch.minimum(j, (st["lens"][:, None] - 1) // 32)
    pages = torch.gather(st["table"], 1, at * 32 // page).long()
    blocks = st["data"].transpose(1, 2)[pages, at % (page // 32)].transpose(1, 2)      # [B, H, nblk, words]
    k, v = _plain_unpack(blocks, D // 64)
    k, v = k.flatten(2, 3), v.flatten(2, 3)                                             # [B, H, nblk * 32, D]
    i = torch.arange(N, device="cuda")
    count = st["cu"][1:] - st["cu"][:-1]
    rows = (st["cu"][:-1, None] + i).clamp(max=st["total"] - 1)
    q = st["q"].float()[rows].reshape(B, N, H, R, D).permute(0, 2, 1, 3, 4).reshape(B, H, N * R, D)
    s = torch.matmul(q, k.transpose(-1, -2).contiguous()) * (1.0 / math.sqrt(D))
    key = (j[:, :, None] * 32 + torch.arange(32, device="cuda")).flatten(1)[:, None, :]
    p = (st["start"][:, None] + i)[:, :, None]
    see = (key <= p) & (key < st["lens"][:, None, None])
    if case["window"]:
        see &= (key > p - case["window"]) | (key < case["sinks"])
    s = s.unflatten(2, (N, R)).masked_fill(~see[:, None, :, None], float("-inf"))
    s = torch.exp(s - s.amax(-1, keepdim=True))
    s = (s / s.sum(-1, keepdim=True)).flatten(2, 3)
    o = torch.matmul(s, v).reshape(B, H, N, R, D).permute(0, 2, 1, 3, 4).reshape(B, N, H * R, D)
    keep = (i < count[:, None]).flatten().nonzero().squeeze(-1)
    return o.flatten(0, 1)[keep].to(DTYPES[case["dtype"]])


def run(state):
    case = state["case"]
    if not own:
        return {"append": _plain_append, "read": _plain_read, "attend": _plain_attend}[case["op"]](state)
    import packed_decode_gemv_amd as vbq
    cache, table = state["cache"], state["table"]
    if case["op"] == "attend":
        return vbq.kv4_attention(cache, state["q"], table, state["lens"], state["cu"], max_q=case["new"],
                                 max_kv=case["kv"], window=case["window"], sinks=case["sinks"],
                                 workspace=state["workspace"])
    if case["op"] == "append":
        vbq.kv4_append(cache, state["k"], state["v"], table, state["start"], state["cu"], max_tokens=case["new"])
    return list(vbq.kv4_read(cache, table, state["start"], state["cu"], state["total"], DTYPES[case["dtype"]],
                             max_tokens=case["new"]))


# ---- the definition in 64 bits -----------------------------------------------------
def _exact_values(data, case, pages, pos, head):
    """Keys and values [n, D] of the tokens at positions `pos` of `pages`, each nibble found by its address."""
    page, H, D = case["page"], case["kv_heads"], case["dim"]
    t, c = (pos % 32)[:, None], torch.arange(D, device="cuda")[None, :]
    g, r = c // 64, c % 64
    base = (((pages * H + head) * (page // 32) + pos % page // 32) * _block_words(case))[:, None]
    G = D // 64
    kw = base + 256 * g + 4 * (16 * (r % 32 // 8) + 4 * (t // 8) + t % 4) + 2 * (t % 8 // 4) + r // 32
    vw = base + 256 * (G + g) + 64 * (t // 8) + r
    words, halves = data.view(-1), data.view(torch.float16).view(-1)
    kc = ((words[kw] >> (4 * (r % 8))) & 15).double()
    vc = ((words[vw] >> (4 * (t % 8))) & 15).double()
    ks = 2 * (base + 512 * G + 32 * g) + t
    vs = 2 * (base + 544 * G + 32 * g) + 8 * (t // 8) + 2 * (t % 4) + t % 8 // 4
    return (halves[ks].double() * kc + halves[ks + 32].double(), halves[vs].double() * vc + halves[vs + 32].double())


def _exact_quantised(x):
    x = x.double()
    x = torch.where(x.isnan(), torch.zeros_like(x), x).clamp(-CLAMP, CLAMP).unflatten(-1, (-1, 64))
    lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    # the scale is the float16 nearest to the float32 quotient of the float32 difference: part of the format
    s = ((hi - lo).float().double() / 15).float().half().double()
    o = lo.float().half().double()
    q = torch.where(s == 0, torch.zeros_like(x), torch.round((x - o) / torch.where(s == 0, torch.ones_like(s), s)))
    return (q.clamp(0, 15) * s + o).flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    kv, new = _lengths(case)
    H, D, page = case["kv_heads"], case["dim"], case["page"]
    R = case["heads"] // H
    if case["op"] == "append":
        return [_exact_quantised(st["k"]), _exact_quantised(st["v"])]
    T = st["total"]
    at = 0
    if case["op"] == "read":
        k = torch.empty(T, H, D, dtype=torch.float64, device="cuda")
        v = torch.empty_like(k)
        for b, (n, m) in enumerate(zip(kv, new)):
            pos = torch.arange(n - m, n, device="cuda")
            pages = st["table"][b].long()[pos // page]
            for h in range(H):
                k[at:at + m, h], v[at:at + m, h] = _exact_values(st["data"], case, pages, pos, h)
            at += m
        return [k, v]
    out = torch.zeros(T, case["heads"], D, dtype=torch.float64, device="cuda")
    for b, (n, m) in enumerate(zip(kv, new)):
        pos = torch.arange(n, device="cuda")
        pages = st["table"][b].long()[pos // page]
        p = torch.arange(n - m, n, device="cuda")
        hidden = pos[None, :] > p[:, None]
        if case["window"]:
            hidden |= (pos[None, :] <= p[:, None] - case["window"]) & (pos[None, :] >= case["sinks"])
        for h in range(H):
            k, v = _exact_values(st["data"], case, pages, pos, h)
            for r in range(h * R, h * R + R):
                s = (st["q"][at:at + m, r].double() @ k.T) / math.sqrt(D)
                s[hidden] = -math.inf
                out[at:at + m, r] = torch.softmax(s, -1) @ v
        at += m
    return out

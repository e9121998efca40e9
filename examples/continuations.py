"""Beam search through one attention layer and a language model head, both packed, over
the 4-bit key/value cache.

    python examples/continuations.py [--beams 8] [--prompt 700] [--steps 24] [--vocab 32001]

A prompt enters once (vbq_gemm, head_norm_rotary, kv4_append, kv4_attention). kv4_fork
makes it the beginning of every beam; then each step decodes all beams together: the
projections (vbq_gemv_batched), norms and rotation of queries and keys
(head_norm_rotary), the append, attention that reads the prompt once for all beams
(kv4_attention_shared), the head (vbq_gemv) and its log probabilities with the most
likely tokens (token_logprobs). The best continuations of all beams are chosen, and
kv4_fork reorders the cache: beams that go on share whole pages, part pages are copied,
pages of beams that ended are free. At the end every beam is decoded again by itself,
token by token, and its score compared.

There is no model around the layer: weights are random, and the layer's output goes to
the head as it is.
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import packed_decode_gemv_amd as vbq  # noqa: E402


class Model:
    def __init__(self, hidden=1024, heads=16, kv_heads=4, dim=64, vocab=32001, seed=0):
        self.hidden, self.heads, self.kv_heads, self.dim, self.vocab = hidden, heads, kv_heads, dim, vocab
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)

        def packed(n, k, gain=1.0):
            widths = rng.choice(np.array([2, 4, 8], np.uint8), size=(n, k // 64), p=[0.2, 0.4, 0.4])
            return vbq.vbq_pack(torch.randn(n, k, generator=gen, device="cuda") * gain * k ** -0.5, widths)

        self.embed = torch.randn(vocab, hidden, generator=gen, device="cuda")
        self.q, self.k, self.v = packed(heads * dim, hidden), packed(kv_heads * dim, hidden), packed(kv_heads * dim, hidden)
        self.o, self.head = packed(hidden, heads * dim), packed(vocab, hidden, 4.0)
        inv_freq = 10000.0 ** (-torch.arange(dim // 2, device="cuda") / (dim // 2))
        weight = 1.0 + 0.1 * torch.randn(2, dim, generator=gen, device="cuda")
        self.rotary = vbq.HeadRotary(dim, inv_freq, q_weight=weight[0], k_weight=weight[1])

    def project(self, x):
        """q, k and v in float32 of rows x (few rows by the GEMV, many by the GEMM)."""
        if len(x) <= vbq.MAX_BATCH:
            q, k, v = vbq.vbq_gemv_batched([self.q, self.k, self.v], [x.half()] * 3)
        else:
            q, k, v = (vbq.vbq_gemm(w, x.bfloat16()) for w in (self.q, self.k, self.v))
        return q.view(-1, self.heads, self.dim), k.view(-1, self.kv_heads, self.dim), v.view(-1, self.kv_heads, self.dim)

    def answer(self, attended):
        """Logits, float32, of the attended heads of few rows."""
        x = vbq.vbq_gemv(self.o, attended.reshape(len(attended), -1).half())
        return vbq.vbq_gemv(self.head, x.half())


class Beams:
    """Sequences over one cache: block table, lengths, how often each page is named."""

    def __init__(self, model, max_beams, max_tokens, page_tokens=64):
        self.model = model
        width = -(-max_tokens // page_tokens)
        pages = 2 * max_beams * width + 1
        self.max_tokens = width * page_tokens
        self.cache = vbq.Kv4Cache(pages, page_tokens, model.kv_heads, model.dim)
        self.table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")

    def fork(self, parents, tokens):
        """The sequences become continuations of `parents`, with pages for that many more tokens each."""
        parents = torch.as_tensor(parents, dtype=torch.int32, device="cuda")
        self.table, self.lens, self.refs = vbq.kv4_fork(self.cache, self.refs, self.table, self.lens, parents,
                                                        reserve=torch.full_like(parents, tokens))

    def enter(self, x, shared=None):
        """x [beams][n][hidden]: every sequence takes n tokens; the attended heads of all of them. shared: how many
        first tokens all sequences have in common."""
        m, (B, n, _) = self.model, x.shape
        q, k, v = m.project(x.reshape(B * n, -1))
        positions = (self.lens[:, None] + torch.arange(n, device="cuda")).int().view(-1)
        q, k = vbq.head_norm_rotary(m.rotary, q, k, positions, q_dtype=torch.float16)
        cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
        vbq.kv4_append(self.cache, k, v, self.table, self.lens, cu, max_tokens=n)
        self.lens = self.lens + n
        if shared is None:
            return vbq.kv4_attention(self.cache, q, self.table, self.lens, cu, n, self.max_tokens)
        groups = torch.tensor([0, B], dtype=torch.int32, device="cuda")
        common = torch.tensor([shared], dtype=torch.int32, device="cuda")
        return vbq.kv4_attention_shared(self.cache, q, self.table, self.lens, cu, groups, common, max_q=n,
                                        max_shared=shared, max_own=self.max_tokens - shared)


def search(model, prompt, beams, steps):
    """Token sequences [beams][steps] and their scores (sums of log probabilities), best first."""
    n = len(prompt)
    s = Beams(model, beams, n + steps + 1)
    s.fork([-1], n)                                        # one empty sequence with pages for the prompt
    attended = s.enter(model.embed[prompt][None])
    r = vbq.token_logprobs(model.answer(attended[-1:]), top=beams)
    scores, tokens = r.top_logprob[0], r.top_index[0].long()
    chosen, parents = tokens[:, None], torch.zeros(beams, dtype=torch.int32, device="cuda")
    for _ in range(steps - 1):
        s.fork(parents, 1)
        attended = s.enter(model.embed[tokens][:, None], shared=n)
        r = vbq.token_logprobs(model.answer(attended), top=beams)
        total = (scores[:, None] + r.top_logprob).view(-1)
        scores, best = torch.topk(total, beams)
        parents = best // beams
        tokens = r.top_index.view(-1)[best].long()
        chosen = torch.cat([chosen[parents], tokens[:, None]], 1)
        parents = parents.int()
    s.cache.check()
    return chosen, scores, s


def score(model, prompt, tokens):
    """The sum of log probabilities of one sequence, decoded by itself."""
    s = Beams(model, 1, len(prompt) + len(tokens) + 1)
    s.fork([-1], len(prompt) + len(tokens))
    attended, total = s.enter(model.embed[prompt][None])[-1:], 0.0
    for t in tokens:
        total += float(vbq.token_logprobs(model.answer(attended), t.view(1)).logprob)
        attended = s.enter(model.embed[t].view(1, 1, -1))
    s.cache.check()
    return total


def run(beams=8, prompt=700, steps=24, vocab=32001, model=None):
    if not 1 <= beams <= vbq.MAX_BATCH:
        raise ValueError(f"beams {beams} outside 1..{vbq.MAX_BATCH}")
    model = model or Model(vocab=vocab)
    gen = torch.Generator(device="cuda").manual_seed(1)
    first = torch.randint(0, model.vocab, (prompt,), generator=gen, device="cuda")
    tokens, scores, s = search(model, first, beams, steps)
    alone = [score(model, first, t) for t in tokens]
    pages = int((s.refs > 0).sum())
    return dict(scores=scores.tolist(), alone=alone, pages=pages, apart=beams * -(-int(s.lens.max()) // s.cache.page_tokens))


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--beams", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=700)
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--vocab", type=int, default=32001)
    a = ap.parse_args()
    r = run(a.beams, a.prompt, a.steps, a.vocab)
    off = max(abs(x - y) for x, y in zip(r["scores"], r["alone"]))
    print(f"{a.beams} beams of {a.steps} tokens after {a.prompt}: best score {r['scores'][0]:.3f}; decoded one by one the "
          f"scores differ by {off:.1e} at most; {r['pages']} pages in use, {r['apart']} without sharing")

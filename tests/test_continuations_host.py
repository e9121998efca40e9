"""Host-side checks of the operators for several continuations of one prompt: sizes, and
arguments that are refused before a GPU is touched."""
import ctypes as C

import pytest

BASE = 0x7F0000000000


def _cache(vbq, **kw):
    d = dict(n_pages=100, page_tokens=64, n_kv_heads=2, head_dim=128, reserved=0, data=BASE, flags=BASE + 256)
    d.update(kw)
    return vbq.vbq_kv4(**d)


def test_rotary_refuses_bad_arguments():
    import packed_decode_gemv_amd as vbq

    def run(plan=(), q=(), k=(), positions=BASE, tokens=3, none=()):
        p = vbq.vbq_head_rotary(**{**dict(head_dim=128, rotary_dim=64, axes=1, interleaved=0, eps=1e-6, reserved=0,
                                          inv_freq=BASE, axis=None, q_weight=BASE, k_weight=None), **dict(plan)})
        rows = dict(in_=BASE, out=BASE, in_token_stride=512, in_head_stride=128, out_token_stride=512, out_head_stride=128,
                    heads=4, in_dtype=0, out_dtype=0, reserved=0)
        return vbq.lib.head_norm_rotary(None if "plan" in none else C.byref(p),
                                        None if "q" in none else C.byref(vbq.vbq_head_rows(**{**rows, **dict(q)})),
                                        None if "k" in none else C.byref(vbq.vbq_head_rows(**{**rows, **dict(k)})),
                                        positions, 3, tokens, None)

    assert run(tokens=0) == 0 and run(tokens=-1) == 2
    assert run(q=dict(heads=0), k=dict(heads=0)) == 0
    for name in ("plan", "q", "k"):
        assert run(none=(name,)) == 1
    for bad, st in ((dict(head_dim=96), 2), (dict(head_dim=320), 2), (dict(head_dim=0), 2), (dict(rotary_dim=8), 2),
                    (dict(rotary_dim=144), 2), (dict(rotary_dim=-16), 2), (dict(axes=0), 1), (dict(axes=256), 1),
                    (dict(interleaved=2), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
                    (dict(eps=float("inf")), 1), (dict(reserved=1), 1), (dict(inv_freq=None), 1),
                    (dict(inv_freq=BASE + 2), 4), (dict(q_weight=BASE + 4), 4)):
        assert run(plan=bad) == st, bad
    for bad, st in ((dict(heads=-1), 2), (dict(heads=65537), 5), (dict(in_=None), 1), (dict(out=None), 1),
                    (dict(in_=BASE + 8), 4), (dict(in_token_stride=4), 4), (dict(out_head_stride=4), 4),
                    (dict(in_dtype=3), 1), (dict(out_dtype=-1), 1), (dict(in_dtype=2, in_head_stride=2), 4),
                    (dict(reserved=1), 1)):
        assert run(q=bad) == st, bad
        assert run(k=bad) == st, bad
    assert run(q=dict(in_dtype=1)) == 1                  # queries and keys of two types
    for bad in (dict(out_dtype=1), dict(out_token_stride=1024), dict(out_head_stride=256)):
        assert run(q=bad) == 1 and run(k=bad) == 1, bad  # in place, but not number for number
    assert run(positions=None) == 1 and run(positions=BASE + 2) == 4


def test_fork_sizes_and_refusals():
    import packed_decode_gemv_amd as vbq
    size = vbq.lib.kv4_fork_workspace
    c = _cache(vbq)
    assert size(C.byref(c), 1, 1, 1) > 0
    assert size(C.byref(c), 65535, 65535, 1 << 20) >= 4 * (3 * 65535 + 100)
    assert size(C.byref(c), 8, 8, 10) <= size(C.byref(c), 9, 8, 10) <= size(C.byref(c), 9, 9, 10) <= size(C.byref(c), 9, 9, 11)
    for bad in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (65536, 1, 1), (1, 65536, 1), (1, 1, (1 << 20) + 1)):
        assert size(C.byref(c), *bad) == -1
    assert size(C.byref(_cache(vbq, page_tokens=48)), 1, 1, 1) == -1 and size(None, 1, 1, 1) == -1

    def run(cache=c, **kw):
        d = dict(batch_in=2, batch_out=3, table_width=4, reserved=0, workspace_bytes=1 << 20)
        for i, n in enumerate(("table_in", "lens_in", "refs_in", "parents", "reserve", "table_out", "lens_out", "refs_out",
                               "workspace")):
            d[n] = BASE + 4096 * i
        d.update(kw)
        return vbq.lib.kv4_fork(cache and C.byref(cache), C.byref(vbq.vbq_kv4_fork(**d)), None)

    assert run(cache=None) == 1 and run(reserved=1) == 1
    large = _cache(vbq, page_tokens=65536, n_kv_heads=4096, head_dim=256)      # pages of 77 GB
    assert run(cache=large) == 5 and size(C.byref(large), 2, 3, 4) == -1
    for bad, st in ((dict(batch_in=0), 2), (dict(batch_out=65536), 5), (dict(table_width=0), 2),
                    (dict(table_width=(1 << 20) + 1), 5), (dict(workspace_bytes=15), 6)):
        assert run(**bad) == st, bad
    for n in ("table_in", "lens_in", "refs_in", "parents", "table_out", "lens_out", "refs_out", "workspace"):
        assert run(**{n: None}) == 1, n
        assert run(**{n: BASE + (1 << 20) + 2}) == 4, n
    for n in ("refs_in", "refs_out", "workspace"):
        assert run(**{n: BASE + (1 << 20) + 4}) == 4, n
    for out in ("table_out", "lens_out", "refs_out", "workspace"):      # an output that is an input, or another output
        for i, other in enumerate(("table_in", "lens_in", "refs_in", "parents", "reserve", "table_out", "lens_out",
                                   "refs_out", "workspace")):
            if other != out:
                assert run(**{out: BASE + 4096 * i}) == 1, (out, other)


def test_shared_attention_refuses_bad_arguments():
    import packed_decode_gemv_amd as vbq
    c = _cache(vbq)

    def pair(a, g):
        d = dict(batch=4, table_width=2, total_q=4, max_q=1, max_kv=0, n_heads=8, dtype=0, causal=1, window=0, sinks=0,
                 scale=0.1, reserved=0, table=BASE, kv_lens=BASE, cu_q=BASE, q=BASE, q_token_stride=1024,
                 q_head_stride=128, out=BASE, lse=None, workspace=BASE, workspace_bytes=1 << 40)
        e = dict(n_groups=1, max_shared=4096, max_own=100, max_group_q=4, cu_groups=BASE, shared=BASE, reserved=0)
        return vbq.vbq_kv4_attn(**{**d, **a}), vbq.vbq_kv4_groups(**{**e, **g})

    def run(a=(), g=(), cache=c):
        x, y = pair(dict(a), dict(g))
        return vbq.lib.kv4_attention_shared(C.byref(cache), C.byref(x), C.byref(y), None)

    def size(a=(), g=()):
        x, y = pair(dict(a), dict(g))
        return vbq.lib.kv4_attention_shared_workspace(C.byref(c), C.byref(x), C.byref(y))

    far = dict(max_shared=1 << 22)                    # too many tokens for each sequence to read them for itself
    assert size(g=far) >= 4 * 4 * 8 * 130 + 8 * 2048
    assert 8 * 2048 <= size(g=dict(max_shared=0)) <= size() < size(g=far)
    assert size(a=dict(n_heads=2 * 33)) > 8 * 2048    # more rows than the kernel for few takes
    for bad, st in ((dict(window=5), 1), (dict(sinks=1), 1), (dict(batch=0), 2), (dict(n_heads=7), 2), (dict(max_q=-1), 2),
                    (dict(batch=65536), 5), (dict(dtype=2), 1), (dict(causal=2), 1), (dict(scale=0.0), 1)):
        assert run(a=bad) == st and size(a=bad) == -1, bad
    for bad, st in ((dict(n_groups=0), 2), (dict(n_groups=65536), 5), (dict(max_shared=-1), 2), (dict(max_own=-1), 2),
                    (dict(max_group_q=-1), 2), (dict(max_own=2 ** 31 - 40), 5), (dict(max_shared=2 ** 31 - 1), 5),
                    (dict(reserved=1), 1)):
        assert run(g=bad) == st and size(g=bad) == -1, bad
    for bad, st in ((dict(q=None), 1), (dict(out=None), 1), (dict(table=None), 1), (dict(workspace=None), 1),
                    (dict(out=BASE + 8), 4), (dict(q_head_stride=4), 4), (dict(workspace_bytes=size() - 1), 6)):
        assert run(a=bad) == st, bad
    for bad, st in ((dict(cu_groups=None), 1), (dict(shared=None), 1), (dict(shared=BASE + 1), 4), (dict(cu_groups=BASE + 2), 4)):
        assert run(g=bad) == st, bad
    assert run(cache=_cache(vbq, head_dim=96)) == 2
    assert run(a=dict(total_q=0)) == 0 and run(a=dict(max_q=0)) == 0
    assert vbq.lib.kv4_attention_shared(C.byref(c), None, None, None) == 1


def test_logprobs_sizes_and_refusals():
    import packed_decode_gemv_amd as vbq
    size = vbq.lib.token_logprobs_workspace
    assert size(0, 100, 5) == 0 and size(1, 100, 5) == 0 and size(4096, 128256, 32) == 0
    assert size(1, 128256, 20) > size(1, 128256, 0) > 4 * 512
    for bad in ((-1, 10, 1), (1, 0, 0), (1, (1 << 30) + 1, 0), (1, 100, 33), (1, 100, -1), (1, 5, 6), (1 << 24, 100, 0)):
        assert size(*bad) == -1, bad

    def run(**kw):
        d = dict(rows=2, vocab=128256, dtype=2, top=3, row_stride=128256, logits=BASE, tokens=BASE, token_bytes=8, reserved=0,
                 logprob=BASE, rank=BASE, entropy=BASE, lse=BASE, top_logprob=BASE, top_index=BASE, workspace=BASE,
                 workspace_bytes=1 << 30)
        d.update(kw)
        return vbq.lib.token_logprobs(C.byref(vbq.vbq_logprobs(**d)), None)

    assert vbq.lib.token_logprobs(None, None) == 1
    assert run(rows=0) == 0
    for bad, st in ((dict(rows=-1), 2), (dict(vocab=0), 2), (dict(top=33), 5), (dict(dtype=3), 1), (dict(dtype=-1), 1),
                    (dict(token_bytes=2), 1), (dict(reserved=1), 1), (dict(logits=None), 1), (dict(logprob=None), 1),
                    (dict(rank=None), 1), (dict(top_logprob=None), 1), (dict(top_index=None), 1), (dict(workspace=None), 1),
                    (dict(logits=BASE + 2), 4), (dict(tokens=BASE + 4), 4), (dict(rank=BASE + 1), 4),
                    (dict(workspace=BASE + 8), 4), (dict(workspace_bytes=100), 6), (dict(vocab=2, top=3), 2)):
        assert run(**bad) == st, bad


def test_the_binding_refuses_before_the_library_is_reached():
    import torch

    import packed_decode_gemv_amd as vbq
    with pytest.raises(ValueError, match="GPU"):
        vbq.HeadRotary(64, torch.ones(32))
    with pytest.raises(ValueError, match="head_dim"):
        vbq.HeadRotary(80, torch.ones(32))
    with pytest.raises(ValueError, match="pairs"):
        vbq.HeadRotary(64, torch.ones(20))
    with pytest.raises(ValueError, match="GPU"):
        vbq.token_logprobs(torch.zeros(2, 10))
    with pytest.raises(ValueError, match="2-D"):
        vbq.token_logprobs(torch.zeros(10))
    for args in ((1, 2 ** 40, 0), (2 ** 33, 10, 0), (1, 10, 11), (-1, 10, 0)):
        with pytest.raises(ValueError, match="refused"):
            vbq.token_logprobs_workspace(*args)


def test_rotary_refuses_more_than_a_launch_holds():
    import packed_decode_gemv_amd as vbq
    p = vbq.vbq_head_rotary(head_dim=64, rotary_dim=0, axes=1, interleaved=0, eps=0.0, reserved=0, inv_freq=None, axis=None,
                            q_weight=None, k_weight=None)
    rows = vbq.vbq_head_rows(in_=BASE, out=BASE, in_token_stride=64, in_head_stride=64, out_token_stride=64,
                             out_head_stride=64, heads=65536, in_dtype=0, out_dtype=0, reserved=0)
    assert vbq.lib.head_norm_rotary(C.byref(p), C.byref(rows), C.byref(rows), None, 0, 2 ** 31 - 1, None) == 5


def test_the_binding_refuses_what_is_no_tensor():
    """On CPU tensors with a stand-in for the plan and the cache: refusals come before the library is called."""
    from types import SimpleNamespace

    import numpy as np
    import torch

    import packed_decode_gemv_amd as vbq
    i32 = torch.int32
    plan = SimpleNamespace(rotary_dim=64, axes=1, head_dim=64, index=-1, _i32=i32, device=torch.device("cpu"))
    q = torch.zeros(3, 2, 64)
    for bad in (None, [0, 1, 2], 7, np.zeros(3, np.int32)):
        with pytest.raises(ValueError, match="positions"):
            vbq.head_norm_rotary(plan, q, None, bad)
    for bad in ([0], np.zeros((3, 2, 64), np.float32), 5):
        for args in ((bad, None), (None, bad)):
            with pytest.raises(ValueError):
                vbq.head_norm_rotary(plan, *args, torch.zeros(3, dtype=i32))
        for kw in (dict(q_out=bad), dict(q_out=bad, q_dtype=torch.float32)):
            with pytest.raises(ValueError):
                vbq.head_norm_rotary(plan, q, None, torch.zeros(3, dtype=i32), **kw)

    cache = SimpleNamespace(n_pages=10, page_tokens=32, n_kv_heads=1, head_dim=64, index=-1, _i32=i32,
                            device=torch.device("cpu"), data=torch.zeros(1, dtype=torch.uint8))
    good = dict(refs=torch.zeros(10, dtype=i32), block_table=torch.zeros(2, 3, dtype=i32), lens=torch.zeros(2, dtype=i32),
                parents=torch.zeros(4, dtype=i32), reserve=torch.zeros(4, dtype=i32), workspace=None)
    for name in good:
        for bad in ([1, 2], 3, np.zeros(2, np.int32)) + (() if name in ("reserve", "workspace") else (None,)):
            with pytest.raises(ValueError):
                vbq.kv4_fork(cache, **{**good, "out": (torch.zeros(4, 3, dtype=i32), torch.zeros(4, dtype=i32),
                                                       torch.zeros(10, dtype=i32)), name: bad})
    with pytest.raises(ValueError):
        vbq.kv4_fork(cache, **good, out=(None, None, None))

    good = dict(q=torch.zeros(2, 1, 64, dtype=torch.float16), block_table=torch.zeros(2, 3, dtype=i32),
                kv_lens=torch.zeros(2, dtype=i32), cu_q=torch.zeros(3, dtype=i32), cu_groups=torch.zeros(2, dtype=i32),
                shared=torch.zeros(1, dtype=i32), out=torch.zeros(2, 1, 64, dtype=torch.float16), workspace=None)
    for name in good:
        for bad in ([1, 2], 3, np.zeros((2, 1, 64), np.float16)) + (() if name in ("out", "workspace") else (None,)):
            with pytest.raises(ValueError):
                vbq.kv4_attention_shared(cache, **{**good, name: bad}, max_q=1, max_shared=1, max_own=1)
    with pytest.raises(ValueError):
        vbq.kv4_attention_shared(cache, **good, lse=[1], max_q=1, max_shared=1, max_own=1)

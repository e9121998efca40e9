"""Host-side checks of the 4-bit key/value cache's entry points: sizes, and
arguments that are refused before a GPU is touched."""
import ctypes as C

import pytest

BASE = 0x7F0000000000


def _cache(vbq, **kw):
    d = dict(n_pages=4, page_tokens=64, n_kv_heads=2, head_dim=128, reserved=0, data=BASE, flags=BASE + 256)
    d.update(kw)
    return vbq.vbq_kv4(**d)


def _range(vbq, **kw):
    d = dict(batch=2, table_width=2, total_tokens=5, max_tokens=3, table=BASE, start=BASE, cu=BASE)
    d.update(kw)
    return vbq.vbq_kv4_range(**d)


def _attn(vbq, **kw):
    d = dict(batch=2, table_width=2, total_q=2, max_q=1, max_kv=4096, n_heads=8, dtype=0, causal=1, window=0, sinks=0,
             scale=0.1, reserved=0, table=BASE, kv_lens=BASE, cu_q=BASE, q=BASE, q_token_stride=1024,
             q_head_stride=128, out=BASE, lse=None, workspace=BASE, workspace_bytes=1 << 40)
    d.update(kw)
    return vbq.vbq_kv4_attn(**d)


def test_page_bytes():
    import packed_decode_gemv_amd as vbq
    size = vbq.lib.kv4_page_bytes
    assert size(32, 1, 64) == 2304                 # 36 bytes per 64 values, keys and values
    assert size(64, 8, 128) == 64 * 8 * 128 * 2 * 9 // 16
    assert size(65536, 4096, 256) == 65536 * 4096 * 256 * 2 * 9 // 16
    for bad in ((16, 1, 64), (48, 1, 64), (131072, 1, 64), (32, 0, 64), (32, 4097, 64), (32, 1, 96), (32, 1, 320),
                (32, 1, 0), (0, 1, 64), (-32, 1, 64)):
        assert size(*bad) == 0


def test_append_and_read_refuse_bad_arguments():
    import packed_decode_gemv_amd as vbq
    L, p = vbq.lib, C.c_void_p(BASE)
    c, r = _cache(vbq), _range(vbq)

    def append(cache=c, rng=r, k=p, v=p, dt=0, kt=256, kh=128, vt=256, vh=128):
        return L.kv4_append(cache and C.byref(cache), rng and C.byref(rng), k, v, dt, kt, kh, vt, vh, None)

    assert append(cache=None) == 1 and append(rng=None) == 1
    assert append(k=None) == 1 and append(v=None) == 1
    assert append(dt=3) == 1 and append(dt=-1) == 1
    assert append(k=C.c_void_p(BASE + 8)) == 4 and append(kt=252) == 4 and append(vh=4) == 4
    assert append(dt=2, kt=2) == 4
    for bad, st in ((dict(page_tokens=48), 2), (dict(head_dim=96), 2), (dict(n_pages=0), 2), (dict(n_pages=2 ** 31), 5),
                    (dict(reserved=1), 1), (dict(data=None), 1), (dict(data=BASE + 4), 4), (dict(flags=BASE + 2), 4),
                    (dict(n_kv_heads=0), 2)):
        cc = _cache(vbq, **bad)
        assert append(cache=cc) == st, bad
        assert L.kv4_read(C.byref(cc), C.byref(r), p, p, 0, None) == st, bad
    for bad, st in ((dict(batch=0), 2), (dict(batch=65536), 5), (dict(table_width=0), 2), (dict(total_tokens=-1), 2),
                    (dict(max_tokens=-1), 2), (dict(table=None), 1), (dict(start=None), 1), (dict(cu=None), 1),
                    (dict(cu=BASE + 1), 4)):
        rr = _range(vbq, **bad)
        assert append(rng=rr) == st, bad
        assert L.kv4_read(C.byref(c), C.byref(rr), p, p, 0, None) == st, bad
    assert L.kv4_read(C.byref(c), C.byref(r), C.c_void_p(BASE + 8), p, 0, None) == 4
    assert L.kv4_read(C.byref(c), C.byref(r), p, p, 5, None) == 1
    # nothing to do: fine, and nothing is launched
    assert append(rng=_range(vbq, total_tokens=0), k=None, v=None) == 0
    assert L.kv4_read(C.byref(c), C.byref(r), None, None, 0, None) == 0


def test_attention_refuses_bad_arguments():
    import packed_decode_gemv_amd as vbq
    L = vbq.lib
    c = _cache(vbq)

    def run(cache=c, **kw):
        return L.kv4_attention(C.byref(cache), C.byref(_attn(vbq, **kw)), None)

    assert L.kv4_attention(None, C.byref(_attn(vbq)), None) == 1
    assert L.kv4_attention(C.byref(c), None, None) == 1
    for bad, st in ((dict(batch=0), 2), (dict(batch=70000), 5), (dict(n_heads=7), 2), (dict(n_heads=0), 2),
                    (dict(max_q=-1), 2), (dict(max_kv=-1), 2), (dict(max_kv=2 ** 31 - 1), 5), (dict(dtype=2), 1),
                    (dict(causal=2), 1), (dict(window=-1), 1), (dict(sinks=-1), 1), (dict(causal=0, window=4), 1),
                    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
                    (dict(max_q=2 ** 30, n_heads=8), 5), (dict(reserved=1), 1)):
        assert run(**bad) == st, bad
        assert L.kv4_attention_workspace(C.byref(c), C.byref(_attn(vbq, **bad))) == -1, bad
    for bad, st in ((dict(table=None), 1), (dict(kv_lens=None), 1), (dict(cu_q=None), 1), (dict(q=None), 1),
                    (dict(out=None), 1), (dict(workspace=None), 1), (dict(workspace=BASE + 8), 4),
                    (dict(q=BASE + 8), 4), (dict(q_token_stride=1020), 4), (dict(q_head_stride=4), 4),
                    (dict(out=BASE + 2), 4), (dict(lse=BASE + 2), 4), (dict(workspace_bytes=100), 6)):
        assert run(**bad) == st, bad
    assert run(cache=_cache(vbq, data=None)) == 1
    assert run(total_q=0) == 0 and run(max_q=0) == 0


@pytest.mark.parametrize("batch,heads,max_q,max_kv,window,sinks",
                         [(1, 8, 1, 131072, 0, 0), (64, 8, 1, 8192, 0, 0), (3, 64, 4096, 9000, 500, 4), (1, 2, 1, 0, 0, 0),
                          (4096, 2, 7, 2 ** 31 - 100, 0, 0)])
def test_workspace_is_bounded_and_grows_with_no_size_beyond_it(batch, heads, max_q, max_kv, window, sinks):
    import packed_decode_gemv_amd as vbq
    c = _cache(vbq)
    n = vbq.lib.kv4_attention_workspace(C.byref(c), C.byref(_attn(vbq, batch=batch, n_heads=heads, max_q=max_q,
                                                                   max_kv=max_kv, window=window, sinks=sinks)))
    assert 0 <= n < 1 << 30


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_a_cache_is_on_a_gpu(device):
    """A buffer elsewhere would reach the kernels as a device pointer."""
    import torch
    import packed_decode_gemv_amd as vbq
    with pytest.raises(ValueError, match="expected a GPU"):
        vbq.Kv4Cache(2, 32, 1, 64, device=device)
    with pytest.raises(ValueError, match="expected a GPU"):
        vbq.Kv4Cache(2, 32, 1, 64, data=torch.zeros(2 * 2304, dtype=torch.uint8, device=device))


def test_attention_refuses_a_scale_that_binary32_does_not_hold_in_base_two():
    """Scores are formed in base two: scale * log2(e) has to be a number."""
    import packed_decode_gemv_amd as vbq
    c = _cache(vbq)
    for scale, ok in ((2.3e38, True), (2.4e38, False), (2.9e38, False), (3.4e38, False), (1e-38, True)):
        a = _attn(vbq, scale=scale)
        assert (vbq.lib.kv4_attention_workspace(C.byref(c), C.byref(a)) >= 0) is ok, scale
        if not ok:
            assert vbq.lib.kv4_attention(C.byref(c), C.byref(a), None) == 1


@pytest.mark.parametrize("sizes", [(4, 2 ** 32 + 32, 1, 64), (4, 32, 2 ** 32 + 1, 64), (4, 32, 1, 2 ** 32 + 64),
                                   (4, 32 - 2 ** 32, 1, 64), (2 ** 32 + 4, 32, 1, 64), (0, 32, 1, 64), (4, 33, 1, 64)])
def test_a_cache_refuses_sizes_beyond_an_int(sizes):
    """They would be cut to 32 bits on their way into the library."""
    import packed_decode_gemv_amd as vbq
    with pytest.raises(ValueError, match="pages take"):
        vbq.Kv4Cache(*sizes, device="cpu")      # (nothing is allocated)


def test_more_workgroups_than_a_launch_takes_are_refused():
    """A launch's first dimension holds 2^32 - 1 threads; what is beyond would be left undone."""
    import packed_decode_gemv_amd as vbq
    L, p = vbq.lib, C.c_void_p(BASE)
    c = _cache(vbq, n_kv_heads=2)
    r = _range(vbq, total_tokens=2 ** 30, max_tokens=2 ** 30)
    assert L.kv4_append(C.byref(c), C.byref(r), p, p, 0, 256, 128, 256, 128, None) == 5
    r = _range(vbq, total_tokens=2 ** 31 - 1, max_tokens=2 ** 31 - 1)
    assert L.kv4_read(C.byref(c), C.byref(r), p, p, 0, None) == 5
    many = _cache(vbq, n_kv_heads=512, head_dim=64)
    for ratio in (1, 16):
        a = _attn(vbq, batch=65535, total_q=65535, max_q=1, n_heads=512 * ratio)
        assert L.kv4_attention(C.byref(many), C.byref(a), None) == 5
        assert L.kv4_attention_workspace(C.byref(many), C.byref(a)) == -1


def test_rows_that_an_int_does_not_hold_with_a_tile_more_are_refused():
    import packed_decode_gemv_amd as vbq
    c = _cache(vbq, n_kv_heads=1)
    for rows, ok in ((2 ** 31 - 1 - 128, True), (2 ** 31 - 1 - 127, False), (2 ** 31 - 1 - 64, False)):
        a = _attn(vbq, batch=1, n_heads=1, max_q=rows, total_q=9)
        assert (vbq.lib.kv4_attention_workspace(C.byref(c), C.byref(a)) >= 0) is ok

"""Refusals of the entry points between a decoder layer's linears (no GPU
needed): argument checks run before any HIP call, so these calls with fake
pointer values launch nothing."""
import ctypes as C

import pytest
import torch

import group_wise_affine_unpack_amd as qa

OK, INVAL, UNSUP, ALIGN = 0, 1, 2, 3
A = 0x10000  # a fake, 16-byte aligned "device" address; never dereferenced


def _msg():
    return qa.lib().qaff_last_error().decode()


def _cache(**kw):
    d = dict(k_packed=A, k_scales=A, k_biases=A, v_packed=A, v_scales=A, v_biases=A, num_pages=4, page_size=16, kv_heads=2,
             head_dim=128, group_size=64, bits=4, dtype=0)
    c = qa.KVCacheArrays(**{**d, **kw})
    return C.byref(c)


_BAD_CACHES = [
    (dict(bits=3), INVAL), (dict(bits=16), INVAL), (dict(group_size=48), INVAL), (dict(head_dim=96), INVAL),
    (dict(head_dim=0), INVAL), (dict(dtype=2), INVAL), (dict(num_pages=0), INVAL), (dict(page_size=0), INVAL),
    (dict(kv_heads=0), INVAL), (dict(head_dim=320), UNSUP), (dict(page_size=24), UNSUP),
    (dict(kv_heads=(1 << 16) + 1), UNSUP), (dict(num_pages=1 << 27), UNSUP), (dict(k_packed=None), INVAL),
    (dict(v_biases=None), INVAL), (dict(v_packed=A + 4), ALIGN), (dict(k_scales=A + 2), ALIGN)]


def _append(cache=None, k=A, v=A, ks=(256, 128), vs=(256, 128), slots=A, T=1):
    return qa.lib().kv_cache_append_affine(cache if cache is not None else _cache(), k, v, *ks, *vs, slots, T, None)


def _read(cache=None, slots=A, k=A, v=A, T=1):
    return qa.lib().kv_cache_read_affine(cache if cache is not None else _cache(), slots, k, v, T, None)


def _attn(cache=None, q=A, qs=(512, 128), table=A, ts=8, pages=8, lens=A, out=A, B=1, heads=4, scale=0.1, window=0):
    return qa.lib().paged_attention_affine(cache if cache is not None else _cache(), q, *qs, table, ts, pages, lens, out, B,
                                           heads, scale, window, None)


@pytest.mark.parametrize("kw,code", _BAD_CACHES)
def test_cache_descriptors(kw, code):
    for call in (_append, _read, _attn):
        assert call(_cache(**kw)) == code
        assert _msg() != ""


def test_null_cache():
    assert qa.lib().kv_cache_read_affine(None, A, A, A, 1, None) == INVAL


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVAL), (dict(T=(1 << 30) + 1), UNSUP), (dict(k=None), INVAL), (dict(v=None), INVAL),
    (dict(slots=None), INVAL), (dict(k=A + 8), ALIGN), (dict(v=A + 2), ALIGN), (dict(slots=A + 4), ALIGN),
    (dict(ks=(-8, 128)), ALIGN), (dict(ks=(256, 4)), ALIGN), (dict(vs=(12, 128)), ALIGN), (dict(T=1 << 28), UNSUP)])
def test_append_arguments(kw, code):
    assert _append(**kw) == code and _msg() != ""


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INVAL), (dict(T=(1 << 30) + 1), UNSUP), (dict(k=None), INVAL), (dict(v=None), INVAL),
    (dict(slots=None), INVAL), (dict(k=A + 8), ALIGN), (dict(slots=A + 4), ALIGN), (dict(T=1 << 28), UNSUP)])
def test_read_arguments(kw, code):
    assert _read(**kw) == code and _msg() != ""


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVAL), (dict(pages=-1), INVAL), (dict(heads=3), INVAL), (dict(heads=0), INVAL),
    (dict(B=65536), UNSUP), (dict(pages=1 << 27), UNSUP), (dict(scale=float("nan")), INVAL),
    (dict(scale=float("inf")), INVAL), (dict(window=-1), INVAL), (dict(q=None), INVAL), (dict(lens=None), INVAL),
    (dict(out=None), INVAL), (dict(table=None), INVAL), (dict(q=A + 8), ALIGN), (dict(out=A + 2), ALIGN),
    (dict(table=A + 2), ALIGN), (dict(lens=A + 1), ALIGN), (dict(qs=(512, 100)), ALIGN), (dict(qs=(-8, 128)), ALIGN),
    (dict(ts=-1), INVAL)])
def test_attention_arguments(kw, code):
    assert _attn(**kw) == code and _msg() != ""


def test_attention_tables_past_31_bits():
    assert _attn(_cache(), pages=(1 << 27)) == UNSUP
    assert _attn(_cache(), pages=(1 << 27) - (1 << 12) + 1) == UNSUP  # (pages of 16: past 2^31 - 2^16 tokens)


def test_attention_rows_past_31_bits():
    # 2^26 pages of 16 tokens by 64 heads: 2^32 tiles
    assert _attn(_cache(num_pages=1 << 26, kv_heads=64), heads=64) == UNSUP


@pytest.mark.parametrize("D,G", [(32, 32), (160, 32), (224, 32)])
def test_attention_head_sizes(D, G):
    assert _attn(_cache(head_dim=D, group_size=G)) == UNSUP


def test_empty_calls_launch_nothing():
    assert _append(T=0, k=None, v=None, slots=None) == OK
    assert _read(T=0, k=None, v=None, slots=None) == OK
    assert _attn(B=0, q=None, table=None, lens=None, out=None) == OK
    assert _msg() == ""


def _norm(fn="rmsnorm", x=A, r=None, w=A, eps=1e-5, h=None, outs=None, M=2, K=64, ld=(64, 64, 64), adt=0, wdt=0):
    outs = outs if outs is not None else ((A,) if fn == "rmsnorm" else (A, A))
    return getattr(qa.lib(), fn)(x, r, w, eps, h, *outs, M, K, *ld, adt, wdt, None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVAL), (dict(K=0), INVAL), (dict(K=(1 << 30) + 1), UNSUP), (dict(adt=2), INVAL), (dict(wdt=3), INVAL),
    (dict(eps=-1e-5), INVAL), (dict(eps=float("nan")), INVAL), (dict(eps=float("inf")), INVAL), (dict(x=None), INVAL),
    (dict(w=None), INVAL), (dict(r=A), INVAL), (dict(h=A), INVAL), (dict(ld=(63, 64, 64)), INVAL),
    (dict(r=A, h=A, ld=(64, 32, 64)), INVAL), (dict(r=A, h=A, ld=(64, 64, 0)), INVAL),
    (dict(ld=(1 << 41, 64, 64)), UNSUP), (dict(x=A + 1), ALIGN), (dict(w=A + 2, wdt=2), ALIGN)])
@pytest.mark.parametrize("fn", ["rmsnorm", "rmsnorm_w4a8"])
def test_norm_arguments(fn, kw, code):
    assert _norm(fn, **kw) == code and _msg() != ""


def test_norm_outputs():
    assert _norm(outs=(None,)) == INVAL
    assert _norm(outs=(A + 1,)) == ALIGN
    assert _norm("rmsnorm_w4a8", outs=(None, A)) == INVAL
    assert _norm("rmsnorm_w4a8", outs=(A, None)) == INVAL
    assert _norm("rmsnorm_w4a8", outs=(A, A + 2)) == ALIGN
    assert _norm(M=0, x=None, w=None, outs=(None,)) == OK


def test_w4a8_codes_arguments():
    f = qa.lib().qgemm_w4a8_codes
    assert f(A, A, A, A, A, None, 1, 64, 48, None) == INVAL
    assert f(A, A, A, A, A, None, -1, 64, 64, None) == INVAL
    assert f(None, A, A, A, A, None, 1, 64, 64, None) == INVAL
    assert f(A, None, A, A, A, None, 1, 64, 64, None) == INVAL
    assert f(A + 8, A, A, A, A, None, 1, 64, 64, None) == ALIGN
    assert f(A, A, A, A, A, None, 1, 64, (1 << 17) + 32, None) == UNSUP
    assert f(A, A, A, A, A, None, 1 << 20, 64, 4096, None) == UNSUP  # codes past 32-bit offsets
    assert f(None, None, None, None, None, None, 0, 64, 64, None) == OK


def test_python_shape_checks():
    k = (torch.zeros(2, 1, 16, 8, dtype=torch.int32), torch.zeros(2, 1, 16, 1, dtype=torch.bfloat16),
         torch.zeros(2, 1, 16, 1, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        qa.AffineKVCache(k, (k[0], k[1][:1], k[2]), 64, 4)
    with pytest.raises(ValueError):
        qa.AffineKVCache(k, (k[0], k[1].half(), k[2].half()), 64, 4)
    with pytest.raises(ValueError):
        qa.AffineKVCache(k, k, 64, 3)
    with pytest.raises(ValueError):  # not on a GPU
        qa.AffineKVCache(k, k, 64, 4)

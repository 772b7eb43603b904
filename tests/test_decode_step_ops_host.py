"""Refusals of the entry points around the paged cache that need no GPU:
argument checks run before any HIP call, so these calls with fake pointer
values launch nothing.  And the oracle's definitions pinned by hand."""
import ctypes as C

import numpy as np
import pytest
import torch

import group_wise_affine_unpack_amd as qa
import oracle.decoder as od

OK, INVAL, UNSUP, ALIGN = 0, 1, 2, 3
A = 0x10000  # a fake, 16-byte aligned "device" address; never dereferenced


def _msg():
    return qa.lib().qaff_last_error().decode()


def _assign(table=A, ts=8, per=8, lens=A, news=A + 64, out=A, free=A, state=A, pages=64, page=16, B=2, slots=A, pos=A, ids=A, T=4):
    return qa.lib().kv_pages_assign(table, ts, per, lens, news, out, free, state, pages, page, B, slots, pos, ids, T, None)


def _trim(table=A, ts=8, per=8, lens=A, news=A + 64, out=A, free=A, state=A, pages=64, page=16, B=2):
    return qa.lib().kv_pages_trim(table, ts, per, lens, news, out, free, state, pages, page, B, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INVAL), (dict(per=-1), INVAL), (dict(pages=0), INVAL), (dict(page=0), INVAL), (dict(page=24), UNSUP),
    (dict(page=1 << 17), UNSUP), (dict(pages=1 << 27), UNSUP), (dict(B=4097), UNSUP), (dict(per=1 << 27, ts=1 << 27), UNSUP),
    (dict(B=4096, per=1 << 20, ts=1 << 20), UNSUP), (dict(ts=7), INVAL), (dict(ts=1 << 41), INVAL), (dict(table=None), INVAL),
    (dict(lens=None), INVAL), (dict(news=None), INVAL), (dict(out=None), INVAL), (dict(free=None), INVAL),
    (dict(state=None), INVAL), (dict(table=A + 2), ALIGN), (dict(lens=A + 1), ALIGN), (dict(state=A + 2), ALIGN),
    (dict(out=A + 64), INVAL)])
def test_pages_argument_errors(kw, code):
    for call in (_assign, _trim):
        assert call(**kw) == code
        assert _msg() != ""


@pytest.mark.parametrize("kw,code", [(dict(T=-1), INVAL), (dict(T=(1 << 30) + 1), UNSUP), (dict(slots=None), INVAL),
                                     (dict(slots=A + 4), ALIGN), (dict(pos=A + 2), ALIGN), (dict(ids=A + 1), ALIGN)])
def test_assign_argument_errors(kw, code):
    assert _assign(**kw) == code


def test_pages_of_nothing():
    assert _assign(B=0, T=0, table=None, lens=None, news=None, out=None, slots=None) == OK
    assert _trim(B=0, table=None, lens=None, news=None, out=None) == OK


def _rot(**kw):
    return C.byref(qa.RotarySpec(**{**dict(inv_freq=A, rotary_dim=64, interleaved=0, magnitude=1.0), **kw}))


def _rotary(rot=None, q=A, qs=(256, 64), k=A + 16, ks=(128, 64), qo=A + 32, qos=(256, 64), ko=A + 48, kos=(128, 64), pos=A, T=1,
            H=4, HK=2, D=64, dt=0):
    return qa.lib().rotary(rot if rot is not None else _rot(), q, *qs, k, *ks, qo, *qos, ko, *kos, pos, T, H, HK, D, dt, None)


def _cache(**kw):
    d = dict(k_packed=A, k_scales=A, k_biases=A, v_packed=A, v_scales=A, v_biases=A, num_pages=4, page_size=16, kv_heads=2,
             head_dim=64, group_size=64, bits=4, dtype=0)
    return C.byref(qa.KVCacheArrays(**{**d, **kw}))


def _fused(rot=None, cache=None, q=A, qs=(256, 64), k=A, ks=(128, 64), v=A, vs=(128, 64), qo=A + 32, qos=(256, 64), pos=A,
           slots=A, T=1, H=4):
    return qa.lib().kv_cache_append_rotary_affine(cache if cache is not None else _cache(), rot if rot is not None else _rot(),
                                                  q, *qs, k, *ks, v, *vs, qo, *qos, pos, slots, T, H, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rot=_rot(rotary_dim=0)), INVAL), (dict(rot=_rot(rotary_dim=31)), INVAL), (dict(rot=_rot(rotary_dim=66)), INVAL),
    (dict(rot=_rot(interleaved=2)), INVAL), (dict(rot=_rot(magnitude=float("nan"))), INVAL),
    (dict(rot=_rot(inv_freq=None)), INVAL), (dict(rot=_rot(inv_freq=A + 4)), ALIGN), (dict(T=-1), INVAL),
    (dict(T=1 << 24), UNSUP), (dict(H=-1), INVAL), (dict(H=4097), UNSUP), (dict(pos=None), INVAL), (dict(pos=A + 2), ALIGN),
    (dict(q=None), INVAL), (dict(k=None), INVAL), (dict(qo=None), INVAL), (dict(q=A + 32, qos=(512, 64)), INVAL)])
def test_rotary_argument_errors(kw, code):
    for call in (_rotary, _fused):
        assert call(**kw) == code, call.__name__
        assert _msg() != ""


@pytest.mark.parametrize("kw,code", [(dict(D=0), INVAL), (dict(D=1025), UNSUP), (dict(HK=-1), INVAL), (dict(HK=4097), UNSUP),
                                     (dict(dt=2), INVAL), (dict(ko=None), INVAL), (dict(q=A + 1), ALIGN), (dict(ks=(-8, 64)), INVAL),
                                     (dict(kos=(1 << 41, 64)), INVAL), (dict(k=A + 48, kos=(64, 128)), INVAL)])
def test_rotary_only_argument_errors(kw, code):
    assert _rotary(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(cache=_cache(bits=3)), INVAL), (dict(cache=_cache(page_size=24)), UNSUP), (dict(cache=_cache(kv_heads=4097)), UNSUP),
    (dict(rot=_rot(rotary_dim=24)), UNSUP), (dict(rot=_rot(rotary_dim=12, interleaved=1)), UNSUP), (dict(v=None), INVAL),
    (dict(slots=None), INVAL), (dict(slots=A + 4), ALIGN), (dict(q=A + 8), ALIGN), (dict(v=A + 2), ALIGN), (dict(qo=A + 8), ALIGN),
    (dict(ks=(100, 64)), ALIGN), (dict(qos=(-64, 64)), ALIGN)])
def test_fused_append_argument_errors(kw, code):
    assert _fused(**kw) == code


def test_null_descriptors():
    assert qa.lib().rotary(None, A, 0, 0, A, 0, 0, A, 0, 0, A, 0, 0, A, 1, 1, 1, 64, 0, None) == INVAL
    assert _rotary(T=0, q=None, k=None, qo=None, ko=None, pos=None) == OK
    assert _rotary(H=0, HK=0, q=None, k=None, qo=None, ko=None) == OK
    assert _fused(T=0, q=None, k=None, v=None, qo=None, pos=None, slots=None) == OK


@pytest.mark.parametrize("args,code", [
    ((A, 0, 1e4, 0, 1, 0, 0, 0), INVAL), ((A, 3, 1e4, 0, 1, 0, 0, 0), INVAL), ((A, 1026, 1e4, 0, 1, 0, 0, 0), UNSUP),
    ((A, 64, 0.0, 0, 1, 0, 0, 0), INVAL), ((A, 64, float("inf"), 0, 1, 0, 0, 0), INVAL), ((A, 64, 1e4, 4, 1, 0, 0, 0), INVAL),
    ((A, 64, 1e4, 1, 0.0, 0, 0, 0), INVAL), ((A, 64, 1e4, 1, float("nan"), 0, 0, 0), INVAL), ((A, 2, 1e4, 2, 2, 0, 0, 0), INVAL),
    ((A, 64, 1e4, 3, 2, 0, 1, 4), INVAL), ((A, 64, 1e4, 3, 2, 100, 4, 4), INVAL), ((A, 64, 1e4, 3, 2, 100, -1, 4), INVAL),
    ((None, 64, 1e4, 0, 1, 0, 0, 0), INVAL), ((A + 4, 64, 1e4, 0, 1, 0, 0, 0), ALIGN)])
def test_frequencies_argument_errors(args, code):
    assert qa.lib().rotary_frequencies(*args, None) == code
    assert _msg() != ""


def test_binding_refusals():
    with pytest.raises(ValueError, match="float64"):
        qa.Rotary(torch.zeros(4))
    with pytest.raises(ValueError, match="scaling"):
        qa.Rotary.make(64, scaling="other", device="cpu")
    pool = qa.KVPagePool(8, 16, "cpu")
    assert pool.state.tolist() == [8, 0, 0, 0] and pool.free_pages.tolist() == list(range(7, -1, -1))
    lens = torch.zeros(2, dtype=torch.int32)
    table = torch.zeros((2, 3), dtype=torch.int32)
    with pytest.raises(ValueError, match="int32"):
        qa.kv_pages_assign(pool, table, lens.long(), lens, 4)
    with pytest.raises(ValueError, match="shape"):
        qa.kv_pages_trim(pool, table, lens, lens[:1])
    with pytest.raises(ValueError, match="on the GPU"):
        qa.kv_pages_trim(pool, table, lens, lens)
    pool.state = pool.state[:2]
    with pytest.raises(ValueError, match="stay as they were made"):
        qa.kv_pages_trim(pool, table, lens, lens)


def test_oracle_pages_by_hand():
    # pages of 16: 10 + 7 tokens open one page, 16 + 1 another, the third sequence finds the stack empty
    table = np.array([[3, -1], [5, -1], [-1, -1]], np.int32)
    t, slots, pos, ids, lens, count, short = od.pages_assign(table, np.array([10, 16, 0]), np.array([7, 1, 2]), np.array([7, 9], np.int32),
                                                             2, 16, 10, 11)
    assert t.tolist() == [[3, 9], [5, 7], [-1, -1]] and count == 0 and short == 1
    assert slots.tolist() == [58, 59, 60, 61, 62, 63, 144, 112, -1, -1, -1]
    assert pos.tolist() == [10, 11, 12, 13, 14, 15, 16, 16, 0, 1, 0] and ids.tolist() == [0] * 7 + [1, 2, 2, -1]
    assert lens.tolist() == [17, 17, 0]
    back, free, lens, count = od.pages_trim(t, lens, np.array([10, 0, 0]), np.array([0, 0, 0], np.int32), 0, 16, 10)
    assert back.tolist() == [[3, -1], [-1, -1], [-1, -1]] and free.tolist() == [7, 5, 9] and lens.tolist() == [10, 0, 0]


def test_oracle_rotary_by_hand():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]], np.float32)
    import oracle
    bits = oracle.f64_to_f16(x.astype(np.float64))
    f = np.array([np.pi / 2, np.pi])
    half, _ = od.rotary(bits, np.array([1]), f, "f16", False)
    assert np.allclose(half[0, 0], [-3, -2, 1, -4, 5])
    pairs, _ = od.rotary(bits, np.array([1]), f, "f16", True, 2.0)
    assert np.allclose(pairs[0, 0], [-4, 2, -6, -8, 5])
    # slow pairs are slowed, fast ones stay
    plain, bands = od.rotary_frequencies(64, 1e4), od.rotary_frequencies(64, 1e4, "bands", 8.0, 8192.0)
    assert bands[0] == plain[0] and np.isclose(bands[-1], plain[-1] / 8)
    based = od.rotary_frequencies(64, 1e4, "base", 8.0)
    assert based[0] == plain[0] and np.isclose(based[-1], plain[-1] / 8)


def _moe(x=A, logits=A, ldt=2, resid=A, y=A, M=1, top_k=2, renorm=1, scale=1.0, **kw):
    d = dict(gate_up_packed=A, gate_up_scales=A, gate_up_biases=A, down_packed=A, down_scales=A, down_biases=A, hidden=256,
             inner=128, num_experts=8, group_size=64, bits=4, dtype=0)
    return qa.lib().qmoe_affine(C.byref(qa.ExpertArrays(**{**d, **kw})), x, logits, ldt, resid, y, M, top_k, renorm, scale, None)


@pytest.mark.parametrize("kw,code", [
    (dict(bits=3), INVAL), (dict(group_size=48), INVAL), (dict(dtype=2), INVAL), (dict(ldt=1), INVAL), (dict(ldt=3), INVAL),
    (dict(num_experts=0), INVAL), (dict(hidden=0), INVAL), (dict(inner=0), INVAL), (dict(hidden=96), INVAL),
    (dict(inner=96), INVAL), (dict(M=-1), INVAL), (dict(M=257), UNSUP), (dict(top_k=0), INVAL), (dict(top_k=9), INVAL),
    (dict(top_k=65, num_experts=128), UNSUP), (dict(renorm=2), INVAL), (dict(scale=float("inf")), INVAL), (dict(scale=float("nan")), INVAL),
    (dict(num_experts=1025), UNSUP), (dict(hidden=65600), UNSUP), (dict(inner=1 << 17), UNSUP),
    (dict(hidden=96, inner=96, group_size=32, bits=2), UNSUP), (dict(x=None), INVAL), (dict(logits=None), INVAL),
    (dict(y=None), INVAL), (dict(gate_up_packed=None), INVAL), (dict(down_biases=None), INVAL), (dict(x=A + 8), ALIGN),
    (dict(y=A + 2), ALIGN), (dict(down_packed=A + 4), ALIGN), (dict(gate_up_scales=A + 2), ALIGN), (dict(logits=A + 2), ALIGN),
    (dict(resid=A + 1), ALIGN)])
def test_moe_argument_errors(kw, code):
    assert _moe(**kw) == code
    assert _msg() != ""


def test_moe_of_nothing():
    assert _moe(M=0, x=None, logits=None, y=None, gate_up_packed=None) == OK
    assert qa.lib().qmoe_affine(None, A, A, 2, None, A, 1, 1, 1, 1.0, None) == INVAL


def test_moe_binding_refusals():
    def triple(e, n, k, dt=torch.float16):
        return torch.zeros((e, n, k // 8), dtype=torch.int32), torch.zeros((e, n, k // 64), dtype=dt), torch.zeros((e, n, k // 64), dtype=dt)
    with pytest.raises(ValueError, match="shape"):
        qa.AffineExperts(triple(2, 256, 64), triple(2, 64, 192), 64, 4)
    with pytest.raises(ValueError, match="dtype"):
        qa.AffineExperts(triple(2, 256, 64), triple(2, 64, 128, torch.bfloat16), 64, 4)
    with pytest.raises(ValueError, match="bits"):
        qa.AffineExperts(triple(2, 256, 64), triple(2, 64, 128), 64, 3)
    with pytest.raises(ValueError, match="rows of up"):
        qa.AffineExperts(triple(2, 255, 64), triple(2, 64, 128), 64, 4)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        qa.AffineExperts(triple(2, 256, 64, torch.float32), triple(2, 64, 128, torch.float32), 64, 4)


def test_oracle_moe_by_hand():
    # one column group, weights 1 and 2 times a unit: y = silu(g) u summed over the inner rows, mixed by the softmax
    import oracle
    one = oracle.f64_to_f16(np.ones((1, 64)))

    def weight(e, n, k, value):
        return (np.zeros((e, n, k // 8), np.uint32), np.zeros((e, n, k // 64), np.uint16),
                np.broadcast_to(oracle.f64_to_f16(np.asarray(value, np.float64)), (e, n, k // 64)).copy())
    up = weight(2, 128, 64, np.array([1 / 64, 1 / 32])[:, None, None])
    down = weight(2, 64, 64, 1 / 64)
    y, _, chosen = od.moe(one, np.array([[0.0, np.log(3)]]), up, down, "f16", 64, 4, 2, True)
    silu = lambda t: t / (1 + np.exp(-t))
    assert chosen == [[1, 0]] and np.allclose(y, 0.25 * silu(1) * 1 + 0.75 * silu(2) * 2)
    y, _, chosen = od.moe(one, np.array([[0.0, np.log(3)]]), up, down, "f16", 64, 4, 1, False, 2.0, one)
    assert chosen == [[1]] and np.allclose(y, 1 + 2 * 0.75 * silu(2) * 2)

"""What oracle.decoder.attention_bound can tell (no GPU): fp32 arithmetic with
11-bit weights stays within it; mistakes that lose a token, a percent of the
scale, or bits of the key biases' sums or of the weights do not."""
import numpy as np
import pytest

import oracle
import oracle.decoder as od
import synth_inputs as si

HALF_STEP = {"bf16": 2.0**-8, "f16": 2.0**-11}
SIZE, D, G = 16, 128, 64


def _case(n, act, bits=8, wide=0.0, key_offset=0.0, far_scale=0.0, seed=0):
    """One sequence, one head.  key_offset: size of a per-channel offset of the keys' biases.  wide: two
    channels of a group with this entry of q and its negative, the others small, so that the sum of q is a small difference.  far_scale: log2 of how far
    one unattended token's value scales stand above the others'."""
    rng = np.random.default_rng((90, n, bits, seed))
    pages = -(-n // SIZE)
    trip = []
    for _ in range(2):
        rows = (pages, 1, SIZE)
        sigma = rng.uniform(0.5, 1.5, (*rows, D // G))
        packed = rng.integers(0, 1 << 32, (*rows, D * bits // 32), dtype=np.uint32)
        trip.append([packed, sigma * 5.5 / (2**bits - 1), -2.75 * sigma])
    q = rng.standard_normal((1, 1, D))
    if wide:
        q[..., 0::G], q[..., 1::G] = wide, -wide
        q.reshape(-1, G)[:, 2:] *= wide / 4000
    k, v = trip
    k[2] = k[2] + key_offset * (1 + 0.3 * rng.standard_normal(k[2].shape))
    if far_scale:
        at = (n // 2 // SIZE, 0, n // 2 % SIZE)
        k[1][at], k[2][at] = 0, -40 * np.sign(q[0, 0].reshape(-1, G).sum(1)) * np.sqrt(D) / np.abs(q[0, 0].reshape(-1, G).sum(1))
        v[1][at] = 2.0**far_scale * 4e-3 * 255 / (2**bits - 1)
    return (si.store(q.astype(np.float32), act), *[(t[0], *(si.store(x.astype(np.float32), act) for x in t[1:])) for t in trip],
            act, G, bits, np.arange(pages, dtype=np.int32)[None], [n], D**-0.5)


def _pieces(x, act, units):
    """x, fp32, as the sum of three 16-bit pieces in units of `units`."""
    left, total = (x * np.float32(units)).astype(np.float32), np.float64(0)
    for _ in range(3):
        piece = oracle.to_f64(si.store(left.astype(np.float32), act), act)
        total = total + piece
        left = (left - piece).astype(np.float32)
    return total / units


def _kernel(case, q_units, own_groups):
    """The kernel's arithmetic in fp32 and f16.  q_units: the power of two that the sums of q are held in, over q's own with its
    largest in [2^14, 2^15).  own_groups: the weights' reference is each group's largest weight times scale, not the largest
    logit and the largest scale by themselves."""
    q, k, v, act, _, bits, table, (n,), scale = case
    f = np.float32
    t = np.arange(n)
    kt, vt = [tuple(a[t // SIZE, 0, t % SIZE] for a in x) for x in (k, v)]
    kc, vc = [od.codes(x[0], bits).reshape(n, -1, G).astype(f) for x in (kt, vt)]
    ks, kb, vs, vb = [oracle.to_f64(x, act).astype(f) for x in (kt[1], kt[2], vt[1], vt[2])]
    qf = oracle.to_f64(q[0, 0], act)
    e = 14 - int(np.floor(np.log2(np.abs(qf).max())))
    qg = (qf * 2.0**e).astype(np.float16).astype(f).reshape(-1, G)
    C = np.einsum("tgi,gi->tg", kc, qg, dtype=f)
    Q = _pieces(qg.sum(1, dtype=f), act, q_units)
    z = ((ks * C).sum(1, dtype=f) + (kb * Q).sum(1).astype(f)) * f(scale * 1.4426950408889634 * 2.0**-e)
    p = np.exp2((z - z.max()).astype(f)).astype(f)
    w = p[:, None] * vs
    if own_groups:
        ref = np.floor(np.log2(np.abs(w).max(0))) - 4
    else:
        ref = np.full(D // G, np.floor(np.log2(np.abs(vs).max())) - 5)
    A = (w * np.exp2(-ref).astype(f)).astype(np.float16).astype(f)
    o = np.einsum("tg,tgi->gi", A, vc, dtype=f) * np.exp2(ref)[:, None] + np.einsum("t,tg->g", p, vb, dtype=f)[:, None]
    return (o / p.sum(dtype=f)).reshape(1, 1, D)


def _share(case, out):
    ref, bound = od.attention_bound(*case)
    return float((np.abs(out - ref) / (bound + 1e-30)).max())


CASES = [dict(n=n, act=act, bits=bits) for n in (1, 40, 1000) for act in ("bf16", "f16") for bits in (2, 4, 8)] + [
    dict(n=200, act="f16", wide=5.0, key_offset=3000.0), dict(n=200, act="bf16", wide=5.0, key_offset=3000.0),
    dict(n=256, act="f16", far_scale=23.0), dict(n=256, act="bf16", far_scale=40.0)]


@pytest.mark.parametrize("kw", CASES)
def test_the_kernels_arithmetic_is_within_the_bound(kw):
    case = _case(**kw)
    assert _share(case, _kernel(case, 2.0**-7, True)) <= 1


@pytest.mark.parametrize("kw", CASES)
def test_outputs_are_those_of_the_definition(kw):
    case = _case(**kw)
    out, bound = od.attention_bound(*case)
    np.testing.assert_allclose(out, od.paged_attention(*case)[0], rtol=1e-9, atol=1e-12)
    assert (bound >= 0).all() and np.isfinite(bound).all()


@pytest.mark.parametrize("n,act,bits", [(40, "f16", 2), (40, "bf16", 4), (200, "bf16", 4), (200, "f16", 8)])
def test_a_token_or_five_percent_of_the_scale_is_told(n, act, bits):
    case = _case(n, act, bits)
    ref, bound = od.attention_bound(*case)
    tol = bound + HALF_STEP[act] * np.abs(ref)
    for wrong in (od.attention_bound(*case, leave_out=(0,))[0], od.attention_bound(*case, leave_out=(-1,))[0],
                  od.attention_bound(*case[:-1], 1.05 * case[-1])[0], 0 * ref):
        assert (np.abs(wrong - ref) > tol).any()


def test_sums_of_q_held_to_sixteen_bits_are_told():
    shares = []
    for seed in range(4):
        case = _case(n=200, act="f16", wide=5.0, key_offset=3000.0, seed=seed)
        shares.append(_share(case, _kernel(case, 2.0**-24, True)))
    assert min(shares) > 1.5


@pytest.mark.parametrize("far", [20.0, 23.0])
def test_weights_below_the_reference_of_an_unattended_scale_are_told(far):
    case = _case(n=256, act="f16", far_scale=far)
    assert _share(case, _kernel(case, 2.0**-7, False)) > 2

"""paged_attention_affine against fp64 within the bound that its own roundings
give (oracle.decoder.attention_bound), half a step of the output's type on top.

Every case first shows on the CPU that its tolerance can tell: the outputs
with the first or the last token left out, or with a scale 5% off, are past
it.  For that the first and the last token of each sequence have keys that
point along a query, so that they hold a good part of its weights."""
import numpy as np
import pytest
import torch

import group_wise_affine_unpack_amd as qa
import oracle
import oracle.decoder as od
import synth_inputs as si
from test_gpu_paged_attention import F16_GRAIN, HALF_STEP, Case

pytestmark = pytest.mark.gpu

LAYOUTS = [(64, 32), (64, 64), (96, 32), (128, 32), (128, 64), (128, 128), (192, 32), (192, 64), (256, 32), (256, 64),
           (256, 128)]
SHARES = [1, 4, 5, 8, 12, 20]


def _mark(c):
    """First and last tokens' keys along the query of the first head of each key head, by about log(tokens)."""
    q = oracle.to_f64(c.q, c.act)
    for b, n in enumerate(c.lens):
        for t in {0, int(n) - 1} if n > 0 else ():
            for j in range(c.kvh):
                row = q[b, j * (c.heads // c.kvh)]
                cols = min(c.D, int((np.log(n) + 1.5) / 2.2 * np.sqrt(c.D)))
                at = (c.table[b, t // c.size], j, t % c.size)
                codes = od.codes(c.k[0][at], c.bits)
                codes[:cols] = np.where(row[:cols] > 0, 2**c.bits - 1, 0)
                words = codes.reshape(-1, 32 // c.bits) << (c.bits * np.arange(32 // c.bits))
                c.k[0][at] = words.sum(-1).astype(np.uint32)


def _ref(c, scale=None, window=0, **kw):
    return od.attention_bound(c.q, c.k, c.v, c.act, c.G, c.bits, c.table, c.lens, c.D**-0.5 if scale is None else scale, window,
                              **kw)


def _check(c, out, scale=None, window=0, what="", planted=True):
    ref, bound = _ref(c, scale, window)
    tol = bound * (1 + HALF_STEP[c.act]) + HALF_STEP[c.act] * np.abs(ref) + (F16_GRAIN if c.act == "f16" else 0)
    if planted:
        s = c.D**-0.5 if scale is None else scale
        for name, wrong in (("first", _ref(c, s, window, leave_out=(0,))), ("last", _ref(c, s, window, leave_out=(-1,))),
                            ("scale", _ref(c, 1.05 * s, window))):
            told = (np.abs(wrong[0] - ref) > tol).any(axis=2)  # [sequence, head]
            for b, n in enumerate(c.lens):
                if n > (1 if name == "scale" else 0):
                    assert told[b].any(), f"{name} of sequence {b} would pass"
    err = np.abs(oracle.to_f64(out.view(torch.int16).cpu().numpy().view(np.uint16), c.act) - ref)
    share = float((err / np.where(tol > 0, tol, 1)).max())
    print(f"[parity] {what} err {err.max():.2e}, at most {share:.2f} of the tolerance", flush=True)
    assert (err <= tol).all(), f"{what}: {share} of the tolerance"


def _run(*a, window=0, scale=None, planted=True, **kw):
    print(f"[case] attention bound {a} {kw} window={window}", flush=True)
    c = Case(*a, **kw)
    _mark(c)
    out = qa.paged_attention_affine(*c.args(), scale=scale, window=window)
    torch.cuda.synchronize()
    _check(c, out, scale, window, str(a[1:7]), planted)


def _cases(shift):
    for i, (D, G) in enumerate(LAYOUTS):
        for j, bits in enumerate((2, 4, 8)):
            yield D, G, bits, SHARES[(i + 2 * j + shift) % 6], ("bf16", "f16")[(i + j + shift) % 2]


@pytest.mark.parametrize("D,G,bits,share,act", list(_cases(0)) + list(_cases(3)))
def test_one_launch(D, G, bits, share, act):
    _run([70, 5, 161], 2 * share, 2, D, G, bits, 16, act=act, seed=50)


@pytest.mark.parametrize("D,G,bits,share,act", list(_cases(1)) + list(_cases(4)))
def test_parts(D, G, bits, share, act):
    _run([700, 0, 33, 260], share, 1, D, G, bits, 16, act=act, seed=51, max_pages=160)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 64, 127, 128, 129, 255, 256, 257, 1000, 2559, 2560])
@pytest.mark.parametrize("max_pages", [None, 160])
def test_lengths(n, max_pages):
    _run([n], 4, 2, 128, 64, 4, 16, seed=52, max_pages=max_pages)


@pytest.mark.parametrize("heads,kvh,n,bits,act", [(8, 1, 20000, 4, "bf16"), (2, 2, 9001, 4, "f16"), (16, 2, 6000, 8, "bf16"),
                                                  (5, 1, 7000, 2, "f16")])
def test_long_sequences(heads, kvh, n, bits, act):
    _run([n], heads, kvh, 128, 64, bits, 64, act=act, seed=53)


@pytest.mark.parametrize("q_std", [8.0, 60.0])
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_peaked_softmax(q_std, act):
    # logits in the tens and hundreds: the few tokens that carry weight are not the marked ones
    _run([300, 65], 4, 2, 128, 64, 8, 16, act=act, seed=54, q_std=q_std, planted=False)


def _offset_keys(c, rng, wide, offset):
    """Queries of a wide pair of channels in each group that nearly cancel, and key biases that vary by thousands: the biases'
    part of a logit is a small difference, to which the sums of q have to be known."""
    q = rng.standard_normal(c.q.shape).reshape(*c.q.shape[:2], -1, c.G)
    q[..., 2:] *= wide / 4000
    q[..., 0], q[..., 1] = wide, -wide
    c.q = si.store(q.reshape(c.q.shape).astype(np.float32), c.act)
    b = oracle.to_f64(c.k[2], c.act)
    c.k[2][:] = si.store((b + offset * (1 + 0.3 * rng.standard_normal(b.shape))).astype(np.float32), c.act)


@pytest.mark.parametrize("pages", [None, 160])
@pytest.mark.parametrize("D,G,bits,share,act", [(128, 64, 4, 4, "f16"), (128, 32, 8, 8, "f16"), (64, 32, 2, 12, "f16"),
                                                (256, 128, 4, 1, "f16"), (96, 32, 8, 20, "f16"), (128, 64, 4, 4, "bf16")])
def test_key_biases_far_from_zero(D, G, bits, share, act, pages):
    c = Case([200, 40, 150], share, 1, D, G, bits, 16, act=act, seed=55, max_pages=pages)
    _offset_keys(c, np.random.default_rng(55), 5.0, 3000.0)
    _check(c, qa.paged_attention_affine(*c.args()), what=f"{D} {G} {bits} {share} {act}", planted=False)


def _at(c, b, t):
    return c.table[b, t // c.size], slice(None), t % c.size


def _set_logits(c, b, ts, z):
    """Keys that give the tokens `ts` a logit of about z in every head (of queries above zero)."""
    for t in ts:
        c.k[1][_at(c, b, t)] = 0
        c.k[2][_at(c, b, t)] = si.store(np.full((c.kvh, c.D // c.G), z / (0.8 * np.sqrt(c.D)), np.float32), c.act)


def _set_values(c, b, ts, factor):
    """The value scales of the tokens `ts` (a group each in `factor`, if it has several) times a power of two."""
    for t in ts:
        for part in (1, 2):
            x = oracle.to_f64(c.v[part][_at(c, b, t)], c.act)
            c.v[part][_at(c, b, t)] = si.store((x * np.asarray(factor)).astype(np.float32), c.act)


def _positive_case(lens, share, D, G, bits, act, pages, seed):
    c = Case(lens, share, 1, D, G, bits, 16, act=act, seed=seed, max_pages=pages, scale_spread=0.1)
    c.q = si.store(np.abs(oracle.to_f64(c.q, act)).astype(np.float32), act)
    return c


KINDS = [(128, 64, 4, 4), (128, 32, 8, 8), (64, 32, 2, 12), (256, 128, 4, 1), (256, 32, 2, 4), (96, 32, 8, 20)]


@pytest.mark.parametrize("pages", [None, 160])
@pytest.mark.parametrize("act,far", [("f16", 13), ("bf16", 40)])
@pytest.mark.parametrize("D,G,bits,share", KINDS)
def test_a_large_scale_without_weight(D, G, bits, share, act, far, pages):
    # one token whose value scales stand far above all others and whose logit is far below them: early, in the middle, last
    c = _positive_case([256, 256, 256], share, D, G, bits, act, pages, 56)
    for b, t in enumerate((0, 100, 255)):
        _set_values(c, b, set(range(256)) - {t}, 2.0**-8)
        _set_values(c, b, [t], 2.0**far / 256 if act == "bf16" else 2.0**far)
        _set_logits(c, b, [t], -100.0)
    _check(c, qa.paged_attention_affine(*c.args()), what=f"{D} {G} {bits} {share} {act}", planted=False)


@pytest.mark.parametrize("pages", [None, 160])
@pytest.mark.parametrize("act,far", [("f16", 22), ("bf16", 50)])
@pytest.mark.parametrize("D,G,bits,share", KINDS[:2] + KINDS[4:])
def test_groups_of_scales_far_apart(D, G, bits, share, act, far, pages):
    # every token's weights count in every group, wide or narrow
    c = _positive_case([256, 40, 17], share, D, G, bits, act, pages, 57)
    factor = 2.0**(10 - np.linspace(0, far, D // G))[None]
    for b, n in enumerate(c.lens):
        _set_values(c, b, range(n), factor)
    _check(c, qa.paged_attention_affine(*c.args()), what=f"{D} {G} {bits} {share} {act}", planted=False)


@pytest.mark.parametrize("pages", [None, 160])
@pytest.mark.parametrize("D,G,bits,share", KINDS)
def test_large_scales_whose_weight_is_gone_later(D, G, bits, share, pages):
    # the first tokens' scales are large and lead at their time; then the logits rise by steps
    c = _positive_case([900, 500], share, D, G, bits, "bf16", pages, 58)
    for b, n in enumerate(c.lens):
        _set_values(c, b, range(40), 2.0**30)
        _set_logits(c, b, range(0, 40), -150.0)
        _set_logits(c, b, range(40, n // 3), -75.3)
        _set_logits(c, b, range(n // 3, n // 2), -37.7)
    _check(c, qa.paged_attention_affine(*c.args()), what=f"{D} {G} {bits} {share}", planted=False)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("share", [4, 12])
@pytest.mark.parametrize("pages", [57, 160])
def test_a_value_scale_that_is_not_finite_leaves_other_groups_their_bits(pages, share, bad):
    # among many steps: new powers of two for its group are none for the others
    c = Case([900, 500], share, 1, 128, 32, 4, 16, seed=59, max_pages=pages, scale_spread=2.0)
    q, cache, table, lens = c.args()
    clean = qa.paged_attention_affine(q, cache, table, lens)
    for t in (0, 70, 450, 899):
        cache.v[1][c.table[0, t // 16], 0, t % 16, 1] = bad
    out = qa.paged_attention_affine(q, cache, table, lens)
    assert torch.equal(out[1], clean[1])
    other = [i for i in range(128) if i // 32 != 1]
    assert torch.equal(out[0][:, other], clean[0][:, other])
    assert not torch.isfinite(out[0, :, 32:64]).all()


@pytest.mark.parametrize("act", ["bf16", "f16"])
@pytest.mark.parametrize("D,G,bits,share", KINDS)
@pytest.mark.parametrize("pages", [1, 160])
def test_a_single_token_is_its_value(D, G, bits, share, act, pages):
    # the largest logit's weights are exact: code * scale + bias, with eight roundings of fp32 (products, sums, joins, the
    # quotient) before the one to the type.  Its p is a power of two but for the roundings of its argument z - mu - 30,
    # which the division by p shows where A's rounding has taken them back: with |z| < 98 (base 2) mu, which is z rounded,
    # and -30 - mu are off by at most 2^-18 each and their sum, about -30, by 2^-20: 9 * 2^-20, times log 2 below 7 * 2^-20
    c = Case([1, 1, 1], share, 1, D, G, bits, 16, act=act, seed=63, max_pages=pages)
    out = qa.paged_attention_affine(*c.args())
    torch.cuda.synchronize()
    at = c.table[:, 0], 0, 0
    packed, scales, biases = (t[at] for t in c.v)
    want = od.values(packed, scales, biases, act, G, bits)[:, None]
    size = (od.codes(packed, bits) * np.repeat(np.abs(oracle.to_f64(scales, act)), G, -1)
            + np.repeat(np.abs(oracle.to_f64(biases, act)), G, -1))[:, None]
    got = oracle.to_f64(out.view(torch.int16).cpu().numpy().view(np.uint16), act)
    keys = od.values(*(t[at] for t in c.k), act, G, bits)
    z = np.einsum("bhd,bd->bh", oracle.to_f64(c.q, act), keys) * D**-0.5 / np.log(2)
    assert np.abs(z).max() < 98
    near = (8 * 2.0**-24 + 7 * 2.0**-20) * size
    tol = HALF_STEP[act] * np.abs(want) + near * (1 + HALF_STEP[act]) + (F16_GRAIN if act == "f16" else 0)
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) / tol).max())

"""GPU parity of paged_attention_affine against fp64 (oracle/decoder.py, whose
`bound` derives how far a kernel on integer codes may be off before its
output's rounding; half a step of the output's type comes on top)."""
import numpy as np
import pytest
import torch

import group_wise_affine_unpack_amd as qa
import oracle.decoder as od
import synth_inputs as si
from gpu_util import TORCH_DT, dev16, host_f64, require_gpu

pytestmark = pytest.mark.gpu

HALF_STEP = {"bf16": 2.0**-8, "f16": 2.0**-11}
F16_GRAIN = 2.0**-25


class Case:
    """A cache of quantized normal rows, queries and a table of shuffled pages."""

    def __init__(self, lens, heads, kvh, D, G, bits, size, act="bf16", seed=0, q_std=1.0, spare=2, max_pages=None,
                 scale_spread=0.5):
        self.dev = require_gpu()
        rng = np.random.default_rng((80, seed, D, G, bits, heads))
        self.heads, self.kvh, self.D, self.G, self.bits, self.size, self.act = heads, kvh, D, G, bits, size, act
        self.lens = np.array(lens, np.int32)
        per = max_pages if max_pages is not None else max(1, -(-int(max(self.lens.max(), 1)) // size))
        self.pages = len(lens) * per + spare
        self.table = rng.permutation(self.pages)[:len(lens) * per].reshape(len(lens), per).astype(np.int32)
        self.k, self.v = (self._triple(rng, scale_spread) for _ in range(2))
        self.q = si.store((q_std * rng.standard_normal((len(lens), heads, D))).astype(np.float32), act)

    def _triple(self, rng, spread):
        rows = (self.pages, self.kvh, self.size)
        packed = rng.integers(0, 1 << 32, (*rows, self.D * self.bits // 32), dtype=np.uint32)
        sigma = np.exp(rng.uniform(-spread, spread, (*rows, self.D // self.G)))
        scales = si.store((sigma * 5.5 / (2**self.bits - 1)).astype(np.float32), self.act)
        biases = si.store((-2.75 * sigma + rng.normal(0, 0.2, sigma.shape)).astype(np.float32), self.act)
        return packed, scales, biases

    def cache(self):
        def put(t):
            return (torch.from_numpy(t[0].view(np.int32)).to(self.dev), dev16(t[1], self.act, self.dev),
                    dev16(t[2], self.act, self.dev))
        return qa.AffineKVCache(put(self.k), put(self.v), self.G, self.bits)

    def args(self):
        return (dev16(self.q, self.act, self.dev), self.cache(), torch.from_numpy(self.table).to(self.dev),
                torch.from_numpy(self.lens).to(self.dev))

    def check(self, out, scale=None, window=0, what=""):
        ref, bound = od.paged_attention(self.q, self.k, self.v, self.act, self.G, self.bits, self.table, self.lens,
                                        self.D**-0.5 if scale is None else scale, window)
        err = np.abs(host_f64(out) - ref)
        tol = bound * (1 + HALF_STEP[self.act]) + HALF_STEP[self.act] * np.abs(ref) + (F16_GRAIN if self.act == "f16" else 0)
        worst = float((err - tol).max())
        print(f"[parity] {what} err {err.max():.2e} of tol {tol[err == err.max()].max():.2e}", flush=True)
        assert worst <= 0, f"{what}: {worst} past the bound"
        return ref


def _run(*a, scale=None, window=0, **kw):
    print(f"[case] attention {a} {kw} scale={scale} window={window}", flush=True)
    c = Case(*a, **kw)
    out = qa.paged_attention_affine(*c.args(), scale=scale, window=window)
    torch.cuda.synchronize()
    return c, c.check(out, scale, window, str(a[1:7]))


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513, 1000])
def test_lengths(n):
    _run([n], 4, 2, 128, 64, 4, 16, seed=1)


@pytest.mark.parametrize("D,G", [(64, 32), (64, 64), (96, 32), (128, 32), (128, 64), (128, 128), (192, 32), (192, 64),
                                 (256, 32), (256, 64), (256, 128)])
@pytest.mark.parametrize("bits", [2, 4, 8])
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_head_sizes_groups_widths_types(D, G, bits, act):
    _run([70, 5, 161], 6, 2, D, G, bits, 16, act=act, seed=2)


@pytest.mark.parametrize("D,G", [(64, 32), (64, 64), (96, 32), (128, 32), (128, 64), (128, 128), (192, 32), (192, 64),
                                 (256, 32), (256, 64), (256, 128)])
@pytest.mark.parametrize("bits", [2, 4, 8])
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_head_sizes_groups_widths_types_in_parts(D, G, bits, act):
    # a table of 2560 tokens: sequences cut into parts and joined
    _run([700, 0, 33, 260], 3, 1, D, G, bits, 16, act=act, seed=30, max_pages=160)


@pytest.mark.parametrize("share", [1, 5, 8, 12])
@pytest.mark.parametrize("D,G", [(64, 32), (64, 64), (96, 32), (128, 32), (128, 64), (128, 128), (192, 32), (192, 64),
                                 (256, 32), (256, 64), (256, 128)])
@pytest.mark.parametrize("bits", [2, 4, 8])
def test_head_sizes_groups_widths_at_other_sharings(D, G, bits, share):
    # one launch, and parts; pages outside the cache and windows that begin inside a tile among them
    act = "f16" if (D // G + bits + share) % 2 else "bf16"
    _run([70, 5, 161], 2 * share, 2, D, G, bits, 16, act=act, seed=40, window=50)
    c = Case([700, 0, 33, 260], share, 1, D, G, bits, 16, act=act, seed=41, max_pages=160)
    c.table[0, 3] = -1
    c.table[3, 16] = c.pages
    c.check(qa.paged_attention_affine(*c.args()))


@pytest.mark.parametrize("n", [1, 16, 31, 127, 128, 129, 255, 256, 257, 1000, 2559, 2560])
def test_lengths_in_parts(n):
    _run([n], 4, 2, 128, 64, 4, 16, seed=31, max_pages=160)


@pytest.mark.parametrize("window", [1, 17, 130, 2100, 2400])
def test_windows_in_parts(window):
    _run([1, 20, 130, 901, 2500], 4, 2, 64, 32, 8, 16, act="f16", seed=32, window=window, max_pages=160)


@pytest.mark.parametrize("heads,kvh", [(17, 1), (40, 1), (33, 11)])
def test_head_sharing_in_parts(heads, kvh):
    _run([700, 129], heads, kvh, 64, 64, 4, 32, seed=33, max_pages=80)


@pytest.mark.parametrize("B,n", [(70, 200), (300, 90), (20, 1200), (40, 300)])
def test_batches_at_every_kernel(B, n):
    # more units than CUs, more sequences than lanes, tables of 1024 tokens, of 2048 and past that
    lens = np.random.default_rng(34).integers(0, n, B)
    for pages in (64, 128, 132):
        _run(list(np.minimum(lens, pages * 16)), 2, 2, 64, 64, 4, 16, seed=34, max_pages=pages)


@pytest.mark.parametrize("heads,kvh", [(1, 1), (3, 3), (2, 1), (7, 1), (16, 1), (17, 1), (40, 1), (71, 1), (32, 8), (33, 11)])
def test_head_sharing(heads, kvh):
    _run([37, 90], heads, kvh, 64, 64, 4, 32, seed=3)


@pytest.mark.parametrize("size", [16, 32, 48, 64, 80, 112, 128, 256, 1024])
def test_page_sizes(size):
    _run([1, size - 1, size, size + 1, 3 * size - 7], 4, 1, 64, 32, 8, size, act="f16", seed=4)


def test_ragged_batch_with_empty_rows():
    _run([0, 700, 1, 0, 33, 4, 1999, 0, 16], 8, 2, 128, 64, 4, 16, seed=5)


def test_every_row_empty():
    c, _ = _run([0, 0, 0], 4, 2, 64, 64, 4, 16, seed=6)


def test_a_table_without_pages():
    c = Case([0, 0], 2, 1, 64, 64, 4, 16, seed=37)
    q, cache, table, _ = c.args()
    lens = torch.tensor([5, 0], dtype=torch.int32, device=c.dev)  # more than the table has
    assert (qa.paged_attention_affine(q, cache, table[:, :0], lens) == 0).all()
    assert qa.paged_attention_affine(q[:0], cache, table[:0], lens[:0]).shape == (0, 2, 64)


def test_negative_and_overlong_lengths():
    # less than nothing is nothing; past the table is the whole table
    c = Case([40, 40, 48], 2, 1, 64, 64, 4, 16, seed=7, max_pages=3)
    q, cache, table, _ = c.args()
    out = qa.paged_attention_affine(q, cache, table, torch.tensor([-5, 40, 10**9], dtype=torch.int32, device=c.dev))
    c.lens = np.array([0, 40, 48], np.int32)
    c.check(out)


@pytest.mark.parametrize("window", [1, 2, 16, 31, 100, 128, 500, 10**12, 2**63 - 1])
def test_windows(window):
    _run([1, 20, 130, 500, 901], 4, 2, 128, 64, 4, 16, seed=8, window=window)


@pytest.mark.parametrize("heads,kvh,n", [(8, 1, 20000), (2, 2, 9001), (16, 2, 6000)])
def test_long_sequences(heads, kvh, n):
    # split over the length and joined
    _run([n], heads, kvh, 128, 64, 4, 64, seed=9)


def test_long_and_short_sequences_together():
    _run([15000, 3, 0, 500, 1] + [40] * 20, 4, 1, 64, 64, 8, 16, act="f16", seed=10, max_pages=950)


@pytest.mark.parametrize("B", [1, 2, 65, 300])
def test_batches(B):
    lens = np.random.default_rng(11).integers(0, 60, B)
    _run(list(lens), 2, 1, 64, 64, 4, 16, seed=11)


@pytest.mark.parametrize("q_std", [8.0, 60.0])
@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_peaked_softmax(q_std, act):
    # logits in the tens and hundreds: one token takes nearly all
    _run([300, 65], 4, 2, 128, 64, 8, 16, act=act, seed=12, q_std=q_std)


@pytest.mark.parametrize("scale", [0.0, 1e-3, 1.0, -0.125])
def test_scales(scale):
    _run([100], 2, 1, 64, 64, 4, 16, seed=13, scale=scale)


def test_logits_that_vanish():
    # queries and a scale whose product is below every fp32: all tokens alike, those of a tile's rest still hidden
    c = Case([37, 64], 2, 1, 64, 64, 4, 16, seed=38)
    c.q = si.store((1e-38 * np.random.default_rng(38).standard_normal((2, 2, 64))).astype(np.float32), "bf16")
    c.check(qa.paged_attention_affine(*c.args(), scale=1e-29), 1e-29)


@pytest.mark.parametrize("pages", [8, 160])
def test_rows_past_4_gib(pages):
    # the same rows in a cache whose code and parameter arrays have them past byte 2^32 (one launch, and parts)
    c = Case([120, 33], 4, 2, 128, 32, 2, 16, seed=39, max_pages=pages)
    q, small, table, lens = c.args()
    base = (1 << 32) // (2 * 16 * 8)  # scales: 2 heads of 16 rows of 4 groups, 2 bytes each
    dev = q.device
    triples = []
    for t in (small.k, small.v):
        new = [torch.empty((base + c.pages, *a.shape[1:]), dtype=a.dtype, device=dev) for a in t]
        for n, a in zip(new, t):
            n[base:] = a
        triples.append(new)
    big = qa.AffineKVCache(*triples, 32, 2)
    out = qa.paged_attention_affine(q, big, table + base, lens)
    assert torch.equal(out, qa.paged_attention_affine(q, small, table, lens))
    c.check(out)


def test_value_scales_over_many_decades():
    # groups whose scales differ by 2^12 either way, the wide ones late and early
    _run([400, 57], 4, 1, 128, 64, 8, 16, seed=14, scale_spread=4.0)


def test_scales_below_zero_and_of_zero():
    # a caller's own cache: flipped groups, constant ones
    c = Case([200, 31], 4, 1, 128, 64, 4, 16, seed=36)
    rng = np.random.default_rng(36)
    for t in (c.k, c.v):
        t[1][rng.random(t[1].shape) < 0.3] ^= 0x8000
        t[1][rng.random(t[1].shape) < 0.1] = 0
    c.check(qa.paged_attention_affine(*c.args()))
    c.v[1][:] = 0
    c.check(qa.paged_attention_affine(*c.args()))


@pytest.mark.parametrize("pos", ["first", "last"])
@pytest.mark.parametrize("n", [1, 16, 31, 64, 129, 700])
def test_the_outermost_tokens_count(pos, n):
    # one token's key is the query itself and its value is far from the others: leaving it out, or taking
    # the slot beside it in, changes the output at once
    c = Case([n], 2, 1, 64, 64, 8, 16, act="f16", seed=15)
    t = 0 if pos == "first" else n - 1
    at = (c.table[0, t // 16], 0, t % 16)
    q = np.tile(np.where(np.arange(64) % 2, 6.0, -6.0), (1, 2, 1)).astype(np.float32)
    c.q = si.f16_bits(q)
    for x, arrays in ((q[0, 0], c.k), (np.linspace(90, 100, 64, dtype=np.float32), c.v)):
        w, s, b = od.quantize_rows(si.f16_bits(x[None]), "f16", 64, 8)
        arrays[0][at], arrays[1][at], arrays[2][at] = w[0], s[0], b[0]
    out = qa.paged_attention_affine(*c.args())
    ref = c.check(out)
    assert (ref > 80).all()


@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -3e38])
@pytest.mark.parametrize("pages", [6, 160])
def test_slots_that_no_sequence_sees_have_no_influence(poison, pages):
    # past the length in the last page, ahead of the window, in other pages
    c = Case([37, 0, 90], 4, 2, 64, 32, 4, 16, seed=16, max_pages=pages)
    q, cache, table, lens = c.args()
    for window in (0, 20):
        clean = qa.paged_attention_affine(q, cache, table, lens, window=window)
        seen = torch.zeros((c.pages, c.size), dtype=torch.bool)
        for b, n in enumerate(c.lens):
            for t in range(max(0, n - window) if window else 0, n):
                seen[c.table[b, t // 16], t % 16] = True
        other = c.cache()
        hide = (~seen).to(c.dev)[:, None, :, None]
        for t in other.k[1:] + other.v[1:]:
            t.masked_fill_(hide, poison)
        assert torch.equal(qa.paged_attention_affine(q, other, table, lens, window=window), clean)


@pytest.mark.parametrize("pages", [7, 160])
def test_table_entries_outside_the_cache_are_left_out(pages):
    c = Case([100, 64, 40], 4, 2, 64, 64, 4, 16, seed=17, max_pages=pages)
    c.table[0, 2], c.table[0, 6] = -1, c.pages
    c.table[1, :4] = [2**31 - 1, -2**31, c.pages + 5, -7]   # nothing left: zeros
    c.table[2, 0] = -3
    out = qa.paged_attention_affine(*c.args())
    ref = c.check(out)
    assert (ref[1] == 0).all() and (host_f64(out)[1] == 0).all()


def test_shared_pages_and_table_rows():
    # two sequences of one prompt: the same pages, and one table row for both (a row stride of 0)
    c = Case([50, 64], 2, 1, 64, 64, 4, 16, seed=18)
    c.table[1] = c.table[0]
    q, cache, table, lens = c.args()
    out = qa.paged_attention_affine(q, cache, table[:1].expand(2, -1), lens)
    c.check(out)


def test_strided_queries_and_tables():
    c = Case([50, 20, 7], 4, 2, 64, 64, 4, 16, seed=19)
    q, cache, table, lens = c.args()
    wide = torch.full((3, 8, 72), 5.0, dtype=torch.bfloat16, device=c.dev)
    wide[:, 2:6, 8:] = q
    tw = torch.full((3, table.shape[1] + 3), 10**6, dtype=torch.int32, device=c.dev)
    tw[:, :-3] = table
    out = torch.empty((3, 4, 64), dtype=torch.bfloat16, device=c.dev)
    got = qa.paged_attention_affine(wide[:, 2:6, 8:], cache, tw[:, :-3], lens, out=out)
    assert got is out
    assert torch.equal(out, qa.paged_attention_affine(q, cache, table, lens))
    c.check(out)


@pytest.mark.parametrize("act", ["bf16", "f16"])
def test_queries_at_the_ends_of_their_range(act):
    # zeros, subnormals, and values near the largest, with a scale that brings the logits back
    c = Case([60] * 4, 2, 1, 64, 64, 8, 16, act=act, seed=20)
    big = 3e38 if act == "bf16" else 65504.0
    x = np.random.default_rng(20).standard_normal((4, 2, 64)).astype(np.float32)
    x[0] = 0
    x[1] *= 1e-39 if act == "bf16" else 1e-7
    x[2] = np.clip(x[2], -1, 1) * big
    c.q = si.store(x, act)
    args = c.args()
    for i, scale in ((0, 0.125), (1, 1e29 if act == "bf16" else 1e6), (2, 1e-30 if act == "bf16" else 1e-5), (3, 0.125)):
        if act == "bf16" and i == 2:
            continue  # sums of such products pass fp32; the scale comes after them
        out = qa.paged_attention_affine(*args, scale=scale)
        ref, bound = od.paged_attention(c.q[i:i + 1], c.k, c.v, act, c.G, c.bits, c.table[i:i + 1], c.lens[i:i + 1], scale)
        err = np.abs(host_f64(out)[i] - ref[0])
        assert (err <= bound[0] * 1.01 + HALF_STEP[act] * np.abs(ref[0]) + F16_GRAIN).all(), (i, err.max())


@pytest.mark.parametrize("pages", [3, 160])
def test_nan_in_a_seen_row_stays_with_its_sequence(pages):
    c = Case([40, 40], 2, 1, 64, 64, 4, 16, seed=21, max_pages=pages)
    q, cache, table, lens = c.args()
    clean = qa.paged_attention_affine(q, cache, table, lens)
    cache.k[1][c.table[0, 1], 0, 3] = float("nan")
    out = qa.paged_attention_affine(q, cache, table, lens)
    assert torch.isnan(out[0]).all() and torch.equal(out[1], clean[1])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("what", [1, 2])
def test_a_value_group_that_is_not_finite_stays_with_its_columns(bad, what):
    c = Case([40, 40], 2, 1, 128, 64, 4, 16, seed=35)
    q, cache, table, lens = c.args()
    clean = qa.paged_attention_affine(q, cache, table, lens)
    cache.v[what][c.table[0, 1], 0, 3, 1] = bad
    out = qa.paged_attention_affine(q, cache, table, lens)
    assert torch.equal(out[0, :, :64], clean[0, :, :64]) and torch.equal(out[1], clean[1])
    assert not torch.isfinite(out[0, :, 64:]).any() if what == 2 else not torch.isfinite(out[0, :, 64:]).all()


def test_same_call_same_bits_and_the_batch_does_not_matter():
    c = Case([3000, 17, 900], 8, 2, 128, 64, 4, 16, seed=22)  # in parts
    args = c.args()
    a = qa.paged_attention_affine(*args)
    for _ in range(3):
        assert torch.equal(qa.paged_attention_affine(*args), a)


@pytest.mark.parametrize("pages", [57, 160])  # one launch; parts and their join
def test_graph_replays_follow_new_lengths(pages):
    c = Case([900, 40, 0], 8, 2, 128, 64, 4, 16, seed=23, max_pages=pages)
    q, cache, table, lens = c.args()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        qa.paged_attention_affine(q, cache, table, lens)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = qa.paged_attention_affine(q, cache, table, lens)
        for new in ([900, 40, 0], [1, 899, 300], [0, 0, 0], [512, 512, 512]):
            lens.copy_(torch.tensor(new, dtype=torch.int32))
            g.replay()
            torch.cuda.synchronize()
            eager = qa.paged_attention_affine(q, cache, table, lens)
            torch.cuda.synchronize()
            assert torch.equal(out, eager), new
    c.lens = np.array([512] * 3, np.int32)
    c.check(out)


def test_two_streams_at_once():
    cases = [Case([2500, 800], 8, 2, 128, 64, 4, 16, seed=24 + i) for i in range(2)]
    args = [c.args() for c in cases]
    refs = [qa.paged_attention_affine(*a) for a in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(qa.paged_attention_affine(*args[i]))
    torch.cuda.synchronize()
    for ref, got in zip(refs, outs):
        assert all(torch.equal(o, ref) for o in got)


def test_python_refusals():
    c = Case([20], 4, 2, 64, 64, 4, 16, seed=26)
    q, cache, table, lens = c.args()
    for bad in ((q[..., :32], cache, table, lens), (q.half(), cache, table, lens), (q, cache, table.long(), lens),
                (q, cache, table, lens.long()), (q, cache, table.repeat(2, 1), lens), (q, cache, table, lens.cpu())):
        with pytest.raises(ValueError):
            qa.paged_attention_affine(*bad)
    for kw in (dict(window=-1), dict(scale=float("nan"))):
        with pytest.raises(qa.QaffError):
            qa.paged_attention_affine(q, cache, table, lens, **kw)
    with pytest.raises(qa.QaffError):
        qa.paged_attention_affine(q[:, :3], cache, table, lens)

"""GPU tests of kv_pages_assign and kv_pages_trim against the oracle's token
by token definition: every output, the whole table (and what lies beside it),
the whole stack and the pool's words, bit for bit."""
import numpy as np
import pytest
import torch

import group_wise_affine_unpack_amd as qa
import oracle.decoder as od
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


class Batch:
    """A pool and a table in which sequences of the given lengths already hold pages."""

    def __init__(self, lens, per, page, spare, dev, seed=0, pad=3):
        rng = np.random.default_rng(seed)
        self.page, self.B, self.per = page, len(lens), per
        had = [min(-(-max(n, 0) // page), per) for n in lens]
        self.pages = max(1, sum(had) + spare)
        order = rng.permutation(self.pages).astype(np.int32)
        self.wide = np.full((self.B, per + pad), -7, np.int32)  # the table is a slice of it
        at = 0
        for b, h in enumerate(had):
            self.wide[b, :h] = order[at:at + h]
            at += h
        self.free = np.full(self.pages, -9, np.int32)
        self.free[:self.pages - at] = order[at:]
        self.count = self.pages - at
        self.lens = np.array(lens, np.int32)
        self.pool = qa.KVPagePool(self.pages, page, dev)
        self.pool.free_pages.copy_(torch.from_numpy(self.free))
        self.pool.state[0] = self.count
        self.wide_d = torch.from_numpy(self.wide).to(dev)
        self.table = self.wide_d[:, :per]
        self.lens_d = torch.from_numpy(self.lens).to(dev)
        self.dev = dev

    def assign(self, news, T, in_place=False):
        """One assign on both sides; checks everything."""
        news = np.array(news, np.int32)
        got = qa.kv_pages_assign(self.pool, self.table, self.lens_d, torch.from_numpy(news).to(self.dev), T,
                                 lens_out=self.lens_d if in_place else None)
        torch.cuda.synchronize()
        table, slots, positions, ids, lens, count, short = od.pages_assign(self.wide[:, :self.per], self.lens, news, self.free,
                                                                          self.count, self.page, self.pages, T)
        for name, g, want in zip(("slots", "positions", "seq_ids", "lens"), got, (slots, positions, ids, lens)):
            assert np.array_equal(g.cpu().numpy(), want), name
        self.wide[:, :self.per], self.count, self.lens, self.lens_d = table, count, lens, got[3]
        self.check(short)
        return got

    def trim(self, keep, in_place=False):
        keep = np.array(keep, np.int32)
        got = qa.kv_pages_trim(self.pool, self.table, self.lens_d, torch.from_numpy(keep).to(self.dev),
                               lens_out=self.lens_d if in_place else None)
        torch.cuda.synchronize()
        short = int(self.pool.state[1])
        table, self.free, self.lens, self.count = od.pages_trim(self.wide[:, :self.per], self.lens, keep, self.free, self.count,
                                                                self.page, self.pages)
        self.wide[:, :self.per] = table
        assert np.array_equal(got.cpu().numpy(), self.lens)
        self.lens_d = got
        self.check(short)

    def check(self, short):
        assert np.array_equal(self.wide_d.cpu().numpy(), self.wide), "table"
        assert np.array_equal(self.pool.free_pages.cpu().numpy(), self.free), "free pages"
        assert self.pool.state.tolist() == [self.count, short, 0, 0]


@pytest.mark.parametrize("B,page,most,new", [(1, 16, 0, 1), (1, 16, 517, 1), (1, 64, 63, 130), (2, 48, 100, 47), (7, 16, 40, 33),
                                             (64, 64, 8000, 5), (65, 32, 300, 64), (300, 128, 2000, 9), (1025, 16, 50, 3),
                                             (4096, 16, 90, 2), (3, 16, 10, 30000)])
def test_assign_then_trim_back(B, page, most, new):
    dev = require_gpu()
    print(f"[case] pages B={B} page={page} lens<={most} new<={new}", flush=True)
    rng = np.random.default_rng((B, page, most))
    lens = rng.integers(0, most + 1, B)
    lens[0] = most
    news = rng.integers(0, new + 1, B)
    news[-1] = new
    per = -(-(most + new) // page) + 1
    x = Batch(lens, per, page, sum(-(-n // page) + 1 for n in news.tolist()), dev, seed=B)
    before = (x.wide.copy(), x.free.copy(), x.count)
    x.assign(news, int(news.sum()) + 5)
    x.trim(lens)
    known = np.arange(len(x.free)) < x.count
    assert x.count == before[2] and np.array_equal(x.free[known], before[1][known])
    fresh = x.wide[:, :per] == -1  # entries that were handed out in between; the others are what they were
    assert np.array_equal(np.where(fresh, 0, x.wide[:, :per]), np.where(fresh, 0, before[0][:, :per]))


def test_growing_and_shrinking_in_place():
    # many steps on one pool, lengths and pool updated in place, some sequences ended and refilled
    dev = require_gpu()
    rng = np.random.default_rng(3)
    x = Batch([0] * 9, 12, 16, 60, dev)
    for step in range(40):
        print(f"[case] step {step}", flush=True)
        if step % 3 == 2:
            x.trim(np.where(rng.random(9) < 0.3, 0, rng.integers(0, 200, 9)), in_place=True)
        else:
            x.assign(rng.integers(0, 30, 9), 9 * 30, in_place=True)
    held = x.wide[:, :12][np.arange(12) < -(-x.lens // 16)[:, None]]
    assert sorted(held.tolist() + x.free[:x.count].tolist()) == list(range(x.pages))  # no page lost or held twice


@pytest.mark.parametrize("spare", [0, 1, 2, 5, 9])
def test_pool_runs_dry(spare):
    # the sequences before the end of the stack keep their pages, those behind it their partly filled ones
    dev = require_gpu()
    x = Batch([5, 16, 0, 31, 7], 6, 16, spare, dev)
    x.assign([40, 1, 20, 1, 3], 70)
    x.assign([1, 1, 1, 1, 1], 5)


def test_lengths_outside_the_table_and_rows_cut():
    dev = require_gpu()
    x = Batch([30, 64, -5, 1000, 63], 4, 16, 20, dev)  # a table of 64 tokens a sequence
    x.assign([100, 3, 10, 4, 2], 130)   # past the capacity: rows without slots
    x = Batch([3, 3, 3], 4, 16, 20, dev)
    x.assign([20, 20, 20], 31)          # fewer rows than tokens
    x = Batch([3, 3, 3], 4, 16, 20, dev)
    x.assign([-4, 2, -(2**31)], 4)      # negative counts for none
    x.assign([2**31 - 1, 2**31 - 1, 5], 50)


def test_nothing_to_do():
    dev = require_gpu()
    x = Batch([17, 3], 3, 16, 4, dev)
    x.assign([0, 0], 0)
    x.assign([0, 0], 9)
    x.trim([17, 9])
    empty = torch.zeros((0, 3), dtype=torch.int32, device=dev)
    none = torch.zeros(0, dtype=torch.int32, device=dev)
    slots, positions, ids, lens = qa.kv_pages_assign(x.pool, empty, none, none, 3)
    assert slots.tolist() == [-1] * 3 and positions.tolist() == [0] * 3 and ids.tolist() == [-1] * 3 and lens.shape == (0,)
    qa.kv_pages_trim(x.pool, empty, none, none)
    x.check(0)


def test_bad_entries_are_dropped():
    # entries and free pages outside the cache give no slots, and do not return to the stack
    dev = require_gpu()
    x = Batch([20, 20], 4, 16, 6, dev)
    x.wide[0, 1] = 10**6
    x.wide_d.copy_(torch.from_numpy(x.wide))
    x.free[x.count - 1] = -3
    x.pool.free_pages.copy_(torch.from_numpy(x.free))
    x.assign([14, 14], 28)
    x.trim([0, 0])
    # counts outside the stack are cut
    x.pool.state[0] = 10**6
    x.count = x.pages
    x.free[:] = np.arange(x.pages)
    x.pool.free_pages.copy_(torch.from_numpy(x.free))
    x.assign([3, 3], 6)
    # the same pages returned twice stop at the stack's end
    y = Batch([64, 64], 4, 16, 0, dev)
    y.pool.state[0] = y.count = 5
    y.trim([0, 0])
    assert y.count == y.pages


def test_captured_step_follows_its_replays():
    # one captured assign whose lengths, table and pool go on from replay to replay, against the oracle
    dev = require_gpu()
    x = Batch([3, 0, 40], 8, 16, 15, dev)
    news = torch.ones(3, dtype=torch.int32, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            slots, positions, ids, _ = qa.kv_pages_assign(x.pool, x.table, x.lens_d, news, 1000, lens_out=x.lens_d)
        for i in range(8):
            n = np.array([1 + i, 16 - 2 * i, 3], np.int32)
            news.copy_(torch.from_numpy(n))
            graph.replay()
            torch.cuda.synchronize()
            table, want, pos, want_ids, x.lens, x.count, short = od.pages_assign(x.wide[:, :8], x.lens, n, x.free, x.count, 16,
                                                                                x.pages, 1000)
            x.wide[:, :8] = table
            assert np.array_equal(slots.cpu().numpy(), want) and np.array_equal(positions.cpu().numpy(), pos)
            assert np.array_equal(ids.cpu().numpy(), want_ids) and np.array_equal(x.lens_d.cpu().numpy(), x.lens)
            x.check(short)


def test_two_pools_on_two_streams():
    dev = require_gpu()
    pools = [Batch([11 * i % 70 for i in range(64)], 40, 16, 3000, dev, seed=i) for i in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    news = torch.full((64,), 500, dtype=torch.int32, device=dev)
    got = []
    for x, s in zip(pools, streams):
        with torch.cuda.stream(s):
            got.append(qa.kv_pages_assign(x.pool, x.table, x.lens_d, news, 32100))
    torch.cuda.synchronize()
    for x, g in zip(pools, got):
        want = od.pages_assign(x.wide[:, :40], x.lens, np.full(64, 500, np.int32), x.free, x.count, 16, x.pages, 32100)
        x.wide[:, :40], x.count = want[0], want[5]
        for a, b in zip(g, want[1:5]):
            assert np.array_equal(a.cpu().numpy(), b)
        x.check(want[6])


def test_more_rows_than_a_pass_of_the_grid():
    # 512 workgroups of 256 rows at most: beyond 131072 rows each goes round again
    dev = require_gpu()
    x = Batch([5, 0, 33], 12600, 16, 20000, dev)
    x.assign([200000, 3, 100000], 300001, in_place=True)  # (and two rows cut)
    x.trim([5, 0, 33], in_place=True)

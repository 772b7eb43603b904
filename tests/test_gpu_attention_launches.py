"""What the header says of paged_attention_affine's launches: up to 160 tokens
(of the window, or of the table) a call is one launch without scratch, so it
may be captured on a stream that has never run one."""
import pytest
import torch

import group_wise_affine_unpack_amd as qa
from test_gpu_paged_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,G,bits", [(256, 64, 8), (256, 32, 4), (192, 64, 8), (128, 64, 4), (64, 32, 2)])
@pytest.mark.parametrize("window,pages", [(1, 40), (145, 40), (146, 40), (160, 40), (0, 10), (10**6, 10)])
def test_short_calls_are_captured_without_an_eager_one(D, G, bits, window, pages):
    c = Case([pages * 16, 3], 4, 1, D, G, bits, 16, seed=60, max_pages=pages)
    args = c.args()
    eager = qa.paged_attention_affine(*args, window=window)  # (on the default stream)
    torch.cuda.synchronize()
    qa.release_workspaces()
    out = torch.empty_like(eager)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        qa.paged_attention_affine(*args, window=window, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
    assert qa.release_workspaces() == 0


def test_the_largest_batch():
    # 65535 sequences: one launch, and shares of the line with a join over all of them (a table of more than 2048 tokens)
    c = Case([32, 1, 17, 0, 29], 4, 2, 64, 64, 4, 16, seed=61, max_pages=2)
    q, cache, table, lens = c.args()
    B = 65535
    at = torch.arange(B, device=c.dev) % 5
    few = qa.paged_attention_affine(q, cache, table, lens)
    long = torch.full((5, 130), -1, dtype=torch.int32, device=c.dev)
    long[:, :2] = table
    for t in (table, long):
        out = qa.paged_attention_affine(q[at], cache, t[at], lens[at])
        torch.cuda.synchronize()
        assert torch.equal(out, few[at])
    with pytest.raises(qa.QaffError):
        qa.paged_attention_affine(q[torch.arange(B + 1, device=c.dev) % 5], cache, table[torch.arange(B + 1, device=c.dev) % 5],
                                  lens[torch.arange(B + 1, device=c.dev) % 5])


@pytest.mark.parametrize("pages", [3, 160])
def test_queries_shared_by_heads_and_sequences(pages):
    # strides of 0: one query for all heads, or for all sequences
    c = Case([48, 33, 5], 8, 2, 64, 64, 4, 16, seed=62, max_pages=pages)
    q, cache, table, lens = c.args()
    for view in (q[:, :1].expand(3, 8, 64), q[:1].expand(3, 8, 64), q[:1, :1].expand(3, 8, 64)):
        assert torch.equal(qa.paged_attention_affine(view, cache, table, lens),
                           qa.paged_attention_affine(view.contiguous(), cache, table, lens))

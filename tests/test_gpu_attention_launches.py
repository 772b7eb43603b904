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

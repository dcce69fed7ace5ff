"""Vocabulary slices in the larger sort, whose later positions hold the tokens of
other slices: runs split in pieces, and pieces added up once more, end at the
slice's last token."""
import pytest
import torch

import gpu_helpers as G
from linear_cross_entropy_tile_amd import flce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["hv", "vh"])
@pytest.mark.parametrize("hot", [0, 95, 96, 202])
def test_slices_of_a_large_batch(layout, hot):
    """Whole numbers, so that every sum is exact: the slices' gradients are the
    whole one's columns, beside an id that fills most of the batch."""
    N, H, V, cuts = 40000, 24, 203, (0, 96, 97, 203)
    g = torch.Generator(device="cuda")
    g.manual_seed(hot)
    tok = torch.randint(0, V, (N,), generator=g, device=G.dev())
    tok[torch.rand(N, generator=g, device=G.dev()) < 0.8] = hot
    tok[::9] = -100
    up = torch.randint(-3, 4, (N, H), generator=g, device=G.dev()).float()
    on = tok >= 0
    want = torch.zeros(V, H, device=G.dev()).index_add_(0, tok[on], up[on])
    w = torch.randn(V, H, generator=g, device=G.dev()).to(torch.bfloat16)
    for b, e in zip(cuts[:-1], cuts[1:]):
        got = flce.embedding_backward(up, tok, e - b, layout=layout, v_begin=b, v_total=V,
                                      grad_dtype="f32")
        assert torch.equal(got if layout == "vh" else got.t(), want[b:e])
        part = w[b:e] if layout == "vh" else w[b:e].t().contiguous()
        out = flce.embedding(part, tok, layout=layout, v_begin=b, v_total=V)["hidden"]
        mine = ((tok >= b) & (tok < e))[:, None]
        assert torch.equal(out, torch.where(mine, w[tok.clamp(min=0)], 0.0))

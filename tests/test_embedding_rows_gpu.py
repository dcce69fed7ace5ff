"""Bits that the embedding leaves or writes beside its values: zero rows are +0
whatever the scale."""
import numpy as np
import pytest
import torch

import gpu_helpers as G
from linear_cross_entropy_tile_amd import flce

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["hv", "vh"])
@pytest.mark.parametrize("N,H", [(7, 8), (40, 2304), (2500, 72), (9000, 136), (9000, 2048)])
@pytest.mark.parametrize("scale", [-0.5, -1.0, 1.0, 3.0])
def test_zero_rows_are_positive_zeros(N, H, scale, layout):
    """Ignored tokens, ids outside the vocabulary and ids of other slices; a zero
    of the weight keeps the sign that its product with the scale has."""
    V, v_begin, v_total = 24, 16, 60
    rng = np.random.default_rng(N + H)
    tok = rng.integers(v_begin, v_begin + V, N)
    tok[::5], tok[1::5], tok[2::5], tok[3::5] = -100, v_total + 3, 2, 59
    w = torch.randn(V, H).to(torch.bfloat16)
    w[:, ::2] = 0.0
    wd = (w if layout == "vh" else w.t().contiguous()).to(G.dev())
    got = flce.embedding(wd, torch.from_numpy(tok).to(G.dev()), layout=layout, scale=scale,
                         v_begin=v_begin, v_total=v_total)["hidden"].cpu().view(torch.int16)
    on = torch.from_numpy((tok >= v_begin) & (tok < v_begin + V))
    assert not bool(got[~on].any())
    rows = w[torch.from_numpy(tok - v_begin)[on]]
    want = (rows.float() * scale).to(torch.bfloat16)
    assert torch.equal(got[on], want.view(torch.int16))

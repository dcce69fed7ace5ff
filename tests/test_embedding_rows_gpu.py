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


@pytest.mark.parametrize("layout", ["hv", "vh"])
@pytest.mark.parametrize("V", [1, 70, 72, 203, 640])
@pytest.mark.parametrize("hidden", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_accumulation_stores_to_used_ids_only(V, hidden, dtype, layout):
    """Ids that no token has hold signalling NaN: any arithmetic on their values,
    and so any store but one of the same bits, would change them. Used ids alone,
    in pairs, in whole groups of eight, and at the borders of the strips of 64."""
    H, N = 264, 500
    rng = np.random.default_rng(V)
    used = np.zeros(V, bool)
    used[::11] = True
    used[[i for i in (8, 9, 62, 63, 64, 65, 127, 128) if i < V]] = True
    used[16:24] = True
    used[V - 1] = True
    if V > 400:
        used[192:256] = True
        used[320:384] = False
    ids = np.nonzero(used)[0]
    tok = np.concatenate([ids, rng.choice(ids, N)])
    tok[1::7] = -100
    used = np.isin(np.arange(V), tok)
    view, signal = ((torch.int16, 0x7F81) if dtype == torch.bfloat16 else (torch.int32, 0x7F800001))
    base = torch.from_numpy(rng.integers(-8, 9, (V, H)).astype(np.float32)).to(dtype)
    base.view(view)[torch.from_numpy(~used)] = signal
    g = torch.from_numpy(rng.integers(-2, 3, (tok.size, H)).astype(np.float32)).to(hidden)
    acc = (base if layout == "vh" else base.t().contiguous()).to(G.dev())
    flce.embedding_backward(g.to(G.dev()), torch.from_numpy(tok).to(G.dev()), V, layout=layout,
                            grad_weight=acc)
    got = (acc if layout == "vh" else acc.t().contiguous()).cpu()
    want = base.clone()
    for v in np.nonzero(used)[0]:  # whole numbers below 2^8 in every partial sum: exact
        want[v] += g[torch.from_numpy(tok == v)].float().sum(0).to(dtype)
    assert torch.equal(got.view(view), want.view(view))


@pytest.mark.parametrize("layout", ["hv", "vh"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_two_streams_add_to_neighbouring_ids(dtype, layout):
    """Two batches without a common id, alternating within every strip and every
    group of 16 bytes, added on two streams at once to one tensor."""
    N, H, V = 20000, 512, 4000
    dev = G.dev()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    base = torch.randint(-8, 9, (V, H) if layout == "vh" else (H, V), generator=gen, device=dev)
    acc = base.to(dtype)
    toks = [2 * torch.randint(0, V // 2, (N,), generator=gen, device=dev) + k for k in (0, 1)]
    ups = [torch.randint(-1, 2, (N, H), generator=gen, device=dev).to(torch.bfloat16)
           for _ in toks]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for s, tok, up in zip(streams, toks, ups):
        with torch.cuda.stream(s):
            flce.embedding_backward(up, tok, V, layout=layout, grad_weight=acc)
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    want = torch.zeros(V, H, device=dev)
    for tok, up in zip(toks, ups):  # whole numbers far below 2^8: exact
        want.index_add_(0, tok, up.float())
    want = base + (want if layout == "vh" else want.t())
    assert want.abs().max() < 256
    assert torch.equal(acc.float(), want)

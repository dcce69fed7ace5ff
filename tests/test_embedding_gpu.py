"""The embedding lookup and its gradient on the GPU against plain computations.

Tolerances. Lookup: bit for bit the fp32 product rounded to bf16 by torch.
Gradient: a sum of n fp32 terms in any order is off by at most (n - 1) 2^-24
times the sum of their magnitudes (to first order), the product with the scale
by 2^-24, and the result's rounding by 2^-8 (bf16) or 2^-24 (fp32) of its value;
accumulation adds one more fp32 rounding of the sum."""
import numpy as np
import pytest
import torch

import gpu_helpers as G
from oracle import operators_oracle as O
from linear_cross_entropy_tile_amd import flce, function

pytestmark = pytest.mark.gpu

HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _tokens(rng, N, V, kind):
    if kind == "same":
        t = np.full(N, V // 2)
    elif kind == "hot":  # a few ids with long runs among rare ones
        t = np.where(rng.random(N) < 0.7, rng.integers(0, min(V, 3), N), rng.integers(0, V, N))
    else:
        t = rng.integers(0, V, N)
    t = t.astype(np.int64)
    if kind == "holes" and N:
        t[rng.random(N) < 0.3] = -100
        t[rng.random(N) < 0.1] = V + 3
        t[rng.random(N) < 0.1] = -7
    return t


def _weight(rng, H, V, layout):
    w = torch.from_numpy(rng.standard_normal((V, H)).astype(np.float32)).to(torch.bfloat16)
    return (w if layout == "vh" else w.t().contiguous()).to(G.dev()), w


def _status(ws):
    return flce.flce_get_status(ws.data_ptr(), torch.cuda.current_stream().cuda_stream)


FORWARD = [(0, 8, 5, "all"), (1, 8, 1, "all"), (1, 2304, 1001, "all"), (31, 72, 7, "holes"),
           (300, 64, 999, "holes"), (511, 200, 640, "all"), (512, 200, 641, "holes"),
           (1025, 136, 4096, "hot"), (4100, 64, 777, "holes"), (9000, 40, 5000, "hot"),
           (16384, 8, 70000, "all"), (20001, 24, 300, "holes"), (33000, 16, 300000, "holes"),
           (700, 4104, 513, "holes"), (2047, 136, 600, "hot"), (2048, 136, 601, "holes"),
           (3000, 72, 4000, "all")]


@pytest.mark.parametrize("layout", ["hv", "vh"])
@pytest.mark.parametrize("N,H,V,kind", FORWARD)
def test_lookup(N, H, V, kind, layout):
    rng = np.random.default_rng(N + H + V)
    tok = _tokens(rng, N, V, kind)
    w, table = _weight(rng, H, V, layout)
    t = torch.from_numpy(tok).to(G.dev())
    keep = (tok >= 0) & (tok < V)
    for scale in (1.0, 13.856, -0.5):
        ws = torch.full((1 << 16,), 255, dtype=torch.uint8, device=G.dev())
        out = flce.embedding(w, t, layout=layout, scale=scale, workspace=ws)
        want = torch.zeros(N, H, dtype=torch.bfloat16)
        want[torch.from_numpy(keep)] = (table[torch.from_numpy(tok[keep])].float()
                                        * torch.tensor(scale)).to(torch.bfloat16)
        assert torch.equal(out["hidden"].cpu(), want), f"scale {scale}"
        assert _status(out["workspace"]) == int(((tok != -100) & ~keep).sum())


@pytest.mark.parametrize("layout", ["hv", "vh"])
def test_lookup_keeps_special_values(layout):
    H, V = 16, 24
    w = torch.randn(V, H).to(torch.bfloat16)
    w[3] = float("inf")
    w[4] = float("nan")
    w[5] = -0.0
    tok = torch.tensor([3, 4, 5, 4, -100, 23])
    wd = (w if layout == "vh" else w.t().contiguous()).to(G.dev())
    out = flce.embedding(wd, tok.to(G.dev()), layout=layout)["hidden"].cpu()
    want = w[tok.clamp(min=0)]
    want[4] = 0
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))


BACKWARD = [(0, 8, 5, "all"), (1, 8, 1, "all"), (33, 16, 1, "same"), (32, 16, 1, "same"),
            (31, 72, 7, "holes"), (64, 8, 3, "same"), (65, 136, 130, "same"),
            (300, 192, 1001, "holes"), (1025, 136, 192, "hot"), (3000, 64, 65, "hot"),
            (9000, 40, 5000, "hot"), (16385, 8, 700, "holes"), (40000, 16, 70001, "hot"),
            (520, 4104, 72, "hot"), (2048, 264, 8, "same"), (30000, 24, 9, "same"), (50000, 16, 40, "hot")]


def _check_grad(got, tok, g, V, scale, layout, dtype, base=None):
    want, mag, count = O.embedding_backward(g, tok, V, scale=scale)
    n = count[:, None].astype(np.float64)
    got = got.float().cpu().numpy().astype(np.float64)
    if layout == "hv":
        got = got.T
    tol = (n + 1) * 2.0 ** -24 * mag
    if base is not None:
        b = base.float().cpu().numpy().astype(np.float64)
        b = b.T if layout == "hv" else b
        unused = count == 0
        assert np.array_equal(got[unused], b[unused], equal_nan=True)
        want = want + b
        tol = tol + 2.0 ** -24 * np.abs(want) * (n > 0)
        got, want, tol = got[~unused], want[~unused], tol[~unused]
    else:
        assert np.all(got[count == 0] == 0.0)
    tol = tol + HALF_STEP[dtype] * (np.abs(want) + tol)
    assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("layout", ["hv", "vh"])
@pytest.mark.parametrize("hidden,dtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"),
                                          ("f32", "f32")])
@pytest.mark.parametrize("N,H,V,kind", BACKWARD)
def test_gradient(N, H, V, kind, hidden, dtype, layout):
    rng = np.random.default_rng(N + H + V)
    tok = _tokens(rng, N, V, kind)
    g = torch.from_numpy(rng.standard_normal((N, H)).astype(np.float32))
    if hidden == "bf16":
        g = g.to(torch.bfloat16)
    scale = float(np.float32(1.5 if N % 2 else 13.856))
    gd, td = g.to(G.dev()), torch.from_numpy(tok).to(G.dev())
    opt = flce.FlceEmbeddingOptions(-100, scale, 1 if layout == "hv" else 0, 0, 0, 0)
    nb = flce.flce_embedding_workspace_size(N, H, V, opt)[1]
    ws = torch.full((nb,), 255, dtype=torch.uint8, device=G.dev())
    kw = dict(layout=layout, scale=scale, workspace=ws)
    got = flce.embedding_backward(gd, td, V, grad_dtype=dtype, **kw)
    assert got.dtype == (torch.float32 if dtype == "f32" else torch.bfloat16)
    assert _status(ws) == int(((tok != -100) & ((tok < 0) | (tok >= V))).sum())
    gh = g.float().numpy()
    _check_grad(got, tok, gh, V, scale, layout, dtype)
    again = flce.embedding_backward(gd, td, V, grad_dtype=dtype, **kw)
    assert torch.equal(got, again)
    # Added to what is there; rows of unused ids keep their bits.
    base = torch.from_numpy(rng.standard_normal(got.shape).astype(np.float32)).to(got.dtype)
    acc = base.to(G.dev())
    out = flce.embedding_backward(gd, td, V, grad_weight=acc, **kw)
    assert out is acc
    _check_grad(acc, tok, gh, V, scale, layout, dtype, base=base)


@pytest.mark.parametrize("layout", ["hv", "vh"])
@pytest.mark.parametrize("V", [70, 72])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_accumulation_leaves_unused_ids_alone(layout, V, dtype):
    H = 24
    base = torch.full((V, H), -0.0).to(dtype)
    base[1::3] = float("nan")
    base[2::7] = float("-inf")
    tok = torch.tensor([0, 6, 6, -100])
    g = torch.ones(4, H, dtype=torch.bfloat16)
    acc = (base if layout == "vh" else base.t().contiguous()).to(G.dev())
    flce.embedding_backward(g.to(G.dev()), tok.to(G.dev()), V, layout=layout, grad_weight=acc)
    got = acc.cpu() if layout == "vh" else acc.cpu().t()
    view = torch.int16 if dtype == torch.bfloat16 else torch.int32
    used = torch.zeros(V, dtype=torch.bool)
    used[[0, 6]] = True
    assert torch.equal(got.contiguous()[~used].view(view), base[~used].view(view))
    assert torch.all(got[0] == 1) and torch.all(got[6] == 2)


@pytest.mark.parametrize("layout", ["hv", "vh"])
def test_gradients_of_infinite_rows_stay_in_their_column(layout):
    """Rows of ignored tokens are not read into any sum, whatever they hold."""
    N, H, V = 200, 16, 40
    tok = torch.arange(N) % V
    tok[::5] = -100
    g = torch.randn(N, H).to(torch.bfloat16)
    g[::5] = float("nan")
    got = flce.embedding_backward(g.to(G.dev()), tok.to(G.dev()), V, layout=layout,
                                  grad_dtype="f32")
    assert bool(torch.isfinite(got).all())


@pytest.mark.parametrize("layout", ["hv", "vh"])
@pytest.mark.parametrize("N", [3000, 17000])
def test_largest_vocabulary(layout, N):
    """Ids up to the library's limit, through both sorts."""
    V, H = (1 << 22) - 256, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    t = torch.randint(0, V, (N,), generator=g, device=G.dev())
    t[:50] = V - 1
    t[50:60] = 0
    w = torch.randn(*((H, V) if layout == "hv" else (V, H)), generator=g, device=G.dev(),
                    dtype=torch.bfloat16)
    out = flce.embedding(w, t, layout=layout)["hidden"]
    rows = w[:, t].t() if layout == "hv" else w[t]
    assert torch.equal(out, rows)
    # Whole numbers: their sums are exact in any order.
    gr = torch.randint(-8, 9, (N, H), generator=g, device=G.dev()).float()
    got = flce.embedding_backward(gr, t, V, layout=layout, grad_dtype="f32")
    want = torch.zeros(V, H, device=G.dev()).index_add_(0, t, gr)
    assert torch.equal(got, want.t() if layout == "hv" else want)


@pytest.mark.parametrize("layout", ["hv", "vh"])
def test_weights_of_more_than_2_32_values(layout):
    """Offsets into the weight and its gradient that pass 32 bits. Every value of
    the gradient is written: the memory it gets held NaN before."""
    V, H, N = (1 << 22) - 256, 1032, 300
    assert V * H > 1 << 32
    shape = (H, V) if layout == "hv" else (V, H)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    w = torch.empty(shape, device=G.dev(), dtype=torch.bfloat16).normal_(generator=g)
    t = torch.randint(0, V, (N,), generator=g, device=G.dev())
    t[::3] = V - 1 - torch.arange(100, device=G.dev()) // 4
    out = flce.embedding(w, t, layout=layout)["hidden"]
    for i, v in enumerate(t.tolist()):
        assert torch.equal(out[i], w[:, v] if layout == "hv" else w[v]), (i, v)
    w.fill_(float("nan"))
    del w
    gr = torch.randint(-8, 9, (N, H), generator=g, device=G.dev()).to(torch.bfloat16)
    got = flce.embedding_backward(gr, t, V, layout=layout)
    ids = sorted(set(t.tolist()))
    for v in ids:  # sums of whole numbers below 2^8: exact, also in bf16
        row = got[:, v] if layout == "hv" else got[v]
        assert torch.equal(row.float(), gr.float()[t == v].sum(0)), v
        row.zero_()
    assert not bool(torch.any(got))


@pytest.mark.parametrize("layout", ["hv", "vh"])
def test_hidden_states_of_more_than_2_32_values(layout):
    """The same for the hidden states and their gradient, at the largest batch."""
    V, H, N = 1000, 2056, 1 << 21
    assert N * H > 1 << 32
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    dev = G.dev()
    w = torch.randn((H, V) if layout == "hv" else (V, H), generator=g, device=dev,
                    dtype=torch.bfloat16)
    t = torch.randint(0, V, (N,), generator=g, device=dev)
    out = flce.embedding(w, t, layout=layout)["hidden"]
    table = w.t().contiguous() if layout == "hv" else w
    for i in range(0, N, 1 << 16):
        assert torch.equal(out[i:i + (1 << 16)], table[t[i:i + (1 << 16)]]), i
    del out
    # Row i, column h holds i % 7 + h % 3: sums are whole numbers below 2^24, exact.
    a = (torch.arange(N, device=dev) % 7).to(torch.bfloat16)
    b = (torch.arange(H, device=dev) % 3).to(torch.bfloat16)
    gr = a[:, None] + b[None, :]
    got = flce.embedding_backward(gr, t, V, layout=layout, grad_dtype="f32")
    tc = t.cpu().numpy()
    sums = np.bincount(tc, weights=np.arange(N) % 7, minlength=V)
    want = sums[:, None] + np.bincount(tc, minlength=V)[:, None] * (np.arange(H) % 3)[None, :]
    got = (got.t() if layout == "hv" else got).cpu().numpy().astype(np.float64)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("layout", ["hv", "vh"])
def test_slices_make_the_whole(layout):
    rng = np.random.default_rng(7)
    N, H, V, cut = 900, 40, 203, 96
    tok = _tokens(rng, N, V, "holes")
    w, table = _weight(rng, H, V, layout)
    t = torch.from_numpy(tok).to(G.dev())
    g = torch.from_numpy(rng.standard_normal((N, H)).astype(np.float32)).to(G.dev())
    whole = flce.embedding(w, t, layout=layout)["hidden"]
    grad = flce.embedding_backward(g, t, V, layout=layout, grad_dtype="f32")
    outs, grads = [], []
    for b, e in ((0, cut), (cut, V)):
        ws = (w[:, b:e] if layout == "hv" else w[b:e]).contiguous()
        out = flce.embedding(ws, t, layout=layout, v_begin=b, v_total=V)
        outs.append(out["hidden"])
        assert _status(out["workspace"]) == int(((tok != -100) & ((tok < 0) | (tok >= V))).sum())
        grads.append(flce.embedding_backward(g, t, e - b, layout=layout, v_begin=b, v_total=V,
                                             grad_dtype="f32"))
    assert torch.equal(outs[0] + outs[1], whole)
    assert torch.equal(torch.cat(grads, 1 if layout == "hv" else 0), grad)


@pytest.mark.parametrize("layout", ["hv", "vh"])
@pytest.mark.parametrize("N", [40, 2500, 17000])
def test_captured_calls_replay(layout, N):
    """Two captured calls that share a workspace, replayed with other inputs
    and eager work between."""
    rng = np.random.default_rng(N)
    H, V = 64, 500
    dev = G.dev()
    w, table = _weight(rng, H, V, layout)
    t = torch.from_numpy(_tokens(rng, N, V, "hot")).to(dev)
    g = torch.randn(N, H, device=dev)
    opt = flce.FlceEmbeddingOptions(-100, 2.0, 1 if layout == "hv" else 0, 1, 1, 0)
    ws = torch.empty(flce.flce_embedding_workspace_size(N, H, V, opt)[1], dtype=torch.uint8,
                     device=dev)

    def step():
        return (flce.embedding(w, t, layout=layout, scale=2.0, workspace=ws)["hidden"],
                flce.embedding_backward(g, t, V, layout=layout, scale=2.0, grad_dtype="f32",
                                        workspace=ws))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, step()))
    for rep in range(3):
        t.copy_(torch.from_numpy(_tokens(rng, N, V, "holes" if rep % 2 else "hot")))
        g.normal_()
        eager = [x.clone() for x in step()]
        for graph, out in graphs:
            for x in out:
                x.fill_(7.0)
            ws.fill_(255)
            graph.replay()
            torch.cuda.synchronize()
            for got, want in zip(out, eager):
                assert torch.equal(got, want)


def test_two_streams_match_alone():
    rng = np.random.default_rng(3)
    dev = G.dev()
    cases = []
    for N, H, V, layout in ((6000, 128, 900, "hv"), (18000, 64, 3000, "vh")):
        t = torch.from_numpy(_tokens(rng, N, V, "hot")).to(dev)
        cases.append((torch.randn(N, H, device=dev), t, V, layout))
    alone = [flce.embedding_backward(g, t, V, layout=lay) for g, t, V, lay in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s, (g, t, V, lay) in zip(streams, cases):
        with torch.cuda.stream(s):
            got.append(flce.embedding_backward(g, t, V, layout=lay))
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        assert torch.equal(a, b)


def test_autograd():
    rng = np.random.default_rng(11)
    N, H, V = 300, 64, 129
    tok = _tokens(rng, N, V, "holes")
    t = torch.from_numpy(tok).to(G.dev())
    for layout in ("hv", "vh"):
        w, _ = _weight(rng, H, V, layout)
        w.requires_grad_(True)
        out = function.embedding(w, t, layout=layout, scale=8.0)
        up = torch.randn(H, N, device=G.dev()).to(torch.bfloat16).t()  # not contiguous
        out.backward(up)
        assert w.grad.dtype == torch.bfloat16 and w.grad.shape == w.shape
        _check_grad(w.grad, tok, up.float().cpu().numpy(), V, 8.0, layout, "bf16")


def test_wrapper_refusals():
    dev = G.dev()
    w = torch.zeros(16, 40, dtype=torch.bfloat16, device=dev)
    t = torch.zeros(4, dtype=torch.int64, device=dev)
    g = torch.zeros(4, 16, dtype=torch.bfloat16, device=dev)
    with pytest.raises(ValueError, match="layout must be"):
        flce.embedding(w, t, layout="v")
    with pytest.raises(ValueError, match="contiguous"):
        flce.embedding(w.t(), t, layout="vh")
    with pytest.raises(ValueError, match="tokens must be"):
        flce.embedding(w, t.int())
    with pytest.raises(ValueError, match="tokens must be on|tokens must be a CUDA"):
        flce.embedding(w, t.cpu())
    with pytest.raises(flce.FlceError, match="BAD_SHAPE"):
        flce.embedding(w, t, v_begin=1)
    with pytest.raises(flce.FlceError, match="MISALIGNED"):
        flce.embedding(torch.zeros(12, 40, dtype=torch.bfloat16, device=dev), t)
    with pytest.raises(ValueError, match="N = 4"):
        flce.embedding_backward(g, t[:3], 40)
    with pytest.raises(ValueError, match=r"grad_weight must be \[16, 40\]"):
        flce.embedding_backward(g, t, 40, grad_weight=torch.zeros(40, 16, device=dev))
    with pytest.raises(ValueError, match="grad_weight must be a bf16"):
        flce.embedding_backward(g, t, 40, grad_weight=w.half())
    with pytest.raises(ValueError, match="workspace must be"):
        flce.embedding_backward(g, t, 40, workspace=torch.zeros(4, device=dev))

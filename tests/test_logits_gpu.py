"""The logits of some rows (flce.logits) on the GPU against the float64 oracle."""
import numpy as np
import pytest
import torch

from linear_cross_entropy_tile_amd import flce
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _inputs(N, H, V, seed, bias=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    h = torch.randn(N, H, generator=g, device=DEV, dtype=torch.bfloat16)
    w = (torch.randn(H, V, generator=g, device=DEV) * H ** -0.5).to(torch.bfloat16)
    return h, w, (torch.randn(V, generator=g, device=DEV) if bias else None)


def _check(out, h, w, b, cap, dtype):
    """H products are summed in fp32 in some order: every sum and the bias round the
    running value, at most the sum of magnitudes, by 2^-24 of it (2^-23 if the matrix
    units cut off), and bf16 rounds the result by 2^-8. The cap is steeper than 1
    nowhere and adds 2^-23 c and three roundings of its result."""
    z, mag = S.logits(h.double().cpu().numpy(), w.double().cpu().numpy(),
                      None if b is None else b.double().cpu().numpy(), cap)
    tol = (h.shape[1] + 8) * 2.0 ** -23 * mag
    if cap > 0:
        tol = tol + 2.0 ** -23 * cap + 4 * 2.0 ** -24 * np.abs(z)
    if dtype == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(z) + tol)
    err = np.abs(out.double().cpu().numpy() - z)
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())


SHAPES = [(1, 8, 1), (1, 8, 7), (3, 16, 8), (2, 24, 9), (1, 64, 127), (5, 40, 128), (17, 96, 129),
          (16, 96, 1000), (33, 128, 1001), (64, 64, 257), (65, 96, 264), (65, 96, 263),
          (70, 32, 8), (129, 200, 520), (257, 72, 256), (300, 40, 250), (1, 4096, 2000),
          (1024, 32, 264), (7, 1032, 130), (40, 2056, 700), (16, 1024, 70001), (20, 520, 20001)]


@pytest.mark.parametrize("N,H,V", SHAPES)
@pytest.mark.parametrize("cap,bias,dtype", [(0.0, False, "f32"), (5.0, True, "bf16")])
def test_logits(N, H, V, cap, bias, dtype):
    h, w, b = _inputs(N, H, V, N + H + V, bias)
    out = flce.logits(h, w, bias=b, softcap=cap, out_dtype=dtype)["logits"]
    assert out.shape == (N, V) and out.dtype == (torch.float32 if dtype == "f32"
                                                 else torch.bfloat16)
    _check(out, h, w, b, cap, dtype)


def test_no_rows():
    h, w, _ = _inputs(0, 64, 100, 1)
    assert flce.logits(h, w)["logits"].shape == (0, 100)


@pytest.mark.parametrize("N,V", [(1, 130), (20, 1001), (66, 264), (30, 70001)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_apart_and_what_lies_between(N, V, dtype):
    """A wider buffer: the rest of its rows stays as it was."""
    h, w, b = _inputs(N, 96, V, 5, True)
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    wide = torch.full((N + 1, V + 13), 7.0, dtype=t, device=DEV)
    out = flce.logits(h, w, bias=b, out_dtype=dtype, out=wide[:N, 3:3 + V])["logits"]
    assert out.data_ptr() == wide[:, 3:].data_ptr()
    _check(out, h, w, b, 0.0, dtype)
    assert (wide[:, :3] == 7).all() and (wide[:, 3 + V:] == 7).all() and (wide[N] == 7).all()


@pytest.mark.parametrize("N,V", [(4, 1000), (4, 1003), (100, 1000), (2, 300)])
def test_infinities_and_nan_stay_in_their_columns_and_rows(N, V):
    """A NaN or infinity of the weight reaches its column, one of hidden its row."""
    h, w, _ = _inputs(N, 1032, V, 9)
    w[5, 3], w[1031, V - 1], w[700, 200] = float("inf"), float("nan"), -float("inf")
    h[1, 1030] = float("nan")
    z = h.double().cpu() @ w.double().cpu()
    out = flce.logits(h, w)["logits"].double().cpu()
    assert torch.equal(torch.isnan(out), torch.isnan(z))
    inf = torch.isinf(z)
    assert torch.equal(torch.isinf(out), inf) and torch.equal(out[inf], z[inf])


def test_matches_the_head():
    """logsumexp and log-probabilities of these logits are the head's."""
    h, w, _ = _inputs(77, 96, 1000, 3)
    y = torch.randint(0, 1000, (77,), device=DEV)
    head = flce.forward(h, w, y, softcap=5.0)
    z = flce.logits(h, w, softcap=5.0)["logits"]
    out = flce.process_logits(z)
    lp = z[torch.arange(77, device=DEV), y] - out["lse"]
    for a, b in ((out["lse"], head["lse"]), (lp, head["logprob"]),
                 (out["entropy"], head["entropy"])):
        assert (a - b).abs().max() < 1e-4


def test_large_offsets():
    """Weight of more than 2^32 bytes, outputs behind element 2^31."""
    V, H = (1 << 22) - 256, 600
    h = torch.randn(3, H, device=DEV, dtype=torch.bfloat16)
    w = torch.empty(H, V, device=DEV, dtype=torch.bfloat16).normal_(0, 0.05)
    out = flce.logits(h, w)["logits"]
    at = torch.tensor([0, 1, V // 2, V - 129, V - 2, V - 1], device=DEV)
    _check(out[:, at], h, w[:, at].contiguous(), None, 0.0, "f32")
    ld = 1 << 30
    wide = torch.empty(3 * ld, device=DEV, dtype=torch.bfloat16)
    rows = wide.view(3, ld)[:, :1000]
    got = flce.logits(h, w[:, :1000].contiguous(), out_dtype="bf16", out=rows)["logits"]
    _check(got, h, w[:, :1000].contiguous(), None, 0.0, "bf16")


@pytest.mark.parametrize("N", [3, 100])
def test_repeats_to_the_bit_on_two_streams_and_captured(N):
    h, w, b = _inputs(N, 2048, 2000, 11, True)
    one = flce.logits(h, w, bias=b)["logits"]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            for _ in range(3):
                got.append(flce.logits(h, w, bias=b)["logits"])
    torch.cuda.synchronize()
    assert all(torch.equal(one, x) for x in got)
    out = torch.zeros_like(one)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    with torch.cuda.stream(streams[0]):
        flce.logits(h, w, bias=b, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        flce.logits(h, w, bias=b, out=out, workspace=ws)
    for k in range(3):
        out.zero_()
        h.mul_(-1.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, flce.logits(h, w, bias=b)["logits"]), k


def test_refusals():
    h, w, b = _inputs(4, 64, 100, 1, True)
    bad = [dict(hidden=h.float()), dict(weight=w[:32]), dict(bias=b[:99]), dict(bias=b.double()),
           dict(out_dtype="f16"), dict(out=torch.empty(4, 99, device=DEV)),
           dict(out=torch.empty(100, 4, device=DEV).t()), dict(out_dtype="bf16",
                                                               out=torch.empty(4, 100, device=DEV)),
           dict(hidden=h.cpu()), dict(weight=w.t().contiguous().t()),
           dict(out=torch.empty(1, 100, device=DEV).expand(4, 100))]
    for kw in bad:
        with pytest.raises(ValueError):
            flce.logits(**{**dict(hidden=h, weight=w), **kw})
    for N in (1025,):
        with pytest.raises(flce.FlceError, match="BAD_SHAPE"):
            flce.logits(h[:1].expand(N, 64).contiguous(), w)
    with pytest.raises(flce.FlceError, match="BAD_SOFTCAP"):
        flce.logits(h, w, softcap=float("nan"))
    with pytest.raises(flce.FlceError, match="MISALIGNED"):
        flce.logits(h[:, :60].contiguous(), w[:60].contiguous())

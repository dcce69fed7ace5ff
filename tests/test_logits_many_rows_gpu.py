"""flce.logits of many rows, where large tiles are used: against the float64 oracle."""
import pytest
import torch

from linear_cross_entropy_tile_amd import flce
from test_logits_gpu import DEV, _check, _inputs

pytestmark = pytest.mark.gpu

# At least 256 blocks of 64 rows by 128 ids; rows around 64, 128, 192 and 256 and their
# multiples, aligned and odd vocabularies, hidden sizes that are no multiple of 32.
SHAPES = [(65, 8, 16264), (65, 32, 16257), (70, 1032, 16400), (100, 24, 16390), (128, 160, 16383),
          (129, 104, 10993), (129, 72, 11000), (192, 96, 10881), (193, 64, 8065), (256, 200, 8200),
          (257, 136, 8065), (257, 128, 8064), (1000, 40, 2049), (1024, 96, 2056), (1024, 96, 1921),
          (1024, 328, 2047), (90, 96, 70001), (300, 520, 20003)]


@pytest.mark.parametrize("N,H,V", SHAPES)
@pytest.mark.parametrize("cap,bias,dtype", [(0.0, False, "f32"), (5.0, True, "bf16")])
def test_logits(N, H, V, cap, bias, dtype):
    h, w, b = _inputs(N, H, V, N + H + V, bias)
    out = flce.logits(h, w, bias=b, softcap=cap, out_dtype=dtype)["logits"]
    _check(out, h, w, b, cap, dtype)


@pytest.mark.parametrize("N,V", [(66, 16392), (66, 16391), (200, 8193), (200, 8200)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_apart_and_what_lies_between(N, V, dtype):
    h, w, b = _inputs(N, 104, V, 5, True)
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    buf = torch.full((N + 1, V + 13), 7.0, dtype=t, device=DEV)
    out = flce.logits(h, w, bias=b, out_dtype=dtype, out=buf[:N, 3:3 + V])["logits"]
    assert out.data_ptr() == buf[:, 3:].data_ptr()
    _check(out, h, w, b, 0.0, dtype)
    assert (buf[:, :3] == 7).all() and (buf[:, 3 + V:] == 7).all() and (buf[N] == 7).all()


@pytest.mark.parametrize("N,V", [(100, 16400), (100, 16403), (200, 8195)])
def test_infinities_and_nan_stay_in_their_columns_and_rows(N, V):
    h, w, _ = _inputs(N, 1032, V, 9)
    w[5, 3], w[1031, V - 1], w[700, 200] = float("inf"), float("nan"), -float("inf")
    h[1, 1030] = float("nan")
    z = h.double().cpu() @ w.double().cpu()
    out = flce.logits(h, w)["logits"].double().cpu()
    assert torch.equal(torch.isnan(out), torch.isnan(z))
    inf = torch.isinf(z)
    assert torch.equal(torch.isinf(out), inf) and torch.equal(out[inf], z[inf])


@pytest.mark.parametrize("V", [16400, 16393])
def test_weight_inside_a_longer_buffer(V):
    """A weight that starts inside of another tensor."""
    N, H = 100, 64
    h, w, _ = _inputs(N, H, V, 21)
    buf = torch.empty(H * V + 8, dtype=torch.bfloat16, device=DEV)
    at = buf[8:].view(H, V)
    at.copy_(w)
    assert torch.equal(flce.logits(h, at)["logits"], flce.logits(h, w)["logits"])


@pytest.mark.parametrize("V", [16400, 16393])
def test_repeats_to_the_bit_and_captured(V):
    N = 150
    h, w, b = _inputs(N, 512, V, 11, True)
    one = flce.logits(h, w, bias=b)["logits"]
    assert all(torch.equal(one, flce.logits(h, w, bias=b)["logits"]) for _ in range(3))
    out = torch.zeros_like(one)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        flce.logits(h, w, bias=b, out=out, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(out, one)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        flce.logits(h, w, bias=b, out=out, workspace=ws)
    for k in range(3):
        out.zero_()
        h.mul_(-1.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, flce.logits(h, w, bias=b)["logits"]), k

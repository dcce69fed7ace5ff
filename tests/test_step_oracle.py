"""The oracle of the operators at the ends of a training step, pinned to closed
forms, library routines and differences."""
import numpy as np
import pytest
import torch

from oracle import step_oracle as S


def test_process_row_by_hand():
    x = np.array([2.0, -2.0, 1.0, 0.5, 3.0])
    y = S.process_row(x, history=[0, 1, 1, 4, 9, -100], prompt=1, repetition=2.0, presence=0.5,
                      frequency=0.25, temperature=0.5, bias=[0, 0, 1, 0, 0],
                      listed=[(3, 1.0), (3, 0.25), (7, 5.0)],
                      allowed=np.array([1, 1, 1, 1, 0], bool))
    # id 0: prompt only, 2/2; id 1: -2*2 - 2*.25 - .5; id 2: bias; id 3: listed twice.
    want = np.array([1.0, -5.0, 2.0, 1.75, -np.inf]) / 0.5
    assert np.allclose(y[:4], want[:4], rtol=0, atol=1e-15) and y[4] == -np.inf


def test_row_stats_against_torch():
    y = torch.randn(301, dtype=torch.float64) * 3
    y[::7] = -float("inf")
    lse, ent, top = S.row_stats(y.numpy())
    p = torch.softmax(y, 0)
    assert abs(lse - float(torch.logsumexp(y, 0))) < 1e-12
    assert abs(ent - float(torch.special.entr(p).sum())) < 1e-12
    assert top == int(y.argmax())
    assert S.row_stats(np.full(4, -np.inf)) == (-np.inf, 0.0, -1)
    assert np.isnan(S.row_stats(np.array([1.0, np.nan, np.inf]))[0])


def test_row_gradient_against_differences():
    rng = np.random.default_rng(3)
    x = rng.normal(size=23) * 2
    hist, allowed = [1, 4, 4, 9, 22], rng.random(23) < 0.8
    kw = dict(history=hist, prompt=2, repetition=1.3, temperature=0.7, allowed=allowed)
    go, gl, ge = rng.normal(size=23), 0.7, -0.4

    def f(x):
        y = S.process_row(x, presence=0.3, frequency=0.2, **kw)
        lse, ent, _ = S.row_stats(y)
        return float((go * np.where(allowed, y, 0)).sum() + gl * lse + ge * ent)

    y = S.process_row(x, presence=0.3, frequency=0.2, **kw)
    g = S.row_gradient(y, go, gl, ge, S.row_slope(x, **kw))
    for i in range(23):
        d = np.zeros(23)
        d[i] = 1e-5
        assert abs((f(x + d) - f(x - d)) / 2e-5 - g[i]) < 1e-8


def test_e4m3_against_torch():
    y = np.concatenate([np.linspace(-448, 448, 20001), np.linspace(-0.02, 0.02, 4001),
                        S.E4M3, (S.E4M3[1:] + S.E4M3[:-1]) / 2]).astype(np.float32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(S.to_e4m3(y), want)
    assert S.E4M3[126] == 448.0


@pytest.mark.parametrize("x", [1.0 + 2.0 ** -9, -3.1415, 0.1, 1e-30])
def test_bf16_rounding(x):
    t = torch.tensor([x], dtype=torch.float32)
    assert S.bf16_nearest(t.numpy())[0] == t.bfloat16().float().item()
    lo = S.bf16_stochastic(t.numpy(), np.array([0], np.uint64))[0]
    hi = S.bf16_stochastic(t.numpy(), np.array([65535], np.uint64))[0]
    part = (float(t) - float(lo)) / (float(hi) - float(lo)) if hi != lo else 0.0
    got = np.array([S.bf16_stochastic(t.numpy(), np.array([b], np.uint64))[0]
                    for b in range(0, 65536, 64)])
    assert set(np.unique(got)) <= {lo, hi} and abs((got == hi).mean() - part) < 2 / 1024


def test_random_bits_are_even_and_independent():
    n = 1 << 16
    streams = [b for t in (0, 1) for s in (1, 2) for b in S.random_bits(12345, s, t, n)]
    for b in streams:
        x = b.astype(np.float64) / 65536
        # Mean and variance of a uniform variable: five standard errors.
        assert abs(x.mean() - 0.5) < 5 * np.sqrt(1 / 12 / n)
        assert abs(x.var() - 1 / 12) < 5 * np.sqrt(1 / 180 / n)
        for bit in range(16):
            assert abs(((b >> np.uint32(bit)) & 1).mean() - 0.5) < 5 * 0.5 / np.sqrt(n)
        assert abs(np.corrcoef(x[1:], x[:-1])[0, 1]) < 5 / np.sqrt(n)
    for i in range(len(streams)):
        for j in range(i):
            c = np.corrcoef(streams[i].astype(float), streams[j].astype(float))[0, 1]
            assert abs(c) < 5 / np.sqrt(n), (i, j)


def test_adamw_against_torch():
    rng = np.random.default_rng(1)
    p, m, v = rng.normal(size=50), np.zeros(50), np.zeros(50)
    q = torch.nn.Parameter(torch.from_numpy(p.copy()))
    opt = torch.optim.AdamW([q], lr=1e-2, betas=(0.9, 0.95), eps=1e-6, weight_decay=0.1)
    for t in range(1, 6):
        g = rng.normal(size=50)
        q.grad = torch.from_numpy(g.copy())
        opt.step()
        p, m, v = S.adamw(p, g, m, v, t, 1e-2, 0.9, 0.95, 1e-6, 0.1)
        f = S.adamw_f32(p, g, m, v, t, 1e-2, 0.9, 0.95, 1e-6, 0.1)
        assert np.abs(p - q.detach().numpy()).max() < 1e-14
        assert all(np.isfinite(a).all() for a in f)


def test_adamw_f32_follows_the_float64_form():
    rng = np.random.default_rng(2)
    p, g, m = (rng.normal(size=1000).astype(np.float32) for _ in range(3))
    v = (rng.random(1000) + 0.1).astype(np.float32)
    a, b = S.adamw(p, g, m, v, 7, 1e-2), S.adamw_f32(p, g, m, v, 7, 1e-2)
    for x, y in zip(a, b[:3]):
        assert np.abs(x - y).max() < 4 * 2.0 ** -24 * max(1.0, np.abs(x).max())


def test_encode_blocks():
    x = np.concatenate([np.linspace(-3, 3, 256), np.full(256, 1e-40), np.linspace(0, 1, 10)])
    codes, scales = S.encode_f32(x)
    assert scales.shape == (3,) and scales[1] == 0 and (codes[256:512] == 0).all()
    # Half a step of three bits of mantissa.
    assert np.abs(codes[:256] * scales[0] - x[:256]).max() <= 3 * 2.0 ** -4 + 1e-6
    assert codes[511 + 10] == 448.0
    tiny = np.array([1.0, 1e-9, 0.0])
    assert list(S.encode_f32(tiny, positive=True)[0]) == [448.0, 2.0 ** -9, 0.0]

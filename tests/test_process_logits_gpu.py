"""Processing of logits (flce.process_logits) on the GPU: the returned logits to the
bit against the definition's fp32 operations, its statistics and the gradient
against the float64 oracle."""
import numpy as np
import pytest
import torch

from linear_cross_entropy_tile_amd import flce, function
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF = float("inf")


def _case(N, V, seed, dtype="f32", longest=40, padded=True, penalties="all", listed=0,
          bias="none", mask="none", temperature=True):
    """(logits, keyword arguments, per-row oracle arguments)."""
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(rng.normal(size=(N, V)) * 3).to(
        torch.float32 if dtype == "f32" else torch.bfloat16).to(DEV)
    lens = [int(rng.integers(0, longest + 1)) for _ in range(N)]
    lens[-1] = 0 if N > 1 else longest
    hist = [rng.integers(0, max(1, min(V, 25)), n) for n in lens]
    for h in hist:  # some ignored, some far
        if len(h) > 3:
            h[1], h[2] = -100, V - 1
    prompt = [int(rng.integers(0, n + 2)) for n in lens]
    kw, rows = {}, [dict() for _ in range(N)]
    if penalties != "none":
        if padded:
            tok = np.full((N, longest + 3), 123456789, np.int64)  # behind the end: not read
            for i, h in enumerate(hist):
                tok[i, :len(h)] = h
            kw["tokens"], kw["lengths"] = torch.from_numpy(tok).to(DEV), torch.tensor(lens).to(DEV)
        else:
            cu = np.concatenate([[0], np.cumsum(lens)])
            kw["tokens"] = torch.from_numpy(np.concatenate(hist).astype(np.int64)).to(DEV)
            kw["cu_seqlens"] = torch.from_numpy(cu).to(DEV)
        kw["prompt_lengths"] = torch.tensor(prompt).to(DEV)
        for i in range(N):
            rows[i].update(history=hist[i], prompt=prompt[i])
        r = (rng.random(N) + 0.7).astype(np.float32)
        kw["repetition_penalty"] = torch.from_numpy(r).to(DEV)
        for i in range(N):
            rows[i]["repetition"] = r[i]
        if penalties == "all":
            p, f = (rng.normal(size=N).astype(np.float32) for _ in range(2))
            kw["presence_penalty"], kw["frequency_penalty"] = (torch.from_numpy(a).to(DEV)
                                                               for a in (p, f))
            for i in range(N):
                rows[i].update(presence=p[i], frequency=f[i])
    if temperature:
        t = (rng.random(N) + 0.5).astype(np.float32)
        t[0] = 0.0
        kw["temperature"] = torch.from_numpy(t).to(DEV)
        for i in range(N):
            rows[i]["temperature"] = t[i]
    if bias != "none":
        b = rng.normal(size=(N, V) if bias == "rows" else V).astype(np.float32)
        kw["bias"] = torch.from_numpy(b).to(DEV)
        for i in range(N):
            rows[i]["bias"] = b[i] if bias == "rows" else b
    if listed:
        k = [int(rng.integers(0, listed + 1)) for _ in range(N)]
        ids = [rng.integers(0, min(V, max(2, n // 3 + 1)), n) for n in k]  # repeats among them
        for a in ids:
            if len(a) > 2:
                a[0], a[1] = -100, V - 1
        val = [rng.normal(size=n).astype(np.float32) for n in k]
        kw["bias_tokens"] = torch.from_numpy(np.concatenate(ids).astype(np.int64)).to(DEV)
        kw["bias_values"] = torch.from_numpy(np.concatenate(val)).to(DEV)
        kw["bias_cu_seqlens"] = torch.from_numpy(np.concatenate([[0], np.cumsum(k)])).to(DEV)
        for i in range(N):
            rows[i]["listed"] = list(zip(ids[i], val[i]))
    if mask != "none":
        words = rng.integers(-2 ** 31, 2 ** 31, (N, -(-V // 32)) if mask == "rows"
                             else -(-V // 32)).astype(np.int32)
        if mask == "rows":
            words[-1] = 0  # a row that allows nothing
        kw["allowed"] = torch.from_numpy(words).to(DEV)
        for i in range(N):
            rows[i]["allowed"] = S.unpack_mask(words[i] if mask == "rows" else words, V)
    return x, kw, rows


def _bits(t):
    return t.float().cpu().numpy()


def _check_forward(x, kw, rows, out, out_dtype):
    lse, ent, top = (out[k].double().cpu().numpy() for k in ("lse", "entropy", "greedy"))
    got = _bits(out["logits"])
    for i, row in enumerate(rows):
        want = S.process_row(_bits(x[i]), dtype=np.float32, **row)
        if out_dtype == "bf16":
            want = S.bf16_nearest(want)
        assert np.array_equal(got[i], want, equal_nan=True), i
        l, e, g = S.row_stats(want)
        assert top[i] == g, (i, top[i], g)
        if not np.isfinite(l):
            assert (np.isnan(l) and np.isnan(lse[i])) or l == lse[i]
            assert (np.isnan(e) and np.isnan(ent[i])) or e == ent[i]
            continue
        # fp32 sums of at most 128 terms a thread, then merges: below 256 roundings
        # of the sums, each exp within (|d| + 4) 2^-24 with |d| weighted by p.
        y = want[np.isfinite(want)].astype(np.float64)
        p = np.exp(y - l)
        spread = float((p * np.abs(y - y.max())).sum())
        assert abs(lse[i] - l) <= 2.0 ** -24 * (300 + 2 * spread + 2 * abs(l)), (i, lse[i] - l)
        assert abs(ent[i] - e) <= 2.0 ** -24 * (300 * (1 + spread) * 2 + 2 * abs(e)
                                                + 3 * float((p * (y - y.max()) ** 2).sum())), i
    return got


CASES = [
    dict(N=1, V=1, longest=2), dict(N=2, V=7, longest=9), dict(N=3, V=8), dict(N=2, V=33),
    dict(N=5, V=1000, penalties="repetition"), dict(N=4, V=2047, listed=9, padded=False),
    dict(N=3, V=2049, bias="shared", mask="shared"), dict(N=6, V=4096, mask="rows", listed=70),
    dict(N=2, V=50257, bias="rows", mask="rows", listed=300, longest=5000),
    dict(N=9, V=5003, penalties="none", mask="rows"), dict(N=3, V=40, listed=1, penalties="none"),
    dict(N=4, V=3001, penalties="none", temperature=False),
    dict(N=300, V=9001, longest=300, padded=False), dict(N=700, V=17000, listed=5, mask="rows"),
    dict(N=1100, V=70, longest=12, padded=False, mask="shared"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c.values())))
@pytest.mark.parametrize("dtype,out_dtype", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"),
                                             ("f32", "bf16")])
def test_forward_and_gradient(case, dtype, out_dtype):
    x, kw, rows = _case(seed=case["N"] + case["V"], dtype=dtype, **case)
    if case["N"] > 100:  # the oracle is a loop over rows
        kw_all, pick = kw, np.unique(np.linspace(0, case["N"] - 1, 23).astype(int))
    else:
        kw_all, pick = kw, np.arange(case["N"])
    before = x.clone()
    out = flce.process_logits(x, out_dtype=out_dtype, **kw_all)
    assert torch.equal(x, before)
    assert flce.flce_get_status(out["workspace"].data_ptr(), 0) == 0
    sub = {k: out[k][torch.from_numpy(pick).to(DEV)] for k in ("logits", "lse", "entropy",
                                                               "greedy")}
    _check_forward(x[torch.from_numpy(pick).to(DEV)], kw, [rows[i] for i in pick], sub, out_dtype)

    rng = np.random.default_rng(1)
    go = torch.from_numpy(rng.normal(size=x.shape)).to(out["logits"].dtype).to(DEV)
    gl, ge = (torch.from_numpy(rng.normal(size=len(x)).astype(np.float32)).to(DEV)
              for _ in range(2))
    plain = flce.process_logits_backward(go, x, **kw)
    full = flce.process_logits_backward(go, x, processed=out["logits"], lse=out["lse"],
                                        entropy=out["entropy"], grad_lse=gl, grad_entropy=ge, **kw)
    only = flce.process_logits_backward(None, x, processed=out["logits"], lse=out["lse"],
                                        grad_lse=gl, **kw)
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    for i in pick:
        sl = {k: v for k, v in rows[i].items() if k in ("history", "prompt", "repetition",
                                                        "temperature", "allowed")}
        f32 = S.row_slope(_bits(x[i]), dtype=np.float32, **sl)
        want = np.where(f32[2], (_bits(go[i]) * f32[0]) * f32[1], np.float32(0))
        want = S.bf16_nearest(want) if dtype == "bf16" else want
        assert np.array_equal(_bits(plain[i]), want), i
        y, slope = _bits(out["logits"][i]), S.row_slope(_bits(x[i]), **sl)
        for got, args in ((full, (_bits(go[i]), float(gl[i]), float(ge[i]))),
                          (only, (np.zeros(len(y)), float(gl[i]), 0.0))):
            g64 = S.row_gradient(y, *args, slope)
            # lse and entropy within 2^-24 (300 (1 + spread) ...) as above: p within
            # 2^-15 of itself for these rows, and a few roundings.
            l, e, _ = S.row_stats(y)
            if l == -np.inf:
                assert (_bits(got[i]) == 0).all()
                continue
            p = np.exp(y.astype(np.float64) - l)
            d = np.abs(np.where(p > 0, y - l, 0.0)) + abs(e) + 1
            size = np.abs(args[0]) + p * (abs(args[1]) + abs(args[2]) * d)
            tol = np.abs(slope[0] * slope[1]) * (8 * 2.0 ** -24 * size + 2.0 ** -14 * p * (
                abs(args[1]) + abs(args[2]) * d)) + half * (np.abs(g64)) * 1.01
            assert (np.abs(_bits(got[i]) - g64) <= tol + 1e-38).all(), i


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_odd_values(dtype):
    """Lowest values as masks, infinities and NaN, allowed and masked ones."""
    V = 3000
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    low = torch.finfo(t).min
    x = torch.randn(8, V, device=DEV).to(t)
    x[0, 10:] = low
    x[1] = low
    x[2, 5], x[2, 2500] = INF, INF
    x[3, 7] = float("nan")
    x[4, 9] = float("nan")   # masked below
    x[5] = -INF
    x[6, 100], x[6, 2900] = float("nan"), float("nan")
    x[7, 0] = -INF
    words = np.full((8, 94), -1, np.int32)
    words[4, 0] = ~(1 << 9)
    allowed = torch.from_numpy(words).to(DEV)
    out = flce.process_logits(x, allowed=allowed)
    rows = [dict(allowed=S.unpack_mask(w, V)) for w in words]
    _check_forward(x, {}, rows, out, dtype)
    assert out["greedy"].tolist()[2:7] == [5, 7, out["greedy"][4].item(), -1, 100]
    assert out["lse"][1].item() == pytest.approx(low, rel=1e-6)
    assert abs(out["entropy"][1].item() - np.log(V)) < 1e-5
    assert torch.isfinite(out["lse"][4]) and out["lse"][2].item() == INF
    # Penalties on infinite and lowest logits follow the same operations.
    tok = torch.tensor([[0, 5, 9]] * 8, device=DEV)
    kw = dict(tokens=tok, lengths=torch.full((8,), 3, device=DEV), repetition_penalty=1.25,
              frequency_penalty=0.5)
    out = flce.process_logits(x, allowed=allowed, **kw)
    for r in rows:
        r.update(history=[0, 5, 9], repetition=1.25, frequency=0.5)
    _check_forward(x, kw, rows, out, dtype)


def test_rows_apart_in_place_and_what_lies_between():
    N, V = 5, 1001
    x, kw, rows = _case(N, V, 4, mask="rows", listed=5)
    wide = torch.full((N + 1, V + 9), 3.0, device=DEV)
    wide[:N, 2:2 + V] = x
    view = wide[:N, 2:2 + V]
    want = flce.process_logits(x, **kw)
    for out in (torch.full((N + 1, V + 4), 5.0, device=DEV), wide):
        target = view if out is wide else out[:N, 1:1 + V]
        got = flce.process_logits(view, out=target, **kw)
        assert all(torch.equal(got[k], want[k]) for k in ("logits", "lse", "entropy", "greedy"))
    assert (wide[:, :2] == 3).all() and (wide[:, 2 + V:] == 3).all() and (wide[N] == 3).all()
    go = torch.randn(N, V, device=DEV)
    g = flce.process_logits_backward(go, x, **kw)
    again = flce.process_logits_backward(go, x, out=go, **kw)
    assert again is go and torch.equal(go, g)


def test_bad_rows_are_refused_on_the_device():
    """Bad offsets: NaN and -1 in their row, counted; the other rows as ever."""
    N, V = 4, 500
    x = torch.randn(N, V, device=DEV)
    tok = torch.randint(0, V, (N, 6), device=DEV)
    good = torch.tensor([6, 0, 3, 2], device=DEV)
    want = flce.process_logits(x, tokens=tok, lengths=good, repetition_penalty=1.5)
    for bad in (-1, 7, 1 << 60, -(1 << 62)):
        lens = good.clone()
        lens[2] = bad
        got = flce.process_logits(x, tokens=tok, lengths=lens, repetition_penalty=1.5)
        g = flce.process_logits_backward(torch.ones_like(x), x, tokens=tok, lengths=lens,
                                         repetition_penalty=1.5)
        assert flce.flce_get_status(got["workspace"].data_ptr(), 0) == 1
        assert torch.isnan(got["logits"][2]).all() and torch.isnan(got["lse"][2])
        assert torch.isnan(got["entropy"][2]) and got["greedy"][2] == -1 and torch.isnan(g[2]).all()
        for i in (0, 1, 3):
            assert all(torch.equal(got[k][i], want[k][i]) for k in ("logits", "lse", "entropy",
                                                                    "greedy"))
            assert not torch.isnan(g[i]).any()
    flat = torch.randint(0, V, (11,), device=DEV)
    for cu, n_bad in (([0, 3, 2, 5, 11], 1), ([0, 3, 5, 12, 11], 2), ([-1, 3, 5, 7, 11], 1),
                      ([0, 3, 5, 7, 12], 1)):
        got = flce.process_logits(x, tokens=flat, cu_seqlens=torch.tensor(cu, device=DEV),
                                  presence_penalty=0.5)
        assert flce.flce_get_status(got["workspace"].data_ptr(), 0) == n_bad
        assert torch.isnan(got["lse"]).sum() == n_bad
    got = flce.process_logits(x, bias_tokens=flat, bias_values=torch.ones(11, device=DEV),
                              bias_cu_seqlens=torch.tensor([0, 3, 2, 5, 11], device=DEV))
    assert flce.flce_get_status(got["workspace"].data_ptr(), 0) == 1
    # Ids outside the vocabulary are passed over and counted.
    tok[0, :3] = torch.tensor([-1, V, 1 << 40])
    got = flce.process_logits(x, tokens=tok, lengths=good, repetition_penalty=1.5,
                              bias_tokens=torch.tensor([V, -100, 3], device=DEV),
                              bias_values=torch.ones(3, device=DEV),
                              bias_cu_seqlens=torch.tensor([0, 2, 2, 2, 3], device=DEV))
    assert flce.flce_get_status(got["workspace"].data_ptr(), 0) == 4


def test_no_rows_and_no_history():
    out = flce.process_logits(torch.empty(0, 10, device=DEV))
    assert out["logits"].shape == (0, 10) and out["lse"].numel() == 0
    assert flce.flce_get_status(out["workspace"].data_ptr(), 0) == 0
    x = torch.randn(2, 50, device=DEV)
    for kw in (dict(tokens=torch.empty(2, 0, dtype=torch.int64, device=DEV),
                    lengths=torch.zeros(2, dtype=torch.int64, device=DEV)),
               dict(tokens=torch.empty(0, dtype=torch.int64, device=DEV),
                    cu_seqlens=torch.zeros(3, dtype=torch.int64, device=DEV))):
        out = flce.process_logits(x, repetition_penalty=2.0, presence_penalty=1.0, **kw)
        assert torch.equal(out["logits"], x)
    out = flce.process_logits(x, repetition_penalty=2.0,
                              tokens=torch.empty(0, dtype=torch.int64, device=DEV),
                              cu_seqlens=torch.tensor([0, 1, 1], device=DEV))
    # Of no tokens, offsets of 1 are outside.
    assert torch.isnan(out["lse"]).all() and torch.isnan(out["logits"]).all()


def test_listed_biases_of_one_id_add_up_in_order():
    """2^24 + 1 + 1 depends on the order in fp32."""
    x = torch.zeros(2, 100, device=DEV)
    vals = [float(2 ** 24), 1.0, 1.0, -float(2 ** 24)] * 40
    rev = vals[::-1]
    tok = torch.full((len(vals) * 2,), 7, device=DEV)
    out = flce.process_logits(x, bias_tokens=tok, bias_values=torch.tensor(vals + rev, device=DEV),
                              bias_cu_seqlens=torch.tensor([0, len(vals), 2 * len(vals)],
                                                           device=DEV))
    want = []
    for v in (vals, rev):
        s = np.float32(0)
        for y in v:
            s = s + np.float32(y)
        want.append(s)
    assert out["logits"][:, 7].tolist() == [float(w) for w in want]


def test_long_history_and_large_offsets():
    """Counts beyond 16 bits, and rows behind element 2^31."""
    V = 1000
    tok = torch.zeros(1, 200000, dtype=torch.int64, device=DEV)
    tok[0, 70000:] = 5
    x = torch.zeros(1, V, device=DEV)
    out = flce.process_logits(x, tokens=tok, lengths=torch.tensor([200000], device=DEV),
                              prompt_lengths=torch.tensor([60000], device=DEV),
                              frequency_penalty=1.0)
    assert out["logits"][0, :6].tolist() == [-10000.0, 0, 0, 0, 0, -130000.0]
    ld = 1 << 30
    wide = torch.zeros(3 * ld, dtype=torch.bfloat16, device=DEV).view(3, ld)
    wide[2, :V] = 2.0
    wide[2, 17] = 3.0
    out = flce.process_logits(wide[:, :V], temperature=0.5)
    assert out["greedy"].tolist() == [0, 0, 17] and out["logits"][2, 17] == 6.0
    got = flce.process_logits(wide[:, :V], out=wide[:, :V], temperature=0.5)
    assert got["greedy"].tolist() == [0, 0, 17] and wide[2, 17] == 6.0 and wide[2, V] == 0


def test_many_rows():
    """More rows than a launch's blocks would take in one dimension."""
    N = 300000
    x = torch.randn(N, 40, device=DEV)
    out = flce.process_logits(x, temperature=2.0)
    assert torch.equal(out["logits"], x * 0.5)
    assert torch.equal(out["greedy"], (x * 0.5).argmax(1))
    assert (out["lse"].double() - torch.logsumexp(x.double() * 0.5, 1)).abs().max() < 2.0 ** -24 * 310


def test_autograd_against_torch():
    """The gradient of a loss on the drawn tokens' log-probabilities, the entropies
    and the logits, against torch's through the same operations in float64."""
    N, V = 6, 333
    x, kw, rows = _case(N, V, 8, mask="rows", listed=6, bias="shared")
    kw["allowed"][-1] = -1
    for i in range(N):
        rows[i]["allowed"] = S.unpack_mask(kw["allowed"][i].cpu().numpy(), V)
    pick = torch.tensor([int(np.flatnonzero(r["allowed"])[3]) for r in rows], device=DEV)
    a = x.clone().requires_grad_(True)
    y, lse, ent, greedy = function.process_logits(a, **kw)
    assert not greedy.requires_grad
    lp = y[torch.arange(N), pick] - lse
    w = torch.linspace(-1, 1, N, device=DEV)
    (w * lp).sum().add(0.3 * (w * ent).sum()).add((y[:, 5:9].clamp(min=-50)).sum()).backward()
    b = x.double().requires_grad_(True)
    cols = []
    for i, r in enumerate(rows):
        f, s, keep = S.row_slope(_bits(x[i]), **{k: r[k] for k in ("history", "prompt", "repetition",
                                                                   "temperature", "allowed")})
        base = torch.from_numpy(S.process_row(_bits(x[i]), **r)).to(DEV)
        f, keep = torch.from_numpy(f * float(s)).to(DEV), torch.from_numpy(keep).to(DEV)
        cols.append(torch.where(keep, base + (b[i] - b[i].detach()) * f, -INF))
    z = torch.stack(cols)
    l64 = torch.logsumexp(z, 1)
    logp = torch.where(torch.isinf(z), 0.0, z - l64[:, None])
    e64 = -(torch.softmax(z, 1) * logp).sum(1)
    wd = w.double()
    ((wd * (z[torch.arange(N), pick] - l64)).sum() + 0.3 * (wd * e64).sum()
     + z[:, 5:9].clamp(min=-50).sum()).backward()
    assert (a.grad.double() - b.grad).abs().max() < 1e-5 * b.grad.abs().max()
    # Only one of the outputs, and upstream gradients that are no dense rows.
    for pickout in range(3):
        a.grad = None
        o = function.process_logits(a, **kw)[pickout]
        torch.where(torch.isfinite(o), o, 0.0).sum().backward()
        assert torch.isfinite(a.grad).all()
    with pytest.raises(ValueError, match="out belongs"):
        function.process_logits(a, out=x)


def test_two_streams_and_two_graphs_with_workspaces_of_their_own():
    x, kw, _ = _case(40, 30011, 3, mask="rows", listed=9, longest=500)
    want = flce.process_logits(x, **kw)
    keys = ("logits", "lse", "entropy", "greedy")
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(flce.process_logits(x, **kw))
    torch.cuda.synchronize()
    assert all(torch.equal(g[k], want[k]) for g in got for k in keys)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = flce.process_logits(x, **kw)
        graphs.append((g, out))
    for k in range(3):
        x.neg_()
        kw["tokens"].add_(k)
        want = flce.process_logits(x, **kw)
        for s, (g, _) in zip(streams, graphs):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            assert all(torch.equal(out[k2], want[k2]) for k2 in keys), k


def test_captured_autograd():
    x = torch.randn(4, 900, device=DEV).requires_grad_(True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y, lse, _, _ = function.process_logits(x, temperature=0.5)
        (y[:, 3] - lse).sum().backward()
        del y, lse
    torch.cuda.current_stream().wait_stream(s)
    eager = x.grad.clone()
    x.grad = torch.zeros_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.grad.zero_()
        y, lse, _, _ = function.process_logits(x, temperature=0.5)
        (y[:, 3] - lse).sum().backward()
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(x.grad, eager)
    # An eager result that is alive on the default stream: refused, not captured. (The
    # captured results would hold the leaf's node on the capture's stream.)
    del y, lse
    keep = function.process_logits(x, temperature=0.5)
    with pytest.raises(RuntimeError, match="still alive"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            function.process_logits(x)
    del keep


def test_refusals():
    x = torch.randn(3, 70, device=DEV)
    tok, n3 = torch.zeros(3, 4, dtype=torch.int64, device=DEV), torch.zeros(
        3, dtype=torch.int64, device=DEV)
    cu = torch.zeros(4, dtype=torch.int64, device=DEV)
    f3 = torch.ones(3, device=DEV)
    bad = [dict(logits=x.half()), dict(logits=x.t()), dict(logits=x[0]), dict(logits=x.cpu()),
           dict(tokens=tok), dict(tokens=tok, cu_seqlens=cu), dict(tokens=tok[0]),
           dict(tokens=tok[:, 0].contiguous(), lengths=n3), dict(lengths=n3),
           dict(tokens=tok[:2], lengths=n3), dict(tokens=tok, lengths=n3[:2]),
           dict(tokens=tok.int(), lengths=n3), dict(tokens=tok[:, :2], lengths=n3),
           dict(tokens=tok, lengths=n3, prompt_lengths=cu), dict(temperature=f3.double()),
           dict(temperature=f3[:2]), dict(bias=f3), dict(bias=torch.ones(2, 70, device=DEV)),
           dict(bias_tokens=n3), dict(bias_tokens=n3, bias_values=f3[:2], bias_cu_seqlens=cu),
           dict(bias_tokens=n3, bias_values=f3, bias_cu_seqlens=n3),
           dict(allowed=n3), dict(allowed=torch.zeros(2, dtype=torch.int32, device=DEV)),
           dict(allowed=torch.zeros(2, 3, dtype=torch.int32, device=DEV)), dict(out_dtype="f64"),
           dict(out=torch.empty(3, 69, device=DEV)), dict(out_dtype="bf16", out=x)]
    for kw in bad:
        with pytest.raises(ValueError):
            flce.process_logits(**{**dict(logits=x), **kw})
    for kw in (dict(temperature=-1.0), dict(temperature=float("nan")),
               dict(repetition_penalty=0.0), dict(presence_penalty=INF)):
        with pytest.raises(flce.FlceError, match="BAD_OPTION"):
            flce.process_logits(x, **kw)
    out = flce.process_logits(x)
    for kw in (dict(grad_lse=f3), dict(grad_entropy=f3, processed=out["logits"], lse=out["lse"]),
               dict(grad_lse=f3[:2], processed=out["logits"], lse=out["lse"]),
               dict(processed=x[:2])):
        with pytest.raises(ValueError):
            flce.process_logits_backward(x, x, **kw)

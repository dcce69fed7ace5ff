"""The policy and the preference loss on the GPU against the float64 oracle.

Tolerance. Kernel and oracle both compute in float64, so they differ by the
float64 roundings of sums of at most some 10^4 terms of order 10 (below 1e-10 of
the largest partial sum, S) and then by the kernel's one rounding to fp32,
2^-24 of the value (2^-150 where it is subnormal)."""
import numpy as np
import pytest
import torch

import gpu_helpers as G
from oracle import operators_oracle as O
from linear_cross_entropy_tile_amd import flce, function

pytestmark = pytest.mark.gpu

V = 1000


def _close(got, want, S=1.0, name=""):
    got = got.detach().cpu().numpy().astype(np.float64)
    want = np.asarray(want, dtype=np.float64)
    assert got.shape == want.shape, name
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        ok = np.abs(got - want) <= 2.0 ** -24 * np.abs(want) + 1e-10 * S + 2.0 ** -149
    bad = ~(same | ok)
    assert not bad.any(), f"{name}: {got[bad][:4]} != {want[bad][:4]} at {np.nonzero(bad)[0][:4]}"


def _cu(lens, start=0):
    return np.concatenate([[start], start + np.cumsum(lens)]).astype(np.int64)


# Sequence lengths: empty ones, single tokens, tile borders (256), many in one
# tile, one over many tiles, up to and beyond the one-block kernel (2048 tokens, 256
# sequences), beyond one block of sequences, beyond 64 of them; padding in front of
# and behind the sequences.
LENGTHS = {
    "one": ([1], 0, 0),
    "empty": ([0, 0], 0, 0),
    "empty_between": ([0, 5, 0, 0, 250, 1, 0, 256, 0], 0, 0),
    "tile_borders": ([256, 255, 1, 257, 512, 1], 0, 0),
    "padded": ([60, 3, 200], 7, 40),
    "small_mixed": ([1, 2, 0, 70, 1, 1, 64, 3, 0, 0, 90] * 4, 5, 9),
    "small_singles": ([1] * 255 + [0], 1, 2),
    "small_limit": ([2000], 10, 38),
    "small_beyond": ([1700, 349], 0, 0),
    "singles": ([1] * 700, 3, 5),
    "long": ([5000], 0, 0),
    "ragged": ([900, 1, 33, 2500, 0, 700, 64], 0, 100),
    "large": ([3000, 1, 0, 4097, 1500, 33, 2048], 11, 300),
    "large_singles": ([1, 2, 0, 1] * 2600, 0, 3),
    "one_large": ([30000], 0, 0),
    "skewed": ([1] * 600 + [16000] + [2] * 300, 0, 0),
    "many": ([1, 0] * 33500, 0, 0),
}


def _inputs(name, seed, holes=True):
    lens, before, after = LENGTHS[name]
    rng = np.random.default_rng(seed)
    cu = _cu(lens, before)
    N = int(cu[-1]) + after
    lp = -rng.exponential(1.0, N).astype(np.float32)
    lab = rng.integers(0, V, N)
    if holes and N:
        lab[rng.random(N) < 0.25] = -100
        lab[rng.random(N) < 0.02] = V + 5
        if len(lens) > 2:
            lab[cu[1]:cu[2]] = -100  # a sequence without a valid token
    x = dict(logprob=lp, labels=lab.astype(np.int64),
             old_logprob=(lp + rng.normal(0, 0.25, N)).astype(np.float32),
             ref_logprob=(lp + rng.normal(0, 0.2, N)).astype(np.float32),
             entropy=rng.exponential(1.0, N).astype(np.float32),
             adv_token=rng.normal(0, 1, N).astype(np.float32),
             adv_seq=rng.normal(0, 1, len(lens)).astype(np.float32), cu=cu)
    x["adv_token"][::17] = 0.0
    # Tokens without a loss hold anything.
    dead = np.ones(N, bool)
    dead[cu[0]:cu[-1]] = False
    dead |= (x["labels"] < 0) | (x["labels"] >= V)
    k = np.nonzero(dead)[0]
    for key, v in (("logprob", np.nan), ("old_logprob", np.inf), ("ref_logprob", -np.inf),
                   ("entropy", np.nan), ("adv_token", np.nan)):
        x[key][k[::2]] = v
    return x


def _up(x):
    return {k: torch.from_numpy(v).to(G.dev()) for k, v in x.items()}


def _invalid(x):
    inside = x["labels"][x["cu"][0]:x["cu"][-1]]
    return int(((inside != -100) & ((inside < 0) | (inside >= V))).sum())


def _status(ws):
    return flce.flce_get_status(ws.data_ptr(), torch.cuda.current_stream().cuda_stream)


POLICY = [
    dict(),
    dict(kl_coef=0.1, entropy_coef=0.01, reduction="sequence_mean"),
    dict(kl_coef=0.1, kl_estimator="k1", reduction="sum", dual_clip=1.1),
    dict(kl_coef=-0.05, kl_estimator="k2", clip_low=0.0, clip_high=0.0, adv="seq"),
    dict(level="sequence", adv="seq", kl_coef=0.02, reduction="sequence_mean", clip_low=0.02,
         clip_high=0.03),
    dict(level="sequence", adv="seq", entropy_coef=0.3, clip_low=1.0, clip_high=0.01,
         dual_clip=1.02),
]


def _policy_call(x, cfg):
    cfg = dict(cfg)
    adv = cfg.pop("adv", "token")
    args = (x["logprob"], x["labels"], x["old_logprob"], x["adv_" + adv])
    kw = dict(cfg, entropy=x["entropy"], ref_logprob=x["ref_logprob"], cu_seqlens=x["cu"],
              advantages_per_sequence=adv == "seq", vocab_size=V)
    return args, kw


@pytest.mark.parametrize("cfg", POLICY, ids=range(len(POLICY)))
@pytest.mark.parametrize("name", LENGTHS)
def test_policy(name, cfg):
    x = _inputs(name, 5)
    args, kw = _policy_call(x, cfg)
    want = O.policy_loss(*args, grad_loss=1.75, **kw)
    S = max(1.0, float(np.nansum(np.abs(want["stats"][:6]))),
            20.0 * len(x["labels"]) if kw.get("reduction") == "sum" else 20.0)
    t = _up(x)
    args, kw = _policy_call(t, cfg)
    nb = flce.flce_policy_workspace_size(len(x["labels"]), len(x["cu"]) - 1)
    ws = torch.full((nb,), 255, dtype=torch.uint8, device=G.dev())
    out = flce.policy_loss(*args, workspace=ws, **kw)
    _close(out["stats"], want["stats"], S, "stats")
    assert torch.equal(out["loss"], out["stats"][:1])
    assert _status(ws) == _invalid(x)
    g = torch.tensor([1.75], device=G.dev())
    bkw = {k: v for k, v in kw.items() if k != "entropy"}
    glp, gent = flce.policy_loss_backward(*args, out["seq_state"], grad_loss=g, **bkw)
    _close(glp, want["grad_logprob"], 1.0, "grad_logprob")
    _close(gent, want["grad_entropy"], 1.0, "grad_entropy")
    ws.fill_(255)
    both = flce.policy_loss_forward_backward(*args, grad_loss=g, workspace=ws, **kw)
    for a, b in ((both["stats"], out["stats"]), (both["grad_logprob"], glp),
                 (both["grad_entropy"], gent)):
        assert torch.equal(a, b)
    assert _status(ws) == _invalid(x)


def test_policy_without_sequences_and_optional_inputs():
    x = _inputs("ragged", 9)
    t = _up(x)
    for cfg in (dict(), dict(reduction="sequence_mean"), dict(reduction="sum", dual_clip=2.0)):
        base = (x["logprob"], x["labels"], x["old_logprob"], x["adv_token"])
        # Without cu_seqlens every token belongs to one sequence.
        keep = np.where((x["labels"] >= 0) & (x["labels"] < V))[0]
        clean = [np.nan_to_num(b, nan=0.5, posinf=0.5, neginf=0.5) if b.dtype == np.float32 else b
                 for b in base]
        td = [torch.from_numpy(c).to(G.dev()) for c in clean]
        want = O.policy_loss(*clean, vocab_size=V, **cfg)
        out = flce.policy_loss_forward_backward(*td, vocab_size=V, **cfg)
        _close(out["stats"], want["stats"], 20.0 * len(keep), str(cfg))
        _close(out["grad_logprob"], want["grad_logprob"])
        assert "grad_entropy" not in out
        one = flce.policy_loss_forward_backward(*td, vocab_size=V, advantages_per_sequence=False,
                                                cu_seqlens=torch.tensor([0, len(clean[0])],
                                                                        device=G.dev()), **cfg)
        assert torch.equal(one["stats"], out["stats"])
    del t


def test_policy_clip_borders_and_overflow():
    """Ratios a rounding step on either side of a bound, ratios that overflow,
    and a zero advantage beside an infinite ratio."""
    eps = 0.2
    old = np.zeros(12, np.float32)
    hi, lo = np.float32(np.log1p(eps)), np.float32(np.log1p(-eps))
    lp = np.array([hi, np.nextafter(hi, np.float32(9)), np.nextafter(hi, np.float32(-9)),
                   lo, np.nextafter(lo, np.float32(9)), np.nextafter(lo, np.float32(-9)),
                   100.0, 100.0, 800.0, 800.0, -800.0, -800.0], dtype=np.float32)
    adv = np.array([1, 1, 1, -1, -1, -1, 1, -1, 0, 1, -1, 1], np.float32)
    lab = np.zeros(12, np.int64)
    with np.errstate(over="ignore", invalid="ignore"):
        for dual in (0.0, 3.0):
            want = O.policy_loss(lp, lab, old, adv, dual_clip=dual, reduction="sum")
            want_g = want["grad_logprob"].astype(np.float32).astype(np.float64)
            out = flce.policy_loss_forward_backward(
                *[torch.from_numpy(a).to(G.dev()) for a in (lp, lab, old, adv)], dual_clip=dual,
                reduction="sum")
            # exp(100) exceeds fp32: the unclipped term is infinite there.
            stats = want["stats"].astype(np.float32).astype(np.float64)
            assert np.array_equal(out["stats"][4:].cpu().numpy(), stats[4:].astype(np.float32))
            if dual:
                _close(out["stats"], stats, 1e4)
            else:
                assert np.isinf(out["stats"][0].item()) and np.isinf(stats[0])
            _close(out["grad_logprob"], want_g, 0.0)


def test_bad_offsets_give_nan_and_are_counted():
    x = _up(_inputs("ragged", 2, holes=False))
    N = x["labels"].numel()
    for bad in ([0, 900, 800, 2000, 2100, 2200, 2300, 2400], [-3, 10, 20, 30, 40, 50, 60, 70],
                [0, 10, 20, 30, 40, 50, 60, N + 1], [1 << 40] * 8,
                [0, 1 << 62, -(1 << 62), 5, 6, 7, 8, 9]):
        x["cu"] = torch.tensor(bad, device=G.dev())
        args, kw = _policy_call(x, dict(entropy_coef=0.1))
        out = flce.policy_loss_forward_backward(*args, **kw)
        assert bool(torch.isnan(out["stats"][:6]).all())
        assert bool((torch.isnan(out["grad_logprob"]) | (out["grad_logprob"] == 0)).all())
        assert _status(out["workspace"]) >= 1
        cu = x["cu"][:7].contiguous()
        y = flce.preference_loss_forward_backward(x["logprob"], x["labels"], cu)
        ok = all(0 <= a <= b <= N for a, b in zip(bad[:6], bad[1:7]))
        assert ok or bool(torch.isnan(y["loss"]).all())


PREF = [
    dict(),
    dict(label_smoothing=0.1, margin=0.5, reduction="sum"),
    dict(beta=2.0, length_normalize=True, margin=-0.3, reduction="none"),
    dict(kind="hinge", beta=0.7, margin=0.2, length_normalize=True),
    dict(kind="ipo", beta=0.3, reduction="none"),
    dict(kind="ipo", length_normalize=True, ref=False),
    dict(ref=False, beta=1.0, reduction="sum", length_normalize=True),
]


@pytest.mark.parametrize("cfg", PREF, ids=range(len(PREF)))
@pytest.mark.parametrize("name", [n for n in LENGTHS if n != "one"])
def test_preference(name, cfg):
    x = _inputs(name, 6)
    if len(x["cu"]) % 2 == 0:
        x["cu"] = np.append(x["cu"], x["cu"][-1])  # an empty last sequence
    cfg = dict(cfg)
    ref = cfg.pop("ref", True)
    P = (len(x["cu"]) - 1) // 2
    rng = np.random.default_rng(1)
    up = rng.normal(size=P if cfg.get("reduction") == "none" else 1).astype(np.float32)
    want = O.preference_loss(x["logprob"], x["labels"], x["cu"],
                             ref_logprob=x["ref_logprob"] if ref else None, grad_loss=up,
                             vocab_size=V, **cfg)
    t = _up(x)
    kw = dict(cfg, vocab_size=V)
    refd = t["ref_logprob"] if ref else None
    nb = flce.flce_preference_workspace_size(len(x["labels"]), P)
    ws = torch.full((nb,), 255, dtype=torch.uint8, device=G.dev())
    out = flce.preference_loss(t["logprob"], t["labels"], t["cu"], ref_logprob=refd, workspace=ws,
                               **kw)
    biggest = max(1.0, float(np.abs(np.concatenate([want["chosen_reward"],
                                                    want["rejected_reward"]])).max()))
    # Through ipo's square an error of the sum counts by twice the gap.
    S = 100.0 * biggest ** 2 * (P if cfg.get("reduction") == "sum" else 1)
    assert _status(ws) == _invalid(x)
    for k in ("loss", "pair_loss", "chosen_reward", "rejected_reward"):
        _close(out[k], want[k], S, k)
    g = torch.from_numpy(up).to(G.dev())
    glp = flce.preference_loss_backward(t["labels"], t["cu"], out["seq_state"], grad_loss=g, **kw)
    _close(glp, want["grad_logprob"], 100.0 * biggest, "grad_logprob")
    ws.fill_(255)
    both = flce.preference_loss_forward_backward(t["logprob"], t["labels"], t["cu"], grad_loss=g,
                                                 ref_logprob=refd, workspace=ws, **kw)
    for k in ("loss", "pair_loss", "chosen_reward", "rejected_reward"):
        assert torch.equal(both[k], out[k]), k
    assert torch.equal(both["grad_logprob"], glp)


def test_preference_extremes():
    """Gaps far into either tail: no overflow, the linear side keeps its value."""
    gaps = np.array([0.0, 1e-6, 40.0, -40.0, 1e4, -1e4, 1e30, -1e30], np.float32)
    P = len(gaps)
    lp = np.concatenate([gaps, np.zeros(P, np.float32)])
    cu = np.arange(2 * P + 1)
    for cfg in (dict(), dict(label_smoothing=0.25), dict(kind="hinge")):
        want = O.preference_loss(lp, np.zeros(2 * P, int), cu, beta=1.0, reduction="none", **cfg)
        out = flce.preference_loss_forward_backward(
            torch.from_numpy(lp).to(G.dev()), torch.zeros(2 * P, dtype=torch.int64, device=G.dev()),
            torch.from_numpy(cu).to(G.dev()), beta=1.0, reduction="none", **cfg)
        # Values relative to a few float64 roundings, then fp32's.
        for k in ("pair_loss", "grad_logprob"):
            got = out[k].cpu().numpy().astype(np.float64)
            w = want[k].astype(np.float32).astype(np.float64)
            assert np.all(np.abs(got - w) <= 2.0 ** -23 * np.abs(w) + 2.0 ** -148), (cfg, k)


@pytest.mark.parametrize("name", ["small_mixed", "ragged", "large"])
def test_captured_calls_replay(name):
    """Captured policy and preference steps that share a workspace, replayed
    with other inputs and eager work between."""
    t = _up(_inputs(name, 3, holes=False))
    if t["cu"].numel() % 2 == 0:
        t["cu"] = torch.cat([t["cu"], t["cu"][-1:]])
        t["adv_seq"] = torch.cat([t["adv_seq"], t["adv_seq"][-1:]])
    for k in ("logprob", "old_logprob", "ref_logprob", "entropy", "adv_token"):
        t[k] = torch.nan_to_num(t[k], 0.1, 0.1, 0.1)
    N, B = t["labels"].numel(), t["cu"].numel() - 1
    ws = torch.empty(max(flce.flce_policy_workspace_size(N, B),
                         flce.flce_preference_workspace_size(N, B // 2)), dtype=torch.uint8,
                     device=G.dev())

    def step():
        args, kw = _policy_call(t, POLICY[1])
        a = flce.policy_loss_forward_backward(*args, workspace=ws, **kw)
        b = flce.preference_loss_forward_backward(t["logprob"], t["labels"], t["cu"],
                                                  ref_logprob=t["ref_logprob"], workspace=ws)
        return [a["stats"], a["grad_logprob"], a["grad_entropy"], b["loss"], b["pair_loss"],
                b["grad_logprob"]]

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
        t["logprob"].normal_(-1.0, 0.3)
        t["labels"].random_(0, V + 30)
        eager = [x.clone() for x in step()]
        for graph, out in graphs:
            for x in out:
                x.fill_(7.0)
            ws.fill_(255)
            graph.replay()
            torch.cuda.synchronize()
            for got, want in zip(out, eager):
                assert torch.equal(got, want)


def test_streams_match_alone():
    xs = [_up(_inputs(n, 4)) for n in ("small_mixed", "large")]

    def step(x):
        args, kw = _policy_call(x, POLICY[1])
        out = flce.policy_loss_forward_backward(*args, **kw)
        return [out["stats"], out["grad_logprob"], out["grad_entropy"]]

    alone = [step(x) for x in xs]
    torch.cuda.synchronize()
    got = []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s, x in zip(streams, xs):
        with torch.cuda.stream(s):
            got.append(step(x))
    torch.cuda.synchronize()
    for a, b in zip(alone, got):
        for p, q in zip(a, b):
            assert torch.equal(p, q)


def test_unaligned_slices():
    """Per-token views that start at any element."""
    x = _inputs("ragged", 8)
    t = _up(x)
    off = {}
    for i, k in enumerate(("logprob", "labels", "old_logprob", "ref_logprob", "entropy",
                           "adv_token", "adv_seq", "cu")):
        pad = torch.zeros(i + 1, dtype=t[k].dtype, device=G.dev())
        off[k] = torch.cat([pad, t[k]])[i + 1:]
    for cfg in POLICY[:2]:
        a, kw = _policy_call(t, cfg)
        b, kwb = _policy_call(off, cfg)
        p = flce.policy_loss_forward_backward(*a, **kw)
        q = flce.policy_loss_forward_backward(*b, **kwb)
        assert torch.equal(p["stats"], q["stats"])
        assert torch.equal(p["grad_logprob"], q["grad_logprob"])


def test_autograd():
    x = _inputs("ragged", 12)
    t = _up(x)
    cfg = POLICY[1]
    args, kw = _policy_call(x, cfg)
    want = O.policy_loss(*args, grad_loss=0.5, **kw)
    args, kw = _policy_call(t, cfg)
    lp, ent = t["logprob"].requires_grad_(True), t["entropy"].requires_grad_(True)
    loss, stats = function.policy_loss(*args, **kw)
    assert loss.dim() == 0 and not stats.requires_grad
    (loss * 0.5).backward()
    _close(stats, want["stats"], 20.0)
    _close(lp.grad, want["grad_logprob"])
    _close(ent.grad, want["grad_entropy"])
    # Only the log-probabilities need a gradient.
    loss, _ = function.policy_loss(lp, t["labels"], t["old_logprob"], t["adv_token"],
                                   cu_seqlens=t["cu"], vocab_size=V)
    g, = torch.autograd.grad(loss, [lp])
    _close(g, O.policy_loss(x["logprob"], x["labels"], x["old_logprob"], x["adv_token"],
                            cu_seqlens=x["cu"], vocab_size=V)["grad_logprob"])
    cu = torch.cat([t["cu"], t["cu"][-1:]])
    P = (cu.numel() - 1) // 2
    for red in ("none", "mean"):
        up = np.linspace(-1, 1, P) if red == "none" else np.ones(1)
        want = O.preference_loss(x["logprob"], x["labels"], cu.cpu().numpy(),
                                 ref_logprob=x["ref_logprob"], reduction=red,
                                 grad_loss=up.astype(np.float32), vocab_size=V)
        loss, chosen, rejected = function.preference_loss(lp, t["labels"], cu,
                                                          ref_logprob=t["ref_logprob"],
                                                          reduction=red, vocab_size=V)
        assert loss.shape == ((P,) if red == "none" else ()) and not chosen.requires_grad
        g, = torch.autograd.grad(loss, [lp], torch.from_numpy(up.astype(np.float32)).to(
            G.dev()).reshape(loss.shape))
        _close(loss.reshape(-1), want["loss"], 1e4)
        _close(rejected, want["rejected_reward"], 1e4)
        _close(g, want["grad_logprob"], 1e3)


def test_wrapper_refusals():
    dev = G.dev()
    x = torch.zeros(6, device=dev)
    y = torch.zeros(6, dtype=torch.int64, device=dev)
    cu = torch.tensor([0, 2, 6], device=dev)
    call = flce.policy_loss
    for kw, msg in [(dict(kl_coef=0.1), "kl_coef needs"), (dict(entropy_coef=0.1), "entropy_coef"),
                    (dict(level="sequence"), "level 'sequence'"),
                    (dict(ref_logprob=x[:5]), "6 element"), (dict(entropy=x.double()), "entropy"),
                    (dict(cu_seqlens=cu.int()), "cu_seqlens"), (dict(cu_seqlens=cu[:1]), "more"),
                    (dict(advantages_per_sequence=True), "advantages must have 1"),
                    (dict(ref_logprob=x.cpu()), "ref_logprob")]:
        with pytest.raises(ValueError, match=msg):
            call(x, y, x, x, **kw)
    with pytest.raises(ValueError, match="contiguous"):
        call(torch.zeros(12, device=dev)[::2], y, x, x)
    with pytest.raises(flce.FlceError, match="BAD_OPTION"):
        call(x, y, x, x, clip_low=1.5)
    with pytest.raises(flce.FlceError, match="BAD_SHAPE"):
        call(x, y, x, x, vocab_size=0)
    with pytest.raises(ValueError, match="seq_state must be"):
        flce.policy_loss_backward(x, y, x, x, torch.zeros(3, 2, dtype=torch.float64, device=dev))
    with pytest.raises(ValueError, match="grad_loss must have 1"):
        flce.policy_loss_forward_backward(x, y, x, x, grad_loss=x)
    with pytest.raises(ValueError, match="even number"):
        flce.preference_loss(x, y, torch.tensor([0, 1, 2, 6], device=dev))
    with pytest.raises(ValueError, match="grad_loss must have 1"):
        flce.preference_loss_forward_backward(x, y, cu, grad_loss=x, reduction="none")
    with pytest.raises(flce.FlceError, match="BAD_OPTION"):
        flce.preference_loss(x, y, cu, kind="ipo", margin=1.0)
    with pytest.raises(ValueError, match="seq_state must have 3"):
        flce.preference_loss_backward(y, cu, torch.zeros(2, dtype=torch.float64, device=dev))

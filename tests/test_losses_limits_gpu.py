"""The losses in batches of more than 2^18 tokens, whose tiles have 256 tokens, up
to the library's limits, against float64 sums over whole arrays.

Tolerance: 2^-24 of the value for the rounding to fp32; beside it 1e-10 of the sum of
the terms' magnitudes for float64 sums of at most 2^21 terms (kernel: chains of some
thousand additions, 2^-53 each; numpy sums pairwise), and for a gradient 1e-9 of its
token weight as in the tests of its precision."""
import numpy as np
import pytest
import torch

import gpu_helpers as G
from linear_cross_entropy_tile_amd import flce

pytestmark = pytest.mark.gpu

MAX = 1 << 21
HALF = 2.0 ** -24 * (1.0 + 2.0 ** -20)


def _mixed():
    rng = np.random.default_rng(0)
    return np.concatenate([np.ones(700, int), [256, 255, 1, 0, 257, 512, 3],
                           np.full(300, 3), [130000], np.zeros(90, int), rng.integers(0, 90, 2000),
                           [1, 60000, 1], rng.integers(20, 300, 301), [0, 0]]).astype(np.int64)


BATCHES = {
    "mixed": lambda: _mixed(),
    "one": lambda: np.array([MAX]),
    "two": lambda: np.array([MAX - 1, 1]),
    "singles": lambda: np.ones(MAX, np.int64),
    "pairs_of_tokens": lambda: np.full(MAX // 2, 2),
    "long_and_singles": lambda: np.concatenate([[1 << 20], np.ones(1 << 20, np.int64)]),
}


def _inputs(name):
    lens = BATCHES[name]()
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    N = int(cu[-1])
    assert N > 1 << 18
    rng = np.random.default_rng(N % 1000)
    lab = rng.integers(0, 1000, N)
    lab[rng.random(N) < 0.2] = -100
    x = dict(lp=-rng.exponential(1.0, N), ent=rng.exponential(1.0, N), adv=rng.normal(0, 1, N))
    x["old"] = x["lp"] + rng.normal(0, 0.25, N)
    x["ref"] = x["lp"] + rng.normal(0, 0.2, N)
    x = {k: v.astype(np.float32) for k, v in x.items()}
    seq = np.repeat(np.arange(lens.size), lens)
    return x, lab, lab >= 0, cu, seq


def _up(v):
    return torch.from_numpy(v).to(G.dev())


def _within(got, want, tol, name):
    got = got.cpu().numpy().astype(np.float64)
    bad = ~(np.abs(got - want) <= HALF * np.abs(want) + tol + 2.0 ** -149)
    assert not bad.any(), f"{name}: {got[bad][:4]} != {want[bad][:4]} at {np.nonzero(bad)[0][:4]}"


@pytest.mark.parametrize("reduction", ["mean", "sequence_mean"])
@pytest.mark.parametrize("name", BATCHES)
def test_policy(name, reduction):
    x, lab, on, cu, seq = _inputs(name)
    B = cu.size - 1
    d = {k: v.astype(np.float64) for k, v in x.items()}
    r, A = np.exp(d["lp"] - d["old"]), d["adv"]
    f = -np.minimum(r * A, np.clip(r, 0.8, 1.3) * A)
    clip = f != -r * A
    df = np.where(clip, 0.0, f)
    k = d["lp"] - d["ref"]
    kl, dkl = np.expm1(-k) + k, -np.expm1(-k)
    n = np.bincount(seq[on], minlength=B).astype(np.float64)
    w = np.full(B, 1.0 / n.sum()) if reduction == "mean" else (
        1.0 / (np.maximum(n, 1.0) * (n > 0).sum()))
    w = np.where(on, w[seq], 0.0)
    terms = [f + 0.05 * kl - 0.01 * d["ent"], f, kl, d["ent"], clip.astype(np.float64),
             d["old"] - d["lp"]]
    t = {key: _up(v) for key, v in x.items()}
    out = flce.policy_loss_forward_backward(
        t["lp"], _up(lab), t["old"], t["adv"], entropy=t["ent"], ref_logprob=t["ref"],
        cu_seqlens=_up(cu), clip_high=0.3, kl_coef=0.05, entropy_coef=0.01, reduction=reduction)
    _within(out["stats"][:6], np.array([(w * v).sum() for v in terms]),
            np.array([1e-10 * (w * np.abs(v)).sum() for v in terms]), "stats")
    assert out["stats"][6].item() == n.sum() and out["stats"][7].item() == (n > 0).sum()
    _within(out["grad_logprob"], w * (df + 0.05 * dkl), 1e-9 * w, "grad_logprob")
    _within(out["grad_entropy"], -0.01 * w, 1e-12 * w, "grad_entropy")
    two = flce.policy_loss(t["lp"], _up(lab), t["old"], t["adv"], entropy=t["ent"],
                           ref_logprob=t["ref"], cu_seqlens=_up(cu), clip_high=0.3, kl_coef=0.05,
                           entropy_coef=0.01, reduction=reduction)
    assert torch.equal(two["stats"], out["stats"])


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("name", [n for n in BATCHES if n != "one"])
def test_preference(name, normalize):
    x, lab, on, cu, seq = _inputs(name)
    if cu.size % 2 == 0:
        cu = np.append(cu, cu[-1])
    P, B = (cu.size - 1) // 2, cu.size - 1
    beta = 0.01
    term = np.where(on, x["lp"].astype(np.float64) - x["ref"].astype(np.float64), 0.0)
    n = np.bincount(seq[on], minlength=B)
    share = 1.0 / np.maximum(n, 1) if normalize else np.ones(B)
    R = np.bincount(seq, term, minlength=B) * share
    mag = np.bincount(seq, np.abs(term), minlength=B) * share
    gap = beta * (R[:P] - R[P:])
    slope = -beta * np.exp(-np.logaddexp(0.0, gap)) / P
    # np.bincount adds one after another: n roundings a sequence at most.
    off = 2.0 ** -52 * n * mag
    off = off[:P] + off[P:] + 1e-12
    t = {key: _up(v) for key, v in x.items()}
    out = flce.preference_loss_forward_backward(t["lp"], _up(lab), _up(cu), ref_logprob=t["ref"],
                                                beta=beta, length_normalize=normalize)
    pair = np.logaddexp(0.0, -gap)
    _within(out["chosen_reward"], beta * R[:P], beta * off, "chosen")
    _within(out["rejected_reward"], beta * R[P:], beta * off, "rejected")
    _within(out["pair_loss"], pair, beta * off + 1e-14, "pair_loss")
    _within(out["loss"], np.array([pair.mean()]), np.array([beta * off.max() + 1e-10 * pair.mean()]),
            "loss")
    both = (np.concatenate([slope, -slope]) * share)[seq]
    tol = (np.concatenate([off, off]) * share * beta * beta / P)[seq] + 1e-12 * np.abs(both)
    _within(out["grad_logprob"], np.where(on, both, 0.0), tol, "grad_logprob")

"""Gradients of the losses to fp32 precision at every batch size: held to the one
rounding to fp32, 2^-24 of the value, whatever the factor of the reduction.

Beside it stand the float64 roundings. Policy: a token's gradient is w (df + c dk)
with df = -exp(d) A and dk of order 1; at the sequence level d is a mean of up to
30000 terms below 2, whose sum is off by at most 30000 * 2^-53 of itself, 4e-12; the
exponential adds 1e-13. With |A| < 6 and |d| < 2 the terms stay below 50, so the
float64 part is below 50 * 5e-12 w < 1e-9 w. Entropy: the product of w, the
coefficient and the upstream gradient, below 2^-50 of it. Preference: the sum of
a sequence of n terms t is off by at most n 2^-53 sum |t| on either side (both add at
most n numbers), which reaches the gradient k share slope(x) through the slope's
Lipschitz constant by the sum: beta^2 / 4 (sigmoid), 0 (hinge, away from x = 1), 2
(ipo); the slope's own float64 error stays below 1e-12 beta (sigmoid, hinge) and
2^-48 of its value (ipo)."""
import numpy as np
import pytest
import torch

import gpu_helpers as G
from oracle import operators_oracle as O
from linear_cross_entropy_tile_amd import flce
from test_losses_gpu import LENGTHS, POLICY, PREF, V, _inputs, _policy_call, _up

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -24 * (1.0 + 2.0 ** -20)   # and what the rounded value's own error adds


def _within(got, want, tol, name):
    got = got.cpu().numpy().astype(np.float64)
    err = np.abs(got - want)
    bad = ~(err <= HALF * np.abs(want) + tol + 2.0 ** -149)
    assert not bad.any(), f"{name}: {got[bad][:4]} != {want[bad][:4]} at {np.nonzero(bad)[0][:4]}"


def _valid(x):
    """(sequence of every token or -1, valid tokens of every sequence)."""
    cu, lab = x["cu"], x["labels"]
    seq = np.searchsorted(cu[1:], np.arange(lab.size), side="right")
    on = (np.arange(lab.size) >= cu[0]) & (seq < cu.size - 1) & (lab >= 0) & (lab < V)
    seq = np.where(on, np.minimum(seq, cu.size - 2), -1)
    return seq, np.bincount(seq[on], minlength=cu.size - 1)


@pytest.mark.parametrize("cfg", POLICY, ids=range(len(POLICY)))
@pytest.mark.parametrize("name", LENGTHS)
def test_policy_gradients(name, cfg):
    x = _inputs(name, 5)
    args, kw = _policy_call(x, cfg)
    want = O.policy_loss(*args, grad_loss=1.75, **kw)
    seq, n = _valid(x)
    red = kw.get("reduction", "mean")
    each = {"mean": np.full(n.size, 1.0 / max(n.sum(), 1)), "sum": np.ones(n.size),
            "sequence_mean": 1.0 / (np.maximum(n, 1) * max((n > 0).sum(), 1))}[red]
    w = 1.75 * np.where(seq >= 0, each[seq], 0.0)
    t = _up(x)
    args, kw = _policy_call(t, cfg)
    out = flce.policy_loss_forward_backward(*args, grad_loss=torch.tensor([1.75], device=G.dev()),
                                            **kw)
    _within(out["grad_logprob"], want["grad_logprob"], 1e-9 * w, "grad_logprob")
    _within(out["grad_entropy"], want["grad_entropy"],
            2.0 ** -50 * np.abs(want["grad_entropy"]), "grad_entropy")


@pytest.mark.parametrize("cfg", PREF, ids=range(len(PREF)))
@pytest.mark.parametrize("name", [n for n in LENGTHS if n != "one"])
def test_preference_gradients(name, cfg):
    x = _inputs(name, 6)
    if len(x["cu"]) % 2 == 0:
        x["cu"] = np.append(x["cu"], x["cu"][-1])
    cfg = dict(cfg)
    ref = cfg.pop("ref", True)
    P = (len(x["cu"]) - 1) // 2
    up = np.random.default_rng(1).normal(size=P if cfg.get("reduction") == "none" else 1)
    up = up.astype(np.float32)
    want = O.preference_loss(x["logprob"], x["labels"], x["cu"],
                             ref_logprob=x["ref_logprob"] if ref else None, grad_loss=up,
                             vocab_size=V, **cfg)["grad_logprob"]
    seq, n = _valid(x)
    on = seq >= 0
    term = np.zeros(on.size)
    term[on] = x["logprob"][on].astype(np.float64)
    if ref:
        term[on] -= x["ref_logprob"][on].astype(np.float64)
    share = 1.0 / np.maximum(n, 1) if cfg.get("length_normalize") else np.ones(n.size)
    off = n * 2.0 ** -53 * np.bincount(seq[on], np.abs(term[on]), minlength=n.size) * share
    gap = 2.0 * (off[:P] + off[P:])          # kernel and oracle
    beta, kind = cfg.get("beta", 0.1), cfg.get("kind", "sigmoid")
    slope = {"sigmoid": beta * beta / 4.0, "hinge": 0.0, "ipo": 2.0}[kind] * gap
    slope += 1e-12 * beta if kind != "ipo" else 0.0
    k = 1.0 / P if cfg.get("reduction", "mean") == "mean" else 1.0
    tol = np.abs(np.broadcast_to(up, (P,))) * k * slope
    tol = (np.concatenate([tol, tol]) * share)[seq] * on + 2.0 ** -48 * np.abs(want)
    t = _up(x)
    out = flce.preference_loss_forward_backward(
        t["logprob"], t["labels"], t["cu"], grad_loss=torch.from_numpy(up).to(G.dev()),
        ref_logprob=t["ref_logprob"] if ref else None, vocab_size=V, **cfg)
    _within(out["grad_logprob"], want, tol, "grad_logprob")

"""The operators together, as a fine-tuning step uses them: the embedding looked
up from the head's own weight, a stand-in model, the fused head, a loss on its
per-token outputs, and both gradients of the tied weight in one tensor. Against
the same step in float64 on the CPU.

Tolerances. Hidden states, logit gradients and grad_hidden pass through bf16
between the operators: 2^-8 of each value, at most four such roundings in a row
here (relative L2 below 2^-6 with room for the sums' own), and a bf16 result."""
import numpy as np
import pytest
import torch

import gpu_helpers as G
import oracle
from oracle import operators_oracle as O
from linear_cross_entropy_tile_amd import flce, function

pytestmark = pytest.mark.gpu

N, H, V = 300, 64, 203
SCALE = 8.0
CU = [0, 70, 70, 131, 200, 241, 290]


def _step_inputs():
    rng = np.random.default_rng(21)
    w = torch.from_numpy((rng.standard_normal((H, V)) * 0.2).astype(np.float32)).to(torch.bfloat16)
    mix = torch.from_numpy((rng.standard_normal((H, H)) / np.sqrt(H)).astype(np.float32))
    tok = rng.integers(0, V, N)
    lab = rng.integers(0, V, N)
    lab[rng.random(N) < 0.3] = -100
    return rng, w, mix.to(torch.bfloat16), tok, lab


def _rel(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


@pytest.mark.parametrize("loss", ["policy", "preference"])
@pytest.mark.parametrize("how", ["calls", "autograd"])
def test_tied_step(loss, how):
    rng, w, mix, tok, lab = _step_inputs()
    dev = G.dev()
    wd, md = w.to(dev), mix.to(dev)
    td, ld = torch.from_numpy(tok).to(dev), torch.from_numpy(lab).to(dev)
    cu = torch.tensor(CU, device=dev)
    old = (-rng.exponential(1.0, N) - 3).astype(np.float32)
    ref = (-rng.exponential(1.0, N) - 3).astype(np.float32)
    adv = rng.normal(size=len(CU) - 1).astype(np.float32)
    dold, dref, dadv = (torch.from_numpy(x).to(dev) for x in (old, ref, adv))
    pol = dict(advantages_per_sequence=True, kl_coef=0.05, kl_estimator="k2", entropy_coef=0.02,
               clip_low=0.9, clip_high=50.0, vocab_size=V)
    pre = dict(beta=0.05, label_smoothing=0.1, vocab_size=V)

    # The step in float64; its clip bounds are wide, so that no token sits near one.
    W, M = w.double().numpy(), mix.double().numpy()
    emb = O.embedding(W.T, tok, scale=SCALE)
    hid = emb @ M
    fw = oracle.forward(hid, W, lab)
    if loss == "policy":
        want = O.policy_loss(fw["logprob"], lab, old, adv, entropy=fw["entropy"], ref_logprob=ref,
                             cu_seqlens=CU, **pol)
        want_loss, glp, gent = want["stats"][0], want["grad_logprob"], want["grad_entropy"]
    else:
        want = O.preference_loss(fw["logprob"], lab, CU, ref_logprob=ref, **pre)
        want_loss, glp, gent = want["loss"][0], want["grad_logprob"], np.zeros(N)
    dh, dw = oracle.backward(hid, W, lab, grad_logprob=glp, grad_entropy=gent)
    dw = dw + O.embedding_backward(dh @ M.T, tok, V, scale=SCALE)[0].T

    if how == "calls":
        e = flce.embedding(wd, td, scale=SCALE)["hidden"]
        x = (e.float() @ md.float()).to(torch.bfloat16)
        out = flce.forward(x, wd, ld)
        if loss == "policy":
            r = flce.policy_loss_forward_backward(out["logprob"], ld, dold, dadv,
                                                  entropy=out["entropy"], ref_logprob=dref,
                                                  cu_seqlens=cu, **pol)
            g, ge = r["grad_logprob"], r["grad_entropy"]
        else:
            r = flce.preference_loss_forward_backward(out["logprob"], ld, cu, ref_logprob=dref,
                                                      **pre)
            g, ge = r["grad_logprob"], None
        gh, gw = flce.backward(x, wd, ld, out["lse"], out["entropy"], g, ge, grad_dtype="f32")
        ge_hidden = gh @ md.float().t().contiguous()
        flce.embedding_backward(ge_hidden, td, V, scale=SCALE, grad_weight=gw)
        got_loss = r["loss"]
    else:
        wp = wd.clone().requires_grad_(True)
        e = function.embedding(wp, td, scale=SCALE)
        x = (e.float() @ md.float()).to(torch.bfloat16)
        lp, ent = function.linear_cross_entropy(x, wp, ld, reduction="none")
        if loss == "policy":
            got_loss, _ = function.policy_loss(lp, ld, dold, dadv, entropy=ent, ref_logprob=dref,
                                               cu_seqlens=cu, **pol)
        else:
            got_loss, _, _ = function.preference_loss(lp, ld, cu, ref_logprob=dref, **pre)
        got_loss.backward()
        gw = wp.grad
    assert abs(got_loss.item() - want_loss) <= 2.0 ** -6 * max(1.0, abs(want_loss))
    assert _rel(gw.float().cpu().numpy(), dw) <= 2.0 ** -6


def _autograd_step(weight, tok, lab, old, adv, cu):
    hidden = torch.tanh(function.embedding(weight, tok, scale=SCALE))
    lp, ent = function.linear_cross_entropy(hidden, weight, lab, reduction="none")
    loss, stats = function.policy_loss(lp, lab, old, adv, entropy=ent, cu_seqlens=cu,
                                       entropy_coef=0.01, advantages_per_sequence=True)
    pref, _, _ = function.preference_loss(lp, lab, cu)
    return loss + pref, stats


def _step_tensors():
    rng, w, _, tok, lab = _step_inputs()
    dev = G.dev()
    old = torch.from_numpy((-rng.exponential(1.0, N) - 3).astype(np.float32)).to(dev)
    adv = torch.from_numpy(rng.normal(size=len(CU) - 1).astype(np.float32)).to(dev)
    return (w.to(dev), torch.from_numpy(tok).to(dev), torch.from_numpy(lab).to(dev), old, adv,
            torch.tensor(CU, device=dev))


def test_captured_autograd_step_replays():
    """Forward and backward through autograd in a captured graph, over a leaf
    that no eager graph holds, replayed with other inputs and eager work
    between; against the same step run eagerly on another leaf."""
    w, tok, lab, old, adv, cu = _step_tensors()

    def eager():
        leaf = w.clone().requires_grad_(True)
        total, stats = _autograd_step(leaf, tok, lab, old, adv, cu)
        total.backward()
        return [total.detach().clone(), stats.clone(), leaf.grad.clone()]

    eager()  # loads what the step needs before the capture
    torch.cuda.synchronize()
    leaf = w.clone().requires_grad_(True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        total, stats = _autograd_step(leaf, tok, lab, old, adv, cu)
        total.backward()
    got = [total.detach(), stats, leaf.grad]
    for rep in range(3):
        tok.random_(0, V)
        w.normal_(0.0, 0.2)
        with torch.no_grad():
            leaf.copy_(w)
        want = eager()
        for x in got:
            x.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


def test_capture_over_a_live_eager_graph_is_refused(monkeypatch):
    """While an eager result lives, a call under capture on another stream is
    refused for the same leaf, by every operator; not for another leaf, on the
    result's own stream, without gradients, or once the result is dropped.
    Nothing is captured here: the query is answered in its place."""
    w, tok, lab, old, adv, cu = _step_tensors()
    weight, lp = w.requires_grad_(True), old.clone().requires_grad_(True)
    calls = {
        "embedding": lambda: function.embedding(weight, tok),
        "policy": lambda: function.policy_loss(lp, lab, old, adv, cu_seqlens=cu,
                                               advantages_per_sequence=True)[0],
        "preference": lambda: function.preference_loss(lp, lab, cu)[0],
    }
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def captured(call):
        with monkeypatch.context() as m, torch.cuda.stream(side):
            m.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
            return call()

    head = lambda: function.linear_cross_entropy(  # noqa: E731
        torch.zeros(N, H, dtype=torch.bfloat16, device=w.device), weight, lab)[0]
    for name, made in (("embedding", calls["embedding"]), ("embedding", head),
                       ("policy", calls["policy"]), ("preference", calls["policy"]),
                       ("policy", calls["preference"])):
        call = calls[name]
        alive = made()
        with pytest.raises(RuntimeError, match="still alive"):
            captured(call)
        with torch.no_grad():
            captured(call)
        with monkeypatch.context() as m:
            m.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
            call()
        other = "embedding" if name != "embedding" else "policy"
        captured(calls[other])
        del alive
        captured(call)
    torch.cuda.synchronize()

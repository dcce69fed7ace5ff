"""The autograd functions with gradients and leaves as other operators make them."""
import pytest
import torch

import gpu_helpers as G
import test_tied_step_gpu as T
from linear_cross_entropy_tile_amd import flce, function

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", ["hv", "vh"])
def test_embedding_takes_a_gradient_at_any_address(layout):
    """A contiguous gradient that starts inside a 16-byte unit: a view that the
    caller passes, and the share that the gradient of a concatenation hands on."""
    N, H, V = 37, 24, 50
    w = torch.randn((H, V) if layout == "hv" else (V, H), device=G.dev()).to(torch.bfloat16)
    tok = torch.arange(N, device=G.dev()) * 3 % V
    leaf = w.clone().requires_grad_(True)
    up = torch.randn(N * H + 1, device=G.dev()).to(torch.bfloat16)
    want = flce.embedding_backward(up[1:].clone().view(N, H), tok, V, layout=layout)
    function.embedding(leaf, tok, layout=layout).backward(up[1:].view(N, H))
    assert torch.equal(leaf.grad, want)
    leaf.grad = None
    head = torch.zeros(1, device=G.dev(), dtype=torch.bfloat16, requires_grad=True)
    out = torch.cat([head, function.embedding(leaf, tok, layout=layout).reshape(-1)])
    out.backward(up)
    assert torch.equal(leaf.grad, want)


def _captured(monkeypatch, stream, call):
    """The call as it would run under a capture on the stream; nothing is
    captured, the query is answered in its place."""
    with monkeypatch.context() as m, torch.cuda.stream(stream):
        m.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
        return call()


def _calls(weight, lp, tok, lab, old, adv, cu):
    return {"embedding": lambda: function.embedding(weight, tok),
            "policy": lambda: function.policy_loss(lp, lab, old, adv, cu_seqlens=cu,
                                                   advantages_per_sequence=True)[0],
            "preference": lambda: function.preference_loss(lp, lab, cu)[0]}


@pytest.mark.parametrize("name", ["embedding", "policy", "preference"])
def test_results_of_a_side_stream_do_not_stop_a_capture(name, monkeypatch):
    """A warm-up on a side stream whose result is still bound: a gradient that is
    added on that stream joins the capture through events, and is not refused.
    One that belongs to the default stream, which no capture can join, is."""
    w, tok, lab, old, adv, cu = T._step_tensors()
    weight, lp = w.requires_grad_(True), old.clone().requires_grad_(True)
    call = _calls(weight, lp, tok, lab, old, adv, cu)[name]
    warm, side = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (warm, side):
        s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        alive = call()
    again = call()  # on the default stream, over the node that the side stream made
    _captured(monkeypatch, side, call)
    del alive, again
    alive = call()
    with pytest.raises(RuntimeError, match="still alive"):
        _captured(monkeypatch, side, call)
    del alive
    torch.cuda.synchronize()


def test_captured_step_with_its_warm_up_still_bound():
    """The usual order: a warm-up on a side stream, its loss still in a variable,
    then forward and backward captured over the same leaf, and replayed with
    other inputs and eager work between."""
    w, tok, lab, old, adv, cu = T._step_tensors()
    leaf = w.clone().requires_grad_(True)
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        bound, _ = T._autograd_step(leaf, tok, lab, old, adv, cu)
        bound.backward()
    torch.cuda.current_stream().wait_stream(warm)
    torch.cuda.synchronize()
    leaf.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        total, stats = T._autograd_step(leaf, tok, lab, old, adv, cu)
        total.backward()
    got = [total.detach(), stats, leaf.grad]
    for rep in range(3):
        tok.random_(0, T.V)
        w.normal_(0.0, 0.2)
        with torch.no_grad():
            leaf.copy_(w)
        other = w.clone().requires_grad_(True)
        t, s = T._autograd_step(other, tok, lab, old, adv, cu)
        t.backward()
        want = [t.detach().clone(), s.clone(), other.grad.clone()]
        del t, s
        for x in got:
            x.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
    assert bool(torch.isfinite(bound))


@pytest.mark.parametrize("holder", ["head", "embedding"])
def test_captured_backward_of_the_head_is_refused_over_a_live_graph(holder, monkeypatch):
    """The head's captured backward over a leaf that a result of the default
    stream holds; its captured forward alone is not refused, nor a backward that
    needs no gradient of that leaf, nor one after the result is dropped."""
    w, tok, lab, old, adv, cu = T._step_tensors()
    weight = w.requires_grad_(True)
    hidden = torch.randn(T.N, T.H, device=w.device).to(torch.bfloat16)
    h = hidden.clone().requires_grad_(True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def eager():
        if holder == "embedding":
            return function.embedding(weight, tok)
        return function.linear_cross_entropy(hidden, weight, lab)[0]

    alive = eager()
    lp, ent = _captured(monkeypatch, side,
                        lambda: function.linear_cross_entropy(h, weight, lab))
    with pytest.raises(RuntimeError, match="still alive"):
        _captured(monkeypatch, side, lambda: (lp + ent).backward(retain_graph=True))
    with pytest.raises(RuntimeError, match="still alive"):
        _captured(monkeypatch, side, lambda: torch.autograd.grad(lp, [weight], retain_graph=True))
    _captured(monkeypatch, side, lambda: torch.autograd.grad(lp, [h], retain_graph=True))
    with torch.cuda.stream(side):
        (lp + ent).backward()  # not captured: allowed
    assert weight.grad is not None and h.grad is not None
    del alive, lp, ent
    _captured(monkeypatch, side,
              lambda: function.linear_cross_entropy(h.detach(), weight, lab)[0].backward())
    torch.cuda.synchronize()


def test_leaves_behind_casts_and_views_are_seen(monkeypatch):
    """A master weight in fp32, cast (and transposed) for the call, has the
    gradient's node of a leaf as much as a direct argument."""
    w, tok, lab, old, adv, cu = T._step_tensors()
    master = w.float().requires_grad_(True)
    wide = old.double().requires_grad_(True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    hidden = torch.randn(T.N, T.H, device=w.device).to(torch.bfloat16)

    def embed():
        return function.embedding(master.to(torch.bfloat16), tok)

    def table():
        return function.embedding((2.0 * master).to(torch.bfloat16).t().contiguous(), tok,
                                  layout="vh")

    def head():
        return function.linear_cross_entropy(hidden, master.to(torch.bfloat16), lab)[0]

    def policy():
        return function.policy_loss(wide.float().view(-1), lab, old, adv, cu_seqlens=cu,
                                    advantages_per_sequence=True)[0]

    def preference():
        return function.preference_loss(wide.float(), lab, cu)[0]

    for made, call in ((embed, table), (head, embed), (policy, preference), (preference, policy)):
        alive = made()
        with pytest.raises(RuntimeError, match="still alive"):
            _captured(monkeypatch, side, call)
        del alive
        _captured(monkeypatch, side, call)
    alive = table()
    with pytest.raises(RuntimeError, match="still alive"):
        _captured(monkeypatch, side, lambda: head().backward())
    del alive
    _captured(monkeypatch, side, lambda: head().backward())
    torch.cuda.synchronize()


class _Halved(torch.autograd.Function):
    """A function of the caller's with an attribute of its own on the node."""

    @staticmethod
    def forward(ctx, x):
        ctx.variable = "its own"
        return 0.5 * x

    @staticmethod
    def backward(ctx, g):
        return 0.5 * g


def test_leaves_on_the_host_and_nodes_of_other_functions():
    """A leaf in host memory that the argument is copied from, and a node of
    another function in between."""
    w, tok, lab, old, adv, cu = T._step_tensors()
    host = w.float().cpu().requires_grad_(True)
    out = function.embedding(host.to(w.device, torch.bfloat16), tok)
    out.backward(torch.ones_like(out))
    ones = torch.ones_like(out)
    want = flce.embedding_backward(ones, tok, T.V)
    assert torch.equal(host.grad, want.float().cpu())
    lp = old.cpu().requires_grad_(True)
    for halved in (lp.to(w.device) * 0.5, _Halved.apply(lp.to(w.device)),
                   _Halved.apply(old.clone().requires_grad_(True))):
        loss, _ = function.policy_loss(halved, lab, old, adv, cu_seqlens=cu,
                                       advantages_per_sequence=True)
        loss.backward()
        function.preference_loss(halved.detach().requires_grad_(True), lab, cu)[0].backward()
    assert bool(torch.isfinite(lp.grad).all())

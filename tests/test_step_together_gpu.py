"""The operators of an RL step together, as they are used: tokens drawn from the
head's processed logits, the policy loss on their log-probabilities, the gradients'
norm and the AdamW update of a tied weight."""
import pytest
import torch

from linear_cross_entropy_tile_amd import flce
from linear_cross_entropy_tile_amd.function import (embedding, linear_cross_entropy, policy_loss,
                                                    process_logits)

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _generate(weight, mix, prompts, steps, allowed, **kw):
    """Greedy continuations of the prompts [N, P] by a model of one matrix; returns
    (tokens [N, P + steps], log-probabilities of the new ones [N, steps])."""
    N, P = prompts.shape
    buf = torch.full((N, P + steps), -100, dtype=torch.int64, device=DEV)
    buf[:, :P] = prompts
    lengths = torch.full((N,), P, dtype=torch.int64, device=DEV)
    plen = lengths.clone()
    logps = []
    for s in range(steps):
        last = buf[:, P + s - 1].contiguous()
        h = flce.embedding(weight, last)["hidden"] @ mix
        z = flce.logits(h, weight, softcap=20.0)["logits"]
        out = flce.process_logits(z, out=z, tokens=buf, lengths=lengths, prompt_lengths=plen,
                                  allowed=allowed, **kw)
        assert flce.flce_get_status(out["workspace"].data_ptr(), 0) == 0
        tok = out["greedy"]
        buf[:, P + s] = tok
        logps.append(out["logits"][torch.arange(N, device=DEV), tok] - out["lse"])
        lengths += 1
    return buf, torch.stack(logps, 1)


def _setup(V=1003, H=64, N=6, P=5):
    g = torch.Generator(device=DEV).manual_seed(1)
    weight = (torch.randn(H, V, generator=g, device=DEV) * 0.3).to(torch.bfloat16)
    mix = (torch.randn(H, H, generator=g, device=DEV) * H ** -0.5).to(torch.bfloat16)
    prompts = torch.randint(0, V, (N, P), generator=g, device=DEV)
    allowed = torch.full((-(-V // 32),), -1, dtype=torch.int32, device=DEV)
    allowed[0] = ~0b111  # ids 0 to 2 are special ones
    return weight, mix, prompts, allowed


def test_generated_tokens_obey_the_processing():
    weight, mix, prompts, allowed = _setup()
    buf, lp = _generate(weight, mix, prompts, 12, allowed, repetition_penalty=1.0,
                        presence_penalty=1000.0)
    new = buf[:, 5:]
    assert (new >= 3).all() and (lp <= 0).all()
    # A presence penalty beyond every logit: no generated token comes twice.
    assert all(row.unique().numel() == 12 for row in new)


def test_behaviour_log_probabilities_are_the_heads():
    """Without penalties the log-probabilities at generation are those of the
    training head on the same tokens: the policy's ratio is 1."""
    weight, mix, prompts, _ = _setup()
    buf, lp = _generate(weight, mix, prompts, 7, None)
    h = flce.embedding(weight, buf[:, 4:-1].reshape(-1))["hidden"] @ mix
    out = flce.forward(h, weight, buf[:, 5:].reshape(-1).contiguous(), softcap=20.0)
    assert (out["logprob"].view(6, 7) - lp).abs().max() < 2e-4


@pytest.mark.parametrize("kind,master", [("f32", True), ("8bit", False)])
def test_training_step(kind, master):
    """Through autograd: the loss's gradients reach the update, whose effect has
    their sign, and an overflow in the batch leaves everything as it was."""
    weight, mix, prompts, allowed = _setup()
    buf, old = _generate(weight, mix, prompts, 8, allowed, temperature=1.0)
    ids, y = buf[:, 4:-1].reshape(-1), buf[:, 5:].reshape(-1).contiguous()
    adv = torch.ones(6, device=DEV)
    adv[3:] = -1
    cu = torch.arange(0, 6 * 8 + 1, 8, device=DEV)
    params = [weight.clone().requires_grad_(True), mix.clone().requires_grad_(True)]
    state = flce.adamw_state(params, kind, master)

    def loss_and_grads(poison=1.0):
        for p in params:
            p.grad = None
        h = embedding(params[0], ids) @ params[1]
        lp, ent = linear_cross_entropy(h, params[0], y, reduction="none", softcap=20.0)
        loss, stats = policy_loss(lp, y, old.reshape(-1), adv, cu_seqlens=cu,
                                  advantages_per_sequence=True)
        (loss * poison).backward()
        return lp.detach().view(6, 8), [p.grad for p in params]

    before, grads = loss_and_grads()
    assert (before - old).abs().max() < 0.05  # the mask is all that differs
    norm = flce.grad_norm(grads, max_norm=1.0)
    with torch.no_grad():
        flce.adamw_step(params, grads, state, lr=2e-3, grad_scale=norm["scale"],
                        rounding="stochastic", seed=1)
    assert int(state["step"]) == 1 and torch.isfinite(norm["norm"]).all()
    after, grads = loss_and_grads()
    change = (after - before).mean(1)
    assert (change[:3] > 0).all() and (change[3:] < 0).all()
    saved = [p.detach().clone() for p in params]
    _, grads = loss_and_grads(float("inf"))
    norm = flce.grad_norm(grads, max_norm=1.0)
    flce.adamw_step(params, grads, state, lr=2e-3, grad_scale=norm["scale"])
    assert int(state["step"]) == 1 and all(torch.equal(a, b) for a, b in zip(params, saved))


def test_loss_on_the_processed_distribution():
    """process_logits under autograd on the head's logits: the gradient raises the
    picked tokens' log-probability."""
    weight, mix, prompts, allowed = _setup()
    h = flce.embedding(weight, prompts[:, 0].contiguous())["hidden"] @ mix
    z = flce.logits(h, weight)["logits"].requires_grad_(True)
    y, lse, ent, tok = process_logits(z, allowed=allowed, temperature=0.7, tokens=prompts,
                                      lengths=torch.full((6,), 5, device=DEV),
                                      repetition_penalty=1.3)
    lp = y[torch.arange(6, device=DEV), tok] - lse
    lp.sum().backward()
    assert (z.grad[:, :3] == 0).all()
    with torch.no_grad():
        moved = flce.process_logits(z + 1e-2 * z.grad, allowed=allowed, temperature=0.7,
                                    tokens=prompts, lengths=torch.full((6,), 5, device=DEV),
                                    repetition_penalty=1.3)
    lp2 = moved["logits"][torch.arange(6, device=DEV), tok] - moved["lse"]
    rise = 1e-2 * z.grad.double().square().sum(1)
    # First order; the second is below the first times the step's size over T^2.
    assert ((lp2 - lp).double() - rise).abs().max() < 0.05 * rise.max() + 1e-5

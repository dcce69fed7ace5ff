"""The losses after bad sequence offsets (they decrease, or leave [0, N]): what
the header promises there, whatever the workspace and the shares that no tile
writes hold. The offsets are values: every access they lead to is clamped."""
import numpy as np
import pytest
import torch

import gpu_helpers as G
from linear_cross_entropy_tile_amd import flce

pytestmark = pytest.mark.gpu

V = 1000

# Lengths, and the offsets (position, value) that break them. An even number of
# sequences, the second half the rejected ones.
BATCHES = {
    "one_block": ([200, 3, 0, 70, 1, 90, 64, 250], [(2, 50), (6, 5000)]),
    "one_block_long": ([1] * 100 + [1700] + [1] * 99, [(60, 900), (150, 20)]),
    "skewed": ([1] * 600 + [16000] + [2] * 301, [(300, 9000), (700, 5000)]),
    "skewed_up": ([2] * 400 + [16000] + [1] * 601, [(100, 12000)]),
    "rejected_only": ([900, 1, 33, 2500, 0, 700], [(5, 100)]),
    "chosen_only": ([900, 1, 33, 2500, 0, 700], [(1, -7)]),
    "large": ([3] * 900 + [290000] + [1] * 99, [(500, 200000), (950, 4000)]),
}


def _inputs(name):
    lens, broken = BATCHES[name]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int64)
    N = int(cu[-1])
    for at, value in broken:
        cu[at] = value
    bad = (cu[:-1] < 0) | (cu[1:] < cu[:-1]) | (cu[1:] > N)
    rng = np.random.default_rng(len(lens))
    lab = rng.integers(0, V, N)
    lab[rng.random(N) < 0.2] = -100
    x = {k: torch.from_numpy(-rng.exponential(1.0, N).astype(np.float32)).to(G.dev())
         for k in ("logprob", "old", "ref", "entropy")}
    x["adv_token"] = torch.from_numpy(rng.normal(size=N).astype(np.float32)).to(G.dev())
    x["adv_seq"] = torch.from_numpy(rng.normal(size=len(lens)).astype(np.float32)).to(G.dev())
    x["labels"] = torch.from_numpy(lab).to(G.dev())
    x["cu"] = torch.from_numpy(cu).to(G.dev())
    return x, bad, lab >= 0


def _status(ws):
    return flce.flce_get_status(ws.data_ptr(), torch.cuda.current_stream().cuda_stream)


def _nan_where_valid(grad, valid):
    g = grad.cpu().numpy()
    return np.isnan(g[valid]).all() and (g[~valid] == 0.0).all()


FILLS = [0, 1, 255]
POLICY = [dict(), dict(level="sequence", adv="seq", reduction="sequence_mean"),
          dict(reduction="sum", adv="seq", kl_coef=0.1, entropy_coef=0.1)]


def _policy(x, cfg):
    cfg = dict(cfg)
    adv = cfg.pop("adv", "token")
    args = (x["logprob"], x["labels"], x["old"], x["adv_" + adv])
    return args, dict(cfg, ref_logprob=x["ref"], cu_seqlens=x["cu"], vocab_size=V,
                      advantages_per_sequence=adv == "seq")


def _workspace(nbytes, fill):
    return torch.full((nbytes,), fill, dtype=torch.uint8, device=G.dev())


@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("name", BATCHES)
def test_policy_counts_bad_sequences(name, fill):
    x, bad, valid = _inputs(name)
    args, kw = _policy(x, POLICY[0])
    ws = _workspace(flce.flce_policy_workspace_size(valid.size, bad.size), fill)
    out = flce.policy_loss(*args, workspace=ws, **kw)
    assert _status(ws) == bad.sum()
    assert bool(torch.isnan(out["loss"]).all()) and bool(torch.isnan(out["stats"][:6]).all())
    ws.fill_(fill)
    flce.policy_loss_forward_backward(*args, workspace=ws, **kw)
    assert _status(ws) == bad.sum()


@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("name", BATCHES)
def test_preference_counts_bad_sequences(name, fill):
    x, bad, valid = _inputs(name)
    P = bad.size // 2
    for red in ("mean", "none"):
        ws = _workspace(flce.flce_preference_workspace_size(valid.size, P), fill)
        out = flce.preference_loss_forward_backward(x["logprob"], x["labels"], x["cu"],
                                                    workspace=ws, reduction=red, vocab_size=V)
        assert _status(ws) == bad.sum()
        assert bool(torch.isnan(out["loss"]).all()) or red == "none"
        assert bool(torch.isnan(out["pair_loss"][torch.from_numpy(bad[:P] | bad[P:])]).all())


@pytest.mark.parametrize("cfg", POLICY, ids=range(len(POLICY)))
@pytest.mark.parametrize("name", BATCHES)
def test_policy_gradients_are_nan_at_every_valid_token(name, cfg):
    """Also at tokens that the broken offsets place in no sequence."""
    x, bad, valid = _inputs(name)
    args, kw = _policy(x, cfg)
    both = flce.policy_loss_forward_backward(*args, entropy=x["entropy"], **kw)
    assert _nan_where_valid(both["grad_logprob"], valid)
    assert _nan_where_valid(both["grad_entropy"], valid)
    out = flce.policy_loss(*args, entropy=x["entropy"], **kw)
    for g in flce.policy_loss_backward(*args, out["seq_state"], **kw):
        assert _nan_where_valid(g, valid)


@pytest.mark.parametrize("reduction", ["mean", "none"])
@pytest.mark.parametrize("name", BATCHES)
def test_preference_gradients_are_nan_at_every_valid_token(name, reduction):
    x, bad, valid = _inputs(name)
    args, kw = (x["logprob"], x["labels"], x["cu"]), dict(reduction=reduction, vocab_size=V)
    both = flce.preference_loss_forward_backward(*args, **kw)
    assert _nan_where_valid(both["grad_logprob"], valid)
    out = flce.preference_loss(*args, **kw)
    assert _nan_where_valid(flce.preference_loss_backward(*args[1:], out["seq_state"], **kw), valid)


def test_nan_upstream_gradient_is_no_bad_offset():
    """A NaN gradient of the loss reaches the tokens of the sequences only."""
    cu = torch.tensor([2, 5, 9], device=G.dev())
    x = -torch.rand(12, device=G.dev())
    lab = torch.zeros(12, dtype=torch.int64, device=G.dev())
    inside = np.zeros(12, bool)
    inside[2:9] = True
    g = torch.full((1,), float("nan"), device=G.dev())
    out = flce.policy_loss_forward_backward(x, lab, x - 0.1, x + 3.0, grad_loss=g, cu_seqlens=cu)
    assert _nan_where_valid(out["grad_logprob"], inside)
    out = flce.preference_loss_forward_backward(x, lab, cu, grad_loss=g)
    assert _nan_where_valid(out["grad_logprob"], inside)


@pytest.mark.parametrize("name", BATCHES)
def test_policy_statistics_are_all_nan(name):
    """The two counts among them: they add up shares that may be undefined."""
    x, bad, valid = _inputs(name)
    args, kw = _policy(x, POLICY[0])
    assert bool(torch.isnan(flce.policy_loss(*args, **kw)["stats"]).all())
    assert bool(torch.isnan(flce.policy_loss_forward_backward(*args, **kw)["stats"]).all())


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
@pytest.mark.parametrize("name", BATCHES)
def test_preference_outputs_of_a_bad_pair_are_nan(name, kind):
    """Both rewards and the loss of a pair, whichever side's offsets are bad."""
    x, bad, valid = _inputs(name)
    P = bad.size // 2
    pair = torch.from_numpy(bad[:P] | bad[P:])
    for norm in (False, True):
        out = flce.preference_loss(x["logprob"], x["labels"], x["cu"], kind=kind,
                                   length_normalize=norm, vocab_size=V)
        for k in ("pair_loss", "chosen_reward", "rejected_reward"):
            assert bool(torch.isnan(out[k].cpu()[pair]).all()), k

"""AdamW steps without a clip factor on gradients that are not finite: their weights
and states are lost, in 8 bits their blocks' states, and nothing else is."""
import numpy as np
import pytest
import torch

from linear_cross_entropy_tile_amd import flce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KW = dict(lr=2e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, seed=3)
NAN, INF = float("nan"), float("inf")
SIZES = [2048 + 100, 7, 5000]
# (tensor, value, gradient): the middle of a block, both ends of one, a short last block,
# a tensor shorter than a block, two in one block.
PLACES = [(0, 300, NAN), (0, 512, INF), (0, 1023, -INF), (0, 2100, NAN), (1, 3, NAN),
          (2, 4096, NAN), (2, 4200, INF)]


def _read(state, key, i):
    """A state as the values that it stands for."""
    t = state[key][i].float()
    if state[key + "_scale"] is not None:
        t = t * state[key + "_scale"][i].repeat_interleave(256)[:t.numel()]
    return t.cpu().numpy()


@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
@pytest.mark.parametrize("dtype,gdtype,master", [
    (torch.float32, torch.float32, False), (torch.bfloat16, torch.bfloat16, True),
    (torch.bfloat16, torch.float32, False)])
@pytest.mark.parametrize("kind", ["f32", "8bit"])
def test_what_a_gradient_that_is_not_finite_reaches(kind, dtype, gdtype, master, rounding):
    gen = torch.Generator(device=DEV).manual_seed(11)
    p0 = [torch.randn(n, generator=gen, device=DEV).to(dtype) for n in SIZES]
    ends = []
    for broken in (False, True):
        params = [p.clone() for p in p0]
        state = flce.adamw_state(params, kind, master)
        gen.manual_seed(12)
        for step in range(2):
            grads = [torch.randn(n, generator=gen, device=DEV).to(gdtype) for n in SIZES]
            if broken and step == 1:
                for i, k, value in PLACES:
                    grads[i][k] = value
            flce.adamw_step(params, grads, state, rounding=rounding, **KW)
        ends.append((params, state))
    (good, good_state), (params, state) = ends
    assert int(state["step"]) == 2
    for i, n in enumerate(SIZES):
        own = np.zeros(n, bool)
        own[[k for t, k, _ in PLACES if t == i]] = True
        reach = own
        if kind == "8bit":
            blocks = np.unique(np.flatnonzero(own) // 256)
            reach = np.isin(np.arange(n) // 256, blocks)
            for key in ("exp_avg_scale", "exp_avg_sq_scale"):
                scales, whole = (s[key][i].cpu().numpy() for s in (state, good_state))
                assert not np.isfinite(scales[blocks]).any(), (i, key)
                other = np.setdiff1d(np.arange(scales.size), blocks)
                assert np.array_equal(scales[other], whole[other]), (i, key)
        for key in ("exp_avg", "exp_avg_sq"):
            got, want = _read(state, key, i), _read(good_state, key, i)
            if kind == "8bit":
                assert np.isnan(got[reach]).all(), (i, key)
            else:
                assert not np.isfinite(got[reach]).any(), (i, key)
            assert np.array_equal(got[~reach], want[~reach]), (i, key)
        # This step's weights come from the moments before they are encoded.
        copies = [(params, good)] + ([(state["master"], good_state["master"])] if master else [])
        for a, b in copies:
            got, want = a[i].float().cpu().numpy(), b[i].float().cpu().numpy()
            assert np.isnan(got[own]).all(), i
            assert np.array_equal(got[~own], want[~own]), i


@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
def test_a_lost_block_stays_lost_and_its_neighbours_go_on(rounding):
    n = 1024
    ends = []
    for value in (0.5, NAN):
        p, g = [torch.ones(n, device=DEV)], [torch.full((n,), 0.5, device=DEV)]
        g[0][256:512] = torch.linspace(-1, 1, 256, device=DEV)
        state = flce.adamw_state(p, "8bit")
        g[0][300] = value
        flce.adamw_step(p, g, state, rounding=rounding, **KW)
        g[0][300] = 0.5
        for _ in range(2):
            flce.adamw_step(p, g, state, rounding=rounding, **KW)
        ends.append((p[0], _read(state, "exp_avg", 0), _read(state, "exp_avg_sq", 0)))
    keep = torch.arange(n, device=DEV) // 256 != 1
    (p, m, v), (q, m1, v1) = ends
    assert torch.isnan(q[~keep]).all() and torch.equal(q[keep], p[keep])
    keep = keep.cpu().numpy()
    for a, b in ((m, m1), (v, v1)):
        assert np.isnan(b[~keep]).all() and np.array_equal(a[keep], b[keep])


def test_a_square_that_overflows_counts_as_infinite_in_8_bits():
    p, g = [torch.ones(512, device=DEV)], [torch.ones(512, device=DEV)]
    g[0][5] = 1e30
    state = flce.adamw_state(p, "8bit")
    flce.adamw_step(p, g, state, **KW)
    assert torch.isfinite(p[0]).all() and np.isfinite(_read(state, "exp_avg", 0)).all()
    v = _read(state, "exp_avg_sq", 0)
    assert np.isnan(v[:256]).all() and np.isfinite(v[256:]).all()

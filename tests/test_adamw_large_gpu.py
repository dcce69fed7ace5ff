"""A tensor of more than 2^32 values: its norm, and an AdamW update of its ends."""
import pytest
import torch

from linear_cross_entropy_tile_amd import flce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_values_behind_2_to_the_32():
    far, n = 1 << 32, 600
    p = torch.zeros(far + n, dtype=torch.bfloat16, device=DEV)
    g = torch.zeros(far + n, dtype=torch.bfloat16, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(1)
    values, grads = (torch.randn(n, generator=gen, device=DEV).bfloat16() for _ in range(2))
    for at in (0, far):
        p[at:at + n], g[at:at + n] = values, grads
    small = [values.clone()]
    small_state, state = flce.adamw_state(small, "8bit"), flce.adamw_state([p], "8bit")
    want = float(2 * grads.double().square().sum()) ** 0.5
    out = flce.grad_norm([g], max_norm=0.25 * want)
    assert abs(out["norm"].item() - want) <= 2.0 ** -23 * want
    assert abs(out["scale"].item() - 0.25) <= 2.0 ** -22
    kw = dict(lr=0.1, weight_decay=0.1, grad_scale=out["scale"])
    for _ in range(2):
        flce.adamw_step(small, [grads], small_state, **kw)
        flce.adamw_step([p], [g], state, **kw)
    for at in (0, far):
        assert torch.equal(p[at:at + n], small[0])
        for key in ("exp_avg", "exp_avg_sq"):
            assert torch.equal(state[key][0][at:at + n].view(torch.uint8),
                               small_state[key][0].view(torch.uint8))
            block = at // 256
            assert torch.equal(state[key + "_scale"][0][block:block + 3],
                               small_state[key + "_scale"][0])
    # Nothing between them has moved.
    assert not p[n:far].any() and not state["exp_avg_scale"][0][3:far // 256].any()
    # The random bits of a value go by all of its index.
    q = flce.adamw_state([p], "f32")
    flce.adamw_step([p], [g], q, rounding="stochastic", seed=1, **kw)
    assert torch.equal(q["exp_avg"][0][:n], q["exp_avg"][0][far:])
    assert not torch.equal(p[:n], p[far:])

"""Options at the ends of what the operators accept."""
import numpy as np
import pytest
import torch

from linear_cross_entropy_tile_amd import flce
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("kind", ["f32", "8bit"])
def test_smallest_eps_and_gradients_of_zero(kind):
    p = [torch.linspace(-2, 2, 300, device=DEV)]
    want = p[0].cpu().numpy() * np.float32(1 - 0.25 * 0.5)
    g = [torch.zeros(300, device=DEV)]
    g[0][7] = 1.0
    state = flce.adamw_state(p, kind)
    flce.adamw_step(p, g, state, lr=0.25, weight_decay=0.5, eps=2.0 ** -126)
    got = p[0].cpu().numpy()
    keep = np.arange(300) != 7
    assert np.array_equal(got[keep], want[keep])
    # The first update of a value is lr; the root and the quotient within 2^-21 of it.
    assert abs(got[7] - (want[7] - 0.25)) <= 0.25 * 2.0 ** -21 + 2.0 ** -23 * abs(want[7])


@pytest.mark.parametrize("softcap", [2.0 ** -127, 1e-30, 3e38])
@pytest.mark.parametrize("N", [3, 70])
def test_smallest_and_largest_cap(softcap, N):
    h = torch.zeros(N, 64, device=DEV, dtype=torch.bfloat16)
    h[1:, 0] = 1.0
    w = torch.zeros(64, 40, device=DEV, dtype=torch.bfloat16)
    w[0] = torch.arange(-20, 20, device=DEV)
    got = flce.logits(h, w, softcap=softcap)["logits"]
    assert (got[0] == 0).all() and (got[1:, 20] == 0).all()
    z = torch.arange(-20, 20, device=DEV).double()
    # The product with a denormal reciprocal is off by 2^-149 at most, c times that in z.
    want = softcap * torch.tanh(z / softcap)
    tol = 2.0 ** -22 * want.abs() + softcap * 2.0 ** -148 * (1 + z.abs()) + 2.0 ** -149
    if softcap < 1:
        tol += 2.0 ** -23 * softcap
    else:
        tol += 2.0 ** -21 * z.abs()  # 1 / c itself: a denormal of 21 bits
    assert ((got[1:].double() - want).abs() <= tol).all()


@pytest.mark.parametrize("repetition,temperature", [(2.0 ** -127, 1.0), (1.0, 2.0 ** -127),
                                                    (3e38, 1.0), (1.0, 3e38)])
def test_smallest_and_largest_divisors(repetition, temperature):
    x = torch.tensor([[0.0, 1.0, -1.0, 2.0 ** -100, -float("inf"), 0.5]], device=DEV)
    tok = torch.arange(5, device=DEV)[None]
    out = flce.process_logits(x, tokens=tok, lengths=torch.tensor([5], device=DEV),
                              repetition_penalty=repetition, temperature=temperature)
    want = S.process_row(x[0].cpu().numpy(), history=range(5), repetition=repetition,
                         temperature=temperature, dtype=np.float32)
    got = out["logits"][0].cpu().numpy()
    assert np.array_equal(got, want) and not np.isnan(got).any()
    assert out["greedy"].item() == int(np.argmax(want))

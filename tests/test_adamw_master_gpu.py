"""Autograd sees that an AdamW step writes to the fp32 copies of bf16 weights."""
import pytest
import torch

from linear_cross_entropy_tile_amd import flce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("kind", ["f32", "8bit"])
def test_a_graph_that_saved_a_copy_refuses_its_backward(kind):
    p = [torch.ones(50, device=DEV, dtype=torch.bfloat16), torch.ones(7, device=DEV)]
    state = flce.adamw_state(p, kind, master=True)
    assert state["master"][1] is None
    copy = state["master"][0].requires_grad_(True)
    loss = (copy * copy).sum()
    with torch.no_grad():
        flce.adamw_step(p, [torch.ones_like(t) for t in p], state)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        flce.adamw_step(p, [torch.ones_like(t) for t in p], state)
    assert int(state["step"]) == 2

"""Tensors that an AdamW step would write twice are refused, wherever they stand."""
import pytest
import torch

from linear_cross_entropy_tile_amd import flce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_one_tensor_in_two_places():
    p = [torch.ones(300, device=DEV, dtype=torch.bfloat16) for _ in range(2)]
    g = [t.clone() for t in p]
    f32, eight = flce.adamw_state(p, master=True), flce.adamw_state(p, "8bit", True)
    bad = [{**f32, "exp_avg_sq": f32["exp_avg"]}, {**f32, "master": f32["exp_avg"]},
           {**f32, "master": [f32["master"][0]] * 2}, {**eight, "master": [None] * 2,
                                                       "exp_avg_sq": eight["exp_avg"][::-1]},
           {**eight, "exp_avg_sq_scale": eight["exp_avg_scale"]},
           {**eight, "exp_avg_scale": [eight["exp_avg_scale"][1]] * 2}]
    for state in bad:
        with pytest.raises(ValueError, match="twice"):
            flce.adamw_step(p, g, state)
    assert int(f32["step"]) == int(eight["step"]) == 0 and all((t == 1).all() for t in p)


def test_empty_tensors_and_missing_copies_are_no_doubles():
    p = [torch.ones(n, device=DEV, dtype=t) for n, t in
         ((0, torch.float32), (5, torch.float32), (0, torch.bfloat16), (7, torch.bfloat16),
          (9, torch.float32))]
    g = [t.clone() for t in p]
    for kind in ("f32", "8bit"):
        state = flce.adamw_state(p, kind, True)
        flce.adamw_step(p, g, state, lr=0.5)
        assert int(state["step"]) == 1 and not any((t == 1).any() for t in p)
        for t in p:
            t.fill_(1)

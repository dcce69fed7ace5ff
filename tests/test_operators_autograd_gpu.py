"""The autograd functions with gradients and leaves as other operators make them."""
import pytest
import torch

import gpu_helpers as G
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

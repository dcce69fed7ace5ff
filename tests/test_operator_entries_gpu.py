"""The operators' C entry points through their Python functions of the same name
(pointers, sizes, options, stream): equal bits with the torch calls, on a stream
of the caller's."""
import pytest
import torch

import gpu_helpers as G
from linear_cross_entropy_tile_amd import flce

pytestmark = pytest.mark.gpu

N, H, V = 300, 64, 203
CU = [0, 70, 70, 131, 200, 241, 290]


def _f32(*shape):
    return torch.full(shape, 7.0, device=G.dev())


def _workspace(nbytes):
    return torch.full((nbytes,), 255, dtype=torch.uint8, device=G.dev())


def _p(*tensors):
    return [t.data_ptr() for t in tensors]


@pytest.fixture
def stream():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        yield s.cuda_stream
    torch.cuda.current_stream().wait_stream(s)


def _tokens():
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    tok = torch.randint(0, V, (N,), generator=g, device=G.dev())
    tok[::7] = -100
    tok[5] = V + 1
    return g, tok


@pytest.mark.parametrize("layout", ["vh", "hv"])
def test_embedding_entries(layout, stream):
    g, tok = _tokens()
    w = torch.randn((V, H) if layout == "vh" else (H, V), generator=g, device=G.dev())
    w = w.to(torch.bfloat16)
    up = torch.randn(N, H, generator=g, device=G.dev())
    opt = flce.FlceEmbeddingOptions(-100, 2.5, flce.FLCE_EMBED_HV if layout == "hv"
                                    else flce.FLCE_EMBED_VH, flce.FLCE_GRAD_F32,
                                    flce.FLCE_GRAD_F32, 1)
    fb, bb = flce.flce_embedding_workspace_size(N, H, V, opt)
    ws = _workspace(max(fb, bb))
    hidden = torch.full((N, H), 7.0, dtype=torch.bfloat16, device=G.dev())
    flce.flce_embedding_forward(*_p(w, tok), N, H, V, 0, V, opt, *_p(hidden, ws), fb, stream)
    kw = dict(layout=layout, scale=2.5)
    assert torch.equal(hidden, flce.embedding(w, tok, **kw)["hidden"])
    assert flce.flce_get_status(ws.data_ptr(), stream) == 1
    gw = w.float()
    flce.flce_embedding_backward(*_p(up, tok), N, H, V, 0, V, opt, *_p(gw, ws), bb, stream)
    assert torch.equal(gw, flce.embedding_backward(up, tok, V, grad_weight=w.float(), **kw))
    with pytest.raises(flce.FlceError, match="flce_embedding_forward: FLCE_ERR_WORKSPACE"):
        flce.flce_embedding_forward(*_p(w, tok), N, H, V, 0, V, opt, *_p(hidden, ws), 16, stream)
    with pytest.raises(flce.FlceError, match="flce_embedding_backward: FLCE_ERR_BAD_SHAPE"):
        flce.flce_embedding_backward(*_p(up, tok), N, H, V, 1, V, opt, *_p(gw, ws), bb, stream)


def test_policy_entries(stream):
    g, lab = _tokens()
    lp, old, ref, ent, adv = (-torch.rand(N, generator=g, device=G.dev()) for _ in range(5))
    cu = torch.tensor(CU, device=G.dev())
    B = len(CU) - 1
    opt = flce.FlcePolicyOptions(-100, 0.2, 0.3, 3.0, 0.1, 0.01, 2, 0, flce.FLCE_REDUCTION_MEAN, 0)
    kw = dict(clip_low=0.2, clip_high=0.3, dual_clip=3.0, kl_coef=0.1, entropy_coef=0.01,
              ref_logprob=ref, cu_seqlens=cu, vocab_size=V)
    want = flce.policy_loss_forward_backward(lp, lab, old, adv, entropy=ent, **kw)
    nb = flce.flce_policy_workspace_size(N, B)
    ws, up = _workspace(nb), torch.ones(1, device=G.dev())
    loss, stats, glp, gent = _f32(1), _f32(8), _f32(N), _f32(N)
    state = torch.zeros(B + 1, 2, dtype=torch.float64, device=G.dev())
    flce.flce_policy_loss_forward(*_p(lp, ent, old, ref, adv, lab, cu), N, B, V, opt,
                                  *_p(loss, stats, state, ws), nb, stream)
    assert torch.equal(stats, want["stats"]) and torch.equal(loss, stats[:1])
    flce.flce_policy_loss_backward(*_p(lp, old, ref, adv, lab, cu), N, B, V, opt,
                                   *_p(state, up, glp, gent), stream)
    assert torch.equal(glp, want["grad_logprob"]) and torch.equal(gent, want["grad_entropy"])
    for t in (loss, stats, glp, gent):
        t.fill_(7.0)
    flce.flce_policy_loss_forward_backward(*_p(lp, ent, old, ref, adv, lab, cu), N, B, V, opt,
                                           *_p(up, loss, stats, glp, gent, ws), nb, stream)
    for got, name in ((loss, "loss"), (stats, "stats"), (glp, "grad_logprob"),
                      (gent, "grad_entropy")):
        assert torch.equal(got, want[name]), name
    with pytest.raises(flce.FlceError, match="flce_policy_loss_forward: FLCE_ERR_NULL_POINTER"):
        flce.flce_policy_loss_forward(None, *_p(ent, old, ref, adv, lab, cu), N, B, V, opt,
                                      *_p(loss, stats, state, ws), nb, stream)


def test_preference_entries(stream):
    g, lab = _tokens()
    lp, ref = (-torch.rand(N, generator=g, device=G.dev()) for _ in range(2))
    cu = torch.tensor(CU, device=G.dev())
    P = (len(CU) - 1) // 2
    opt = flce.FlcePreferenceOptions(-100, 0.3, 0.1, 0.2, 0, 1, flce.FLCE_REDUCTION_SUM)
    want = flce.preference_loss_forward_backward(lp, lab, cu, ref_logprob=ref, beta=0.3,
                                                 label_smoothing=0.1, margin=0.2,
                                                 length_normalize=True, reduction="sum",
                                                 vocab_size=V)
    nb = flce.flce_preference_workspace_size(N, P)
    ws, up = _workspace(nb), torch.ones(1, device=G.dev())
    loss, pair, chosen, rejected, glp = _f32(1), _f32(P), _f32(P), _f32(P), _f32(N)
    state = torch.zeros(2 * P + 1, dtype=torch.float64, device=G.dev())
    outs = ((loss, "loss"), (pair, "pair_loss"), (chosen, "chosen_reward"),
            (rejected, "rejected_reward"), (glp, "grad_logprob"))
    flce.flce_preference_loss_forward(*_p(lp, ref, lab, cu), N, P, V, opt,
                                      *_p(loss, pair, chosen, rejected, state, ws), nb, stream)
    flce.flce_preference_loss_backward(*_p(lab, cu), N, P, V, opt, *_p(state, up, glp), stream)
    for got, name in outs:
        assert torch.equal(got, want[name]), name
        got.fill_(7.0)
    flce.flce_preference_loss_forward_backward(*_p(lp, ref, lab, cu), N, P, V, opt,
                                               *_p(up, loss, pair, chosen, rejected, glp, ws), nb,
                                               stream)
    for got, name in outs:
        assert torch.equal(got, want[name]), name
    with pytest.raises(flce.FlceError, match="flce_preference_loss_backward: FLCE_ERR_BAD_SHAPE"):
        flce.flce_preference_loss_backward(*_p(lab, cu), N, 0, V, opt, *_p(state, up, glp), stream)

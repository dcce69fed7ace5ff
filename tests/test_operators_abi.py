"""Argument checks of the embedding, policy and preference entry points on the
host (no device work), and of their torch wrappers."""
import ctypes

import pytest
import torch

from linear_cross_entropy_tile_amd import flce, function

A = 0x1000
BIG = 1 << 40


def _embed(fn="forward", **kw):
    o = dict(ii=-100, scale=1.0, layout=1, hdt=0, gdt=0, acc=0)
    a = dict(x=A, tokens=A, N=4, H=8, V=10, vb=0, vt=10, out=A, ws=A, wsb=BIG)
    for k, v in kw.items():
        (o if k in o else a)[k] = v
    opt = flce.FlceEmbeddingOptions(o["ii"], o["scale"], o["layout"], o["hdt"], o["gdt"], o["acc"])
    f = flce.lib().flce_embedding_forward if fn == "forward" else flce.lib().flce_embedding_backward
    return f(a["x"], a["tokens"], a["N"], a["H"], a["V"], a["vb"], a["vt"], ctypes.byref(opt),
             a["out"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("fn", ["forward", "backward"])
@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(tokens=None), 1), (dict(out=None), 1), (dict(ws=None), 1),
    (dict(N=-1), 2), (dict(N=(1 << 21) + 1), 2), (dict(H=0), 2), (dict(V=0), 2),
    (dict(V=(1 << 22)), 2), (dict(vb=-1), 2), (dict(vb=1), 2), (dict(vt=9), 2),
    (dict(vb=(1 << 63) - 1), 2), (dict(vb=(1 << 63) - 5), 2),
    (dict(vt=1 << 23), 2),
    (dict(H=12), 4), (dict(x=A + 8), 4), (dict(out=A + 4), 4), (dict(ws=A + 8), 4),
    (dict(tokens=A + 4), 4), (dict(wsb=16), 5),
    (dict(scale=float("nan")), 9), (dict(scale=float("inf")), 9), (dict(scale=1e39), 9),
    (dict(layout=2), 9), (dict(hdt=2), 9), (dict(gdt=-1), 9), (dict(acc=2), 9),
])
def test_embedding_rejects(fn, kw, code):
    assert _embed(fn, **kw) == code


def _policy_opt(**kw):
    o = dict(ii=-100, lo=0.2, hi=0.2, dual=0.0, kl=0.0, ent=0.0, est=2, level=0, red=1, aps=0)
    o.update(kw)
    return flce.FlcePolicyOptions(o["ii"], o["lo"], o["hi"], o["dual"], o["kl"], o["ent"],
                                  o["est"], o["level"], o["red"], o["aps"])


def _policy(which, **kw):
    a = dict(lp=A, e=A, old=A, ref=A, adv=A, lab=A, cu=A, N=4, B=2, V=10, g=None, loss=None, stats=A,
             state=A, glp=A, gent=A, ws=A, wsb=BIG)
    o = {k: kw.pop(k) for k in list(kw) if k not in a}
    a.update(kw)
    opt = ctypes.byref(_policy_opt(**o))
    L = flce.lib()
    if which == "forward":
        return L.flce_policy_loss_forward(a["lp"], a["e"], a["old"], a["ref"], a["adv"], a["lab"],
                                          a["cu"], a["N"], a["B"], a["V"], opt, a["loss"],
                                          a["stats"], a["state"], a["ws"], a["wsb"], None)
    if which == "backward":
        return L.flce_policy_loss_backward(a["lp"], a["old"], a["ref"], a["adv"], a["lab"],
                                           a["cu"], a["N"], a["B"], a["V"], opt, a["state"],
                                           a["g"], a["glp"], a["gent"], None)
    return L.flce_policy_loss_forward_backward(a["lp"], a["e"], a["old"], a["ref"], a["adv"],
                                               a["lab"], a["cu"], a["N"], a["B"], a["V"], opt,
                                               a["g"], a["loss"], a["stats"], a["glp"], a["gent"], a["ws"],
                                               a["wsb"], None)


POLICY_BAD = [
    (dict(lp=None), 1), (dict(old=None), 1), (dict(adv=None), 1), (dict(lab=None), 1),
    (dict(kl=0.1, ref=None), 1),
    (dict(N=-1), 2), (dict(N=(1 << 21) + 1), 2), (dict(B=0), 2), (dict(B=(1 << 21) + 1), 2),
    (dict(V=0), 2), (dict(V=1 << 22), 2), (dict(cu=None), 2),
    (dict(red=0), 3), (dict(red=4), 3),
    (dict(lp=A + 2), 4), (dict(lab=A + 4), 4), (dict(cu=A + 4), 4), (dict(adv=A + 1), 4),
    (dict(lo=-0.1), 9), (dict(lo=1.1), 9), (dict(hi=-1.0), 9), (dict(hi=float("inf")), 9),
    (dict(lo=float("nan")), 9), (dict(dual=1.0), 9), (dict(dual=-2.0), 9),
    (dict(kl=float("nan")), 9), (dict(ent=float("inf")), 9), (dict(est=3), 9), (dict(level=2), 9),
    (dict(aps=2), 9), (dict(level=1, aps=0), 9), (dict(level=1, aps=1, cu=None, B=1), 9),
]


@pytest.mark.parametrize("which", ["forward", "backward", "both"])
@pytest.mark.parametrize("kw,code", POLICY_BAD)
def test_policy_rejects(which, kw, code):
    assert _policy(which, **kw) == code


@pytest.mark.parametrize("which,kw,code", [
    ("forward", dict(stats=None), 1), ("forward", dict(state=None), 1),
    ("forward", dict(ws=None), 1), ("forward", dict(ent=0.1, e=None), 1),
    ("forward", dict(wsb=300), 5), ("forward", dict(state=A + 4), 4), ("forward", dict(ws=A + 8), 4),
    ("forward", dict(loss=A + 2), 4),
    ("backward", dict(state=None), 1), ("backward", dict(glp=None), 1),
    ("backward", dict(gent=A + 2), 4),
    ("both", dict(glp=None), 1), ("both", dict(stats=None), 1), ("both", dict(wsb=300), 5),
])
def test_policy_rejects_outputs(which, kw, code):
    assert _policy(which, **kw) == code


def _pref(which, **kw):
    a = dict(lp=A, ref=A, lab=A, cu=A, N=4, P=2, V=10, g=None, loss=A, pair=A, c=A, r=A, state=A,
             glp=A, ws=A, wsb=BIG)
    o = dict(ii=-100, beta=0.1, eps=0.0, margin=0.0, kind=0, norm=0, red=1)
    for k, v in kw.items():
        (o if k in o else a)[k] = v
    opt = ctypes.byref(flce.FlcePreferenceOptions(o["ii"], o["beta"], o["eps"], o["margin"],
                                                  o["kind"], o["norm"], o["red"]))
    L = flce.lib()
    if which == "forward":
        return L.flce_preference_loss_forward(a["lp"], a["ref"], a["lab"], a["cu"], a["N"], a["P"],
                                              a["V"], opt, a["loss"], a["pair"], a["c"], a["r"],
                                              a["state"], a["ws"], a["wsb"], None)
    if which == "backward":
        return L.flce_preference_loss_backward(a["lab"], a["cu"], a["N"], a["P"], a["V"], opt,
                                               a["state"], a["g"], a["glp"], None)
    return L.flce_preference_loss_forward_backward(a["lp"], a["ref"], a["lab"], a["cu"], a["N"],
                                                   a["P"], a["V"], opt, a["g"], a["loss"],
                                                   a["pair"], a["c"], a["r"], a["glp"], a["ws"],
                                                   a["wsb"], None)


@pytest.mark.parametrize("which", ["forward", "backward", "both"])
@pytest.mark.parametrize("kw,code", [
    (dict(lab=None), 1), (dict(cu=None), 1),
    (dict(N=-1), 2), (dict(N=(1 << 21) + 1), 2), (dict(P=0), 2), (dict(P=(1 << 20) + 1), 2),
    (dict(V=0), 2), (dict(red=3), 3), (dict(lab=A + 4), 4), (dict(cu=A + 2), 4),
    (dict(beta=0.0), 9), (dict(beta=-1.0), 9), (dict(beta=float("nan")), 9),
    (dict(beta=float("inf")), 9), (dict(eps=-0.1), 9), (dict(eps=0.6), 9),
    (dict(margin=float("inf")), 9), (dict(kind=3), 9), (dict(kind=-1), 9),
    (dict(kind=1, eps=0.1), 9), (dict(kind=2, eps=0.1), 9), (dict(kind=2, margin=0.1), 9),
    (dict(norm=2), 9),
])
def test_preference_rejects(which, kw, code):
    assert _pref(which, **kw) == code


@pytest.mark.parametrize("which,kw,code", [
    ("forward", dict(lp=None), 1), ("forward", dict(loss=None), 1), ("forward", dict(pair=None), 1),
    ("forward", dict(c=None), 1), ("forward", dict(r=None), 1), ("forward", dict(state=None), 1),
    ("forward", dict(ws=None), 1), ("forward", dict(wsb=300), 5),
    ("forward", dict(state=A + 4), 4), ("backward", dict(state=None), 1),
    ("backward", dict(glp=None), 1), ("both", dict(glp=None), 1), ("both", dict(lp=None), 1),
])
def test_preference_rejects_outputs(which, kw, code):
    assert _pref(which, **kw) == code


def test_workspace_sizes():
    opt = flce.FlceEmbeddingOptions(-100, 1.0, 1, 0, 0, 0)
    f, b = flce.flce_embedding_workspace_size(8192, 2304, 256000, opt)
    # sorted keys and positions; strip starts and the split runs' fp32 rows.
    assert f >= 8 * 8192 and b >= f + 4 * 4001 + 8 * 256 * 2304
    assert flce.flce_embedding_workspace_size(0, 8, 1, opt)[0] >= 256
    assert flce.flce_policy_workspace_size(0, 1) >= 256
    assert flce.flce_policy_workspace_size(1 << 21, 1 << 21) >= 48 * 2 * (1 << 21)
    assert flce.flce_preference_workspace_size(1 << 21, 1 << 20) >= 24 * 2 * (1 << 21)
    for bad in [(-1, 1), (1, 0), ((1 << 21) + 1, 1)]:
        with pytest.raises(flce.FlceError):
            flce.flce_policy_workspace_size(*bad)
        with pytest.raises(flce.FlceError):
            flce.flce_preference_workspace_size(*bad)


def test_wrappers_reject_host_tensors_and_options():
    w = torch.zeros(8, 10, dtype=torch.bfloat16)
    t = torch.zeros(4, dtype=torch.int64)
    x = torch.zeros(4)
    with pytest.raises(ValueError, match="weight must be a CUDA"):
        flce.embedding(w, t)
    with pytest.raises(ValueError, match="grad_hidden must be a bf16 or fp32"):
        flce.embedding_backward(torch.zeros(4, 8, dtype=torch.float16), t, 10)
    with pytest.raises(ValueError, match="labels must be a CUDA"):
        flce.policy_loss(x, t, x, x)
    with pytest.raises(ValueError, match="level must be one of"):
        flce.policy_loss(x, t, x, x, level="word")
    with pytest.raises(ValueError, match="reduction must be one of"):
        flce.policy_loss(x, t, x, x, reduction="none")
    with pytest.raises(ValueError, match="kl_estimator must be one of"):
        flce.policy_loss_forward_backward(x, t, x, x, kl_estimator="k4")
    with pytest.raises(TypeError):
        flce.policy_loss(x, t, x, x, clip=0.2)
    # The autograd functions keep no workspace for their backward.
    for fn, args in ((function.policy_loss, (x, t, x, x)), (function.preference_loss, (x, t, t))):
        with pytest.raises(TypeError, match="workspace"):
            fn(*args, workspace=x)
    with pytest.raises(ValueError, match="kind must be one of"):
        flce.preference_loss(x, t, t, kind="margin")
    with pytest.raises(ValueError, match="logprob must be a CUDA"):
        flce.preference_loss(x, t, t)

"""The float64 oracle of the embedding, policy loss and preference loss: its
gradients against central differences of its values, and closed forms."""
import numpy as np
import pytest

from oracle import operators_oracle as O

CU = [0, 5, 5, 9, 16, 20]  # an empty sequence among them


def _policy_inputs(seed, N=22):
    r = np.random.default_rng(seed)
    lp = -r.exponential(1.0, N)
    lab = r.integers(0, 50, N)
    lab[[1, 9, 10, 11]] = -100
    lab[13] = 99
    return dict(logprob=lp, labels=lab, old_logprob=lp + r.normal(0, 0.3, N),
                ref_logprob=lp + r.normal(0, 0.2, N), entropy=r.exponential(1.0, N),
                advantages=r.normal(0, 1, N), vocab_size=60)


@pytest.mark.parametrize("reduction", ["mean", "sum", "sequence_mean"])
@pytest.mark.parametrize("level", ["token", "sequence"])
@pytest.mark.parametrize("kl", ["k1", "k2", "k3"])
@pytest.mark.parametrize("dual", [0.0, 1.2])
def test_policy_gradient_is_the_difference_quotient(reduction, level, kl, dual):
    x = _policy_inputs(3)
    kw = dict(cu_seqlens=CU, level=level, reduction=reduction, kl_coef=0.3, kl_estimator=kl,
              entropy_coef=0.07, dual_clip=dual)
    if level == "sequence":
        x["advantages"] = x["advantages"][:5]
        kw["advantages_per_sequence"] = True
    got = O.policy_loss(**x, **kw)
    h = 1e-6
    for name, grad in (("logprob", got["grad_logprob"]), ("entropy", got["grad_entropy"])):
        for t in range(22):
            v = []
            for s in (h, -h):
                y = dict(x)
                y[name] = x[name].copy()
                y[name][t] += s
                v.append(O.policy_loss(**y, **kw)["stats"][0])
            # Second-order error of the quotient: h^2 |f'''| / 6 and 2^-53 |f| / h.
            assert abs((v[0] - v[1]) / (2 * h) - grad[t]) < 1e-8
    assert np.all(got["grad_logprob"][[1, 9, 10, 11, 13, 20, 21]] == 0.0)


def test_policy_closed_forms():
    one = dict(labels=[1], entropy=[2.0], ref_logprob=[-1.0], entropy_coef=0.5)
    for r, A, dual, want, clip in [(1.5, 1.0, 0, -1.2, 1), (1.1, 1.0, 0, -1.1, 0),
                                   (0.5, 1.0, 0, -0.5, 0), (0.5, -1.0, 0, 0.8, 1),
                                   (5.0, -1.0, 0, 5.0, 0), (5.0, -1.0, 3.0, 3.0, 1),
                                   (5.0, 0.0, 3.0, 0.0, 0)]:
        st = O.policy_loss(logprob=[-1.0], old_logprob=[-1.0 - np.log(r)], advantages=[A],
                           dual_clip=dual, **one)["stats"]
        assert np.allclose(st, [want - 1.0, want, 0.0, 2.0, clip, -np.log(r), 1, 1], atol=1e-14)


@pytest.mark.parametrize("kind,kw", [("sigmoid", {}), ("sigmoid", dict(label_smoothing=0.2,
                                                                       margin=0.3)),
                                     ("hinge", dict(margin=0.1)), ("ipo", {})])
@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
@pytest.mark.parametrize("normalize", [False, True])
def test_preference_gradient_is_the_difference_quotient(kind, kw, reduction, normalize):
    r = np.random.default_rng(5)
    cu = [0, 4, 4, 9, 15, 18, 20]
    lp = -r.exponential(1.0, 21)
    ref = lp + r.normal(0, 0.5, 21)
    lab = r.integers(0, 9, 21)
    lab[[2, 10]] = -100
    up = r.normal(size=3) if reduction == "none" else np.array([1.7])
    kw = dict(kw, kind=kind, reduction=reduction, length_normalize=normalize, beta=0.4,
              ref_logprob=ref, labels=lab, cu_seqlens=cu, grad_loss=up)
    got = O.preference_loss(lp, **kw)
    h = 1e-6
    for t in range(21):
        v = []
        for s in (h, -h):
            y = lp.copy()
            y[t] += s
            v.append(float((O.preference_loss(y, **kw)["loss"] * up).sum()))
        assert abs((v[0] - v[1]) / (2 * h) - got["grad_logprob"][t]) < 1e-8


def test_embedding_gradient_is_the_transpose():
    r = np.random.default_rng(1)
    table, g = r.normal(size=(7, 4)), r.normal(size=(9, 4))
    tok = np.array([3, 0, 3, -100, 9, 6, 3, 0, -1])
    out = O.embedding(table, tok, scale=1.5)
    grad, mag, count = O.embedding_backward(g, tok, 7, scale=1.5)
    assert np.isclose((out * g).sum(), (table * grad).sum(), rtol=1e-13)
    assert count.tolist() == [2, 0, 0, 3, 0, 0, 1] and np.all(mag >= np.abs(grad) - 1e-15)
    half = (O.embedding(table[:3], tok, scale=1.5, v_begin=0)
            + O.embedding(table[3:], tok, scale=1.5, v_begin=3))
    assert np.array_equal(half, out)

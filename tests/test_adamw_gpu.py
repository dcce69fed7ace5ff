"""Norm of the gradients and AdamW (flce.grad_norm, flce.adamw_step) on the GPU
against the oracle: moments, codes and scales to the bit, weights within the
update's rounding."""
import numpy as np
import pytest
import torch

from linear_cross_entropy_tile_amd import flce
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KW = dict(lr=2e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
SIZES = [1, 7, 8, 255, 256, 257, 4095, 4096, 4097, 70001, 0, 3]
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _tensors(sizes, dtype, gen, std=1.0, shift=0):
    """One tensor a size, each ``shift`` elements behind an aligned address."""
    out = []
    for n in sizes:
        t = torch.empty(n + shift, device=DEV, dtype=TYPES[dtype])[shift:]
        t.copy_(torch.randn(n, generator=gen, device=DEV) * std)
        out.append(t)
    return out


def _np(t):
    return t.detach().float().cpu().numpy().reshape(-1)


def _snapshot(state):
    return {k: (None if v is None else v.clone() if isinstance(v, torch.Tensor)
                else [None if t is None else t.clone() for t in v]) for k, v in state.items()}


def _check(params, grads, state, before, p0, kw, scale=1.0, rounding="nearest", seed=0):
    t = int(state["step"])
    assert t == int(before["step"]) + 1
    eight = before["exp_avg_scale"] is not None
    mismatched = total = 0
    for i, (p, g) in enumerate(zip(params, grads)):
        n = p.numel()
        if n == 0:
            continue
        m0, v0 = _np(before["exp_avg"][i]), _np(before["exp_avg_sq"][i])
        if eight:
            blk = np.arange(n) // 256
            m0 = m0 * _np(before["exp_avg_scale"][i])[blk]
            r0 = v0 * _np(before["exp_avg_sq_scale"][i])[blk]
            v0 = r0 * r0
        w = before["master"][i] if before["master"] is not None else None
        start = _np(p0[i] if w is None else w)
        p1, m1, v1, r1, change = S.adamw_f32(start, _np(g), m0, v0, t, grad_scale=scale, **kw)
        bits = S.random_bits(seed, t, i, n) if rounding == "stochastic" else (None,) * 3
        if eight:
            for kind, x, b, pos in (("exp_avg", m1, bits[1], False), ("exp_avg_sq", r1, bits[2],
                                                                      True)):
                codes, scales = S.encode_f32(x, b, pos)
                assert np.array_equal(_np(state[kind + "_scale"][i]), scales), (i, kind)
                assert np.array_equal(_np(state[kind][i]), codes.astype(np.float32)), (i, kind)
        else:
            assert np.array_equal(_np(state["exp_avg"][i]), m1), i
            assert np.array_equal(_np(state["exp_avg_sq"][i]), v1), i
        # The update's root and reciprocal are within 1 ulp (2^-23) each, twice counted
        # by the products around them; the two last operations round to the nearest.
        tol = 8 * 2.0 ** -23 * change + 2.0 ** -23 * (np.abs(p1) + change)
        got = _np(p)
        if w is not None:
            assert (np.abs(_np(state["master"][i]) - p1) <= tol).all(), i
            assert np.array_equal(got, S.bf16_nearest(_np(state["master"][i]))), i
        elif p.dtype == torch.float32:
            assert (np.abs(got - p1) <= tol).all(), i
        elif rounding == "nearest":
            assert (np.abs(got - p1) <= tol + 2.0 ** -8 * np.abs(p1) + 1e-38).all(), i
        else:
            want = S.bf16_stochastic(p1, bits[0])
            off = got != want
            # Where the last bits of p1 differ, a value next to a border may go the other way.
            assert (np.abs(got - p1)[off] <= (2.0 ** -7 * np.abs(p1) + tol)[off]).all(), i
            mismatched, total = mismatched + int(off.sum()), total + n
    # tol is some 2^-22 of a weight, a border's width 2^-8 of it: one in 2^12 at most.
    assert mismatched <= 4 + total / 1024


@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("dtype,gdtype,kind,master,rounding", [
    ("f32", "f32", "f32", False, "nearest"), ("bf16", "bf16", "f32", False, "nearest"),
    ("bf16", "f32", "f32", False, "stochastic"), ("bf16", "bf16", "f32", True, "stochastic"),
    ("f32", "bf16", "8bit", False, "nearest"), ("bf16", "bf16", "8bit", False, "stochastic"),
    ("bf16", "f32", "8bit", True, "stochastic"), ("f32", "f32", "8bit", False, "stochastic"),
    ("bf16", "f32", "8bit", False, "nearest"), ("bf16", "bf16", "8bit", True, "nearest"),
])
def test_steps(dtype, gdtype, kind, master, rounding, shift):
    gen = torch.Generator(device=DEV).manual_seed(len(dtype) + shift)
    params = _tensors(SIZES, dtype, gen, 1.0, shift)
    state = flce.adamw_state(params, kind, master)
    assert (state["master"] is not None) == master
    if shift:  # states at odd addresses too
        for k in ("exp_avg", "exp_avg_sq"):
            state[k] = [torch.zeros(t.numel() + shift, device=DEV, dtype=t.dtype)[shift:]
                        for t in state[k]]
    for s in range(3):
        grads = _tensors(SIZES, gdtype, gen, 10.0 ** -s, shift)
        grads[5][:] = 0
        before, p0 = _snapshot(state), [p.clone() for p in params]
        scale = torch.tensor([0.37], device=DEV) if s else None
        seed = 5 + (s << 40)
        flce.adamw_step(params, grads, state, grad_scale=scale, rounding=rounding, seed=seed, **KW)
        _check(params, grads, state, before, p0, KW, np.float32(0.37) if s else 1.0, rounding, seed)


def test_many_tensors_of_mixed_types():
    """More tensors than a launch's table holds, types and master copies mixed."""
    gen = torch.Generator(device=DEV).manual_seed(2)
    sizes = [(i * 37) % 600 for i in range(130)]
    params = [t for i, n in enumerate(sizes)
              for t in _tensors([n], "bf16" if i % 3 else "f32", gen)]
    grads = [t for i, n in enumerate(sizes)
             for t in _tensors([n], "bf16" if i % 2 else "f32", gen)]
    for kind in ("f32", "8bit"):
        state = flce.adamw_state(params, kind, master=True)
        state["master"][4] = None  # a bf16 tensor without a copy among those with one
        before, p0 = _snapshot(state), [p.clone() for p in params]
        flce.adamw_step(params, grads, state, rounding="stochastic", seed=3, **KW)
        _check(params, grads, state, before, p0, KW, rounding="stochastic", seed=3)
    out = flce.grad_norm(grads, max_norm=0.5)
    want = np.sqrt(sum(float(g.double().square().sum()) for g in grads))
    assert abs(out["norm"].item() - want) <= 2.0 ** -23 * want
    assert abs(out["scale"].item() - 0.5 / want) <= 2.0 ** -23 * 0.5 / want


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sizes", [[1], [5, 0, 8], [4096], [4097], [100003, 1], [9000001, 17],
                                   [0]])
def test_norm(sizes, dtype):
    gen = torch.Generator(device=DEV).manual_seed(sum(sizes))
    for shift in (0, 1):
        grads = _tensors(sizes, dtype, gen, 3.0, shift)
        want = float(sum(g.double().square().sum() for g in grads) ** 0.5)
        for most in (0.0, 1e9, 0.25):
            out = flce.grad_norm(grads, max_norm=most)
            # Rounded to fp32 once; the float64 sum's own error is far below.
            assert abs(out["norm"].item() - want) <= 2.0 ** -23 * want
            s = min(1.0, most / want) if most and want else 1.0
            assert abs(out["scale"].item() - s) <= 2.0 ** -23
        again = flce.grad_norm(grads, max_norm=0.25)
        assert torch.equal(out["norm"], again["norm"]) and torch.equal(out["scale"], again["scale"])


def test_norm_of_extreme_values():
    """Squares that fp32 cannot hold; infinities and NaN make the factor NaN."""
    for value in (3e38, 1e-40, 1e-30):
        g = [torch.full((1000,), value, device=DEV)]
        want = float(g[0].double().square().sum().sqrt())
        out = flce.grad_norm(g, max_norm=1.0)
        assert out["norm"].item() == (np.float32(want) if want < 3.4e38 else np.inf)
        assert not torch.isnan(out["scale"]).any()
    for value in (float("inf"), float("nan"), -float("inf")):
        g = [torch.ones(10, device=DEV), torch.ones(5000, device=DEV, dtype=torch.bfloat16)]
        g[1][4999] = value
        for most in (0.0, 1.0):
            out = flce.grad_norm(g, max_norm=most)
            assert torch.isnan(out["scale"]).all() and not torch.isfinite(out["norm"]).any()


@pytest.mark.parametrize("kind", ["f32", "8bit"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_factor_that_is_not_finite_changes_nothing(kind, value):
    gen = torch.Generator(device=DEV).manual_seed(1)
    params, grads = _tensors([300, 5000], "bf16", gen), _tensors([300, 5000], "bf16", gen)
    state = flce.adamw_state(params, kind, master=True)
    flce.adamw_step(params, grads, state, **KW)
    before, p0 = _snapshot(state), [p.clone() for p in params]
    grads[0][5] = value
    scale = flce.grad_norm(grads, max_norm=1.0)["scale"]
    flce.adamw_step(params, grads, state, grad_scale=scale, **KW)
    assert int(state["step"]) == 1
    flat = lambda s: [t for v in s.values() if v is not None  # noqa: E731
                      for t in (v if isinstance(v, list) else [v]) if t is not None]
    for a, b in zip(flat(state) + params, flat(before) + p0):
        assert torch.equal(a.view(torch.uint8) if a.element_size() == 1 else a,
                           b.view(torch.uint8) if b.element_size() == 1 else b)


def test_against_torch_over_many_steps():
    """fp32 weights follow torch.optim.AdamW over 50 steps in float64: each step's
    update is within 2^-19 of itself and rounds the weight by 2^-24 of it."""
    gen = torch.Generator(device=DEV).manual_seed(4)
    p = _tensors([2000, 33], "f32", gen)
    ref = [torch.nn.Parameter(t.double()) for t in p]
    opt = torch.optim.AdamW(ref, lr=1e-2, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    state = flce.adamw_state(p)
    lr = torch.tensor([1e-2], device=DEV)
    for _ in range(50):
        g = _tensors([2000, 33], "f32", gen)
        for r, x in zip(ref, g):
            r.grad = x.double()
        opt.step()
        flce.adamw_step(p, g, state, lr=lr, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
    # The moments' own rounding, 2^-22 of them after a mean of 20 steps, moves an update
    # by as much of itself; an update is below 3 lr.
    assert max((a.double() - b).abs().max() for a, b in zip(p, ref)) < 50 * (
        3e-2 * 2.0 ** -19 + 4 * 2.0 ** -23)


def test_stochastic_rounding_moves_weights_that_nearest_leaves():
    """An update of 1/32 of a bf16 step: lost in every step, or kept on average."""
    n = 1 << 16
    moved = {}
    for rounding in ("nearest", "stochastic"):
        p = [torch.ones(n, device=DEV, dtype=torch.bfloat16)]
        state = flce.adamw_state(p)
        for s in range(32):
            flce.adamw_step(p, [torch.ones(n, device=DEV)], state, lr=2.0 ** -13,
                            weight_decay=0.0, rounding=rounding, seed=9)
        moved[rounding] = float((1.0 - p[0].double()).mean())
    assert moved["nearest"] == 0.0
    # 32 steps of 2^-13, each rounded by less than 2^-8: five standard errors.
    assert abs(moved["stochastic"] - 32 * 2.0 ** -13) < 5 * 2.0 ** -9 * 32 ** 0.5 / n ** 0.5


def test_eight_bit_states_follow_fp32_ones():
    """A second moment that decays by 5 % a step follows it on average under
    stochastic rounding, though a code's steps are up to 12 % apart."""
    gen = torch.Generator(device=DEV).manual_seed(7)
    n = 1 << 14
    p = [torch.zeros(n, device=DEV)]
    s8, s32 = flce.adamw_state(p, "8bit"), flce.adamw_state(p)
    q = [torch.zeros(n, device=DEV)]
    for k in range(30):
        g = _tensors([n], "f32", gen, 1.0 if k < 5 else 0.02)
        flce.adamw_step(p, g, s8, rounding="stochastic", seed=k, **KW)
        flce.adamw_step(q, g, s32, **KW)
    r8 = s8["exp_avg_sq"][0].float() * s8["exp_avg_sq_scale"][0].repeat_interleave(256)
    r32 = s32["exp_avg_sq"][0].sqrt()
    # Roots: each step rounds by up to 12 %, 25 times, but independently over values.
    assert abs(float(r8.mean() / r32.mean()) - 1) < 0.02
    assert (r8 > 0).all()


def test_captured_step_on_a_side_stream():
    """Norm, clip and update in a graph: the step's count, the learning rate and the
    factor follow the device over replays."""
    gen = torch.Generator(device=DEV).manual_seed(3)
    sizes = [5000, 77]
    params, grads = _tensors(sizes, "bf16", gen), _tensors(sizes, "bf16", gen)
    eager, lr = [p.clone() for p in params], torch.tensor([1e-2], device=DEV)
    state, state2 = flce.adamw_state(params, "8bit", True), flce.adamw_state(eager, "8bit", True)
    kw = dict(beta1=0.9, beta2=0.95, rounding="stochastic", seed=77)

    def step(ps, st):
        norm = flce.grad_norm(grads, max_norm=1.0)
        flce.adamw_step(ps, grads, st, lr=lr, grad_scale=norm["scale"], **kw)
        return norm["norm"]

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = step(params, state)
    for k in range(4):
        lr.mul_(0.5)
        for g in grads:
            g.mul_(-1.5)
        graph.replay()
        torch.cuda.synchronize()
        want = step(eager, state2)
        assert torch.equal(norm, want) and int(state["step"]) == k + 1
        for a, b in zip(params + state["master"] + state["exp_avg_scale"],
                        eager + state2["master"] + state2["exp_avg_scale"]):
            assert torch.equal(a, b), k


def test_two_streams_update_two_lists_at_once():
    gen = torch.Generator(device=DEV).manual_seed(3)
    lists = [(_tensors([60001], "f32", gen), _tensors([60001], "f32", gen)) for _ in range(2)]
    want = []
    for p, g in lists:
        q = [t.clone() for t in p]
        st = flce.adamw_state(q)
        for _ in range(5):
            flce.adamw_step(q, g, st, **KW)
        want.append(q)
    states = [flce.adamw_state(p) for p, _ in lists]
    streams = [torch.cuda.Stream() for _ in lists]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s, (p, g), st in zip(streams, lists, states):
            with torch.cuda.stream(s):
                flce.adamw_step(p, g, st, **KW)
    torch.cuda.synchronize()
    for (p, _), q in zip(lists, want):
        assert torch.equal(p[0], q[0])


def test_step_counts_far_along():
    """Corrections after 2^40 steps are 1; the count goes on."""
    p, g = [torch.ones(10, device=DEV)], [torch.ones(10, device=DEV)]
    state = flce.adamw_state(p)
    state["step"].fill_(1 << 40)
    flce.adamw_step(p, g, state, lr=0.5, beta1=0.5, beta2=0.5, eps=0.0, weight_decay=0.0)
    # m = 1/2, v = 1/2: the update is lr sqrt(1/2).
    assert int(state["step"]) == (1 << 40) + 1
    assert abs(p[0][0].item() - (1 - 0.5 * 0.5 ** 0.5)) < 4 * 2.0 ** -24


def test_denormal_gradients_without_eps():
    """g = 1e-21, whose square is a denormal: the root is taken exactly enough."""
    p, g = [torch.ones(8, device=DEV)], [torch.full((8,), 1e-21, device=DEV)]
    for kind in ("f32", "8bit"):
        q = [p[0].clone()]
        state = flce.adamw_state(q, kind)
        flce.adamw_step(q, g, state, lr=0.25, beta1=0.0, beta2=0.0, eps=0.0, weight_decay=0.0)
        # v = 1e-42 is a multiple of 2^-149 within 2^-150, a part of 7e-4 of it.
        assert abs(q[0][0].item() - 0.75) < 0.25 * 1e-3


def test_a_step_between_forward_and_backward_is_noticed():
    """Autograd sees the update: a graph that saved the weight refuses its backward."""
    w = torch.ones(50, device=DEV, requires_grad=True)
    loss = (w * w).sum()
    state = flce.adamw_state([w])
    with torch.no_grad():
        flce.adamw_step([w], [torch.ones(50, device=DEV)], state)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():
        p = [torch.ones(50, device=DEV)]
        flce.adamw_step(p, [torch.ones(50, device=DEV)], flce.adamw_state(p))


def test_refusals():
    p = [torch.ones(300, device=DEV), torch.ones(4, device=DEV, dtype=torch.bfloat16)]
    g = [t.clone() for t in p]
    st = flce.adamw_state(p)
    s8 = flce.adamw_state(p, "8bit", True)
    ok = dict(params=p, grads=g, state=st)
    bad = [dict(params=p[0]), dict(params=[]), dict(params=[t.cpu() for t in p]),
           dict(params=[t.half() for t in p]), dict(grads=g[:1]), dict(grads=[g[0][:299], g[1]]),
           dict(grads=[torch.ones(300, 2, device=DEV)[:, 0], g[1]]),
           dict(grad_scale=torch.ones(2, device=DEV)), dict(lr=torch.ones(1, device=DEV).double()),
           dict(rounding="up"), dict(params=[p[0], p[0][:4]]),
           dict(params=[p[0], p[0]], grads=[g[0], g[0]]),
           dict(state={**st, "exp_avg": [st["exp_avg"][0], st["exp_avg"][0][:4]]}),
           dict(state={**st, "exp_avg": s8["exp_avg"]}),
           dict(state={**st, "exp_avg_sq": st["exp_avg"][:1]}),
           dict(state={**st, "step": torch.zeros(1, device=DEV)}),
           dict(state={**s8, "exp_avg_scale": [t[:1] for t in s8["exp_avg_scale"]]}),
           dict(state={**st, "master": [p[0], None]}),
           dict(state={**st, "master": [None]})]
    for kw in bad:
        with pytest.raises(ValueError):
            flce.adamw_step(**{**ok, **kw})
    for kw in (dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1e-8), dict(lr=float("nan")),
               dict(weight_decay=float("inf")), dict(lr=1e300)):
        with pytest.raises(flce.FlceError, match="BAD_OPTION"):
            flce.adamw_step(**{**ok, **kw})
    for bad_state in ("16bit", None):
        with pytest.raises(ValueError):
            flce.adamw_state(p, bad_state)
    with pytest.raises(ValueError):
        flce.grad_norm([])
    with pytest.raises(ValueError):
        flce.grad_norm(p[0])
    with pytest.raises(flce.FlceError, match="BAD_OPTION"):
        flce.grad_norm(g, max_norm=-1.0)
    assert int(st["step"]) == 0 and (p[0] == 1).all()

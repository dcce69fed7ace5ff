"""Argument checks of the entry points for logits, their processing, the gradients'
norm and AdamW on the host (no device work), of their torch wrappers, and their
planner under sanitizers (tests/host/step_plan_check.cpp)."""
import ctypes
import os
import shutil
import subprocess
import tempfile

import pytest
import torch

from linear_cross_entropy_tile_amd import flce, function

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x1000
BIG = 1 << 40
NAN, INF = float("nan"), float("inf")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_step_planner_under_sanitizers():
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "step_plan_check")
        cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer",
               "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
               "-I" + os.path.join(ROOT, "include"),
               "-I" + os.path.join(ROOT, "linear_cross_entropy_tile_amd", "csrc"),
               os.path.join(ROOT, "tests", "host", "step_plan_check.cpp"), "-o", exe]
        subprocess.run(cmd, check=True, capture_output=True, text=True)
        env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
                   UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
        res = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=300)
        assert res.returncode == 0, res.stdout + res.stderr
        assert "failures: 0" in res.stdout, res.stdout


def _logits(**kw):
    a = dict(h=A, w=A, b=None, N=4, H=8, V=10, cap=0.0, dt=1, out=A, ld=10, ws=A, wsb=BIG)
    a.update(kw)
    return flce.lib().flce_logits(a["h"], a["w"], a["b"], a["N"], a["H"], a["V"], a["cap"],
                                  a["dt"], a["out"], a["ld"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(h=None), 1), (dict(w=None), 1), (dict(out=None), 1), (dict(ws=None), 1),
    (dict(N=-1), 2), (dict(N=1025), 2), (dict(H=0), 2), (dict(H=(1 << 20) + 8), 2),
    (dict(V=0), 2), (dict(V=1 << 22, ld=1 << 22), 2), (dict(ld=9), 2), (dict(ld=1 << 41), 2),
    (dict(H=12), 4), (dict(h=A + 8), 4), (dict(w=A + 2), 4), (dict(out=A + 2), 4),
    (dict(b=A + 2), 4), (dict(ws=A + 8), 4), (dict(wsb=100), 5), (dict(cap=NAN), 6),
    (dict(cap=INF), 6), (dict(dt=2), 9), (dict(N=0, ws=None), 1),
])
def test_logits_rejects(kw, code):
    assert _logits(**kw) == code


def test_logits_of_no_rows_launch_nothing():
    assert _logits(N=0, h=None, w=None, out=None) == 0


def _options(**kw):
    o = flce.FlceProcessOptions()
    for k, v in {**dict(ignore_index=-100, tokens=A, tokens_size=40, tokens_stride=10, offsets=A,
                        repetition_penalty=1.5, temperature=1.0, bias_stride=0, logits_dtype=1,
                        out_dtype=1), **kw}.items():
        setattr(o, k, v)
    return o


def _process(which, **kw):
    a = dict(x=A, ld=10, N=4, V=10, out=2 * A, ldo=10, lse=A, ent=A, top=A, ws=A, wsb=BIG,
             grad=3 * A, ldg=10, go=2 * A, gl=None, ge=None)
    own = {k: kw.pop(k) for k in list(kw) if k in a}
    a.update(own)
    opt = ctypes.byref(_options(**kw))
    if which == "forward":
        return flce.lib().flce_process_logits(a["x"], a["ld"], a["N"], a["V"], opt, a["out"],
                                              a["ldo"], a["lse"], a["ent"], a["top"], a["ws"],
                                              a["wsb"], None)
    g = flce.FlceProcessGrads(a["go"], a["ldo"], a["gl"], a["ge"], a["out"], a["ldo"], a["lse"],
                              a["ent"])
    return flce.lib().flce_process_logits_backward(ctypes.byref(g), a["x"], a["ld"], a["N"],
                                                   a["V"], opt, a["grad"], a["ldg"], a["ws"],
                                                   a["wsb"], None)


@pytest.mark.parametrize("which", ["forward", "backward"])
@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(ws=None), 1), (dict(offsets=None), 1), (dict(tokens=None), 1),
    (dict(bias_offsets=A, bias_count=3), 1), (dict(bias_tokens=A), 1),
    (dict(bias_offsets=A, bias_count=3, bias_tokens=A), 1),
    (dict(N=-1), 2), (dict(N=(1 << 21) + 1), 2), (dict(V=0), 2), (dict(V=1 << 22), 2),
    (dict(ld=9), 2), (dict(ldo=9), 2), (dict(tokens_stride=11), 2), (dict(tokens_stride=-1), 2),
    (dict(tokens_size=-1), 2), (dict(tokens_size=39), 2), (dict(bias=A, bias_stride=9), 2),
    (dict(allowed=A, allowed_stride=-1), 2), (dict(bias_count=-1), 2),
    (dict(tokens_size=1 << 62, tokens_stride=1 << 61), 2),
    (dict(tokens=A + 4), 4), (dict(offsets=A + 4), 4), (dict(prompt_lengths=A + 4), 4),
    (dict(repetition=A + 2), 4), (dict(presence=A + 1), 4), (dict(frequency=A + 2), 4),
    (dict(temperatures=A + 2), 4), (dict(bias=A + 2), 4), (dict(allowed=A + 2), 4),
    (dict(x=A + 2), 4), (dict(ws=A + 8), 4), (dict(wsb=300), 5),
    (dict(repetition_penalty=0.0), 9), (dict(repetition_penalty=-1.0), 9),
    (dict(repetition_penalty=NAN), 9), (dict(repetition_penalty=INF), 9),
    (dict(presence_penalty=INF), 9), (dict(frequency_penalty=NAN), 9),
    (dict(temperature=-0.5), 9), (dict(temperature=NAN), 9), (dict(logits_dtype=2), 9),
    (dict(out_dtype=-1), 9),
])
def test_process_rejects(which, kw, code):
    assert _process(which, **kw) == code


@pytest.mark.parametrize("which,kw,code", [
    ("forward", dict(out=None), 1), ("forward", dict(out=2 * A + 2), 4),
    ("forward", dict(lse=A + 2), 4), ("forward", dict(ent=A + 1), 4),
    ("forward", dict(top=A + 4), 4),
    ("forward", dict(out=A, out_dtype=0), 9), ("forward", dict(out=A, ldo=11), 9),
    ("backward", dict(grad=None), 1), ("backward", dict(gl=A, out=None), 1),
    ("backward", dict(gl=A, lse=None), 1), ("backward", dict(ge=A, ent=None), 1),
    ("backward", dict(grad=3 * A + 2), 4), ("backward", dict(gl=A + 2), 4),
    ("backward", dict(ldg=9), 2), ("backward", dict(grad=2 * A, ldg=12), 9),
    ("backward", dict(grad=2 * A, logits_dtype=0), 9),
])
def test_process_rejects_outputs(which, kw, code):
    assert _process(which, **kw) == code


def test_process_rejects_no_options():
    assert flce.lib().flce_process_logits(A, 10, 4, 10, None, A, 10, A, A, A, A, BIG, None) == 1
    o = _options()
    assert flce.lib().flce_process_logits_backward(None, A, 10, 4, 10, ctypes.byref(o), A, 10, A,
                                                   BIG, None) == 1


def _norm(**kw):
    a = dict(g=[A, A], n=[4, 5], d=[0, 1], count=2, most=1.0, norm=A, scale=A, ws=A, wsb=BIG)
    a.update(kw)
    n = max(1, len(a["n"]))
    return flce.lib().flce_grad_norm((ctypes.c_void_p * n)(*a["g"]) if a["g"] else None,
                                     (ctypes.c_int64 * n)(*a["n"]), (ctypes.c_int * n)(*a["d"]),
                                     a["count"], a["most"], a["norm"], a["scale"], a["ws"],
                                     a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(g=[A, None]), 1), (dict(g=None), 1), (dict(norm=None), 1), (dict(ws=None), 1),
    (dict(count=-1), 2), (dict(count=(1 << 20) + 1), 2), (dict(n=[4, -1]), 2),
    (dict(n=[4, (1 << 35) + 1]), 2), (dict(g=[A + 1, A]), 4), (dict(g=[A, A + 2]), 4),
    (dict(norm=A + 2), 4), (dict(scale=A + 2), 4), (dict(ws=A + 4), 4), (dict(wsb=260), 5),
    (dict(d=[0, 2]), 9), (dict(most=-1.0), 9), (dict(most=NAN), 9), (dict(most=INF), 9),
])
def test_norm_rejects(kw, code):
    assert _norm(**kw) == code


def _adamw(**kw):
    """The second of two tensors, the lists, options and arguments as ``kw`` says."""
    t = dict(size=10, param=A, grad=A, master=None, exp_avg=A, exp_avg_sq=A, exp_avg_scale=None,
             exp_avg_sq_scale=None, param_dtype=0, grad_dtype=0)
    o = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, state_dtype=0,
             rounding=0, seed=0)
    a = dict(tensors=True, count=2, without=None, opt=True, lrd=None, scale=None, step=A, ws=A,
             wsb=BIG)
    for k, v in kw.items():
        next(d for d in (t, o, a) if k in d)[k] = v
    first = dict(t, size=10, param=A, grad=A, master=None, exp_avg=A, exp_avg_sq=A,
                 exp_avg_scale=A, exp_avg_sq_scale=A, param_dtype=1, grad_dtype=1)
    kinds = {"size": ctypes.c_int64, "param_dtype": ctypes.c_int, "grad_dtype": ctypes.c_int}
    arrays = [(kinds.get(k, ctypes.c_void_p) * 2)(first[k], t[k]) for k in t]
    table = flce.FlceAdamwList(a["count"], *[
        None if a["without"] == k else ctypes.addressof(x) for k, x in zip(t, arrays)])
    return flce.lib().flce_adamw_step(ctypes.byref(table) if a["tensors"] else None,
                                      ctypes.byref(flce.FlceAdamwOptions(*o.values()))
                                      if a["opt"] else None, a["lrd"], a["scale"], a["step"],
                                      a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(tensors=False), 1), (dict(opt=False), 1), (dict(step=None), 1), (dict(ws=None), 1),
    (dict(param=None), 1), (dict(grad=None), 1), (dict(exp_avg=None), 1),
    (dict(exp_avg_sq=None), 1), (dict(state_dtype=1), 1),
    (dict(state_dtype=1, exp_avg_scale=A), 1), (dict(without="size"), 1),
    (dict(without="param"), 1), (dict(without="grad"), 1), (dict(without="exp_avg"), 1),
    (dict(without="exp_avg_sq"), 1), (dict(without="param_dtype"), 1),
    (dict(without="grad_dtype"), 1),
    (dict(without="exp_avg_scale", state_dtype=1, exp_avg_sq_scale=A), 1),
    (dict(count=-1), 2), (dict(count=(1 << 20) + 1), 2), (dict(size=-1), 2),
    (dict(size=(1 << 35) + 1), 2),
    (dict(param=A + 1), 4), (dict(grad=A + 1), 4), (dict(grad=A + 2, grad_dtype=1), 4),
    (dict(master=A + 2), 4), (dict(exp_avg=A + 2), 4), (dict(exp_avg_sq=A + 1), 4),
    (dict(state_dtype=1, exp_avg_scale=A + 2, exp_avg_sq_scale=A), 4),
    (dict(step=A + 4), 4), (dict(lrd=A + 2), 4), (dict(scale=A + 1), 4), (dict(ws=A + 8), 4),
    (dict(wsb=300), 5),
    (dict(lr=NAN), 9), (dict(lr=INF), 9), (dict(lr=1e39), 9), (dict(beta1=1.0), 9),
    (dict(beta1=-0.1), 9), (dict(beta2=1.0), 9), (dict(beta2=NAN), 9), (dict(eps=-1.0), 9),
    (dict(eps=1e39), 9), (dict(weight_decay=NAN), 9), (dict(weight_decay=1e50), 9),
    (dict(state_dtype=2), 9), (dict(rounding=2), 9), (dict(param_dtype=2), 9),
    (dict(grad_dtype=-1), 9), (dict(master=A, param_dtype=1), 9),
])
def test_adamw_rejects(kw, code):
    assert _adamw(**kw) == code


def test_workspace_sizes():
    assert flce.flce_logits_workspace_size(1, 4096, 128256) >= 256
    # Tiles: 256 tokens of the hidden rows; splits: fp32 sums.
    assert flce.flce_logits_workspace_size(200, 4096, 128256) >= 256 * 4096 * 2
    assert flce.flce_logits_workspace_size(8, 4096, 1000) >= 2 * 4 * 8 * 1000
    assert flce.flce_process_workspace_size(0, 1) >= 256
    assert flce.flce_process_workspace_size(64, 128256) >= 64 * 16 * 32
    assert flce.flce_adamw_workspace_size() == flce._ADAMW_BYTES
    n = (ctypes.c_int64 * 2)(10, 1 << 30)
    assert flce.flce_grad_norm_workspace_size(n, 2) >= 8 * 4096
    assert flce.flce_grad_norm_workspace_size(None, 0) >= 256
    for f, args in ((flce.flce_logits_workspace_size, (1025, 8, 8)),
                    (flce.flce_logits_workspace_size, (1, 12, 8)),
                    (flce.flce_process_workspace_size, (-1, 8)),
                    (flce.flce_process_workspace_size, (1, 0)),
                    (flce.flce_grad_norm_workspace_size, (None, 1))):
        with pytest.raises(flce.FlceError):
            f(*args)


def test_wrappers_reject_host_tensors():
    x, w = torch.zeros(4, 8), torch.zeros(8, 10, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="hidden must be a CUDA"):
        flce.logits(x.bfloat16(), w)
    with pytest.raises(ValueError, match="logits must be a CUDA"):
        flce.process_logits(x)
    with pytest.raises(ValueError, match="logits must be a CUDA"):
        flce.process_logits_backward(x, x)
    with pytest.raises(TypeError):
        flce.process_logits(x, top_k=5)
    with pytest.raises(ValueError, match="logits must be a CUDA"):
        function.process_logits(x)
    with pytest.raises(ValueError, match="workspace belongs"):
        function.process_logits(x, workspace=x)
    with pytest.raises(ValueError, match=r"grads\[0\] must be a CUDA"):
        flce.grad_norm([x])
    with pytest.raises(ValueError, match="params must have a tensor"):
        flce.adamw_state([])
    with pytest.raises(ValueError, match="params must be a list"):
        flce.adamw_step(x, [x], {})
    with pytest.raises(ValueError, match="state must be one of"):
        flce.adamw_state([x], "4bit")

"""The operators at the ends of a training step from plain C99 (tests/c_abi/
flce_step_check.c, built with gcc against include/flce.h and the in-tree library), run as
a child process; and their C entry points through the Python functions of the same name:
equal bits with the torch calls, on a stream of the caller's."""
import ctypes
import os
import subprocess

import pytest
import torch

from linear_cross_entropy_tile_amd import flce

pytestmark = pytest.mark.gpu

BIN = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c_abi", "flce_step_check")
DEV = "cuda:0"


def test_c_program():
    assert os.path.exists(BIN), f"{BIN} missing: run __graft_entry__.build() first"
    res = subprocess.run([BIN], capture_output=True, text=True, timeout=120)
    print(res.stdout, res.stderr, flush=True)
    assert res.returncode == 0, res.stdout + res.stderr
    assert "flce_step_check ok" in res.stdout


@pytest.fixture
def stream():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        yield s.cuda_stream
    torch.cuda.current_stream().wait_stream(s)


def _workspace(nbytes):
    return torch.full((nbytes,), 255, dtype=torch.uint8, device=DEV)


def test_logits_and_processing_entries(stream):
    N, H, V = 5, 64, 203
    h = torch.randn(N, H, device=DEV, dtype=torch.bfloat16)
    w = torch.randn(H, V, device=DEV, dtype=torch.bfloat16)
    ws = _workspace(flce.flce_logits_workspace_size(N, H, V))
    z = torch.empty(N, V, device=DEV)
    flce.flce_logits(h.data_ptr(), w.data_ptr(), None, N, H, V, 3.0, flce.FLCE_GRAD_F32,
                     z.data_ptr(), V, ws.data_ptr(), ws.numel(), stream)
    assert torch.equal(z, flce.logits(h, w, softcap=3.0)["logits"])

    tok, lens = torch.randint(0, V, (N, 9), device=DEV), torch.full((N,), 7, device=DEV)
    opt = flce.FlceProcessOptions(ignore_index=-100, tokens=tok.data_ptr(), tokens_size=9 * N,
                                  tokens_stride=9, offsets=lens.data_ptr(),
                                  repetition_penalty=1.5, frequency_penalty=0.5, temperature=0.7,
                                  logits_dtype=1, out_dtype=1)
    kw = dict(tokens=tok, lengths=lens, repetition_penalty=1.5, frequency_penalty=0.5,
              temperature=0.7)
    ws = _workspace(flce.flce_process_workspace_size(N, V))
    y, lse = torch.empty_like(z), torch.empty(N, device=DEV)
    flce.flce_process_logits(z.data_ptr(), V, N, V, opt, y.data_ptr(), V, lse.data_ptr(), None,
                             None, ws.data_ptr(), ws.numel(), stream)
    want = flce.process_logits(z, **kw)
    assert torch.equal(y, want["logits"]) and torch.equal(lse, want["lse"])
    assert flce.flce_get_status(ws.data_ptr(), stream) == 0
    g, gz = torch.randn(N, V, device=DEV), torch.empty_like(z)
    up = flce.FlceProcessGrads(grad_out=g.data_ptr(), ld_grad_out=V)
    flce.flce_process_logits_backward(up, z.data_ptr(), V, N, V, opt, gz.data_ptr(), V,
                                      ws.data_ptr(), ws.numel(), stream)
    assert torch.equal(gz, flce.process_logits_backward(g, z, **kw))


def test_update_entries(stream):
    p, g = torch.randn(1000, device=DEV), torch.randn(1000, device=DEV)
    q = p.clone()
    state = flce.adamw_state([q])
    m, v = torch.zeros(1000, device=DEV), torch.zeros(1000, device=DEV)
    step = torch.zeros(1, dtype=torch.int64, device=DEV)
    sizes, dtypes = (ctypes.c_int64 * 1)(1000), (ctypes.c_int * 1)(flce.FLCE_GRAD_F32)

    def one(t):
        return (ctypes.c_void_p * 1)(t.data_ptr())

    ws = _workspace(max(flce.flce_grad_norm_workspace_size(sizes, 1),
                        flce.flce_adamw_workspace_size()))
    out = torch.empty(2, device=DEV)
    flce.flce_grad_norm(one(g), sizes, dtypes, 1, 1.0, out.data_ptr(), out[1:].data_ptr(),
                        ws.data_ptr(), ws.numel(), stream)
    norm = flce.grad_norm([g], max_norm=1.0)
    assert torch.equal(out[:1], norm["norm"]) and torch.equal(out[1:], norm["scale"])
    keep = [sizes, one(p), one(g), one(m), one(v), dtypes]
    a = [ctypes.addressof(x) for x in keep]
    table = flce.FlceAdamwList(1, a[0], a[1], a[2], None, a[3], a[4], None, None, a[5], a[5])
    opt = flce.FlceAdamwOptions(1e-2, 0.9, 0.95, 1e-8, 0.1, flce.FLCE_STATE_F32,
                                flce.FLCE_ROUND_NEAREST, 0)
    flce.flce_adamw_step(table, opt, None, out[1:].data_ptr(), step.data_ptr(), ws.data_ptr(),
                         ws.numel(), stream)
    flce.adamw_step([q], [g], state, lr=1e-2, beta2=0.95, weight_decay=0.1,
                    grad_scale=norm["scale"])
    assert torch.equal(p, q) and torch.equal(m, state["exp_avg"][0]) and int(step) == 1

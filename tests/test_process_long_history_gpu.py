"""Histories around the 32767 tokens from which on they are counted in 32 bits, in
vocabularies on both sides of a slice and of half a slice, with ids outside the
vocabulary: logits to the bit against the definition's fp32 operations, statistics
against float64, and the count of what is no id."""
import numpy as np
import pytest
import torch

from linear_cross_entropy_tile_amd import flce
from oracle import step_oracle as S

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
LENGTHS = [33001, 4, 32767, 32768, 0, 40000]
I64 = np.iinfo(np.int64)


def _history(rng, V, n, ignore):
    """n tokens: few ids all over the vocabulary (the ends of slices and of their halves
    among them), ignored ones and such as are no ids."""
    marks = [0, 1, 5, V - 1, V // 2] + [b + k for b in range(1024, V, 1024) for k in (-1, 0)][-12:]
    ids = np.unique(np.clip(marks + rng.integers(0, V, 9).tolist(), 0, V - 1))
    h = rng.choice(ids, n)
    if n > 100:
        none = [V, V + 1, V + 44, V + 1024, V + 1068, V + 1069, V + 2048, V + 4096, -1, 1 << 31,
                (1 << 32) + 1, 1 << 40, -(1 << 40), I64.min, I64.max, ignore]
        at = rng.choice(n, 6 * len(none), replace=False)
        h[at] = none * 6
    return h


def _case(N, V, seed, listed, ignore):
    rng = np.random.default_rng(seed)
    lens = [int(rng.integers(0, 9)) for _ in range(N)]
    for k, n in enumerate(LENGTHS):  # the long rows lie apart
        lens[k * N // len(LENGTHS)] = n
    hist = [_history(rng, V, n, ignore) for n in lens]
    prompt = [n // 3 for n in lens]
    r, p, f = (0.7 + rng.random(N), rng.normal(size=N), rng.normal(size=N) * 1e-3)
    r, p, f = (a.astype(np.float32) for a in (r, p, f))
    kw = dict(tokens=torch.from_numpy(np.concatenate(hist).astype(np.int64)).to(DEV),
              cu_seqlens=torch.from_numpy(np.concatenate([[0], np.cumsum(lens)])).to(DEV),
              prompt_lengths=torch.tensor(prompt, device=DEV),
              repetition_penalty=torch.from_numpy(r).to(DEV),
              presence_penalty=torch.from_numpy(p).to(DEV),
              frequency_penalty=torch.from_numpy(f).to(DEV), ignore_index=ignore)
    rows = [dict(history=hist[i], prompt=prompt[i], repetition=r[i], presence=p[i],
                 frequency=f[i], ignore_index=ignore) for i in range(N)]
    if listed:
        ids = [rng.integers(0, V, 5) for _ in range(N)]
        for a in ids:
            a[1] = a[0]
            a[2] = V + 7
        val = [rng.normal(size=5).astype(np.float32) for _ in range(N)]
        kw.update(bias_tokens=torch.from_numpy(np.concatenate(ids)).to(DEV),
                  bias_values=torch.from_numpy(np.concatenate(val)).to(DEV),
                  bias_cu_seqlens=torch.arange(0, 5 * N + 1, 5, device=DEV))
        for i in range(N):
            rows[i]["listed"] = list(zip(ids[i], val[i]))
    no_ids = sum(int(((h != ignore) & ((h < 0) | (h >= V))).sum()) for h in hist)
    return kw, rows, no_ids + (N if listed else 0)


# Six rows take slices of 2048 ids, and the larger batches slices of 4096.
@pytest.mark.parametrize("listed", [False, True], ids=["history", "listed"])
@pytest.mark.parametrize("N,V", [
    (6, 1), (6, 1000), (6, 1023), (6, 1024), (6, 1025), (6, 2047), (6, 2048), (6, 2049),
    (6, 3001), (6, 50257), (1030, 1000), (1030, 2047), (1030, 2048), (1030, 2049), (1030, 4095),
    (1030, 4096), (520, 4097), (520, 6143), (520, 6144), (520, 6145), (80, 50257)])
def test_rows_on_both_sides_of_32_bit_counts(N, V, listed):
    ignore = 5 if V % 2 else -100  # an id of the vocabulary may be the one to pass over
    kw, rows, no_ids = _case(N, V, N + V, listed, ignore)
    x = torch.randn(N, V, generator=torch.Generator(device=DEV).manual_seed(V), device=DEV) * 3
    before = x.clone()
    out = flce.process_logits(x, **kw)
    assert flce.flce_get_status(out["workspace"].data_ptr(), 0) == no_ids
    assert torch.equal(x, before)
    grad = flce.process_logits_backward(torch.ones_like(x), x, **{
        k: v for k, v in kw.items() if not k.startswith("bias")})
    long = {k * N // len(LENGTHS) for k in range(len(LENGTHS))}
    for i in sorted(long | {1, N - 1}):
        xi = x[i].cpu().numpy()
        want = S.process_row(xi, dtype=np.float32, **rows[i])
        assert np.array_equal(out["logits"][i].cpu().numpy(), want), i
        lse, entropy, greedy = S.row_stats(want)
        assert out["greedy"][i].item() == greedy, i
        # fp32 sums of at most 16 terms a thread, then merges: below 256 roundings of
        # them, and each exp within (|d| + 4) 2^-24 with |d| weighted by p.
        y = want.astype(np.float64)
        p = np.exp(y - lse)
        d = np.abs(y - y.max())
        spread = float((p * d).sum())
        assert abs(out["lse"][i].item() - lse) <= 2.0 ** -24 * (300 + 2 * spread + 2 * abs(lse)), i
        assert abs(out["entropy"][i].item() - entropy) <= 2.0 ** -24 * (
            600 * (1 + spread) + 2 * abs(entropy) + 3 * float((p * d * d).sum())), i
        first, second, _ = S.row_slope(xi, dtype=np.float32, **{
            k: rows[i][k] for k in ("history", "prompt", "repetition", "ignore_index")})
        assert np.array_equal(grad[i].cpu().numpy(), first * second), i


def test_what_lies_behind_the_vocabulary_changes_no_result():
    """A long history's ids of 1000 .. 8000 are none of a vocabulary of 1000."""
    V = 1000
    x = torch.randn(2, V, device=DEV)
    tok = torch.full((2, 40000), 7, dtype=torch.int64, device=DEV)
    kw = dict(lengths=torch.tensor([40000, 40000], device=DEV), frequency_penalty=1e-4,
              presence_penalty=0.5)
    want = flce.process_logits(x, tokens=tok, **kw)
    tok[:, 100:7100] = torch.arange(1000, 8000, device=DEV)
    tok[:, 7100:14100] = -torch.arange(1000, 8000, device=DEV)
    tok[:, 14100:] = 7
    got = flce.process_logits(x, tokens=tok, **kw)
    assert flce.flce_get_status(got["workspace"].data_ptr(), 0) == 2 * 14000
    keep = torch.arange(V, device=DEV) != 7
    assert torch.equal(got["logits"][:, keep], want["logits"][:, keep])
    n = np.float32(26000) * np.float32(1e-4)
    x7 = (x[:, 7].cpu().numpy() - n) - np.float32(0.5)
    assert np.array_equal(got["logits"][:, 7].cpu().numpy(), x7)
    y = got["logits"].double()
    assert torch.equal(got["greedy"], y.argmax(1))
    assert (got["lse"].double() - torch.logsumexp(y, 1)).abs().max() < 2.0 ** -24 * 330


def test_the_longest_row_and_a_longer_one():
    """2^31 - 1 occurrences are counted; a row of one more is refused."""
    most = (1 << 31) - 1
    tok = torch.zeros(1, most + 1, dtype=torch.int64, device=DEV)
    x = torch.ones(1, 3, device=DEV)
    kw = dict(tokens=tok, frequency_penalty=2.0 ** -20)
    out = flce.process_logits(x, lengths=torch.tensor([most], device=DEV), **kw)
    # The count rounds to 2^31 in fp32.
    assert out["logits"].tolist() == [[1.0 - 2048.0, 1.0, 1.0]] and out["greedy"].item() == 1
    assert flce.flce_get_status(out["workspace"].data_ptr(), 0) == 0
    packed = dict(tokens=tok[0], cu_seqlens=torch.tensor([0, most + 1], device=DEV))
    for history in (dict(tokens=tok, lengths=torch.tensor([most + 1], device=DEV)), packed):
        out = flce.process_logits(x, frequency_penalty=2.0 ** -20, **history)
        grad = flce.process_logits_backward(x, x, frequency_penalty=2.0 ** -20, **history)
        assert flce.flce_get_status(out["workspace"].data_ptr(), 0) == 1
        assert torch.isnan(out["logits"]).all() and out["greedy"].item() == -1
        assert torch.isnan(grad).all()

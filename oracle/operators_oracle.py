"""Float64 oracle of the operators beside the head: embedding, policy loss and
preference loss, written from their definitions (include/flce.h) with plain
loops over the sequences. Inputs are numpy arrays; every result is float64.
"""
from __future__ import annotations

import numpy as np


def _valid(labels, ignore_index, V):
    labels = np.asarray(labels)
    return (labels != ignore_index) & (labels >= 0) & (labels < V)


# ---------------------------------------------------------------- embedding

def embedding(table, tokens, scale=1.0, ignore_index=-100, v_begin=0, v_total=None):
    """scale * table[token - v_begin] for a table [V,H] (the slice [v_begin,
    v_begin + V) of v_total ids), zero rows for the other tokens."""
    table = np.asarray(table, dtype=np.float64)
    out = np.zeros((len(tokens), table.shape[1]))
    for i, x in enumerate(tokens):
        if x != ignore_index and v_begin <= x < v_begin + table.shape[0]:
            out[i] = scale * table[x - v_begin]
    return out


def embedding_backward(grad_hidden, tokens, V, scale=1.0, ignore_index=-100, v_begin=0):
    """(grad [V,H], sum of |terms| [V,H], positions [V]) of the lookup."""
    g = np.asarray(grad_hidden, dtype=np.float64)
    out = np.zeros((V, g.shape[1]))
    mag = np.zeros_like(out)
    count = np.zeros(V, dtype=np.int64)
    for i, x in enumerate(tokens):
        if x != ignore_index and v_begin <= x < v_begin + V:
            out[x - v_begin] += scale * g[i]
            mag[x - v_begin] += np.abs(scale * g[i])
            count[x - v_begin] += 1
    return out, mag, count


# ---------------------------------------------------------------- policy loss

def _policy_term(d, A, clip_low, clip_high, dual_clip):
    """(value, derivative by d, clipped) of the clipped policy term."""
    if A == 0.0:
        return 0.0, 0.0, False
    r = np.exp(d)
    value = -min(r * A, min(max(r, 1.0 - clip_low), 1.0 + clip_high) * A)
    clipped = value != -r * A
    if A < 0.0 and dual_clip > 0.0 and value > -dual_clip * A:
        value, clipped = -dual_clip * A, True
    return value, (0.0 if clipped else -r * A), clipped


def _kl(x, estimator):
    if estimator == "k1":
        return x, 1.0
    if estimator == "k2":
        return 0.5 * x * x, x
    return np.expm1(-x) + x, -np.expm1(-x)


def policy_loss(logprob, labels, old_logprob, advantages, entropy=None, ref_logprob=None,
                cu_seqlens=None, advantages_per_sequence=False, clip_low=0.2, clip_high=0.2,
                dual_clip=0.0, kl_coef=0.0, kl_estimator="k3", entropy_coef=0.0, level="token",
                reduction="mean", ignore_index=-100, vocab_size=(1 << 22) - 256, grad_loss=1.0):
    """{"stats" [8], "grad_logprob" [N], "grad_entropy" [N]}."""
    f64 = np.float64
    lp = np.asarray(logprob, dtype=f64)
    N = lp.size
    valid = _valid(labels, ignore_index, vocab_size)
    cu = [0, N] if cu_seqlens is None else [int(c) for c in cu_seqlens]
    seqs = []
    for s in range(len(cu) - 1):
        seqs.append([t for t in range(cu[s], cu[s + 1]) if valid[t]])
    n = sum(len(t) for t in seqs)
    q = sum(1 for t in seqs if t)
    stats = np.zeros(8)
    glp, gent = np.zeros(N), np.zeros(N)
    for s, tok in enumerate(seqs):
        if not tok:
            continue
        w = {"mean": 1.0 / n, "sum": 1.0, "sequence_mean": 1.0 / (len(tok) * q)}[reduction]
        d = {t: lp[t] - f64(old_logprob[t]) for t in tok}
        if level == "sequence":
            mean_d = sum(d.values()) / len(tok)
        for t in tok:
            A = f64(advantages[s if advantages_per_sequence else t])
            pg, dpg, clip = _policy_term(mean_d if level == "sequence" else d[t], A, clip_low,
                                         clip_high, dual_clip)
            kl = dkl = 0.0
            if ref_logprob is not None:
                kl, dkl = _kl(lp[t] - f64(ref_logprob[t]), kl_estimator)
            ent = f64(entropy[t]) if entropy is not None else 0.0
            loss = pg + (kl_coef * kl if kl_coef else 0.0) - (entropy_coef * ent
                                                              if entropy_coef else 0.0)
            stats[:6] += w * np.array([loss, pg, kl, ent, float(clip), -d[t]])
            glp[t] = grad_loss * w * (dpg + (kl_coef * dkl if kl_coef else 0.0))
            gent[t] = -grad_loss * w * entropy_coef
    stats[6], stats[7] = n, q
    return {"stats": stats, "grad_logprob": glp, "grad_entropy": gent}


# ---------------------------------------------------------------- preference loss

def preference_loss(logprob, labels, cu_seqlens, ref_logprob=None, kind="sigmoid", beta=0.1,
                    label_smoothing=0.0, margin=0.0, length_normalize=False, reduction="mean",
                    ignore_index=-100, vocab_size=(1 << 22) - 256, grad_loss=None):
    """{"loss" [1] or [P], "pair_loss", "chosen_reward", "rejected_reward" [P],
    "grad_logprob" [N]}."""
    lp = np.asarray(logprob, dtype=np.float64)
    ref = np.zeros_like(lp) if ref_logprob is None else np.asarray(ref_logprob, dtype=np.float64)
    valid = _valid(labels, ignore_index, vocab_size)
    cu = [int(c) for c in cu_seqlens]
    P = (len(cu) - 1) // 2
    R, share, toks = np.zeros(2 * P), np.ones(2 * P), []
    for s in range(2 * P):
        tok = [t for t in range(cu[s], cu[s + 1]) if valid[t]]
        toks.append(tok)
        if length_normalize and tok:
            share[s] = 1.0 / len(tok)
        R[s] = sum(lp[t] - ref[t] for t in tok) * share[s]
    pair, slope = np.zeros(P), np.zeros(P)
    for i in range(P):
        gap = R[i] - R[P + i]
        x = beta * gap - margin
        if kind == "sigmoid":
            e = label_smoothing
            pair[i] = (1 - e) * np.logaddexp(0.0, -x) + e * np.logaddexp(0.0, x)
            sig = np.exp(-np.logaddexp(0.0, -x))
            slope[i] = beta * (sig - (1 - e)) if e else -beta * np.exp(-np.logaddexp(0.0, x))
        elif kind == "hinge":
            pair[i] = max(0.0, 1.0 - x)
            slope[i] = -beta if x < 1.0 else 0.0
        else:
            pair[i] = (gap - 1.0 / (2.0 * beta)) ** 2
            slope[i] = 2.0 * (gap - 1.0 / (2.0 * beta))
    up = np.ones(P if reduction == "none" else 1) if grad_loss is None else np.asarray(
        grad_loss, dtype=np.float64)
    k = 1.0 / P if reduction == "mean" else 1.0
    glp = np.zeros_like(lp)
    for s in range(2 * P):
        i = s % P
        g = up[i if reduction == "none" else 0] * k * slope[i] * share[s]
        for t in toks[s]:
            glp[t] = g if s < P else -g
    loss = pair if reduction == "none" else np.array([k * pair.sum()])
    return {"loss": loss, "pair_loss": pair, "chosen_reward": beta * R[:P],
            "rejected_reward": beta * R[P:], "grad_logprob": glp}

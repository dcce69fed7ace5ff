"""Performance cases of the operators next to the fused head: the scaled
embedding lookup with its gradient by sorted tokens (``embedding``), the
clipped policy loss with a KL term (``policy``) and the paired preference loss
(``preference``).

Each case runs in one of two forms on the same inputs: ``own = False`` computes
the operator from elementary torch operations (32 bits, 64 for long sums,
comparisons against a clip border and differences that cancel), ``own = True``
calls this package. ``exact`` evaluates the definition in 64 bits.

Definitions. Embedding: hidden_i = scale * E[token_i] (row token_i of a [V,H]
table, or column token_i of the head's [H,V] weight), zero for ignored tokens;
its gradient is scale * (sum over the positions of a token of grad_hidden_i).
Policy loss: with d = logprob - old_logprob (its mean over a sequence at the
"sequence" level), ratio r = exp(d), advantage A and x = logprob - ref_logprob,
  token loss = -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A)
               (at most -dual_clip A where A < 0 and dual_clip is on)
               + kl_coef * kl(x) - entropy_coef * entropy,
averaged over valid tokens, summed, or averaged within and then over sequences.
Preference loss: R_s = the sum (or mean) over a sequence of logprob -
ref_logprob, x = beta (R_chosen - R_rejected) - margin, and
  sigmoid: -(1 - eps) log sigmoid(x) - eps log sigmoid(-x),  hinge: max(0, 1 - x),
  ipo: (R_chosen - R_rejected - 1 / (2 beta))^2.
"""
import math
import random

import numpy as np
import torch

own = False

IGNORE = -100
GEN_DEVICE = "cuda"


# ---------------------------------------------------------------- cases

def _emb(name, direction, layout, N, H, V, zipf, scale, grad="bf16", ignored=0.0):
    return {"name": name, "op": "embedding", "direction": direction, "layout": layout, "N": N,
            "H": H, "V": V, "zipf": zipf, "scale": scale, "grad": grad, "ignored": ignored}


def _pol(name, direction, B, lo, hi, prompt, level, reduction, kl, kl_coef, entropy_coef, dual):
    return {"name": name, "op": "policy", "direction": direction, "B": B, "lo": lo, "hi": hi,
            "prompt": prompt, "level": level, "reduction": reduction, "kl": kl,
            "kl_coef": kl_coef, "entropy_coef": entropy_coef, "dual": dual}


def _pref(name, direction, P, lo, hi, prompt, kind, beta, smoothing, margin, normalize, reduction,
          ref):
    return {"name": name, "op": "preference", "direction": direction, "P": P, "lo": lo, "hi": hi,
            "prompt": prompt, "kind": kind, "beta": beta, "smoothing": smoothing,
            "margin": margin, "normalize": normalize, "reduction": reduction, "ref": ref}


def listed():
    return [
        # One decoding step of 16 sequences through a tied, capped head's weight.
        _emb("embed_decode_tied", "forward", "hv", 16, 2304, 256000, 1.1, 48.0),
        # A prompt batch through the same weight: columns gathered from [H,V].
        _emb("embed_prompt_tied", "forward", "hv", 8192, 2304, 256000, 1.1, 48.0),
        # A rollout batch (16 x 2048 tokens) from a table of its own.
        _emb("embed_rollout_table", "forward", "vh", 32768, 5120, 152064, 1.1, 1.0),
        # The embedding's share of a tied weight's gradient, training step.
        _emb("embed_grad_tied", "backward", "hv", 8192, 2304, 256000, 1.1, 48.0),
        # Mid-size table, fp32 gradient, a tenth of the tokens ignored.
        _emb("embed_grad_table_f32", "backward", "vh", 4096, 4096, 32000, 0.0, 1.0, "f32", 0.1),
        # Small odd vocabulary: no row of the weight is aligned.
        _emb("embed_grad_odd", "backward", "hv", 300, 192, 1001, 0.0, 13.856, "bf16", 0.1),
        # A few short answers: latency of one loss call with its gradients.
        _pol("policy_small", "train", 4, 60, 140, 0.25, "token", "mean", "k3", 0.04, 0.0, 0.0),
        # 16 rollouts of 2048 with a 512-token prompt, entropy bonus, dual clip.
        _pol("policy_rollout", "train", 16, 2048, 2048, 0.25, "token", "sequence_mean", "k3",
             0.001, 0.001, 3.0),
        # Sequence-level ratios over ragged answers, through autograd.
        _pol("policy_sequence", "autograd", 256, 100, 2000, 0.25, "sequence", "sequence_mean",
             "k2", 0.01, 0.0, 0.0),
        # A whole rollout step: 2 M tokens in a thousand ragged sequences.
        _pol("policy_large", "train", 1000, 200, 3900, 0.2, "token", "mean", "k3", 0.001, 0.001,
             0.0),
        # A micro-batch of four pairs.
        _pref("preference_small", "autograd", 4, 40, 200, 0.3, "sigmoid", 0.1, 0.1, 0.0, False,
              "mean", True),
        # A thousand sequences, length-normalised, no reference model.
        _pref("preference_large", "train", 500, 200, 3900, 0.3, "sigmoid", 2.0, 0.0, 1.0, True,
              "mean", False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embedding", "policy", "preference"])
    if op == "embedding":
        direction = rng.choice(["forward", "backward"])
        layout = rng.choice(["hv", "vh"])
        H = 8 * _log_int(rng, 8, 640)
        V = _log_int(rng, 700, 256000)
        N = _log_int(rng, 1, 32768)
        if direction == "backward":
            while H * V > 2304 * 256000:
                H = max(8, H // 16 * 8)
        return _emb("drawn", direction, layout, N, H, V, rng.choice([0.0, 0.7, 1.1]),
                    rng.choice([1.0, 0.5, round(math.sqrt(H), 3)]), rng.choice(["bf16", "f32"]),
                    rng.choice([0.0, 0.1, 0.5]))
    lo = _log_int(rng, 1, 1500)
    hi = lo + _log_int(rng, 1, 2500)
    prompt = rng.choice([0.0, 0.1, 0.25, 0.5])
    # At most two million tokens, as in the largest listed case.
    most = 2000000 // hi
    if op == "policy":
        B = min(_log_int(rng, 1, 1000), most)
        level = rng.choice(["token", "token", "sequence"])
        return _pol("drawn", rng.choice(["train", "autograd", "forward"]), B, lo, hi, prompt,
                    level, rng.choice(["mean", "sum", "sequence_mean"]),
                    rng.choice(["none", "k1", "k2", "k3"]), rng.choice([0.001, 0.02, 0.1]),
                    rng.choice([0.0, 0.001, 0.01]), rng.choice([0.0, 2.0, 3.0]))
    kind = rng.choice(["sigmoid", "sigmoid", "hinge", "ipo"])
    return _pref("drawn", rng.choice(["train", "autograd", "forward"]), min(_log_int(rng, 1, 500), most // 2),
                 lo, hi, prompt, kind, rng.choice([0.05, 0.1, 0.5]),
                 rng.choice([0.0, 0.1]) if kind == "sigmoid" else 0.0,
                 rng.choice([0.0, 0.5]) if kind != "ipo" else 0.0, rng.random() < 0.4,
                 rng.choice(["mean", "sum", "none"]), rng.random() < 0.8)


def _lengths(case):
    """Sequence lengths of a case, the same for every seed."""
    n = case["B"] if case["op"] == "policy" else 2 * case["P"]
    rng = random.Random(f"{n} {case['lo']} {case['hi']}")
    return [rng.randint(case["lo"], case["hi"]) for _ in range(n)]


# ---------------------------------------------------------------- inputs

def _token_probs(V, s):
    p = np.arange(1, V + 1, dtype=np.float64) ** (-s)
    return p / p.sum()


def _tokens(gen, N, V, zipf, ignored):
    if zipf > 0.0:
        cdf = torch.from_numpy(np.cumsum(_token_probs(V, zipf))).to(GEN_DEVICE)
        u = torch.rand(N, generator=gen, device=GEN_DEVICE, dtype=torch.float64)
        t = torch.searchsorted(cdf, u).clamp_(max=V - 1)
    else:
        t = torch.randint(0, V, (N,), generator=gen, device=GEN_DEVICE)
    if ignored > 0.0:
        t = torch.where(torch.rand(N, generator=gen, device=GEN_DEVICE) < ignored,
                        torch.full_like(t, IGNORE), t)
    return t


def prepare(case, seed):
    gen = torch.Generator(device=GEN_DEVICE)
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        x = torch.randn(*shape, generator=gen, device=GEN_DEVICE, dtype=dtype)
        return x.mul_(std) if std != 1.0 else x

    st = {"case": case}
    if case["op"] == "embedding":
        N, H, V = case["N"], case["H"], case["V"]
        st["tokens"] = _tokens(gen, N, V, case["zipf"], case["ignored"])
        if case["direction"] == "forward":
            shape = (H, V) if case["layout"] == "hv" else (V, H)
            st["weight"] = normal(*shape, std=0.05, dtype=torch.bfloat16)
        else:
            st["grad_hidden"] = normal(N, H, std=1e-3, dtype=torch.bfloat16)
        return st

    lens = _lengths(case)
    cu = np.zeros(len(lens) + 1, dtype=np.int64)
    np.cumsum(lens, out=cu[1:])
    N = int(cu[-1])
    st["cu_seqlens"] = torch.from_numpy(cu).to(GEN_DEVICE)
    # The prompt, the first part of each sequence, carries no loss.
    starts = torch.from_numpy(np.repeat(cu[:-1], lens)).to(GEN_DEVICE)
    plen = torch.from_numpy(np.repeat((np.array(lens) * case["prompt"]).astype(np.int64),
                                      lens)).to(GEN_DEVICE)
    in_prompt = torch.arange(N, device=GEN_DEVICE) - starts < plen
    labels = torch.randint(0, 32000, (N,), generator=gen, device=GEN_DEVICE)
    st["labels"] = torch.where(in_prompt, torch.full_like(labels, IGNORE), labels)
    zero = torch.zeros((), device=GEN_DEVICE)
    # Log-probabilities of sampled tokens: most near 0, a tail of unlikely ones.
    lp = -(torch.rand(N, generator=gen, device=GEN_DEVICE).clamp_(min=1e-6).log_().neg_())
    st["logprob"] = torch.where(in_prompt, zero, lp)
    if case["op"] == "policy":
        # The rollout's policy is a few steps behind, the reference further.
        drift = 0.15 if case["level"] == "token" else 0.5
        st["old_logprob"] = torch.where(in_prompt, zero, lp + normal(N, std=drift))
        st["ref_logprob"] = (torch.where(in_prompt, zero, lp + normal(N, std=0.2))
                             if case["kl"] != "none" else None)
        st["entropy"] = (torch.where(in_prompt, zero, normal(N).abs_())
                         if case["entropy_coef"] != 0.0 else None)
        # Group-normalised rewards: one advantage a sequence, or one a token.
        st["advantages"] = normal(len(lens) if case["level"] == "sequence" else N)
    else:
        st["ref_logprob"] = (torch.where(in_prompt, zero, lp + normal(N, std=0.2))
                             if case["ref"] else None)
    if case["direction"] == "autograd":
        st["logprob"].requires_grad_(True)
        if st.get("entropy") is not None:
            st["entropy"].requires_grad_(True)
    return st


# ---------------------------------------------------------------- this package

def _run_own(st):
    from linear_cross_entropy_tile_amd import flce, function
    c = st["case"]
    if c["op"] == "embedding":
        if c["direction"] == "forward":
            return flce.embedding(st["weight"], st["tokens"], layout=c["layout"],
                                  scale=c["scale"])["hidden"]
        return flce.embedding_backward(st["grad_hidden"], st["tokens"], c["V"],
                                       layout=c["layout"], scale=c["scale"],
                                       grad_dtype=c["grad"])
    if c["op"] == "policy":
        kw = dict(entropy=st["entropy"], ref_logprob=st["ref_logprob"],
                  cu_seqlens=st["cu_seqlens"], dual_clip=c["dual"],
                  kl_coef=c["kl_coef"] if c["kl"] != "none" else 0.0,
                  kl_estimator=c["kl"] if c["kl"] != "none" else "k3",
                  entropy_coef=c["entropy_coef"], level=c["level"],
                  advantages_per_sequence=c["level"] == "sequence", reduction=c["reduction"])
        args = (st["logprob"], st["labels"], st["old_logprob"], st["advantages"])
        if c["direction"] == "autograd":
            loss, stats = function.policy_loss(*args, **kw)
            wrt = [t for t in (st["logprob"], st["entropy"]) if t is not None]
            return ([loss.detach().reshape(1), stats[:6], stats[6:]]
                    + list(torch.autograd.grad(loss, wrt)))
        if c["direction"] == "forward":
            out = flce.policy_loss(*args, **kw)
            return [out["loss"], out["stats"][:6], out["stats"][6:]]
        out = flce.policy_loss_forward_backward(*args, **kw)
        grads = [out["grad_logprob"]]
        if st["entropy"] is not None:
            grads.append(out["grad_entropy"])
        return [out["loss"], out["stats"][:6], out["stats"][6:]] + grads
    kw = dict(ref_logprob=st["ref_logprob"], kind=c["kind"], beta=c["beta"],
              label_smoothing=c["smoothing"], margin=c["margin"],
              length_normalize=c["normalize"], reduction=c["reduction"])
    args = (st["logprob"], st["labels"], st["cu_seqlens"])
    if c["direction"] == "autograd":
        loss, chosen, rejected = function.preference_loss(*args, **kw)
        up = torch.ones_like(loss)
        grad, = torch.autograd.grad(loss, [st["logprob"]], up)
        return [loss.detach().reshape(-1), chosen, rejected, grad]
    if c["direction"] == "forward":
        out = flce.preference_loss(*args, **kw)
        return [out["loss"], out["chosen_reward"], out["rejected_reward"]]
    out = flce.preference_loss_forward_backward(*args, **kw)
    return [out["loss"], out["chosen_reward"], out["rejected_reward"], out["grad_logprob"]]


# ---------------------------------------------------------------- plain torch

def _plain_embedding(st):
    c = st["case"]
    tok = st["tokens"]
    valid = tok != IGNORE
    idx = torch.where(valid, tok, torch.zeros_like(tok))
    if c["direction"] == "forward":
        w = st["weight"]
        rows = w[idx] if c["layout"] == "vh" else w[:, idx].t()
        return torch.where(valid[:, None], rows.float() * c["scale"], 0.0).to(torch.bfloat16)
    g = torch.where(valid[:, None], st["grad_hidden"].float(), 0.0)
    dw = torch.zeros(c["V"], c["H"], device=g.device)
    dw.index_add_(0, idx, g)
    dw *= c["scale"]
    if c["layout"] == "hv":
        dw = dw.t()
    return dw.to(torch.float32 if c["grad"] == "f32" else torch.bfloat16).contiguous()


def _sequence_ids(cu, N):
    return torch.searchsorted(cu[1:], torch.arange(N, device=cu.device), right=True)


def _clipped(d, A, dual):
    """(policy term, its derivative in d, clipped) of log ratios d (64 bits)."""
    A32 = A.float()
    r = torch.exp(d.float())
    over = (A > 0) & (d > math.log1p(0.2))
    under = (A < 0) & (d < math.log1p(-0.2))
    far = (A < 0) & (d > math.log(dual)) if dual > 0.0 else torch.zeros_like(over)
    bound = torch.where(over, 1.2, torch.where(under, 0.8, dual)).float()
    clipped = over | under | far
    live = torch.where(A32 == 0, torch.zeros_like(A32), -r * A32)
    return (torch.where(clipped, -bound * A32, live),
            torch.where(clipped, torch.zeros_like(live), live), clipped)


def _plain_policy(st):
    c = st["case"]
    lp, cu = st["logprob"].detach(), st["cu_seqlens"]
    N, B = lp.numel(), cu.numel() - 1
    valid = st["labels"] != IGNORE
    seq = _sequence_ids(cu, N)

    def per_seq(x):
        out = torch.zeros(B, dtype=torch.float64, device=lp.device)
        return out.index_add_(0, seq, torch.where(valid, x.double(), 0.0))

    n_s = per_seq(torch.ones_like(lp))
    n, n_seq = n_s.sum(), (n_s > 0).sum()
    d = lp.double() - st["old_logprob"].double()
    if c["level"] == "sequence":
        mean_d = per_seq(d) / n_s.clamp(min=1.0)
        pg, dpg, clip = (t[seq] for t in _clipped(mean_d, st["advantages"], c["dual"]))
    else:
        pg, dpg, clip = _clipped(d, st["advantages"], c["dual"])
    kl = dkl = torch.zeros_like(lp)
    if st["ref_logprob"] is not None:
        x = lp.double() - st["ref_logprob"].double()
        if c["kl"] == "k1":
            kl, dkl = x.float(), torch.ones_like(lp)
        elif c["kl"] == "k2":
            kl, dkl = (0.5 * x * x).float(), x.float()
        else:
            e = torch.expm1(-x)
            kl, dkl = (e + x).float(), (-e).float()
    ent = st["entropy"].detach() if st["entropy"] is not None else torch.zeros_like(lp)
    kl_coef = c["kl_coef"] if c["kl"] != "none" else 0.0
    loss_t = pg + kl_coef * kl - c["entropy_coef"] * ent
    if c["reduction"] == "mean":
        w = (1.0 / n.clamp(min=1.0)).expand(B)
    elif c["reduction"] == "sum":
        w = torch.ones_like(n_s)
    else:
        w = 1.0 / (n_s.clamp(min=1.0) * n_seq.clamp(min=1))
    terms = [loss_t, pg, kl, ent, clip, -d]
    stats = torch.stack([(w * per_seq(t)).sum() for t in terms] + [n, n_seq.double()]).float()
    out = [stats[0:1].clone(), stats[:6], stats[6:]]
    if c["direction"] != "forward":
        wt = torch.where(valid, w[seq], 0.0).float()
        out.append(torch.where(valid, wt * (dpg + kl_coef * dkl), 0.0))
        if st["entropy"] is not None:
            out.append(-wt * c["entropy_coef"])
    return out


def _plain_preference(st):
    c = st["case"]
    lp, cu = st["logprob"].detach(), st["cu_seqlens"]
    N, P = lp.numel(), c["P"]
    valid = st["labels"] != IGNORE
    seq = _sequence_ids(cu, N)
    zeros = torch.zeros(2 * P, dtype=torch.float64, device=lp.device)
    x = lp.double()
    if st["ref_logprob"] is not None:
        x = x - st["ref_logprob"].double()
    R = zeros.index_add(0, seq, torch.where(valid, x, 0.0))
    norm = torch.ones_like(zeros)
    if c["normalize"]:
        norm = zeros.index_add(0, seq, valid.double()).clamp(min=1.0)
        R = R / norm
    diff = R[:P] - R[P:]
    z = c["beta"] * diff - c["margin"]
    if c["kind"] == "sigmoid":
        e = c["smoothing"]
        tail = torch.log1p(torch.exp(-z.abs()))
        loss = (1 - e) * (tail + (-z).clamp(min=0)) + e * (tail + z.clamp(min=0))
        slope = c["beta"] * (1.0 / (1.0 + torch.exp(-z)) - (1 - e))
    elif c["kind"] == "hinge":
        loss = (1 - z).clamp(min=0)
        slope = torch.where(z < 1, -c["beta"], 0.0).double()
    else:
        t = diff - 0.5 / c["beta"]
        loss, slope = t * t, 2 * t
    out = [(c["beta"] * R[:P]).float(), (c["beta"] * R[P:]).float()]
    scale = 1.0
    if c["reduction"] == "none":
        out = [loss.float()] + out
    elif c["reduction"] == "sum":
        out = [loss.sum().reshape(1).float()] + out
    else:
        scale = 1.0 / P
        out = [loss.mean().reshape(1).float()] + out
    if c["direction"] != "forward":
        coef = (scale * torch.cat([slope, -slope]) / norm).float()
        out.append(torch.where(valid, coef[seq], 0.0))
    return out


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "embedding":
        return _plain_embedding(state)
    return _plain_policy(state) if op == "policy" else _plain_preference(state)


# ---------------------------------------------------------------- 64-bit definition

def _exact_embedding(c, st):
    tok = st["tokens"]
    keep = torch.nonzero(tok >= 0).reshape(-1)
    if c["direction"] == "forward":
        out = torch.zeros(c["N"], c["H"], dtype=torch.float64, device=tok.device)
        table = st["weight"] if c["layout"] == "vh" else st["weight"].t()
        out[keep] = table[tok[keep]].double() * c["scale"]
        return out
    # Sums by running totals over the positions in token order.
    order = keep[torch.argsort(tok[keep], stable=True)]
    ids, counts = torch.unique_consecutive(tok[order], return_counts=True)
    dw = torch.zeros(c["V"], c["H"], dtype=torch.float64, device=tok.device)
    if order.numel():
        ends = torch.cumsum(counts, 0)
        for h0 in range(0, c["H"], 512):
            run_sum = torch.cumsum(st["grad_hidden"][order, h0:h0 + 512].double(), 0)
            total = run_sum[ends - 1]
            total[1:] -= run_sum[ends[:-1] - 1]
            dw[ids, h0:h0 + 512] = total * c["scale"]
    return dw if c["layout"] == "vh" else dw.t().contiguous()


def _segment_sums(x, bounds):
    run_sum = np.concatenate([[0.0], np.cumsum(x, dtype=np.longdouble)])
    return (run_sum[bounds[1:]] - run_sum[bounds[:-1]]).astype(np.float64)


def _exact_policy(c, st):
    def host(t):
        return None if t is None else t.detach().cpu().numpy().astype(np.float64)

    lp, old, ref, ent = (host(st[k]) for k in ("logprob", "old_logprob", "ref_logprob", "entropy"))
    bounds = st["cu_seqlens"].cpu().numpy()
    lens = np.diff(bounds)
    on = (st["labels"].cpu().numpy() >= 0).astype(np.float64)
    count = _segment_sums(on, bounds)
    logr = lp - old
    adv = host(st["advantages"])
    if c["level"] == "sequence":
        logr_used = np.repeat(_segment_sums(on * logr, bounds) / np.maximum(count, 1), lens)
        adv = np.repeat(adv, lens)
    else:
        logr_used = logr
    ratio = np.exp(logr_used)
    inner = np.minimum(ratio * adv, np.clip(ratio, 0.8, 1.2) * adv)
    flat = ratio * adv > inner
    if c["dual"] > 0.0:
        floor = c["dual"] * adv
        flat = flat | ((adv < 0) & (inner < floor))
        inner = np.where(adv < 0, np.maximum(inner, floor), inner)
    policy = -inner
    slope = np.where(flat, 0.0, -ratio * adv)
    kl = dkl = np.zeros_like(lp)
    if ref is not None:
        x = lp - ref
        kl, dkl = {"k1": lambda: (x, np.ones_like(x)),
                   "k2": lambda: (x * x / 2, x),
                   "k3": lambda: (np.exp(np.longdouble(-x)) + x - 1, -np.expm1(-x))}[c["kl"]]()
        kl = kl.astype(np.float64)
    ec, kc = c["entropy_coef"], c["kl_coef"] if c["kl"] != "none" else 0.0
    e = ent if ent is not None else np.zeros_like(lp)
    if c["reduction"] == "mean":
        weight = np.full(len(lens), 1.0 / max(count.sum(), 1.0))
    elif c["reduction"] == "sum":
        weight = np.ones(len(lens))
    else:
        weight = 1.0 / (np.maximum(count, 1.0) * max((count > 0).sum(), 1))
    tw = np.repeat(weight, lens) * on

    def reduce(x):
        return float(np.sum((tw * x).astype(np.longdouble)))

    stats = [reduce(policy + kc * kl - ec * e), reduce(policy), reduce(kl), reduce(e),
             reduce(flat.astype(np.float64)), reduce(-logr), count.sum(), float((count > 0).sum())]
    out = [torch.tensor(x, dtype=torch.float64) for x in (stats[:1], stats[:6], stats[6:])]
    if c["direction"] != "forward":
        out.append(torch.from_numpy(tw * (slope + kc * dkl)))
        if ent is not None:
            out.append(torch.from_numpy(-ec * tw))
    return [t.to(GEN_DEVICE) for t in out]


def _exact_preference(c, st):
    P = c["P"]
    bounds = st["cu_seqlens"].cpu().numpy()
    on = st["labels"].cpu().numpy() >= 0
    x = st["logprob"].detach().cpu().numpy().astype(np.float64)
    if st["ref_logprob"] is not None:
        x = x - st["ref_logprob"].cpu().numpy().astype(np.float64)
    score = _segment_sums(np.where(on, x, 0.0), bounds)
    each = np.ones(2 * P)
    if c["normalize"]:
        each = 1.0 / np.maximum(_segment_sums(on.astype(np.float64), bounds), 1.0)
        score = score * each
    gap = score[:P] - score[P:]
    m = c["beta"] * gap - c["margin"]
    if c["kind"] == "sigmoid":
        eps = c["smoothing"]
        loss = (1 - eps) * np.logaddexp(0.0, -m) + eps * np.logaddexp(0.0, m)
        dm = -(1 - eps) / (1 + np.exp(m)) + eps / (1 + np.exp(-m))
        dgap = dm * c["beta"]
    elif c["kind"] == "hinge":
        loss, dgap = np.maximum(0.0, 1 - m), np.where(m < 1, -c["beta"], 0.0)
    else:
        loss = (gap - 1 / (2 * c["beta"])) ** 2
        dgap = 2 * (gap - 1 / (2 * c["beta"]))
    red = {"none": loss, "sum": np.array([loss.sum()]), "mean": np.array([loss.mean()])}
    out = [red[c["reduction"]], c["beta"] * score[:P], c["beta"] * score[P:]]
    if c["direction"] != "forward":
        part = dgap / P if c["reduction"] == "mean" else dgap
        out.append(np.where(on, np.repeat(np.concatenate([part, -part]) * each, np.diff(bounds)),
                            0.0))
    return [torch.from_numpy(np.ascontiguousarray(o)).to(GEN_DEVICE) for o in out]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "embedding":
        return _exact_embedding(case, st)
    return _exact_policy(case, st) if case["op"] == "policy" else _exact_preference(case, st)


# ---------------------------------------------------------------- work

def work(case):
    if case["op"] == "embedding":
        N, H, V = case["N"], case["H"], case["V"]
        live = N * (1.0 - case["ignored"])
        if case["direction"] == "forward":
            p = _token_probs(V, case["zipf"])
            distinct = float(np.sum(-np.expm1(live * np.log1p(-np.minimum(p, 1 - 1e-12)))))
            return {"bytes": 8 * N + 2 * distinct * H + 2 * N * H, "flops": live * H}
        out = 4 if case["grad"] == "f32" else 2
        return {"bytes": 8 * N + 2 * live * H + out * V * H, "flops": live * H}
    lens = _lengths(case)
    N, S = sum(lens), len(lens)
    grad = case["direction"] != "forward"
    if case["op"] == "policy":
        # labels, logprob, old_logprob; the reference, entropy and advantages
        # where they are given a token; the gradients.
        per = 8 + 4 + 4 + (4 if case["level"] == "token" else 0)
        per += 4 if case["kl"] != "none" else 0
        per += 4 if case["entropy_coef"] != 0.0 else 0
        per += (4 + (4 if case["entropy_coef"] != 0.0 else 0)) if grad else 0
        return {"bytes": per * N + 12 * S + 36, "flops": 40 * N}
    per = 8 + 4 + (4 if case["ref"] else 0) + (4 if grad else 0)
    return {"bytes": per * N + 16 * S, "flops": 4 * N}

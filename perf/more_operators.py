"""Performance cases of the operators at the two ends of a training step on the
fused head: the logits of the rows that are sampled next (``logits``), their
penalties, biases and masks (``process``), and the update of the weights
(``adamw``).

Each case runs in one of two forms on the same inputs: ``own = False`` computes
the operator from elementary torch operations (32 bits, 64 for the gradients'
norm and the bias corrections), ``own = True`` calls this package. ``exact``
evaluates the definition in 64 bits.

Definitions.
  logits   z[i,v] = cap(sum_h hidden[i,h] weight[h,v] + bias[v]), cap(z) =
           c tanh(z / c) with a cap c, else z.
  process  In row i, with n(v) the occurrences of v in the generated part of the
           row's history and seen(v) those anywhere in it, a logit x becomes
             x > 0 ? x / r : x r   if seen          (repetition)
             - frequency n(v), - presence if n(v)
             + bias[v] + the row's listed biases of v
             / temperature, and -inf where the row's mask forbids v,
           in this order. Beside it come the logsumexp, the entropy and the first
           largest value of the row as it is returned (after rounding). The
           gradient is that of the returned logits with respect to the logits.
  adamw    With t the step, s the clip factor min(1, max_norm / norm) of the norm
           over all gradients, g = s grad,
             m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
             p = (1 - lr wd) p - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps).
           States in 8 bits: for each 256 values of a tensor, m and sqrt(v) as
           e4m3 codes times a scale (the largest code is 448); a second moment
           above zero takes the smallest code at least. Rounding to bf16 or to a
           code is to the nearest, or stochastic with the bits of a hash of the
           seed, the step, the tensor and the element.
"""
import math
import random

import torch

own = False

GEN_DEVICE = "cuda"
BLOCK = 256
BETA1, BETA2, EPS, DECAY, LR = 0.9, 0.95, 1e-8, 0.1, 1e-4
TINY = 2.0 ** -100


# ---------------------------------------------------------------- cases

def _log(name, N, H, V, cap, bias, out):
    return {"name": name, "op": "logits", "N": N, "H": H, "V": V, "cap": cap, "bias": bias,
            "out": out}


def _proc(name, direction, N, V, dtype, out, history, padded, penalties, listed_bias, dense_bias,
          mask):
    return {"name": name, "op": "process", "direction": direction, "N": N, "V": V, "dtype": dtype,
            "out": out, "history": history, "padded": padded, "penalties": penalties,
            "listed_bias": listed_bias, "dense_bias": dense_bias, "mask": mask}


def _adam(name, layers, H, V, dtype, grad, state, master, clip, rounding):
    return {"name": name, "op": "adamw", "layers": layers, "H": H, "V": V, "dtype": dtype,
            "grad": grad, "state": state, "master": master, "clip": clip, "rounding": rounding}


def listed():
    return [
        # One sequence being generated: the weight is read for a single row.
        _log("logits_one", 1, 4096, 128256, 0.0, False, "bf16"),
        # A decoding batch on the capped head with its large vocabulary.
        _log("logits_decode_capped", 16, 2304, 256000, 30.0, False, "f32"),
        # Odd vocabulary: no row of the weight is aligned; a bias per id.
        _log("logits_odd_bias", 61, 768, 50257, 0.0, True, "f32"),
        # A large decoding batch (256 rollouts at once).
        _log("logits_rollouts", 256, 5120, 152064, 0.0, False, "bf16"),
        # One short chat: latency of a single row.
        _proc("process_one", "forward", 1, 32000, "f32", "f32", 300, True, "repetition", 0, False,
              "none"),
        # A served batch with everything: penalties, listed biases, a mask a row.
        _proc("process_served", "forward", 64, 128256, "f32", "f32", 4096, True, "all", 100, False,
              "rows"),
        # Rollouts in packed histories, 16 bits in and out, one mask for all rows.
        _proc("process_rollouts", "forward", 512, 152064, "bf16", "bf16", 2048, False, "all", 0,
              False, "shared"),
        # Gradient through the processed distribution, odd vocabulary.
        _proc("process_grad_odd", "backward", 300, 50257, "f32", "f32", 700, False, "all", 0, True,
              "rows"),
        # Adapters: a few small tensors, all in 32 bits; launches count.
        _adam("adamw_adapters", 2, 64, 0, "f32", "f32", "f32", False, True, "nearest"),
        # A small model of 97 tensors, 16-bit weights with a 32-bit copy.
        _adam("adamw_model", 16, 1280, 32000, "bf16", "bf16", "f32", True, True, "nearest"),
        # The tied weight alone, stochastic rounding instead of a copy.
        _adam("adamw_tied", 0, 2304, 256000, "bf16", "bf16", "f32", False, False, "stochastic"),
        # The same with states in 8 bits, and a norm over it.
        _adam("adamw_tied_8bit", 0, 2304, 256000, "bf16", "bf16", "8bit", False, True,
              "stochastic"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logits", "process", "adamw"])
    if op == "logits":
        N, H, V = _log_int(rng, 1, 256), 8 * _log_int(rng, 8, 640), _log_int(rng, 700, 256000)
        while H * V > 5120 * 152064:
            H = max(8, H // 16 * 8)
        return _log("drawn", N, H, V, rng.choice([0.0, 0.0, 5.0, 30.0]), rng.random() < 0.3,
                    rng.choice(["f32", "bf16"]))
    if op == "process":
        N, V = _log_int(rng, 1, 512), _log_int(rng, 700, 256000)
        N = max(1, min(N, 512 * 152064 // V // 2))
        dtype = rng.choice(["f32", "bf16"])
        return _proc("drawn", rng.choice(["forward", "forward", "backward"]), N, V, dtype,
                     rng.choice([dtype, "f32"]), _log_int(rng, 1, 8192), rng.random() < 0.5,
                     rng.choice(["none", "repetition", "all"]), rng.choice([0, 0, 10, 300]),
                     rng.random() < 0.3, rng.choice(["none", "shared", "rows"]))
    layers = rng.choice([0, 0, 1, 4, 24])
    H = 8 * _log_int(rng, 2, 288)
    V = _log_int(rng, 700, 256000) if layers == 0 or rng.random() < 0.7 else 0
    while H * V + 12 * layers * H * H > 2304 * 256000:
        H = max(8, H // 16 * 8)
    dtype = rng.choice(["f32", "bf16"])
    return _adam("drawn", layers, H, V, dtype, rng.choice([dtype, "f32"]),
                 rng.choice(["f32", "8bit"]), dtype == "bf16" and rng.random() < 0.5,
                 rng.random() < 0.6, rng.choice(["nearest", "stochastic"]))


def _shapes(case):
    """Weights of a case: a table, and per layer an attention's and a mlp's
    matrices with the gains of two norms."""
    H, V = case["H"], case["V"]
    layer = [(H,), (3 * H, H), (H, H), (H,), (4 * H, H), (H, 4 * H)]
    return ([(H, V)] if V else []) + layer * case["layers"]


def _lengths(case):
    """Histories' lengths of a case, the same for every seed; the last one of
    several is empty."""
    rng = random.Random(f"{case['N']} {case['history']}")
    lens = [rng.randint((case["history"] + 1) // 2, case["history"]) for _ in range(case["N"])]
    if len(lens) > 1:
        lens[-1] = 0
    return lens


# ---------------------------------------------------------------- inputs

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def prepare(case, seed):
    gen = torch.Generator(device=GEN_DEVICE)
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        x = torch.randn(*shape, generator=gen, device=GEN_DEVICE, dtype=dtype)
        return x.mul_(std) if std != 1.0 else x

    def uniform(n, lo, hi):
        return torch.rand(n, generator=gen, device=GEN_DEVICE) * (hi - lo) + lo

    st = {"case": case}
    if case["op"] == "logits":
        N, H, V = case["N"], case["H"], case["V"]
        st["hidden"] = normal(N, H, dtype=torch.bfloat16)
        st["weight"] = normal(H, V, std=0.05, dtype=torch.bfloat16)
        st["bias"] = normal(V, std=0.5) if case["bias"] else None
        return st

    if case["op"] == "process":
        N, V = case["N"], case["V"]
        st["logits"] = normal(N, V, std=3.0, dtype=_TYPES[case["dtype"]])
        lens = torch.tensor(_lengths(case), device=GEN_DEVICE)
        # Ids of a text: few of them make up most of it.
        width = int(case["history"])
        u = torch.rand(N, width, generator=gen, device=GEN_DEVICE, dtype=torch.float64)
        ids = (V * u ** 4).long().clamp_(max=V - 1)
        st["lengths"] = st["cu_seqlens"] = None
        if case["padded"]:
            st["tokens"], st["lengths"] = ids, lens
        else:
            st["tokens"] = ids[torch.arange(width, device=GEN_DEVICE) < lens[:, None]]
            st["cu_seqlens"] = torch.nn.functional.pad(torch.cumsum(lens, 0), (1, 0))
        st["prompt_lengths"] = lens // 3
        st["repetition"] = uniform(N, 1.0, 1.5)
        st["presence"] = uniform(N, 0.0, 1.0)
        st["frequency"] = uniform(N, 0.0, 0.5)
        st["temperature"] = uniform(N, 0.5, 1.5)
        if case["penalties"] != "all":
            st["presence"] = st["frequency"] = None
        if case["penalties"] == "none":
            st["repetition"] = None
        st["bias_tokens"] = st["bias_values"] = st["bias_cu_seqlens"] = None
        if case["listed_bias"]:
            k = case["listed_bias"]
            st["bias_tokens"] = torch.randint(0, V, (N * k,), generator=gen, device=GEN_DEVICE)
            st["bias_values"] = normal(N * k, std=2.0)
            st["bias_cu_seqlens"] = torch.arange(0, N * k + 1, k, device=GEN_DEVICE)
        st["bias"] = normal(V, std=0.5) if case["dense_bias"] else None
        st["allowed"] = None
        if case["mask"] != "none":
            words = -(-V // 32)
            shape = (words,) if case["mask"] == "shared" else (N, words)
            st["allowed"] = torch.randint(-2 ** 31, 2 ** 31, shape, generator=gen,
                                          device=GEN_DEVICE).int()
        if case["direction"] == "backward":
            st["grad"] = normal(N, V, std=1e-3, dtype=_TYPES[case["out"]])
        return st

    # Each kind of values lies in one buffer, its tensors at multiples of 256
    # with zeros between them.
    sizes = [math.prod(s) for s in _shapes(case)]
    room = [-(-n // BLOCK) * BLOCK for n in sizes]
    starts = [sum(room[:k]) for k in range(len(room))]
    total = sum(room)

    def views(flat):
        return [flat[a:a + n].view(s) for a, n, s in zip(starts, sizes, _shapes(case))]

    def scales(flat):
        return [flat[a // BLOCK:(a + n) // BLOCK] for a, n in zip(starts, room)]

    def live(x):
        if sizes != room:
            for a, n, k in zip(starts, sizes, room):
                x[a + n:a + k] = 0
        return x

    flat = {"params": live(normal(total, std=0.05, dtype=_TYPES[case["dtype"]])),
            "grads": live(normal(total, std=1e-3, dtype=_TYPES[case["grad"]]))}
    if case["master"]:
        flat["master"] = live(flat["params"].float() + normal(total, std=1e-5))
    # Moments as they stand after a few steps.
    if case["state"] == "f32":
        flat["exp_avg"] = live(normal(total, std=3e-4))
        flat["exp_avg_sq"] = live(normal(total, std=6e-4).square_().add_(1e-8))
    else:
        e4m3 = torch.float8_e4m3fn
        flat["exp_avg"] = live(normal(total, std=120.0).clamp_(-448, 448)).to(e4m3)
        flat["exp_avg_sq"] = live(normal(total, std=120.0).abs_().clamp_(30, 448)).to(e4m3)
        flat["exp_avg_scale"] = uniform(total // BLOCK, 2e-6, 3e-6)
        flat["exp_avg_sq_scale"] = uniform(total // BLOCK, 4e-6, 6e-6)
    st["params"], st["grads"] = views(flat["params"]), views(flat["grads"])
    st["state"] = {"step": torch.full((1,), 9, dtype=torch.int64, device=GEN_DEVICE)}
    for kind in ("master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
        cut = scales if kind.endswith("scale") else views
        st["state"][kind] = cut(flat[kind]) if kind in flat else None
    st["flat"], st["room"], st["seed"] = flat, room, seed
    return st


# ---------------------------------------------------------------- this package

def _process_arguments(st):
    return dict(tokens=st["tokens"], cu_seqlens=st["cu_seqlens"], lengths=st["lengths"],
                prompt_lengths=st["prompt_lengths"],
                repetition_penalty=1.0 if st["repetition"] is None else st["repetition"],
                presence_penalty=0.0 if st["presence"] is None else st["presence"],
                frequency_penalty=0.0 if st["frequency"] is None else st["frequency"],
                temperature=st["temperature"], bias=st["bias"], bias_tokens=st["bias_tokens"],
                bias_values=st["bias_values"], bias_cu_seqlens=st["bias_cu_seqlens"],
                allowed=st["allowed"])


def _updated(st):
    """All that a step writes."""
    return [v for k, v in st["flat"].items() if k != "grads"] + [st["state"]["step"]]


def _run_own(st):
    from linear_cross_entropy_tile_amd import flce
    c = st["case"]
    if c["op"] == "logits":
        return flce.logits(st["hidden"], st["weight"], bias=st["bias"], softcap=c["cap"],
                           out_dtype=c["out"])["logits"]
    if c["op"] == "process":
        if c["direction"] == "backward":
            return flce.process_logits_backward(st["grad"], st["logits"],
                                                **_process_arguments(st))
        out = flce.process_logits(st["logits"], out_dtype=c["out"], **_process_arguments(st))
        return [out[k] for k in ("logits", "lse", "entropy", "greedy")]
    norm = []
    scale = None
    if c["clip"]:
        out = flce.grad_norm(st["grads"], max_norm=1.0)
        norm, scale = [out["norm"], out["scale"]], out["scale"]
    flce.adamw_step(st["params"], st["grads"], st["state"], lr=LR, beta1=BETA1, beta2=BETA2,
                    eps=EPS, weight_decay=DECAY, grad_scale=scale, rounding=c["rounding"],
                    seed=st["seed"])
    return norm + _updated(st)


# ---------------------------------------------------------------- plain torch

def _plain_logits(st):
    c = st["case"]
    z = st["hidden"].float() @ st["weight"].float()
    if st["bias"] is not None:
        z += st["bias"]
    if c["cap"] > 0.0:
        z = c["cap"] * torch.tanh(z / c["cap"])
    return z.to(_TYPES[c["out"]])


def _history(st):
    """(occurrences in the generated part, whether seen) of every id, [N,V]."""
    c = st["case"]
    N, V = c["N"], c["V"]
    if c["padded"]:
        ids, lens = st["tokens"], st["lengths"]
        at = torch.arange(ids.shape[1], device=ids.device).expand_as(ids)
        row = torch.arange(N, device=ids.device)[:, None].expand_as(ids)
        there = at < lens[:, None]
        ids, at, row = ids[there], at[there], row[there]
    else:
        ids, cu = st["tokens"], st["cu_seqlens"]
        row = torch.searchsorted(cu[1:], torch.arange(ids.numel(), device=ids.device), right=True)
        at = torch.arange(ids.numel(), device=ids.device) - cu[row]
    flat = row * V + ids
    made = at >= st["prompt_lengths"][row]
    counts = torch.zeros(N * V, dtype=torch.int32, device=ids.device)
    counts.index_add_(0, flat, made.int())
    seen = torch.zeros(N * V, dtype=torch.bool, device=ids.device)
    seen[flat] = True
    return counts.view(N, V), seen.view(N, V)


def _mask(st):
    V = st["case"]["V"]
    bit = torch.arange(V, device=st["logits"].device)
    return ((st["allowed"][..., bit // 32] >> (bit % 32).int()) & 1) != 0


def _plain_process(st):
    c = st["case"]
    N, V = c["N"], c["V"]
    x = st["logits"].float()
    counts = None
    inv_t = 1.0 / st["temperature"][:, None]
    if c["penalties"] != "none":
        counts, seen = _history(st)
        r = st["repetition"][:, None]
        slope = torch.where(seen, torch.where(x > 0, 1.0 / r, r), 1.0)
    if c["direction"] == "backward":
        g = st["grad"].float()
        if counts is not None:
            g = g * slope
        g = g * inv_t
        if st["allowed"] is not None:
            g = torch.where(_mask(st), g, 0.0)
        return g.to(_TYPES[c["dtype"]])
    if counts is not None:
        x = x * slope
    if c["penalties"] == "all":
        x = x - st["frequency"][:, None] * counts
        x = torch.where(counts > 0, x - st["presence"][:, None], x)
    if st["bias"] is not None:
        x = x + st["bias"]
    if st["bias_tokens"] is not None:
        k = c["listed_bias"]
        rows = torch.arange(N, device=x.device).repeat_interleave(k)
        more = torch.zeros(N * V, dtype=torch.float64, device=x.device)
        more.index_add_(0, rows * V + st["bias_tokens"], st["bias_values"].double())
        x = x + more.view(N, V).float()
    x = x * inv_t
    if st["allowed"] is not None:
        x = torch.where(_mask(st), x, -math.inf)
    out = x.to(_TYPES[c["out"]])
    x = out.float()
    m = x.amax(1, keepdim=True)
    d = torch.where(m == -math.inf, -math.inf, x - m)
    e = torch.exp(d)
    s = e.sum(1)
    lse = m[:, 0] + torch.log(s)
    u = torch.where(e > 0, e * d, 0.0).sum(1)
    entropy = torch.where(s > 0, torch.log(s) - u / s, 0.0)
    return [out, lse, entropy, torch.argmax(x, 1)]


def _mix(x):
    """A 32-bit hash of values below 2^32 held in int64."""
    x = x ^ (x >> 16)
    x = (x * 0x9E3779B1) & 0xFFFFFFFF
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _plain_random(st):
    """Three streams of 16 random bits (weights, first and second moments), for
    all values of all tensors."""
    mask = 0xFFFFFFFF
    step = st["state"]["step"]
    room = torch.tensor(st["room"], device=step.device)
    total = sum(st["room"])
    seed = torch.full_like(step, st["seed"])
    key = _mix((seed & mask) ^ _mix((seed >> 32) & mask))
    key = _mix(key ^ (step & mask))
    keys = _mix((key + torch.arange(len(room), device=step.device) * 0x6A09E667) & mask)
    starts = torch.cumsum(room, 0) - room
    at = torch.arange(total, device=step.device)
    if len(room) > 1:
        keys = keys.repeat_interleave(room, output_size=total)
        at = at - starts.repeat_interleave(room, output_size=total)
    h1 = _mix((at & mask) ^ _mix(keys ^ (at >> 32)))
    h2 = ((h1 ^ 0x6A09E667) * 0x9E3779B1) & mask
    h2 = h2 ^ (h2 >> 16)
    return (h1 >> 16).int(), (h2 >> 16).int(), (h2 & 0xFFFF).int()


def _to_code(y, bits):
    """e4m3 codes of y (|y| <= 448): to the nearest, or stochastic with 16 random
    bits a value."""
    if bits is None:
        return y.to(torch.float8_e4m3fn)
    b = y.abs().view(torch.int32)
    large = ((b + (bits << 4)) & -(1 << 20)).view(torch.float32)
    small = torch.floor(y.abs() * 512.0 + bits.float() * 2.0 ** -16) * 2.0 ** -9
    return torch.copysign(torch.where(y.abs() >= 2.0 ** -6, large, small), y).to(
        torch.float8_e4m3fn)


def _plain_adamw(st):
    c, step, flat = st["case"], st["state"]["step"], st["flat"]
    g = flat["grads"].float()
    out = []
    if c["clip"]:
        norm = g.double().square().sum().sqrt()
        scale = torch.clamp(1.0 / norm, max=1.0).float()
        out = [norm.float().reshape(1), scale.reshape(1)]
        g = g * scale
    step += 1
    t = step.double()
    rise = (LR / (1.0 - BETA1 ** t)).float()
    root = (1.0 / torch.sqrt(1.0 - BETA2 ** t)).float()
    m, v = flat["exp_avg"].float(), flat["exp_avg_sq"].float()
    if c["state"] == "8bit":
        m = (m.view(-1, BLOCK) * flat["exp_avg_scale"][:, None]).view(-1)
        v = (v.view(-1, BLOCK) * flat["exp_avg_sq_scale"][:, None]).square().view(-1)
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * g) * (1.0 - BETA2)
    p = flat["master" if c["master"] else "params"].float()
    r = torch.sqrt(v)
    p = p * (1.0 - LR * DECAY) - rise * (m / (r * root + EPS))
    loose = c["dtype"] == "bf16" and not c["master"]
    bits = (None, None, None)
    if c["rounding"] == "stochastic" and (loose or c["state"] == "8bit"):
        bits = _plain_random(st)
    if c["master"]:
        flat["master"].copy_(p)
    if loose and bits[0] is not None:
        p = ((p.view(torch.int32) + bits[0]) & -65536).view(torch.float32)
    flat["params"].copy_(p)
    if c["state"] == "f32":
        flat["exp_avg"].copy_(m)
        flat["exp_avg_sq"].copy_(v)
        return out + _updated(st)
    for kind, x, rnd in (("exp_avg", m, bits[1]), ("exp_avg_sq", r, bits[2])):
        x = x.view(-1, BLOCK)
        top = x.abs().amax(1, keepdim=True)
        live = top >= TINY
        y = torch.where(live, x * (448.0 / top), 0.0)
        code = _to_code(y, None if rnd is None else rnd.view(-1, BLOCK))
        if kind == "exp_avg_sq":
            code = torch.where((y > 0) & (code.float() == 0), 2.0 ** -9, code.float())
        flat[kind].copy_(code.reshape(-1))
        flat[kind + "_scale"].copy_(torch.where(live, top / 448.0, 0.0)[:, 0])
    return out + _updated(st)


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "logits":
        return _plain_logits(state)
    return _plain_process(state) if op == "process" else _plain_adamw(state)


# ---------------------------------------------------------------- 64-bit definition

def _exact_logits(c, st):
    z = torch.empty(c["N"], c["V"], dtype=torch.float64, device=GEN_DEVICE)
    h = st["hidden"].double()
    for v0 in range(0, c["V"], 16384):
        z[:, v0:v0 + 16384] = h @ st["weight"][:, v0:v0 + 16384].double().contiguous()
    if st["bias"] is not None:
        z += st["bias"].double()
    return torch.tanh(z / c["cap"]) * c["cap"] if c["cap"] else z


def _exact_process(c, st):
    N, V = c["N"], c["V"]
    lens = _lengths(c)
    if c["padded"]:
        histories = [st["tokens"][i, :lens[i]] for i in range(N)]
    else:
        histories = torch.split(st["tokens"], lens)
    rows = []
    for i in range(N):
        x = st["logits"][i].double()
        slope = torch.ones_like(x)
        if c["penalties"] != "none":
            h = histories[i]
            ids = torch.unique(h)
            r = float(st["repetition"][i])
            slope[ids] = torch.where(x[ids] > 0, 1.0 / r, r).double()
        t = float(st["temperature"][i])
        keep = None
        if st["allowed"] is not None:
            words = st["allowed"] if c["mask"] == "shared" else st["allowed"][i]
            keep = ((words[:, None] >> torch.arange(32, device=words.device, dtype=torch.int32))
                    & 1).reshape(-1)[:V].bool()
        if c["direction"] == "backward":
            g = st["grad"][i].double() * slope / t
            rows.append(g if keep is None else g * keep)
            continue
        x = x * slope
        if c["penalties"] == "all":
            ids, n = torch.unique(h[int(st["prompt_lengths"][i]):], return_counts=True)
            x[ids] -= float(st["frequency"][i]) * n + float(st["presence"][i])
        if st["bias"] is not None:
            x = x + st["bias"].double()
        if c["listed_bias"]:
            k = c["listed_bias"]
            x = x.index_add(0, st["bias_tokens"][i * k:i * k + k],
                            st["bias_values"][i * k:i * k + k].double())
        x = x / t
        rows.append(x if keep is None else x.masked_fill(~keep, -math.inf))
    full = torch.stack(rows)
    if c["direction"] == "backward":
        return full
    # The statistics are those of the row as it is returned.
    seen = full.to(_TYPES[c["out"]]).double()
    p = torch.softmax(seen, 1)
    entropy = -(p * torch.where(p > 0, torch.log_softmax(seen, 1), 0.0)).sum(1)
    return [full, torch.logsumexp(seen, 1), entropy, None]


def _exact_adamw(c, st):
    state = st["state"]
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in st["grads"]))
    scale = min(1.0, 1.0 / norm) if c["clip"] else 1.0
    t = int(state["step"]) + 1
    new = {k: v.double() for k, v in st["flat"].items() if k != "grads"}
    at = 0
    for k, param in enumerate(st["params"]):
        n = param.numel()
        g = st["grads"][k].double().reshape(-1) * scale
        m, v = state["exp_avg"][k].double().reshape(-1), state["exp_avg_sq"][k].double().reshape(-1)
        if c["state"] == "8bit":
            m = m * state["exp_avg_scale"][k].double().repeat_interleave(BLOCK)[:n]
            v = (v * state["exp_avg_sq_scale"][k].double().repeat_interleave(BLOCK)[:n]) ** 2
        m += (1.0 - BETA1) * (g - m)
        v += (1.0 - BETA2) * (g * g - v)
        p = (state["master"][k] if c["master"] else param).double().reshape(-1)
        p = p - LR * (DECAY * p + (m / (1 - BETA1 ** t))
                      / ((v / (1 - BETA2 ** t)).sqrt() + EPS))
        for kind in ("params", "master") if c["master"] else ("params",):
            new[kind][at:at + n] = p
        if c["state"] == "f32":
            new["exp_avg"][at:at + n] = m
            new["exp_avg_sq"][at:at + n] = v
        else:
            # What a code stands for before it is rounded.
            for kind, x in (("exp_avg", m), ("exp_avg_sq", v.sqrt())):
                s = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK).abs().amax(1) / 448
                new[kind][at:at + n] = x / s.repeat_interleave(BLOCK)[:n]
                new[kind + "_scale"][at // BLOCK:at // BLOCK + s.numel()] = s
        at += st["room"][k]
    out = [torch.tensor([norm]), torch.tensor([scale])] if c["clip"] else []
    return [o.double() for o in out] + list(new.values()) + [None]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "logits":
        return _exact_logits(case, st)
    return _exact_process(case, st) if case["op"] == "process" else _exact_adamw(case, st)


# ---------------------------------------------------------------- work

_BYTES = {"f32": 4, "bf16": 2}


def work(case):
    if case["op"] == "logits":
        N, H, V = case["N"], case["H"], case["V"]
        return {"bytes": 2 * H * V + 2 * N * H + (4 * V if case["bias"] else 0)
                + _BYTES[case["out"]] * N * V, "flops": 2 * N * H * V}
    if case["op"] == "process":
        N, V = case["N"], case["V"]
        b = N * V * (_BYTES[case["dtype"]] + _BYTES[case["out"]])
        if case["direction"] == "backward":
            b += N * V * _BYTES[case["dtype"]] if case["penalties"] != "none" else 0
        else:
            b += 16 * N + 12 * N * case["listed_bias"] + (4 * V if case["dense_bias"] else 0)
        if case["penalties"] != "none":
            b += 8 * sum(_lengths(case))
        if case["mask"] != "none":
            b += -(-V // 32) * 4 * (N if case["mask"] == "rows" else 1)
        return {"bytes": b, "flops": 10 * N * V}
    n = sum(math.prod(s) for s in _shapes(case))
    # With a norm the gradients are read twice unless a cache holds them.
    per = _BYTES[case["grad"]] + 2 * _BYTES[case["dtype"]]
    per += 16 if case["state"] == "f32" else 4 + 16 / BLOCK
    per += 8 - _BYTES[case["dtype"]] if case["master"] else 0
    return {"bytes": per * n, "flops": 20 * n}

"""Oracle of the operators at the two ends of a training step: logits to sample
from, their processing with its gradient, the gradients' norm and the AdamW
update, written from their definitions (include/flce.h) with numpy.

Functions named ``*_f32`` follow the definition's sequence of fp32 operations,
one rounding each, and state the exact bits; the others are float64.
"""
from __future__ import annotations

import numpy as np

F = np.float32


# ---------------------------------------------------------------- logits

def logits(hidden, weight, bias=None, softcap=0.0):
    """(z [N,V], sum of |terms| before the cap [N,V])."""
    h, w = np.asarray(hidden, np.float64), np.asarray(weight, np.float64)
    z, mag = h @ w, np.abs(h) @ np.abs(w)
    if bias is not None:
        z, mag = z + bias, mag + np.abs(bias)
    return (softcap * np.tanh(z / softcap) if softcap > 0 else z), mag


# ---------------------------------------------------------------- processing of logits

def _row_terms(V, history, prompt, ignore_index):
    """(seen [V], generated occurrences [V]) of one row."""
    seen, made = np.zeros(V, bool), np.zeros(V, np.int64)
    for j, t in enumerate(history):
        if t != ignore_index and 0 <= t < V:
            seen[t] = True
            made[t] += j >= prompt
    return seen, made


def unpack_mask(words, V):
    w = np.asarray(words).astype(np.uint32)
    return ((w[:, None] >> np.arange(32, dtype=np.uint32)) & 1).reshape(-1)[:V].astype(bool)


def process_row(x, history=(), prompt=0, repetition=1.0, presence=0.0, frequency=0.0,
                temperature=1.0, bias=None, listed=(), allowed=None, ignore_index=-100,
                dtype=np.float64):
    """One row, in float64, or with dtype float32 by the definition's fp32
    operations (reciprocals, products and sums in its order)."""
    T = dtype
    x = np.asarray(x, T).copy()
    V = x.size
    seen, made = _row_terms(V, history, prompt, ignore_index)
    r, t = T(repetition), T(temperature)
    with np.errstate(all="ignore"):
        inv_r, inv_t = T(1) / r, T(1) if t == 0 else T(1) / t
        x = np.where(seen, x * np.where(x > 0, inv_r, r), x).astype(T)
        x = np.where(made > 0, (x - T(frequency) * made.astype(T)) - T(presence), x).astype(T)
        if bias is not None:
            x = x + np.asarray(bias, T)
        if len(listed):
            extra = np.zeros(V, T)
            for tok, val in listed:
                if tok != ignore_index and 0 <= tok < V:
                    extra[tok] = extra[tok] + T(val)
            x = x + extra
        x = x * inv_t
    if allowed is not None:
        x = np.where(allowed, x, T(-np.inf))
    return x


def row_slope(x, history=(), prompt=0, repetition=1.0, temperature=1.0, allowed=None,
              ignore_index=-100, dtype=np.float64):
    """What a logit is multiplied by: (the first factor, the second, 0 or 1)."""
    T = dtype
    seen, _ = _row_terms(len(x), history, prompt, ignore_index)
    r = T(repetition)
    first = np.where(seen, np.where(np.asarray(x) > 0, T(1) / r, r), T(1))
    second = T(1) if temperature == 0 else T(1) / T(temperature)
    return first, second, (np.ones(len(x), bool) if allowed is None else allowed)


def row_stats(y):
    """(lse, entropy, greedy) of a returned row, float64."""
    y = np.asarray(y, np.float64)
    if np.isnan(y).any():
        return np.nan, np.nan, int(np.argmax(np.isnan(y)))
    m = y.max()
    if m == -np.inf:
        return -np.inf, 0.0, -1
    if m == np.inf:
        return np.inf, np.nan, int(np.argmax(y))
    e = np.exp(y - m)
    s = e.sum()
    d = np.where(e > 0, y - m, 0.0)
    return m + np.log(s), np.log(s) - (e * d).sum() / s, int(np.argmax(y))


def row_gradient(y, grad_out, grad_lse, grad_entropy, slope):
    """d(grad_out . y + grad_lse lse + grad_entropy entropy) / d logits."""
    first, second, keep = slope
    lse, entropy, _ = row_stats(y)
    g = np.asarray(grad_out, np.float64).copy()
    if lse != -np.inf:
        p = np.exp(np.asarray(y, np.float64) - lse)
        d = np.where(p > 0, np.asarray(y, np.float64) - lse, 0.0)
        g = g + p * (grad_lse - grad_entropy * (d + entropy))
    return np.where(keep, g * first * second, 0.0)


# ---------------------------------------------------------------- random bits, codes

def hash32(x):
    x = np.asarray(x, np.uint32)
    with np.errstate(over="ignore"):
        x = x ^ (x >> np.uint32(16))
        x = x * np.uint32(0x9E3779B1)
        x = x ^ (x >> np.uint32(15))
        x = x * np.uint32(0xBB67AE85)
    return x ^ (x >> np.uint32(16))


def random_bits(seed, step, tensor, n):
    """(weights, first, second moments): 16 bits for each of the first n values of
    a tensor (n below 2^32)."""
    u = np.uint32
    with np.errstate(over="ignore"):
        key = hash32(u(seed & 0xFFFFFFFF) ^ hash32(u(seed >> 32)))
        key = hash32(key ^ u(step & 0xFFFFFFFF))
        key = hash32(np.asarray([key], u) + u((tensor * 0x6A09E667) & 0xFFFFFFFF))
        key = hash32(key)  # the upper half of the value's index is 0
        h = hash32(np.arange(n, dtype=u) ^ key)
        g = (h ^ u(0x6A09E667)) * u(0x9E3779B1)
    g = g ^ (g >> u(16))
    return h >> u(16), g >> u(16), g & u(0xFFFF)


#: Values of the non-negative e4m3 codes 0 .. 126 (127 is NaN).
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10)
                 for c in range(127)])


def to_e4m3(y, bits=None):
    """Values of the codes of y (fp32, |y| <= 448): nearest, ties to the even code, or
    with 16 random bits a value the code below, or above where bits / 2^16 is at
    least 1 - the part cut off."""
    a = np.abs(np.asarray(y, np.float64))
    lo = np.clip(np.searchsorted(E4M3, a, side="right") - 1, 0, 126)
    hi = np.minimum(lo + 1, 126)
    step = np.where(hi > lo, E4M3[hi] - E4M3[lo], 1.0)
    part = (a - E4M3[lo]) / step
    if bits is None:
        up = (part > 0.5) | ((part == 0.5) & (lo % 2 == 1))
    else:
        up = part + bits.astype(np.float64) * 2.0 ** -16 >= 1.0
        # Below the smallest normal code the sum is one of fp32 values.
        small = np.floor((a * 512).astype(F) + bits.astype(F) * F(2.0 ** -16)) > lo
        up = np.where(a < 2.0 ** -6, small, up)
    return np.copysign(E4M3[np.where(up, hi, lo)], y)


def bf16_nearest(x):
    b = np.asarray(x, F).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(F)


def bf16_stochastic(x, bits):
    b = np.asarray(x, F).view(np.uint32).astype(np.uint64)
    return ((b + bits) & 0xFFFF0000).astype(np.uint32).view(F)


# ---------------------------------------------------------------- AdamW

def adamw_f32(p, g, m, v, step, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01,
              grad_scale=1.0):
    """(p, m, v, sqrt v, |change of p|) after step ``step`` by the definition's fp32
    operations; the square root and the quotient rounded to the nearest."""
    b1, b2 = F(beta1), F(beta2)
    g = np.asarray(g, F) * F(grad_scale)
    m = np.asarray(m, F) * b1 + g * F(1.0 - beta1)
    v = np.asarray(v, F) * b2 + (g * g) * F(1.0 - beta2)
    r = np.sqrt(v)
    rise, root = F(lr / (1.0 - beta1 ** step)), F(1.0 / np.sqrt(1.0 - beta2 ** step))
    change = rise * (m / (r * root + F(eps)))
    return np.asarray(p, F) * F(1.0 - lr * weight_decay) - change, m, v, r, np.abs(change)


def adamw(p, g, m, v, step, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01,
          grad_scale=1.0):
    """(p, m, v) after step ``step`` in float64."""
    g = np.asarray(g, np.float64) * grad_scale
    m = beta1 * np.asarray(m, np.float64) + (1 - beta1) * g
    v = beta2 * np.asarray(v, np.float64) + (1 - beta2) * g * g
    denom = np.sqrt(v / (1 - beta2 ** step)) + eps
    p = np.asarray(p, np.float64)
    return p - lr * weight_decay * p - lr / (1 - beta1 ** step) * m / denom, m, v


def encode_f32(x, bits=None, positive=False, block=256):
    """(values of the codes, scales) of fp32 values in blocks."""
    x = np.asarray(x, F)
    codes, scales = np.zeros(x.size), np.zeros(-(-x.size // block), F)
    for b in range(scales.size):
        s = slice(b * block, (b + 1) * block)
        top = np.abs(x[s]).max()
        if top >= 2.0 ** -100:
            y = x[s] * (F(448) * (F(1) / top))
            c = to_e4m3(y, None if bits is None else bits[s])
            codes[s] = np.where((y > 0) & (c == 0), 2.0 ** -9, c) if positive else c
            scales[b] = top * F(1 / 448)
    return codes, scales

"""Plain fp64 statements of the attention-layer operators, for the tests: one
row at a time, on the CPU, from the definitions in include/gdn2_attn.h."""
import math

import numpy as np

#: unit roundoff of the 16-bit types: half the spacing of values in [1, 2)
UNIT = {"torch.bfloat16": 2.0 ** -8, "torch.float16": 2.0 ** -11}


def f64(t):
    return t.detach().double().cpu().numpy()


def norm_rope(x, positions, inv_freq, weight=None, norm=True, interleaved=False, factor=1.0, eps=1e-6):
    """x [T, H, D] (fp64 array) normed and rotated."""
    x = np.array(x, dtype=np.float64)
    if norm:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        if weight is not None:
            x = x * weight
    y = x.copy()
    half = 0 if inv_freq is None else len(inv_freq)
    for t in range(x.shape[0]):
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            # exact reduction: a Python integer times a rational frequency
            turns = math.fmod(int(positions[t]) * float(inv_freq[i]), 2 * math.pi) if abs(
                int(positions[t])) < 2 ** 24 else reduced(int(positions[t]), float(inv_freq[i]))
            c, s = math.cos(turns) * factor, math.sin(turns) * factor
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, a] * s + x[t, :, b] * c
    return y


def reduced(position, freq):
    """position * freq modulo 2 pi for large positions, in exact integers with 2 pi to 200 bits."""
    from fractions import Fraction
    two_pi = Fraction(2 * 31415926535897932384626433832795028841971693993751058209749445923, 10 ** 64)
    x = Fraction(freq) * position
    return float(x - two_pi * (x // two_pi))


def attention(q, k_cache, v_cache, table, kv_lens, cu, scale, causal=True, window=-1):
    """(out, lse, spread): spread = sum_c softmax_c |v_c|, the scale of the
    error that rounding each weight brings.  All arrays fp64 or integers."""
    T, HQ, D = q.shape
    page_size, HKV = k_cache.shape[1], k_cache.shape[2]
    out, spread = np.zeros((T, HQ, D)), np.zeros((T, HQ, D))
    lse = np.full((T, HQ), -np.inf)
    for n in range(len(cu) - 1):
        new, length = int(cu[n + 1] - cu[n]), int(kv_lens[n])
        if new == 0 or length == 0:
            continue
        c = np.arange(length)
        pages, slots = table[n][c // page_size], c % page_size
        for j in range(new):
            place = length - new + j
            seen = np.ones(length, dtype=bool)
            if causal:
                seen &= c <= place
                if window >= 0:
                    seen &= c >= place - window
            if not seen.any():
                continue
            t = int(cu[n]) + j
            for hk in range(HKV):
                ks, vs = k_cache[pages[seen], slots[seen], hk], v_cache[pages[seen], slots[seen], hk]
                hs = slice(hk * (HQ // HKV), (hk + 1) * (HQ // HKV))
                x = q[t, hs] @ ks.T * scale
                m = x.max(-1, keepdims=True)
                e = np.exp(x - m)
                z = e.sum(-1, keepdims=True)
                out[t, hs] = e @ vs / z
                spread[t, hs] = e @ np.abs(vs) / z
                lse[t, hs] = (m + np.log(z))[:, 0]
    return out, lse, spread

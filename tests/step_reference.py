"""64-bit references of the steps around the attention (norm and rotation, masked attention, token
scores) for the tests, and the error bounds they use."""
from __future__ import annotations

import math

import numpy as np
import torch

from q8_reference import HALF

U = 2.0 ** -24                       # half a step of float32, relative


def frequencies(rd, theta, scaling="none", factor=1.0, n=0, low=0.0, high=0.0):
    """Angle per position of each pair, and the amplitude, pair by pair from the definitions."""
    out, amp = [], 1.0
    if scaling == "yarn":
        low, high = low or 1.0, high or 32.0
        at = [rd * math.log(n / (2 * math.pi * t)) / (2 * math.log(theta)) for t in (high, low)]
        a, b = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rd - 1)
        amp = 0.1 * math.log(factor) + 1
    if scaling == "bands":
        low, high = low or 1.0, high or 4.0
    for i in range(rd // 2):
        base = theta * factor ** (rd / (rd - 2)) if scaling == "ntk" else theta
        f = base ** (-2 * i / rd)
        if scaling == "linear":
            f /= factor
        elif scaling == "yarn":
            if i >= b and i > a:
                f /= factor
            elif i > a:
                part = (i - a) / (b - a)
                f = f * (1 - part) + f / factor * part
        elif scaling == "bands":
            turns = n * f / (2 * math.pi)
            if turns <= low:
                f /= factor
            elif turns < high:
                part = (turns - low) / (high - low)
                f = f * part + f / factor * (1 - part)
        out.append(f)
    return out, amp


def _mod_turn(pos, f):
    """pos * f / 2 pi modulo one turn, exactly in the rationals from the doubles f and 2 pi."""
    from fractions import Fraction
    turn = Fraction(f) / Fraction(2 * math.pi)
    return np.vectorize(lambda p: float((int(p) * turn) % 1), otypes=[float])(pos)


def rotate(x, weight, eps, pos, freq, amp, interleaved):
    """x [n, H, d] (torch), pos [n] ints: normed and rotated rows in float64, and the bound of the error of
    a float32 computation (before any rounding to the output's type)."""
    x = x.detach().cpu().double().numpy()
    n, H, d = x.shape
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight.detach().cpu().double().numpy()
    rd = 2 * len(freq)
    y, size = x.copy(), np.abs(x)
    if rd:
        turns = np.stack([_mod_turn(np.asarray(pos), f) for f in freq], -1)[:, None]       # [n, 1, rd/2]
        c, s = amp * np.cos(2 * np.pi * turns), amp * np.sin(2 * np.pi * turns)
        one = np.arange(0, rd, 2) if interleaved else np.arange(rd // 2)
        two = one + (1 if interleaved else rd // 2)
        a, b = x[..., one], x[..., two]
        y[..., one], y[..., two] = a * c - b * s, a * s + b * c
        size[..., one] = size[..., two] = abs(amp) * (np.abs(a) + np.abs(b))
    # norm: 128 squares added 16 or fewer in a row, then by halves (<= 21 roundings, halved by the root), root,
    # quotient, two products: < 16; rotation: cosine and sine off by 4 half steps with the amplitude and by the
    # angle's 2^-25 of a quarter turn; two products and a sum: < 8; the last position's own rounding of the
    # frequency, 2^-53 of the angle in turns for positions below 2^31: 2^-20 turns of f <= 1 / 2 pi
    far = 0.0 if not rd else float(np.max(np.abs(np.asarray(pos, np.float64)))) * max(freq) * 2.0 ** -52
    return y, (24 * U + far) * size


def masked_attention(q, slots, k_pool, v_pool, scale, lo, hi, pos=None, slopes=None, cap=0.0, drop_none=False):
    """One request: q [n, Hq, d] (torch), slots [T], pools [slots, Hkv, d] (torch), lo / hi [n].  Keys outside a row's
    range are not looked at.  Returns the output and the bound of its error, float64 [n, Hq, d]."""
    dt = q.dtype
    q = q.detach().cpu().double().numpy()
    kp, vp = k_pool.detach().cpu().double().numpy(), v_pool.detach().cpu().double().numpy()
    n, hq, d = q.shape
    slots = np.asarray(slots, np.int64)
    T, hkv = len(slots), kp.shape[1]
    g = hq // hkv
    out, tol = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    inside = (slots >= 0) & (slots < len(kp))
    for i in range(n):
        t = np.arange(max(0, int(lo[i])), min(T, int(hi[i])))
        if drop_none:
            t = t[slots[t] != -1]
        if not len(t):
            continue
        at, ok = np.where(inside[t], slots[t], 0), inside[t][:, None]
        for h in range(hq):
            k, v = (np.where(ok, p[at, h // g], 0.0) for p in (kp, vp))
            with np.errstate(all="ignore"):
                dot = k @ q[i, h] * scale
                s = cap * np.tanh(dot / cap) if cap > 0 else dot
                size = np.abs(k) @ np.abs(q[i, h]) * abs(scale)
                # products of d terms in float32 (an MMA's additions may cut instead of round), the scale's
                # and the base's roundings
                ds = 2 * d * U * size.max() + 4 * U * np.abs(dot).max()
                if cap > 0:
                    # its quotient, tanh and product: 2^-22 of the cap, above 512 2^-20 of itself
                    ds = ds + (10 * U * cap if cap <= 512 else 20 * U * np.abs(dot).max())
                if slopes is not None:
                    bias = float(slopes[h]) * np.abs(float(pos[i]) - t)
                    s = s - bias
                    ds = ds + 4 * U * np.abs(bias).max()
                ds = ds + 4 * U * np.abs(s).max()
                p = np.exp(s - s.max())
                p = p / p.sum()
                o, A = p @ v, p @ np.abs(v)
                rel = 2 * ds + len(t) * U + 2.0 ** -21
                if dt == torch.bfloat16:
                    rel = rel + HALF[dt]                       # the weights, rounded before the product with V
                out[i, h] = o
                tol[i, h] = 1.01 * (HALF[dt] * (np.abs(o) + rel * A) + rel * A) + 1e-30
    return out, tol


def token_scores(x, temperature):
    """x [rows, V] (torch): log probabilities and entropy in float64, the order of the tokens, and the bounds of the
    errors of a log probability (per token) and of the entropy."""
    x = x.detach().cpu().double().numpy()
    R, V = x.shape
    with np.errstate(all="ignore"):
        y = x / temperature
        m = y.max(-1, keepdims=True)
        e = np.exp(y - m)
        S = e.sum(-1, keepdims=True)
        lp = y - m - np.log(S)
        p = e / S
        H = -np.where(p > 0, p * lp, 0.0).sum(-1)
        H = np.where(np.isnan(lp).any(-1) | np.isnan(S[:, 0]), np.nan, H)
        d = np.where(p > 0, np.minimum(np.abs(y - m), 140.0), 0.0)
        # a weight 2^d: d off by 3 roundings of itself, exp2 by 2^-22; sums of V weights through threads, warps and
        # CTAs (every thread adds at most V / 32 + 8 of them one after the other, then < 20 halvings and moves)
        rel = (p * (3 * U * 1.45 * d)).sum(-1) + 2.0 ** -21 + (V / 32 + 40) * U * (V <= 4096) + (V / 512 + 40) * U
        tol_lp = rel[:, None] + 4 * U * (np.abs(y - m) + np.abs(np.log(S)) + 1)
        mean_d = (p * d).sum(-1)
        tol_h = rel * (1 + 3 * mean_d) + (p * d * 8 * U * 1.45 * (1 + d)).sum(-1) + 8 * U * (1 + np.abs(np.log(S[:, 0])))
    key = np.where(np.isnan(x), -np.inf, x) + 0.0
    # NaN behind -infinity
    order = np.stack([np.lexsort((np.arange(V), np.isnan(x[r]), -key[r])) for r in range(R)]) if R else np.zeros((0, V), int)
    return lp, H, order, tol_lp, tol_h

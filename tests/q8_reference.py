"""64-bit reference of the 8-bit KV pool for the tests, and the error bounds they use."""
from __future__ import annotations

import numpy as np
import torch

E_MIN, E_MAX = -50, 38
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative


def e4m3_values():
    """The 256 values of the format (code 0x7f and 0xff are NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


VALUES = e4m3_values()


def quantise(x):
    """Codes (uint8) and scale bytes (uint8) of rows x [..., d] (a torch tensor), and which rows are
    poisoned.  Nearest code by search over the format's values, ties to the even code."""
    x = x.detach().cpu().double().numpy()
    top = np.abs(x).max(-1)
    finite = np.isfinite(x).all(-1)
    e = np.full(top.shape, E_MIN)
    for _ in range(E_MAX - E_MIN):
        with np.errstate(invalid="ignore"):
            e = np.where((top > 448 * 2.0 ** e) & (e < E_MAX), e + 1, e)
    bad = ~finite | ~(top <= 448 * 2.0 ** float(E_MAX))
    y = np.where(bad[..., None], 0.0, x) / 2.0 ** e[..., None].astype(float)
    pos = VALUES[:127]                                # ascending codes 0..126
    a = np.abs(y)
    hi = np.clip(np.searchsorted(pos, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.signbit(y), code | 128, code)
    code = np.where(bad[..., None], 0, code)
    return code.astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8), bad


def values(codes, scale):
    """float64 values of codes [..., d] with scale bytes [...]."""
    f = np.where(scale > E_MAX + 127, np.nan, 2.0 ** (scale.astype(float) - 127))
    f = np.where(scale == 0, 0.0, f)
    return VALUES[codes] * f[..., None]


def random_pool(num_slots, hkv, d, g, spread=0.4):
    """A filled pool (CPU tensors: codes k, v, scales) and its values as float64 arrays."""
    out, scale = [], []
    for _ in range(2):
        x = torch.randn((num_slots, hkv, d), generator=g) * torch.exp(spread * torch.randn((num_slots, hkv, 1), generator=g))
        c, s, _ = quantise(x)
        out.append(torch.from_numpy(c))
        scale.append(torch.from_numpy(s))
    kv_scale = torch.stack(scale, -1).contiguous()
    vals = [values(o.numpy(), s.numpy()) for o, s in zip(out, scale)]
    return out[0], out[1], kv_scale, vals[0], vals[1]


def attention(q, slots, kval, vval, scale, drop_none=False):
    """One request: q [n, Hq, d] (torch), slots [T] ints; a slot outside the pool is a zero row, with
    drop_none -1 is no key.  Returns the output and the bound of its error for outputs in q's
    dtype, both float64 [n, Hq, d]."""
    dt = q.dtype
    q = q.detach().cpu().double().numpy()
    n, hq, d = q.shape
    slots = np.asarray(slots, np.int64)
    if drop_none:
        slots = slots[slots != -1]
    T = len(slots)
    out, tol = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    if T == 0:
        return out, tol
    inside = (slots >= 0) & (slots < len(kval))
    k = np.where(inside[:, None, None], kval[np.where(inside, slots, 0)], 0.0)
    v = np.where(inside[:, None, None], vval[np.where(inside, slots, 0)], 0.0)
    g = hq // kval.shape[1]
    for h in range(hq):
        kh, vh = k[:, h // g], v[:, h // g]
        s = q[:, h] @ kh.T * scale
        with np.errstate(invalid="ignore"):
            p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        out[:, h] = p @ vh
        A = p @ np.abs(vh)
        dot = np.abs(q[:, h]) @ np.abs(kh).T * abs(scale)
        # float32 sums of d products and T probabilities, the base-2 argument (2 roundings of a
        # logit), exp2 to 2^-22
        ds = (d * 2.0 ** -24) * dot.max(-1) + 2 * 2.0 ** -24 * 1.5 * np.abs(s).max(-1)
        rel = 2 * ds + T * 2.0 ** -24 + 2.0 ** -21
        if dt == torch.bfloat16:
            # queries carried as two e4m3 terms: off by at most 2^-17 of the row's largest; the
            # probabilities rounded to bf16
            ds = 2.0 ** -17 * np.abs(q[:, h]).max(-1) * np.abs(kh).sum(-1).max() * abs(scale)
            rel = rel + 2 * ds + HALF[dt]
        tol[:, h] = 1.01 * (HALF[dt] * (np.abs(out[:, h]) + rel[:, None] * A) + rel[:, None] * A) + 1e-30
    return out, tol


def assert_attention(got, want, tol, what=""):
    got = np.asarray(got, np.float64)
    assert got.shape == want.shape, (got.shape, want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN pattern differs"
    live = ~np.isnan(want)
    over = (np.abs(got - want) - tol)[live]
    assert not (over > 0).any(), f"{what}: {np.sum(over > 0)} elements, worst {over.max():.3e} over its bound"

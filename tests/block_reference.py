"""Plain 64-bit restatements of the 8-bit store and of the bounds of the
attention over it, from the definitions in include/mac.h; numpy, no library
code."""
import math

import numpy as np

from serving_reference import E4M3, _nearest_even

PAGE, D = 16, 128
E_MIN, E_MAX = -60, 60


def e4m3(x):
    """The nearest e4m3 value, ties to even, at most 448; NaN where x is not finite."""
    x = np.asarray(x, np.float64)
    ok = np.isfinite(x)
    y = E4M3[_nearest_even(np.abs(np.where(ok, x, 0.0)), E4M3)]
    return np.where(ok, np.copysign(y, x), np.nan)


def need(x):
    """The smallest e in E_MIN .. E_MAX with every finite |x| at most 448 2^e."""
    top = np.abs(x[np.isfinite(x)]).max(initial=0.0)
    e = E_MIN
    while e < E_MAX and top > 448.0 * 2.0 ** e:
        e += 1
    return e


class Store:
    """Codes by (page, K or V, head, offset) as their values, and exponents."""

    def __init__(self, num_pages, kv_heads):
        self.code = np.zeros((num_pages, 2, kv_heads, PAGE, D))
        self.exp = np.full((num_pages, 2, kv_heads), E_MIN)

    def append(self, k, v, slots):
        k, v, slots = np.asarray(k, np.float64), np.asarray(v, np.float64), np.asarray(slots)
        inside = (slots >= 0) & (slots < len(self.code) * PAGE)
        for page in sorted(set(int(s) // PAGE for s in slots[inside])):
            here = {int(s) % PAGE: t for t, s in enumerate(slots) if inside[t] and int(s) // PAGE == page}  # the last one
            for w, x in enumerate((k, v)):
                for h in range(k.shape[1]):
                    old = self.exp[page, w, h]
                    e = need(np.stack([x[t, h] for t in here.values()]))
                    if 0 in here:
                        self.code[page, w, h] = 0
                    else:
                        e = max(e, old)
                        self.code[page, w, h] = e4m3(self.code[page, w, h] * 2.0 ** float(old - e))
                    for off, t in here.items():
                        with np.errstate(invalid="ignore"):
                            self.code[page, w, h, off] = e4m3(x[t, h] / 2.0 ** float(e))
                    self.exp[page, w, h] = e

    def gather(self, slots):
        """(k, v) [tokens, kv_heads, 128]; zeros where there is no slot."""
        slots = np.asarray(slots)
        inside = (slots >= 0) & (slots < len(self.code) * PAGE)
        p, o = np.where(inside, slots, 0) // PAGE, np.where(inside, slots, 0) % PAGE
        x = self.code[p, :, :, o] * 2.0 ** self.exp[p].astype(float)[..., None]        # [tokens, 2, heads, 128]
        x[~inside] = 0.0
        return x[:, 0], x[:, 1]


def attention(q, keys, values, ev, scale):
    """q [n_query, heads, 128] over a request's keys, values [len, kv_heads, 128]; ev [len, kv_heads] the exponent of each
    token's value scale.  Returns out, lse and what the bounds need: mag = sum max(p, 2^-23 r / 2^ev) |v| / sum p, where
    r is the row's largest p 2^ev, and the largest sum |q k| scale."""
    nq, H, _ = q.shape
    n, Hkv, _ = keys.shape
    G = H // Hkv
    out, lse = np.zeros((nq, H, D)), np.full((nq, H), -np.inf)
    mag, top = np.zeros((nq, H, D)), np.zeros((nq, H))
    for i in range(nq):
        seen = n - (nq - 1) + i
        if seen <= 0:
            continue
        for h in range(H):
            k, v, e = keys[:seen, h // G], values[:seen, h // G], ev[:seen, h // G].astype(float)
            s = k @ q[i, h] * scale
            m = s.max()
            p = np.exp(s - m)
            l = p.sum()
            out[i, h] = p @ v / l
            lse[i, h] = m + math.log(l)
            r = (s / math.log(2) + e).max() - m / math.log(2)            # log2 of the largest p 2^ev
            mag[i, h] = np.maximum(p, 2.0 ** np.clip(r - 23 - e, -1000, 1000)) @ np.abs(v) / l
            top[i, h] = (np.abs(k) @ np.abs(q[i, h])).max() * scale
    return out, lse, mag, top


def attention_tolerance(out, mag, top, lse, n):
    """Bounds on the kernel's error per element of out and of lse.

    out is rounded to bf16: 2^-8 of it.  A weight is w = 2^(s + ev - low) with low at least 9 and at most 15 below the
    row's largest s + ev, rounded to f16: within 2^-11 of it, or, below f16's smallest normal 2^-14, within 2^-25,
    which is at most 2^-34 = 2^-11 2^-23 of the largest weight: together 2^-11 mag.  A score is 8 fp32 accumulations of
    16 products (each within 2^-23 of sum |q k|) times an fp32 factor, itself rounded twice: 8 * 2^-23 top + 3 * 2^-23
    |score| <= 12 * 2^-23 top; the difference low - ev and the one with the score are rounded, each to 2^-24 of at most
    1.45 top + 80 log2 units, together 2^-23 (1.45 top + 80) ln 2 <= 2^-23 (1.1 top + 56); the exponential is good to
    2^-21.  Weight and normaliser are each off by that sum.  Sums over n tokens add at most n / 16 accumulations
    per row and the merges, under 64 + n / 16 in all, each 2^-23 of mag (and 2^-23 of the normaliser)."""
    d = 2.0 ** -23 * (14 * top + 56) + 2.0 ** -21
    acc = (64 + n / 16) * 2.0 ** -23
    return (2.0 ** -8 * np.abs(out) + mag * (2.0 ** -11 + 2 * d + 2 * acc)[..., None] + 1e-30,
            d + acc + 2.0 ** -21 * np.abs(np.where(np.isfinite(lse), lse, 0.0)) + 2.0 ** -22)

"""Plain 64-bit restatements of the operators around the decode step, for the
tests: the norm and rotation, one step of page bookkeeping, the 4-bit format
and attention.  Written from the definitions in include/mac.h; numpy and torch
on the CPU, no library code."""
import math

import numpy as np
import torch

PAGE, D, BLOCK = 16, 128, 16

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# the finite non-negative e4m3 values in code order: 2^-9 steps below 2^-6, then 8 steps per power of two
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] +
                [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:119])


def _nearest_even(x, grid):
    """Index of the grid value nearest to x, ties to the even index (the even significand), saturating."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    up, down = grid[hi] - x, x - grid[lo]
    return np.where(up < down, hi, np.where(up > down, lo, np.where(lo % 2 == 0, lo, hi)))


def stored(x, scale=1.0):
    """The values the 4-bit store holds for x [..., 128] (numpy float64)."""
    x = np.asarray(x, np.float64) / scale
    b = x.reshape(-1, BLOCK)
    bad = ~np.isfinite(b).all(axis=1)
    safe = np.where(bad[:, None], 0.0, b)
    s = E4M3[_nearest_even(np.abs(safe).max(axis=1) / 6.0, E4M3)][:, None]
    q = np.divide(np.abs(safe), s, out=np.zeros_like(safe), where=s > 0)
    y = np.sign(safe) * E2M1[_nearest_even(q, E2M1)] * s
    y[bad] = np.nan
    return (y * scale).reshape(x.shape)


def norm_rope(x, w, pos, rotary, base, interleaved, eps):
    """(y, rotated y) in float64: x [T, heads, 128], pos [T]."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    r = y.clone()
    for i in range(rotary // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)
        t = pos.double() * base ** (-2.0 * i / rotary)
        c, s = torch.cos(t)[:, None], torch.sin(t)[:, None]
        r[..., a] = y[..., a] * c - y[..., b] * s
        r[..., b] = y[..., b] * c + y[..., a] * s
    return y, r


def page_step(lengths, new, table, ring, state, max_tokens):
    """One step, request by request.  Returns (lengths, state, starts, positions, slots, table, ring, status)."""
    table, ring = np.array(table, np.int64), np.array(ring, np.int64)
    B, P, N = len(lengths), table.shape[1], len(ring)
    head, count = int(state[0]), int(state[1])
    status, at, want, taken, freed = 0, 0, 0, 0, []
    ok_state = 0 <= head < N and 0 <= count <= N
    if not ok_state:
        status |= 4
    out = [int(x) for x in lengths]
    starts, pos, slot = [0], [0] * max_tokens, [-1] * max_tokens
    free = count if ok_state else 0
    for b in range(B):
        n, old = int(new[b]), int(lengths[b])
        have = -(-old // PAGE) if old >= 0 else 0
        m = max(n, 0)
        if old < 0 or old > PAGE * P:
            status |= 4
            old, granted = 0, False
        elif n < 0:
            freed += [int(p) for p in table[b, :have]]
            out[b], granted = 0, False
        else:
            need = -(-(old + n) // PAGE) - have
            granted = False
            if have + need > P:
                status |= 2
            elif at + n > max_tokens:
                status |= 8
            else:
                want += need
                if need and want > free:
                    status |= 1
                else:
                    granted = True
                    for c in range(need):
                        table[b, have + c] = ring[(head + want - need + c) % N]
                    if need:
                        taken = want
                    out[b] = old + n
        for i in range(m):
            if at + i >= max_tokens:
                break
            p = old + i
            pos[at + i] = p
            if granted:
                page = int(table[b, p // PAGE])
                if 0 <= page < N:
                    slot[at + i] = page * PAGE + p % PAGE
                else:
                    status |= 4
        at += m
        starts.append(min(at, max_tokens))
    if ok_state:
        back = len(freed)
        if count + back <= N:
            for c, p in enumerate(freed):
                ring[(head + count + c) % N] = p
                if not 0 <= p < N:
                    status |= 4
        else:
            status |= 16
            back = 0
        state = [(head + taken) % N, count - taken + back]
    elif freed:
        status |= 16
    return [np.array(x, np.int64) for x in (out, state, starts, pos, slot, table, ring, [status])]


def attention(q, keys, values, scale):
    """q [n_query, heads, 128] of one request over its keys, values [len, kv_heads, 128], all float64 numpy.  Returns
    out, lse, and per output row the quantities the tolerances need: sum max(p, 2^-23 p_max) |v| / sum p [.., 128] and
    the largest sum |q k| scale."""
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
            k, v = keys[:seen, h // G], values[:seen, h // G]
            s = k @ q[i, h] * scale
            m = s.max()
            p = np.exp(s - m)
            l = p.sum()
            out[i, h] = p @ v / l
            lse[i, h] = m + math.log(l)
            mag[i, h] = np.maximum(p, 2.0 ** -23) @ np.abs(v) / l
            top[i, h] = (np.abs(k) @ np.abs(q[i, h])).max() * scale
    return out, lse, mag, top


def attention_tolerance(out, mag, top, lse, n):
    """Bounds on the kernel's error per element of out and of lse.

    out is rounded to bf16: 2^-8 of it.  Each weight is rounded to f16, held times 2^9 against a reference that
    is no larger than the row's largest score: within 2^-11 of the weight, or, where that is below f16's smallest normal
    2^-14, within the subnormals' half step 2^-25, which is 2^-34 = 2^-11 2^-23 of the largest weight.  Together at most
    2^-11 sum max(p, 2^-23 p_max) |v| / sum p =: 2^-11 mag.  A score is a sum of 128 products in fp32 (8 accumulations of 16, each rounded or cut at
    2^-23 of sum |q k|), times an fp32 scale: within 16 * 2^-23 * top + 2^-22 |score| <= 18 * 2^-23 * top; the weight
    and its normaliser then are each off by that, plus 2^-21 of the exponential.  The sums over the n tokens add at
    most n / 16 accumulations per row plus the merges (under 64 + n / 16 in all), each 2^-23 of mag."""
    d = 18 * 2.0 ** -23 * top + 2.0 ** -21
    acc = (64 + n / 16) * 2.0 ** -23
    return (2.0 ** -8 * np.abs(out) + mag * (2.0 ** -11 + 2 * d + 2 * acc)[..., None] + 1e-30,
            d + acc + 2.0 ** -21 * np.abs(np.where(np.isfinite(lse), lse, 0.0)) + 2.0 ** -22)

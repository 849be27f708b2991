"""A restatement of the prompt attention kernel's work split, for the tests."""
TOK, EXTRA = 128, 4


def seen(n, m, lag, i):
    return min(max(m - n - lag + i + 1, 0), m)


def items(seqs, G, Hkv, lag):
    """Items in order, from those of the most blocks down: (sequence, head, tile, blocks of tile A, of tile B, first block on the edge)."""
    T, out = 128 // G, []
    for b, (n, m) in enumerate(seqs):
        for tile in reversed(range(-(-n // (2 * T)))):
            nblk = []
            for x in range(2):
                t = min(T, n - (2 * tile + x) * T)
                nblk.append(-(-seen(n, m, lag, (2 * tile + x) * T + t - 1) // TOK) if t > 0 else 0)
            edge = seen(n, m, lag, 2 * tile * T) // TOK
            out += [(b, h, tile, nblk[0], nblk[1], edge) for h in range(Hkv)]
    return sorted(out, key=lambda it: -cost(it))


def cost(it):
    return EXTRA + max(it[3], it[4], 1)


def split(its, grid):
    """(rounds, prefix of the line's costs, quotas) as each CTA derives them."""
    rounds = max(len(its) // grid - 1, 0)
    load = [sum(cost(its[r * grid + (grid - 1 - c if r & 1 else c)]) for r in range(rounds)) for c in range(grid)]
    line = its[rounds * grid:]
    pre = [0]
    for it in line:
        pre.append(pre[-1] + cost(it))
    total = pre[-1]
    lo, hi = 0, max(load) + -(-total // grid)
    while lo < hi:
        mid = (lo + hi) // 2
        if sum(max(mid - x, 0) for x in load) >= total:
            hi = mid
        else:
            lo = mid + 1
    quota, at = [], 0
    for x in load:
        quota.append(min(at, total))
        at = min(at + max(hi - x, 0), total)
    # a bound among an item's extra blocks, or behind them, moves to its beginning
    for c, q in enumerate(quota):
        start = max((p for p in pre[:-1] if p <= q), default=0)
        if q < total and q - start <= EXTRA:
            quota[c] = start
    return rounds, load, pre, quota + [total]


def walk(its, grid, c, sp):
    """CTA c's pieces: (item, first block, last block + 1, partial slot or -1)."""
    rounds, _, pre, quota = sp
    for r in range(rounds):
        i = r * grid + (grid - 1 - c if r & 1 else c)
        yield i, 0, max(its[i][3], its[i][4]), -1
    at, end = quota[c], quota[c + 1]
    lo, hi = 0, len(pre) - 1
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if pre[mid] <= at else (lo, mid)
    k = lo
    while at < end:
        it = its[rounds * grid + k]
        start, stop = pre[k], pre[k] + cost(it)
        begins, ends = start >= at, stop <= end
        j0, j1, slot = 0, max(it[3], it[4]), -1
        if not (begins and ends):
            slot, j0, j1 = (1 if begins else 0), max(at - start - EXTRA, 0), min(j1, end - start - EXTRA)
        yield rounds * grid + k, j0, j1, slot
        at = min(stop, end)
        k += 1


def spans(its, grid, sp):
    """The items that the second kernel merges: item -> (first CTA, last CTA)."""
    rounds, _, pre, quota = sp
    out = {}
    for k in range(len(pre) - 1):
        for c in range(grid):
            if quota[c] <= pre[k] < quota[c + 1] and pre[k + 1] > quota[c + 1]:
                d = c
                while quota[d + 1] < pre[k + 1]:
                    d += 1
                out[rounds * grid + k] = (c, d)
    return out

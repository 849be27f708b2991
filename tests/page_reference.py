"""A plain restatement of one step of page bookkeeping with rejected drafts and
refused releases, for the tests.  Written from the definitions in
include/mac.h, request by request; no library code."""
import numpy as np

PAGE = 16


def pages(tokens):
    return -(-tokens // PAGE)


def step(lengths, new, table, ring, state, max_tokens, rejected=None):
    """Returns (lengths, state, starts, positions, slots, table, ring, status, unreleased)."""
    table, ring = np.array(table, np.int64), np.array(ring, np.int64)
    B, P, N = len(lengths), table.shape[1], len(ring)
    head, count = int(state[0]), int(state[1])
    ok_state = 0 <= head < N and 0 <= count <= N
    status = 0 if ok_state else 4
    free = count if ok_state else 0
    old = [int(x) for x in lengths]
    out, unreleased = list(old), [0] * B
    back = [int(rejected[b]) if rejected is not None and new[b] >= 0 else 0 for b in range(B)]
    good = [0 <= old[b] <= PAGE * P and 0 <= back[b] <= old[b] for b in range(B)]
    kept = [old[b] - back[b] if good[b] else 0 for b in range(B)]
    granted, fresh, gives = [False] * B, [0] * B, [[] for _ in range(B)]
    at, want, taken, begin = 0, 0, 0, []
    # who gets what
    for b in range(B):
        n = max(int(new[b]), 0)
        begin.append(at)
        at += n
        if not good[b]:
            status |= 4
            continue
        held = pages(old[b])
        if new[b] < 0:
            gives[b] = [int(p) for p in table[b, :held]]
            out[b] = 0
            continue
        after = pages(kept[b] + n)
        need = max(after - held, 0)
        if after > P:
            status |= 2
        elif at > max_tokens:
            status |= 8
        else:
            want += need
            if need and want > free:
                status |= 1
            else:
                granted[b], fresh[b] = True, want - need
                if need:
                    taken = want
        out[b] = kept[b] + n if granted[b] else kept[b]
        left = pages(out[b])
        if left < held:
            gives[b] = [int(p) for p in table[b, left:held]]
    # what cannot be given back stays where it is: all of it, or a request that holds an id outside the pool
    room = ok_state and free + sum(map(len, gives)) <= N
    if not room and any(gives):
        status |= 16
    for b in range(B):
        stuck = gives[b] and (not room or any(not 0 <= p < N for p in gives[b]))
        if stuck:
            if room:
                status |= 4
            if new[b] < 0:
                unreleased[b] = old[b]
            else:
                out[b], granted[b], kept[b] = old[b], False, old[b]
            gives[b] = []
    # tables and slots
    pos, slot = [0] * max_tokens, [-1] * max_tokens
    for b in range(B):
        held = pages(old[b]) if good[b] else 0
        if granted[b]:
            for c in range(pages(out[b]) - held):
                table[b, held + c] = ring[(head + fresh[b] + c) % N]
                if not 0 <= table[b, held + c] < N:
                    status |= 4
        for i in range(max(int(new[b]), 0)):
            if begin[b] + i >= max_tokens:
                break
            p = kept[b] + i
            pos[begin[b] + i] = p
            if granted[b]:
                page = int(table[b, p // PAGE])
                if 0 <= page < N:
                    slot[begin[b] + i] = page * PAGE + p % PAGE
                else:
                    status |= 4
    starts = [min(x, max_tokens) for x in begin + [at]]
    freed = [p for g in gives for p in g]
    for c, p in enumerate(freed):
        ring[(head + free + c) % N] = p
    if ok_state:
        state = [(head + taken) % N, count - taken + len(freed)]
    return [np.array(x, np.int64) for x in (out, state, starts, pos, slot, table, ring, [status], unreleased)]

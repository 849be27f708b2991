"""The prompt attention's work split on the CPU: every block of every item is
done once, partial results land where the second kernel looks for them, and
the CTAs' loads are level."""
import random

import pytest

import prompt_split as S


def _cases():
    yield [(16, 16)], 4, 8, 0
    yield [(0, 5), (1, 1), (0, 0)], 1, 1, 0
    yield [(300, 300)], 7, 4, 400
    yield [(32768, 32768)], 4, 8, 0
    yield [(2048, 32768), (509, 8700)], 4, 8, 0
    yield [(512, 32768)], 4, 8, 64
    yield [(1, 100000)] * 9, 8, 1, 0
    yield [(5, 2)], 128, 2, 0
    r = random.Random(7)
    for _ in range(60):
        G, Hkv = r.choice([1, 2, 3, 4, 7, 8, 16, 32, 100, 128]), r.choice([1, 2, 3, 8])
        seqs = []
        for _ in range(r.choice([1, 2, 5, 40])):
            n = int(2 ** r.uniform(0, 12)) * (r.random() < 0.9)
            seqs.append((n, max(n + int(2 ** r.uniform(0, 14)) * (r.random() < 0.4) - (r.random() < 0.1) * r.randint(0, 50), 0)))
        yield seqs, G, Hkv, r.choice([0, 0, 1, 64, 5000])


@pytest.mark.parametrize("grid", [152, 7, 256])
def test_every_block_once_and_level_loads(grid):
    for seqs, G, Hkv, lag in _cases():
        its = S.items(seqs, G, Hkv, lag)
        if not its:
            continue
        sp = S.split(its, grid)
        rounds, load, pre, quota = sp
        assert len(pre) - 1 < 2 * grid and quota[0] == 0 and all(a <= b for a, b in zip(quota, quota[1:]))
        done, slots, work = {}, {}, []
        for c in range(grid):
            w = 0
            for i, j0, j1, slot in S.walk(its, grid, c, sp):
                assert 0 <= j0 <= j1 and (slot < 0 or j0 < j1)
                done.setdefault(i, []).append((j0, j1, c, slot))
                if slot >= 0:
                    assert (c, slot) not in slots           # one partial per CTA and slot
                    slots[c, slot] = i
                w += max(j1 - j0, 1) + (S.EXTRA if j0 == 0 else 0)
            work.append(w)
        assert sorted(done) == list(range(len(its)))
        merged = S.spans(its, grid, sp)
        for i, parts in done.items():
            parts.sort(key=lambda x: x[2])
            assert parts[0][0] == 0 and parts[-1][1] == max(its[i][3], its[i][4])
            assert all(a[1] == b[0] for a, b in zip(parts, parts[1:]))
            if len(parts) == 1:
                assert parts[0][3] == -1 and i not in merged
            else:
                first, last = merged[i]
                assert parts[0][2] == first and parts[-1][2] == last and parts[0][3] == 1
                assert all(x[3] == 0 for x in parts[1:])
                # a CTA between them without a share says so itself
                assert set(range(first, last + 1)) - {x[2] for x in parts} <= {c for c in range(grid) if quota[c] == quota[c + 1]}
        if max(load) * grid <= sum(load) + pre[-1]:
            # a share may pass the level by a block, and by the extra blocks that moved to it
            assert max(work) - sum(work) / grid <= 2 + S.EXTRA

"""The prompt attention's work split as the kernel numbers its items, by levels
that are coarse where sequences are long; and the constants that the
restatement in prompt_split.py shares with the kernel."""
import os
import re

import pytest

import prompt_split as S

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_computation_gb300", "csrc")
LEVELS = 2048


def _constants():
    out = {}
    for name in ("mac_prompt.cuh", "mac_prompt_attention.cu"):
        for key, value in re.findall(r"constexpr int (\w+) = (\d+);", open(os.path.join(CSRC, name)).read()):
            out[key] = int(value)
    return out


def test_the_restatements_constants_are_the_kernels():
    c = _constants()
    assert (c["kTok"], c["kPExtra"], c["kPLevels"], c["kPLineRows"]) == (S.TOK, S.EXTRA, LEVELS, 1)
    its = S.items([(64 * 1000, 64 * 1000)], 4, 1, 0)
    assert len(its) == 1000 and S.split(its, 152)[0] == 1000 // 152 - c["kPLineRows"]
    assert c["kPMaxCtas"] >= 152 and c["kPRows"] == 2 * 128


class Numbered:
    """Items as the kernel numbers them: tiles_from, level_of, item_at and blocks_at restated."""

    def __init__(self, seqs, G, Hkv, lag):
        self.T, self.Hkv = 128 // G, Hkv
        self.q = [(n, m - n - lag) for n, m in seqs]
        top = max((self.blocks(s, self.tiles(s) - 1) for s in self.q if s[0] > 0), default=0)
        self.shift = 0
        while top >> self.shift >= LEVELS:
            self.shift += 1
        self.levels = (top >> self.shift) + 1
        self.above = [sum(self.tiles_from(s, k << self.shift) for s in self.q) * Hkv for k in range(self.levels + 1)]

    def tiles(self, s):
        return (s[0] + 2 * self.T - 1) // (2 * self.T)

    def seen(self, s, token):
        return (max(s[1] + token + 1, 0) + S.TOK - 1) // S.TOK

    def blocks(self, s, tile):
        return max(self.seen(s, min((tile + 1) * 2 * self.T, s[0]) - 1), 1)

    def tiles_from(self, s, blocks):
        tiles = self.tiles(s)
        if blocks <= 1:
            return tiles
        need = (blocks - 1) * S.TOK + 1 - s[1]
        if need > s[0]:
            return 0
        return tiles if need <= 0 else tiles - (need - 1) // (2 * self.T)

    def level(self, i):
        lo, hi = 0, self.levels
        while hi - lo > 1:
            mid = (lo + hi) >> 1
            lo, hi = (mid, hi) if self.above[mid] > i else (lo, mid)
        return lo

    def item(self, i):
        k = self.level(i)
        place = i - self.above[k + 1]
        for b, s in enumerate(self.q):
            high = self.tiles_from(s, (k + 1) << self.shift)
            own = (self.tiles_from(s, k << self.shift) - high) * self.Hkv
            if place < own:
                down, head = divmod(place, self.Hkv)
                tile = self.tiles(s) - 1 - high - down
                tok0, T = 2 * tile * self.T, self.T
                ta, tb = min(T, s[0] - tok0), max(min(T, s[0] - tok0 - T), 0)
                return (b, head, tile, self.seen(s, tok0 + ta - 1), self.seen(s, tok0 + T + tb - 1) if tb else 0)
            place -= own
        raise AssertionError(i)


def _split(num, its, grid):
    """S.split with the whole items' loads by their levels, as the kernel adds them up."""
    rounds = max(len(its) // grid - 1, 0)
    load = [sum((num.level(r * grid + (grid - 1 - c if r & 1 else c)) << num.shift) + S.EXTRA for r in range(rounds))
            for c in range(grid)]
    pre = [0]
    for it in its[rounds * grid:]:
        pre.append(pre[-1] + S.cost(it))
    total, live = pre[-1], load
    level = -(-total // grid)
    while rounds:                                       # the mean over those that are not past it
        level = -(-(sum(live) + total) // len(live))
        left = [x for x in live if x < level]
        if len(left) == len(live):
            break
        live = left
    quota, at = [], 0
    for x in load:
        quota.append(min(at, total))
        at += max(level - x, 0)
    assert at >= total
    for c, q in enumerate(quota):
        start = max((p for p in pre[:-1] if p <= q), default=0)
        if q < total and q - start <= S.EXTRA:
            quota[c] = start
    return rounds, load, pre, quota + [total]


@pytest.mark.parametrize("seqs,G,Hkv,lag,shift", [
    ([(300, 300), (17, 900), (0, 4), (2000, 2000)], 4, 2, 0, 0),
    ([(262144, 262144)], 8, 1, 0, 1),
    ([(40, 300001), (100, 100), (3, 262200), (1, 5), (70, 270000), (0, 9)], 2, 2, 0, 1),
    ([(30000, 600000), (5, 5), (9000, 9000)], 7, 1, 64, 2),
    ([(2000, 1200000)] * 3 + [(500, 500)], 32, 1, 0, 3),
    ([(20000, 262143)], 1, 4, 0, 1), ([(20000, 262016)], 1, 4, 0, 0)])
@pytest.mark.parametrize("grid", [152, 7])
def test_items_by_levels_cover_every_block_once(seqs, G, Hkv, lag, shift, grid):
    num = Numbered(seqs, G, Hkv, lag)
    assert num.shift == shift and num.levels <= LEVELS
    its = [num.item(i) for i in range(num.above[0])]
    want = S.items(seqs, G, Hkv, lag)
    assert sorted(its) == sorted(it[:5] for it in want)
    big = [max(it[3], it[4], 1) >> shift for it in its]
    assert big == sorted(big, reverse=True) and big == [num.level(i) for i in range(len(its))]
    if shift == 0:                                      # then the order of costs is that of the restatement
        assert [S.cost(it) for it in its] == [S.cost(it) for it in want]
    sp = _split(num, its, grid)
    rounds, load, pre, quota = sp
    assert len(pre) - 1 < 2 * grid and quota[0] == 0 and all(a <= b for a, b in zip(quota, quota[1:]))
    if shift == 0:
        assert sp == S.split(want, grid)
    done = {}
    for c in range(grid):
        slots = set()
        for i, j0, j1, slot in S.walk(its, grid, c, sp):
            assert 0 <= j0 <= j1 and (slot < 0 or j0 < j1) and slot not in slots
            if slot >= 0:
                slots.add(slot)
            done.setdefault(i, []).append((c, j0, j1, slot))
    assert sorted(done) == list(range(len(its)))
    merged = S.spans(its, grid, sp)
    for i, parts in done.items():
        assert parts[0][1] == 0 and parts[-1][2] == max(its[i][3], its[i][4])
        assert all(a[2] == b[1] for a, b in zip(parts, parts[1:]))
        if len(parts) == 1:
            assert parts[0][3] == -1 and i not in merged
        else:
            assert merged[i] == (parts[0][0], parts[-1][0]) and [p[3] for p in parts] == [1] + [0] * (len(parts) - 1)

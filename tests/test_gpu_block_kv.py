"""The 8-bit store and the attention over it on the GPU, against 64-bit
restatements of their definitions (block_reference.py, where the tolerances are
derived); stored values are compared exactly."""
import numpy as np
import pytest
import torch

import block_reference as BR
from test_gpu_serving_ops import BF16, _randn

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def _np(t):
    return t.double().cpu().numpy()


def _sized(shape, seed, spread=2.0):
    """Tokens [n, heads, 128] whose sizes differ by powers of two of `spread` standard deviation."""
    r = np.random.default_rng(seed)
    return (torch.from_numpy(r.standard_normal(shape) * 2.0 ** (spread * r.standard_normal((shape[0], shape[1], 1))))
            ).to(BF16)


# ---- the store -------------------------------------------------------------------

def _round(cache, ref, k, v, slots, every):
    cache.append(k.cuda(), v.cuda(), _i32(slots))
    ref.append(_np(k), _np(v), slots)
    for got, want in zip(cache.gather(_i32(every)), ref.gather(every)):
        np.testing.assert_array_equal(_np(got), want)


@pytest.mark.parametrize("T,Hkv,pages", [(1, 1, 1), (7, 8, 3), (64, 3, 4), (333, 2, 40), (1024, 2, 80), (1025, 2, 80),
                                         (2500, 1, 200), (4096, 4, 256)])
def test_store_in_any_order(T, Hkv, pages):
    """Tokens anywhere in any pages, two calls behind one another (pages started anew, pages that grow, pages that keep
    their scale), on both sides of the length where the append changes its form."""
    from kv_cache_computation_gb300 import BlockKV
    cache, ref = BlockKV(Hkv, Hkv, num_pages=pages), BR.Store(pages, Hkv)
    every = np.arange(pages * 16)
    for seed in (1, 2, 3):
        slots = np.random.default_rng(seed).permutation(pages * 16)[:T]
        slots[T // 2] = -3 if T > 1 else slots[0]
        _round(cache, ref, _sized((T, Hkv, 128), seed), _sized((T, Hkv, 128), 10 + seed), slots, every)
    cache.sync()


@pytest.mark.parametrize("first,T,pages", [(0, 64, 9), (0, 40, 9), (3, 61, 9), (16, 16, 9), (5, 7, 9), (0, 2064, 130),
                                           (7, 2051, 130)])
def test_store_whole_pages(first, T, pages):
    """Runs of consecutive tokens that start and end inside a page, then token by token as in decoding."""
    from kv_cache_computation_gb300 import BlockKV
    Hkv = 2
    cache, ref = BlockKV(Hkv, Hkv, num_pages=pages), BR.Store(pages, Hkv)
    order = np.random.default_rng(4).permutation(pages)
    every = (order[:, None] * 16 + np.arange(16)).reshape(-1)
    if first:
        _round(cache, ref, _sized((first, Hkv, 128), 5), _sized((first, Hkv, 128), 6), every[:first], every)
    _round(cache, ref, _sized((T, Hkv, 128), 7), _sized((T, Hkv, 128), 8), every[first:first + T], every)
    for t in range(first + T, min(first + T + 20, pages * 16)):
        _round(cache, ref, _sized((1, Hkv, 128), 100 + t, 4.0), _sized((1, Hkv, 128), 200 + t, 4.0), every[t:t + 1], every)


def test_store_values_at_every_border():
    """Ties between codes, 448 times a power of two and its neighbours, the smallest codes, what saturates, what is
    below every scale, zeros of both signs."""
    from kv_cache_computation_gb300 import BlockKV
    vals = [448.0, 450.0, 446.0, 224.0, 225.0, 17.0, 17.5, 18.5, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9, 3.0 * 2.0 ** -10,
            0.0, -0.0, 2.0 ** -6, 15.0 * 2.0 ** -10, 1.0, 1.0625, 1.1875]
    tops = [448.0, 450.0, 449.0, 2.0 ** 60, 448.0 * 2.0 ** 60, 2.0 ** 69, 2.0 ** 127, 2.0 ** -52, 2.0 ** -60, 2.0 ** -69,
            2.0 ** -71, 2.0 ** -133, 0.0, 0.875, 0.88]
    k = torch.zeros(len(tops), 1, 128)
    for t, top in enumerate(tops):
        k[t, 0, 0] = top
        for i, x in enumerate(vals):
            y = x * (top / 448.0 if top else 1e-30)
            k[t, 0, 2 * i + 1], k[t, 0, 2 * i + 2] = y, -y
    k = k.to(BF16)
    cache, ref = BlockKV(1, 1, num_pages=len(tops)), BR.Store(len(tops), 1)
    slots = np.arange(len(tops)) * 16
    _round(cache, ref, k, k.flip(0), slots, np.arange(len(tops) * 16))
    _round(cache, ref, k.roll(1, 0), k, slots + 3, np.arange(len(tops) * 16))     # every page meets another size
    _round(cache, ref, k.roll(2, 0), k.flip(0), slots + 1, np.arange(len(tops) * 16))


def test_store_nonfinite_duplicates_bad_slots_and_strides():
    from kv_cache_computation_gb300 import BlockKV, MacError
    cache, ref = BlockKV(4, 2, num_pages=3), BR.Store(3, 2)
    wide = _randn((9, 2 * 2 * 128 + 8), 9)
    wide[1, 5] = float("nan")
    wide[2, 256 + 20] = float("-inf")
    wide[3, 128:256] = float("inf")
    x = wide.cuda()
    slots = np.array([0, 31, 7, 48, 31, 2 ** 31 - 1, 7, 33, -5])      # two past the store, two twice
    cache.append(x[:, :256], x[:, 256:512], _i32(slots))
    ref.append(_np(wide[:, :256].reshape(9, 2, 128)), _np(wide[:, 256:512].reshape(9, 2, 128)), slots)
    every = np.concatenate((np.arange(48), [-1, 47, 3]))
    for got, want in zip(cache.gather(_i32(every)), ref.gather(every)):
        np.testing.assert_array_equal(_np(got), want)
    with pytest.raises(MacError, match="slot"):
        cache.sync()
    cache.sync()                                                        # reported once
    got = cache.gather(_i32([0, 48, 1, 1]))[0]
    assert (got[1] == 0).all()
    with pytest.raises(MacError, match="slot"):
        cache.sync()


def test_store_beyond_32_bit_offsets():
    """The last pages of a store of more than 2^32 bytes."""
    from kv_cache_computation_gb300 import BlockKV
    pages, Hkv = 140000, 8
    cache = BlockKV(Hkv, Hkv, num_pages=pages)
    assert cache.sizes["store"] > 2 ** 32
    ref = BR.Store(2, Hkv)
    base = (pages - 2) * 16
    for seed, slots in ((1, np.arange(20)), (2, np.arange(20, 32))):
        k, v = _sized((len(slots), Hkv, 128), seed), _sized((len(slots), Hkv, 128), 9 + seed)
        cache.append(k.cuda(), v.cuda(), _i32(base + slots))
        ref.append(_np(k), _np(v), slots)
    for got, want in zip(cache.gather(_i32(base + np.arange(32))), ref.gather(np.arange(32))):
        np.testing.assert_array_equal(_np(got), want)
    table = _i32([[pages - 2, pages - 1]])
    q = _randn((1, Hkv, 128), 5)
    out, lse = cache.attention(q.cuda(), table, _i32([32]))
    K, V = ref.gather(np.arange(32))
    ev = np.repeat(ref.exp[:, 1], 16, 0)
    o, l, mag, top = BR.attention(_np(q), K, V, ev, 1 / np.sqrt(128))
    to, tl = BR.attention_tolerance(o, mag, top, l, 32)
    assert (np.abs(_np(out) - o) <= to).all() and (np.abs(_np(lse) - l) <= tl).all()


# ---- attention -------------------------------------------------------------------

class Case:
    """Requests of given lengths in a store of shuffled pages, and their 64-bit counterparts."""

    def __init__(self, lens, H, Hkv, nq, seed=0, qscale=1.5, scale=0.0, spread=1.0):
        from kv_cache_computation_gb300 import BlockKV
        r = np.random.default_rng(seed)
        self.lens, self.scale, self.nq = list(lens), scale or 1 / np.sqrt(128), nq
        pages = [-(-n // 16) for n in lens]
        total = sum(pages) + 3
        perm = r.permutation(total)
        self.table = np.full((len(lens), max(max(pages), 1)), -1, np.int64)
        at = 0
        for b, p in enumerate(pages):
            self.table[b, :p] = perm[at:at + p]
            at += p
        self.cache = BlockKV(H, Hkv, num_pages=total, max_batch=len(lens), max_query=nq, sm_scale=scale)
        # what slots past a request's length hold must have no effect: a store full of NaN
        nan = torch.full((total * 16, Hkv, 128), float("nan"), dtype=BF16).cuda()
        self.cache.append(nan, nan, torch.arange(total * 16, dtype=torch.int32).cuda())
        self.k, self.v, self.ev = [], [], []
        for b, n in enumerate(lens):
            k, v = _sized((n, Hkv, 128), 100 + seed + b, spread), _sized((n, Hkv, 128), 200 + seed + b, spread)
            t = np.arange(n)
            slots = self.table[b, t // 16] * 16 + t % 16
            self.cache.append(k.cuda(), v.cuda(), _i32(slots))
            tail = np.arange(n, -(-n // 16) * 16)
            if len(tail):                       # the last page's other slots: NaN again
                self.cache.append(nan[:len(tail)], nan[:len(tail)], _i32(self.table[b, tail // 16] * 16 + tail % 16))
            K, V, E = np.zeros((n, Hkv, 128)), np.zeros((n, Hkv, 128)), np.zeros((n, Hkv), int)
            for x, out, ex in ((_np(k), K, None), (_np(v), V, E)):
                for p in range(0, n, 16):
                    for h in range(Hkv):
                        e = BR.need(x[p:p + 16, h])
                        out[p:p + 16, h] = BR.e4m3(x[p:p + 16, h] / 2.0 ** e) * 2.0 ** e
                        if ex is not None:
                            ex[p:p + 16, h] = e
            self.k.append(K)
            self.v.append(V)
            self.ev.append(E)
        self.q = _randn((len(lens), nq, H, 128), 300 + seed, qscale)
        self.dev = dict(q=self.q.cuda(), page_table=_i32(self.table), lengths=_i32(lens))

    def run(self, **kw):
        return self.cache.attention(**{**self.dev, **kw})

    def check(self, out, lse, requests=None):
        for b in range(len(self.lens)) if requests is None else requests:
            o, l, mag, top = BR.attention(_np(self.q[b]), self.k[b], self.v[b], self.ev[b], self.scale)
            to, tl = BR.attention_tolerance(o, mag, top, l, self.lens[b])
            go, gl = _np(out[b]).reshape(o.shape), _np(lse[b]).reshape(l.shape)
            assert (np.abs(go - o) <= to).all(), (b, self.lens[b], np.abs(go - o).max(), (np.abs(go - o) - to).max())
            empty = np.isneginf(l)
            assert (np.isneginf(gl) == empty).all()
            assert (np.abs(gl[~empty] - l[~empty]) <= tl[~empty]).all(), (b, self.lens[b])


@pytest.mark.parametrize("H,Hkv,nq", [(1, 1, 1), (8, 8, 1), (32, 8, 1), (6, 2, 1), (8, 1, 1), (9, 1, 1), (16, 1, 1),
                                      (28, 2, 1), (17, 1, 1), (32, 1, 1), (24, 8, 4), (4, 4, 8), (12, 4, 3), (2, 1, 16),
                                      (28, 4, 3), (4, 4, 32)])
def test_attention_head_layouts(H, Hkv, nq):
    c = Case([1, 16, 31, 0, 47, 200, 33], H, Hkv, nq, seed=H + nq)
    c.check(*c.run())
    c.cache.sync()


@pytest.mark.parametrize("lens", [[1], [0], [2], [15], [17], [32], [5000], [4096, 1, 0, 777], [0, 0, 0], [33] * 40,
                                  [3] * 300, [1, 3000] * 5])
def test_attention_lengths(lens):
    c = Case(lens, 8, 2, 1, seed=len(lens))
    c.check(*c.run(), requests=range(0, len(lens), max(1, len(lens) // 10)))


@pytest.mark.parametrize("H,Hkv,nq", [(4, 1, 1), (48, 4, 1), (20, 1, 1), (60, 2, 1)])
def test_attention_cut_at_any_place(H, Hkv, nq):
    """Short requests, some without tokens: with more and more of them the cut of the line falls on every place of a group,
    its beginning and what counts for a piece's own cost included."""
    lens = np.random.default_rng(H).integers(0, 150, 420).tolist()
    c = Case(lens, H, Hkv, nq, seed=H)
    for B in list(range(1, 420, 23)) + [420]:
        out, lse = c.run(q=c.dev["q"][:B], page_table=c.dev["page_table"][:B], lengths=c.dev["lengths"][:B])
        c.check(out, lse, requests=range(B) if B == 420 else range(0, B, 5))
    c.cache.sync()


@pytest.mark.parametrize("H,Hkv,nq", [(32, 8, 1), (16, 1, 1), (32, 1, 1), (28, 4, 3)])
def test_attention_long(H, Hkv, nq):
    c = Case([30001], H, Hkv, nq, seed=3)
    c.check(*c.run())


@pytest.mark.parametrize("qscale,scale", [(0.0, 0.0), (1e-30, 0.0), (60.0, 0.0), (3e4, 1e-4), (1.0, 5.0), (1.0, 1e-8)])
def test_attention_score_ranges(qscale, scale):
    c = Case([500, 70], 8, 2, 1, seed=21, qscale=qscale, scale=scale)
    c.check(*c.run())


@pytest.mark.parametrize("H,nq,spread", [(4, 1, 8.0), (12, 1, 8.0), (20, 1, 8.0), (32, 1, 8.0), (7, 3, 8.0), (4, 1, 15.0)])
def test_attention_pages_of_very_different_scale(H, nq, spread):
    """Pages whose keys and values differ by many powers of two: the reference follows the products, and a page of small
    values with the largest scores counts as much as the definition says.  (Queries small enough that scores stay
    within some hundreds.)"""
    c = Case([400, 100], H, 1, nq, seed=61, qscale=2.0 ** -(2 * spread), spread=spread)
    c.check(*c.run())


@pytest.mark.parametrize("H", [4, 12, 20, 32])
def test_attention_zero_values_beside_others(H):
    """Whole pages of zero values (the smallest scale) that take nearly all of the weight, and requests of nothing else."""
    c = Case([200, 64], H, 1, 1, seed=63)
    n = 200
    k, v = _randn((n, 1, 128), 5), _randn((n, 1, 128), 6)
    d = torch.sign(_randn((128,), 7))
    k[32:64] = 0.3 * d
    v[32:64] = 0
    q = (d * 0.5).expand(1, 1, H, 128).to(BF16)
    t = np.arange(n)
    for b, (kb, vb) in enumerate(((k, v), (k[:64], torch.zeros_like(v[:64])))):
        m = len(kb)
        c.cache.append(kb.cuda(), vb.cuda(), _i32(c.table[b, t[:m] // 16] * 16 + t[:m] % 16))
        st = BR.Store(-(-m // 16), 1)
        st.append(_np(kb), _np(vb), t[:m])
        c.k[b], c.v[b] = st.gather(t[:m])
        c.ev[b] = np.repeat(st.exp[:, 1], 16, 0)[:m]
    c.q = q.repeat(2, 1, 1, 1)
    c.dev["q"] = c.q.cuda()
    out, lse = c.run()
    c.check(out, lse)
    assert (out[1] == 0).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("qscale", [2.0 ** 20, 2.0 ** 24, 2.0 ** 26, 1e15, 1e30])
@pytest.mark.parametrize("H,n", [(4, 5000), (12, 200), (20, 200), (32, 200)])
def test_attention_scores_beyond_the_significand(H, n, qscale):
    """Scores of 2^20 to 2^100 leave all weight to the row's largest: the output is that token's value (rounded to bf16,
    its weight 1 to 2^-11 by f16) and the lse its score.  The second largest has no weight where it is further below
    than both scores' errors, 64 log2 units more included."""
    c = Case([n], H, 1, 1, seed=17, qscale=qscale, spread=0.0)
    out, lse = c.run()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    q, k, v = _np(c.q[0, 0]), c.k[0][:, 0], c.v[0][:, 0]
    s = (k @ q.T) * c.scale
    err = 2.0 ** -23 * 14 * (np.abs(k) @ np.abs(q.T)).max(0) * c.scale
    order = np.argsort(s, axis=0)
    best, second = order[-1], order[-2]
    at = np.arange(H)
    clear = s[best, at] - s[second, at] > 2 * err + 64
    assert clear.sum() >= H // 2
    want = v[best]
    assert (np.abs(_np(out[0, 0]) - want) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(want) + 1e-12)[clear].all()
    gl = _np(lse[0, 0])
    assert (np.abs(gl - s[best, at]) <= err + 2.0 ** -21 * np.abs(gl))[clear].all()


def test_attention_nonfinite_tokens_stay_in_their_request():
    c = Case([40, 50, 60], 4, 2, 1, seed=41)
    nan = torch.full((1, 2, 128), float("nan"), dtype=BF16).cuda()
    c.cache.append(nan, nan, _i32([int(c.table[1, 1]) * 16 + 3]))                    # token 19 of request 1
    out, lse = c.run()
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    c.check(out, lse, requests=[0, 2])


@pytest.mark.parametrize("H,Hkv,nq,n,bad", [
    (2, 1, 4, 40, [(39, 0, 3)]), (8, 2, 3, 34, [(33, 1, 0), (32, 0, 127)]), (4, 1, 4, 18, [(17, 0, 85), (15, 0, 86)]),
    (4, 4, 2, 33, [(32, 2, 1), (31, 3, 2)]), (7, 1, 3, 700, [(699, 0, 6), (698, 0, 102)]),
    (2, 1, 16, 20, [(19, 0, 64), (6, 0, 0)]), (4, 2, 2, 2, [(1, 1, 3)])])
def test_attention_nonfinite_values_of_later_drafts(H, Hkv, nq, n, bad):
    """A drafted token whose values hold an infinity: the queries before it stay finite, those from it on get NaN in that
    element, and only there."""
    c = Case([n, 5 + nq], H, Hkv, nq, seed=71)
    for tok, h, el in sorted(bad):
        again = range(tok, n) if tok % 16 == 0 else [tok]           # a page that is started anew loses what it held
        for t in again:
            k, v = c.k[0][t:t + 1], c.v[0][t:t + 1].copy()          # stored values are fixed points of the format
            if t == tok:
                v[0, h, el] = np.inf
                c.v[0][t, h, el] = np.nan
            c.cache.append(torch.from_numpy(k).to(BF16).cuda(), torch.from_numpy(v).to(BF16).cuda(),
                           _i32([int(c.table[0, t // 16]) * 16 + t % 16]))
        if tok % 16 == 0:
            for g in range(Hkv):
                c.ev[0][tok:, g] = BR.need(c.v[0][tok:, g])
    out, lse = c.run()
    c.check(out, lse, requests=[1])
    v = c.v[0]
    o, l, mag, top = BR.attention(_np(c.q[0]), c.k[0], np.nan_to_num(v), c.ev[0], c.scale)
    to, tl = BR.attention_tolerance(o, mag, top, l, n)
    seen = np.zeros(o.shape, bool)
    for i in range(nq):
        seen[i] = np.repeat(np.isnan(v[:n - (nq - 1) + i]).any(0), H // Hkv, 0)
    assert seen.any() and not seen.all()
    go = _np(out[0])
    np.testing.assert_array_equal(np.isnan(go), seen)
    assert (np.abs(go - o) <= to)[~seen].all()
    assert (np.abs(_np(lse[0]) - l) <= tl).all()


@pytest.mark.parametrize("H,nq,n", [(4, 1, 300), (4, 1, 9000), (12, 1, 300), (32, 1, 300), (2, 3, 77), (6, 4, 300)])
def test_attention_rows_of_very_different_magnitude(H, nq, n):
    c = Case([n], H, 1, nq, seed=100 + H + nq)
    q = c.q.float()
    for i in range(nq):
        for h in range(H):
            q[0, i, h] *= (1.0, 1e15, 1.0, 1e-30, 1.0, 1e30)[(i + h) % 6]
    c.q = q.to(BF16)
    c.dev["q"] = c.q.cuda()
    out, lse = c.run()
    c.check(out, lse)
    if nq > 1:
        c.dev["q"][0, nq - 1] *= 2.0 ** 60
        out2, lse2 = c.run()
        assert torch.equal(out2[0, :nq - 1], out[0, :nq - 1]) and torch.equal(lse2[0, :nq - 1], lse[0, :nq - 1])


@pytest.mark.parametrize("H,n", [(4, 7), (4, 3000), (12, 100), (20, 100), (32, 100)])
def test_attention_nonfinite_queries_give_nan_in_their_row(H, n):
    c = Case([n], H, 1, 1, seed=81)
    bad = [0, 1, H - 1]
    for row, x in zip(bad, ("-inf", "inf", "nan")):
        c.q[0, 0, row, 77] = float(x)
    c.dev["q"] = c.q.cuda()
    out, lse = c.run()
    assert torch.isnan(out[0, 0, bad]).all() and torch.isnan(lse[0, 0, bad]).all()
    good = [r for r in range(H) if r not in bad]
    o, l, mag, top = BR.attention(_np(c.q[0])[:, good], c.k[0], c.v[0], c.ev[0], c.scale)
    to, tl = BR.attention_tolerance(o, mag, top, l, n)
    assert (np.abs(_np(out[0])[:, good] - o) <= to).all() and (np.abs(_np(lse[0])[:, good] - l) <= tl).all()


def test_attention_reports_bad_pages_and_lengths():
    from kv_cache_computation_gb300 import MacError
    c = Case([40, 50, 60], 4, 2, 1, seed=61)
    good = c.run()
    bad = c.dev["page_table"].clone()
    bad[1, 2] = c.cache.num_pages
    out = c.run(page_table=bad)
    with pytest.raises(MacError, match="page"):
        c.cache.sync()
    for b in (0, 2):
        assert torch.equal(out[0][b], good[0][b])
    for n in (-1, 16 * c.table.shape[1] + 1):
        ln = c.dev["lengths"].clone()
        ln[2] = n
        out = c.run(page_table=torch.clamp(c.dev["page_table"], min=0), lengths=ln)
        with pytest.raises(MacError, match="length"):
            c.cache.sync()
        c.check(*out, requests=[0, 1])
    c.check(*c.run())


def test_strided_table_given_outputs_and_three_dim_q():
    c = Case([70, 0, 9, 0], 8, 2, 1, seed=51)
    wide = torch.full((4, c.table.shape[1] + 5), -1, dtype=torch.int32).cuda()
    wide[:, :c.table.shape[1]] = c.dev["page_table"]
    buf = torch.full((6, 8, 128), 7.0, dtype=BF16).cuda()
    out, lse = c.cache.attention(c.dev["q"][:, 0].contiguous(), wide[:, :c.table.shape[1]], c.dev["lengths"], out=buf[:4])
    c.check(out, lse)
    assert (buf[4:] == 7.0).all() and (out[1] == 0).all() and torch.isneginf(lse[3]).all()
    out2, none = c.run(want_lse=False)
    assert none is None and torch.equal(out2[:, 0], out)


def test_reproducible_captured_and_on_another_stream():
    """Two runs agree bit for bit; captured appends and attention serve other tokens and lengths when replayed; another
    stream; a scratch shared by layers of different sizes."""
    from kv_cache_computation_gb300 import BlockKV
    c = Case([900, 40, 0, 300], 8, 2, 1, seed=81)
    a, b = c.run(), c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    s = torch.cuda.Stream()
    d = c.run(stream=s)
    s.synchronize()
    assert torch.equal(d[0], a[0])
    other = BlockKV(8, 2, num_pages=1500, max_batch=4)
    small = BlockKV(8, 2, num_pages=9, max_batch=4, share=other)
    ref, ref2 = BR.Store(1500, 2), BR.Store(9, 2)
    T = 2000
    k, v, slots = (torch.zeros((T, 2, 128), dtype=BF16).cuda(), torch.zeros((T, 2, 128), dtype=BF16).cuda(),
                   torch.full((T,), -1, dtype=torch.int32).cuda())
    lens, table = torch.zeros(1, dtype=torch.int32).cuda(), torch.arange(126, dtype=torch.int32).cuda()[None]
    q = _randn((1, 8, 128), 3).cuda()

    def step():
        other.append(k, v, slots)                           # more than the scan takes: through the marks
        small.append(k[:20], v[:20], torch.clamp(slots[:20], max=9 * 16 - 1))
        return other.attention(q, table, lens)
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out, lse = step()
    for seed in range(3):
        r = np.random.default_rng(seed)
        at = np.concatenate((r.permutation(16 * 126)[:1900], np.full(100, -1)))
        if seed == 0:
            at[:1900] = np.arange(1900)
        kk, vv = _sized((T, 2, 128), 30 + seed), _sized((T, 2, 128), 40 + seed)
        k.copy_(kk), v.copy_(vv), slots.copy_(torch.from_numpy(at.astype(np.int32))), lens.fill_(1900)
        graph.replay()
        torch.cuda.synchronize()
        ref.append(_np(kk), _np(vv), at)
        ref2.append(_np(kk[:20]), _np(vv[:20]), np.minimum(at[:20], 9 * 16 - 1))
        every = np.arange(1900)
        K, V = ref.gather(every)
        for got, want in zip(other.gather(_i32(every)), (K, V)):
            np.testing.assert_array_equal(_np(got), want)
        for got, want in zip(small.gather(_i32(np.arange(144))), ref2.gather(np.arange(144))):
            np.testing.assert_array_equal(_np(got), want)
        o, l, mag, top = BR.attention(_np(q), K, V, np.repeat(ref.exp[:, 1], 16, 0)[:1900], 1 / np.sqrt(128))
        to, tl = BR.attention_tolerance(o, mag, top, l, 1900)
        assert (np.abs(_np(out) - o) <= to).all() and (np.abs(_np(lse) - l) <= tl).all()
    other.sync()


def test_refusals_on_the_gpu():
    from kv_cache_computation_gb300 import BlockKV, MacError, QkvRotary, QuantKV
    c = Case([40, 50], 4, 2, 2, seed=71)
    q, t, n = c.dev["q"], c.dev["page_table"], c.dev["lengths"]
    with pytest.raises(MacError):                                   # more query tokens than the handle was made for
        c.cache.attention(torch.zeros(2, 3, 4, 128, dtype=BF16).cuda(), t, n)
    with pytest.raises(MacError):                                   # more requests
        c.cache.attention(q.repeat(2, 1, 1, 1), t.repeat(2, 1), n.repeat(2))
    for kw in (dict(q=q.float()), dict(q=q[..., :64]), dict(q=q.transpose(1, 2)), dict(page_table=t.long()),
               dict(page_table=t[:1]), dict(lengths=n.long()), dict(lengths=n.cpu()), dict(out=q.float())):
        with pytest.raises((TypeError, ValueError)):
            c.run(**kw)
    k, s = torch.zeros(3, 2, 128, dtype=BF16).cuda(), torch.zeros(3, dtype=torch.int32).cuda()
    for a in ((k, k[:2], s), (k, k, s[:2]), (k.float(), k, s), (k.cpu(), k, s), (k, k, s.long()), (k[..., :64], k, s)):
        with pytest.raises((TypeError, ValueError)):
            c.cache.append(*a)
    with pytest.raises(MacError):                                   # a token stride that is no multiple of 16 bytes
        c.cache.append(torch.zeros(3, 2 * 128 + 4, dtype=BF16).cuda()[:, :256], k, s)
    with pytest.raises(ValueError):
        c.cache.decode_step_qkv(QkvRotary(8, 2), torch.zeros(2, 8 * 128, dtype=BF16).cuda(), n, n, t, n)
    with pytest.raises(ValueError):                                 # too small a scratch to share
        BlockKV(4, 2, num_pages=50000, share=c.cache)
    with pytest.raises(ValueError):                                 # a scratch of the other kind
        BlockKV(4, 2, num_pages=1, share=QuantKV(4, 2, num_pages=1))
    c.cache.append(k[:0], k[:0], s[:0])                             # nothing to do is no error
    assert c.cache.gather(s[:0])[0].shape == (0, 2, 128)
    assert c.cache.attention(q[:0], t[:0], n[:0])[0].shape == (0, 2, 4, 128)
    c.check(*c.run())


# ---- the operators together ---------------------------------------------------------

@pytest.mark.parametrize("n_query,capture", [(1, False), (3, False), (1, True), (3, True)])
def test_serving_steps_together(n_query, capture):
    """Six steps of a padded batch (an idle slot; a request finishes and its slot is taken again; drafts rejected) from
    projections to outputs."""
    from kv_cache_computation_gb300 import BlockKV, QkvRotary, new_page_pool, page_step
    B, H, Hkv, P, N = 4, 8, 2, 8, 40
    rot = QkvRotary(H, Hkv, base=10000.0)
    cache = BlockKV(H, Hkv, num_pages=N, max_batch=B, max_query=n_query)
    ref = BR.Store(N, Hkv)
    ring, state = new_page_pool(N)
    lens, table = torch.zeros(B, dtype=torch.int32).cuda(), torch.zeros((B, P), dtype=torch.int32).cuda()
    w = _randn(128, 1).cuda(), _randn(128, 2).cuda()
    s = page_step(lens, _i32([45, 16, 3, 0]), table, ring, state, max_tokens=80, in_place=True)
    x = _randn((80, (H + 2 * Hkv) * 128), 3).cuda()
    _, _, k, v = rot(x, s.positions, *w)
    cache.append(k, v, s.slots)                          # the padding's slots are -1
    ref.append(_np(k), _np(v), s.slots.cpu().numpy())
    qkv = torch.zeros((B * n_query, (H + 2 * Hkv) * 128), dtype=BF16).cuda()
    new, rejected = torch.zeros(B, dtype=torch.int32).cuda(), torch.zeros(B, dtype=torch.int32).cuda()

    def step():
        st = page_step(lens, new, table, ring, state, max_tokens=B * n_query, in_place=True, rejected=rejected)
        return st, cache.decode_step_qkv(rot, qkv, st.positions, st.slots, table, st.lengths, *w, starts=st.starts)
    run = step
    if capture:
        step()                                           # no request has a new token: nothing changes
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = step()

        def run():
            graph.replay()
            return res
    for t in range(6):
        new.copy_(_i32([n_query, n_query, -1 if t == 2 else n_query, 0 if t < 4 else n_query]))
        rejected.copy_(_i32([n_query - 1 if t else 0, 0, 0, 0]))
        qkv.copy_(_randn(tuple(qkv.shape), 50 + t, 1.0 + t))
        st, (out, lse) = run()
        cache.sync()
        assert int(st.status) == 0
        first = st.starts.cpu().numpy()
        for b in range(B):
            rows = slice(b * n_query, (b + 1) * n_query)
            n = int(st.lengths[b])
            if first[b + 1] - first[b] != n_query:
                assert (out[b] == 0).all() and torch.isneginf(lse[b]).all()
                continue
            at = slice(int(first[b]), int(first[b + 1]))
            _, q, kn, vn = rot(qkv[rows], st.positions[at], *w)
            ref.append(_np(kn), _np(vn), st.slots[at].cpu().numpy())
        for b in range(B):                               # every request's tokens are stored before any attends
            if first[b + 1] - first[b] != n_query:
                continue
            n, rows, at = int(st.lengths[b]), slice(b * n_query, (b + 1) * n_query), slice(int(first[b]), int(first[b + 1]))
            _, q, _, _ = rot(qkv[rows], st.positions[at], *w)
            slots = table[b].cpu().numpy()[np.arange(n) // 16] * 16 + np.arange(n) % 16
            K, V = ref.gather(slots)
            o, l, mag, top = BR.attention(_np(q), K, V, ref.exp[slots // 16, 1], 1 / np.sqrt(128))
            to, tl = BR.attention_tolerance(o, mag, top, l, n)
            assert (np.abs(_np(out[b]) - o) <= to).all() and (np.abs(_np(lse[b]) - l) <= tl).all()

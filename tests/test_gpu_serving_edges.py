"""Edges of the operators around the decode step on the GPU: non-finite values
beside what they must not reach, slots without new tokens, rejected drafts,
refused releases, queries of very different magnitude, shared scratch."""
import numpy as np
import pytest
import torch

import page_reference as PR
import serving_reference as R
from test_gpu_serving_ops import BF16, Case, _check_rope, _randn

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


# ---- norm and rotation -------------------------------------------------------

@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("T,rotary,inter", [(3, 0, False), (3, 64, False), (3, 64, True), (3, 8, True), (130, 104, False),
                                            (310, 96, False), (310, 96, True), (310, 40, True), (310, 0, False)])
def test_rope_leaves_unrotated_elements_alone(T, rotary, inter, norm):
    """An infinity or NaN behind the rotated elements stays where it is: every other element of that part is what the
    definition gives, and without a norm nothing of the row's rotated part changes either."""
    from kv_cache_computation_gb300 import QkvRotary
    H, Hkv = 3, 1
    x = _randn((T, (H + 2 * Hkv) * 128), 1).view(T, H + 2 * Hkv, 128)
    # token t, head h: one element behind the rotated ones
    for t in range(T):
        for h in range(H + Hkv):
            at = rotary + (7 * t + 31 * h) % (128 - rotary)
            x[t, h, at] = (float("inf"), float("-inf"), float("nan"), 2.0)[(t + h) % 4]
    pos = torch.arange(T, dtype=torch.int32) + 5
    w = (_randn(128, 2).abs() + 0.5).to(BF16) if norm else None
    dw = None if w is None else w.cuda()
    rot = QkvRotary(H, Hkv, rotary_dim=rotary, base=10000.0, interleaved=inter)
    q_pre, q_post, k, _ = rot(x.reshape(T, -1).cuda(), pos.cuda(), dw, dw)
    for got, src in ((q_post, x[:, :H]), (k, x[:, H:H + Hkv]), (q_pre, x[:, :H])):
        y, r = R.norm_rope(src, w, pos, rotary, 10000.0, inter, 1e-6)
        want = y if got is q_pre else r
        g = got.double().cpu()
        for test in (torch.isnan, torch.isposinf, torch.isneginf):
            assert torch.equal(test(g), test(want)), test
        fine = torch.isfinite(want)
        mag = torch.where(torch.isfinite(y), y.abs(), 0.0)
        half = rotary // 2
        if half and got is not q_pre:
            a, b = ((slice(0, rotary, 2), slice(1, rotary, 2)) if inter else (slice(0, half), slice(half, rotary)))
            mag[..., a] = mag[..., b] = mag[..., a] + mag[..., b]
        _check_rope(torch.where(fine, g, 0.0), torch.where(fine, want, 0.0), "finite elements", mag)
        if not norm:
            same = torch.isnan(src[..., rotary:]) | (got.cpu()[..., rotary:] == src[..., rotary:])
            assert same.all()


# ---- attention over the store ------------------------------------------------

@pytest.mark.parametrize("qscale", [2.0 ** 20, 2.0 ** 22, 2.0 ** 23, 2.0 ** 24, 2.0 ** 25, 2.0 ** 26, 2.0 ** 28, 1e15, 1e30])
@pytest.mark.parametrize("H,n", [(4, 5000), (12, 200), (20, 200), (32, 200)])
def test_attention_scores_beyond_the_significand(H, n, qscale):
    """Scores of 2^20 to 2^100 leave all weight to the row's largest: the output is that token's value (rounded to
    bf16, its weight 1 to 2^-11 by f16) and the lse its score (18 * 2^-23 of sum |q k| as derived for the smaller
    ones).  The second largest has no weight where it is further below than both scores' errors, 64 log2 units
    more included."""
    c = Case([n], H, 1, 1, seed=17, qscale=qscale)
    out, lse = c.run()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    q, k, v = c.q[0, 0].double().numpy(), c.k[0][:, 0], c.v[0][:, 0]
    s = (k @ q.T) * c.scale
    err = 18 * 2.0 ** -23 * (np.abs(k) @ np.abs(q.T)).max(0) * c.scale
    order = np.argsort(s, axis=0)
    best, second = order[-1], order[-2]
    at = np.arange(H)
    clear = s[best, at] - s[second, at] > 2 * err + 64
    assert clear.sum() >= H // 2
    go, gl = out[0, 0].double().cpu().numpy(), lse[0, 0].double().cpu().numpy()
    want = v[best]
    assert (np.abs(go - want) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(want) + 1e-12)[clear].all()
    assert (np.abs(gl - s[best, at]) <= err + 2.0 ** -21 * np.abs(gl))[clear].all()


@pytest.mark.parametrize("H,nq,n", [(4, 1, 300), (4, 1, 9000), (12, 1, 300), (20, 1, 300), (32, 1, 300), (32, 1, 9000),
                                    (2, 3, 77), (6, 4, 300)])
def test_attention_rows_of_very_different_magnitude(H, nq, n):
    """Heads and drafted tokens of one group from 1e-30 to 1e30: a row's result does not depend on the others' size, and
    a later draft's query does not change an earlier one's result by a bit."""
    c = Case([n], H, 1, nq, seed=100 + H + nq)
    q = c.q.float()
    for i in range(nq):
        for h in range(H):
            # at most 1e30 against the store's values of about 1; every other row keeps its ordinary size
            q[0, i, h] *= (1.0, 1e15, 1.0, 1e-30, 1.0, 1e30)[(i + h) % 6]
    c.q = q.to(BF16)
    c.dev["q"] = c.q.cuda()
    out, lse = c.run()
    c.check(out, lse)
    if nq > 1:
        c.dev["q"][0, nq - 1] *= 2.0 ** 60
        out2, lse2 = c.run()
        assert torch.equal(out2[0, :nq - 1], out[0, :nq - 1]) and torch.equal(lse2[0, :nq - 1], lse[0, :nq - 1])


# ---- a step from its projection --------------------------------------------------

@pytest.mark.parametrize("what", ["queries", "requests", "no_token", "columns", "overlap", "lengths_type", "lengths_shape",
                                  "table_type"])
def test_a_refused_step_stores_nothing(what):
    """Every argument that the step's attention refuses is refused before its append."""
    from kv_cache_computation_gb300 import MacError, QkvRotary, QuantKV
    H, Hkv, B, nq = 4, 2, 2, 1
    cache = QuantKV(H, Hkv, num_pages=4, max_batch=B, max_query=2)
    rot = QkvRotary(H, Hkv)
    table, lens = _i32([[0, 1], [2, 3]]), _i32([1, 1])
    if what == "queries":
        nq = 3
    elif what == "requests":
        B, table, lens = 3, _i32([[0, 1], [2, 3], [1, 0]]), _i32([1, 1, 1])
    elif what == "no_token":
        nq = 0
    elif what == "columns":
        table = table[:, :0]
    elif what == "overlap":
        table = table[:1].expand(2, 2)
    elif what == "lengths_type":
        lens = lens.long()
    elif what == "lengths_shape":
        lens = lens[:, None]
    elif what == "table_type":
        table = table.long()
    qkv = _randn((B * nq, (H + 2 * Hkv) * 128), 3).cuda()
    slots = torch.arange(B * nq, dtype=torch.int32).cuda() * 16
    with pytest.raises((TypeError, ValueError, MacError)):
        cache.decode_step_qkv(rot, qkv, torch.zeros_like(slots), slots, table, lens)
    k, v = cache.gather(torch.arange(64, dtype=torch.int32).cuda())
    assert (k == 0).all() and (v == 0).all()
    cache.sync()


# ---- errors and shared scratch -----------------------------------------------------

def test_a_refusal_carries_no_earlier_text():
    from kv_cache_computation_gb300 import MacError, QuantKV
    a = QuantKV(4, 2, num_pages=2)
    z, bad = torch.zeros((1, 2, 128), dtype=BF16).cuda(), _i32([99])
    wide = torch.zeros((2, 2 * 128 + 4), dtype=BF16).cuda()
    for call in (lambda: a.attention(torch.zeros((2, 4, 128), dtype=BF16).cuda(), _i32([[0], [0]]), _i32([0, 0])),
                 lambda: a.append(wide[:, :256], wide[:, :256], _i32([0, 1]))):
        a.append(z, z, bad)
        with pytest.raises(MacError, match="slot"):
            a.sync()
        with pytest.raises(MacError) as e:
            call()
        assert "slot" not in str(e.value)


def test_a_shared_scratch_keeps_unread_reports():
    """A layer made on another's scratch does not clear what that one has yet to report; a scratch whose handles are gone
    starts without reports."""
    from kv_cache_computation_gb300 import MacError, QuantKV
    a = QuantKV(4, 2, num_pages=2)
    z = torch.zeros((1, 2, 128), dtype=BF16).cuda()
    a.append(z, z, _i32([99]))
    b = QuantKV(8, 2, num_pages=3, max_query=2, share=a)
    with pytest.raises(MacError, match="slot"):
        a.sync()
    b.sync()
    b.append(z, z, _i32([99]))
    with pytest.raises(MacError, match="slot"):             # one word: whoever asks first
        a.sync()
    b.sync()
    b.append(z, z, _i32([99]))
    a.close()
    with pytest.raises(MacError, match="slot"):             # the owner's end does not end the sharing
        b.sync()
    b.append(z, z, _i32([99]))
    torch.cuda.synchronize()
    scratch = b._scratch
    b.close()
    c = QuantKV(4, 2, num_pages=2, share=type("Q", (), dict(device=scratch.device, _scratch=scratch))())
    c.sync()


# ---- page bookkeeping ----------------------------------------------------------------

NAMES = ("lengths", "free_state", "starts", "positions", "slots", "table", "ring", "status", "unreleased")


def _step(lens, new, table, ring, state, T, in_place, **kw):
    """page_step as numpy arrays, in the order of the reference's."""
    from kv_cache_computation_gb300 import page_step
    ln, tab, rg, st = _i32(lens), _i32(table), _i32(ring), _i32(state)
    s = page_step(ln, _i32(new), tab, rg, st, max_tokens=T, in_place=in_place, **kw)
    assert len(s) == 6 and (s.unreleased is not None) == in_place
    out = [s.lengths, s.free_state, s.starts, s.positions, s.slots, tab, rg, s.status]
    return [x.cpu().numpy().astype(np.int64) for x in out + ([s.unreleased] if in_place else [])]


def _agree(got, want):
    for a, b, name in zip(got, want, NAMES):
        np.testing.assert_array_equal(a, b, err_msg=name)


@pytest.mark.parametrize("T", [10, 1500])
@pytest.mark.parametrize("state,bits", [([5, 8], 16), ([0, 7], 16), ([8, 3], 20), ([-1, 3], 20), ([0, 9], 20), ([2, 4], 16), ([2, 3], 0)])
def test_refused_release_in_place_keeps_what_it_holds(state, bits, T):
    """Finished requests of five pages, for which a ring of eight that holds more than three has no room: their lengths come
    back beside the zeros."""
    lens, new = [20, 5, 0, 33], [-1, 1, -3, -2]
    table = [[1, 2, 0], [3, 0, 0], [0, 0, 0], [4, 5, 6]]
    for in_place in (False, True):
        want = PR.step(lens, new, table, np.arange(8), state, T)
        got = _step(lens, new, table, np.arange(8), state, T, in_place)
        _agree(got, want)
        assert int(got[7][0]) & ~1 == bits
        if in_place:
            assert list(got[8]) == ([20, 0, 0, 33] if bits else [0] * 4)


@pytest.mark.parametrize("T", [12, 3000])
@pytest.mark.parametrize("where", [[(3, 0)], [(3, 2), (0, 1)], [(3, 1), (5, 0), (5, 3)], [(5, 3)]])
def test_ids_outside_the_pool_stay_out_of_the_ring(where, T):
    """A finished request that holds an id outside the pool frees nothing; the others' pages follow one another in the
    ring, and what the ring counts as free is of the pool."""
    lens = [40, 3, 30, 40, 16, 64]
    table = np.array([[0, 1, 2, -1], [3, -1, -1, -1], [4, 5, -1, -1], [6, 7, 8, -1], [9, -1, -1, -1], [10, 11, 12, 13]])
    ring = np.full(16, -9)
    ring[[15, 0]] = 14, 15
    new = [-1, 1, -2, -1, 1, -1]
    for k, (b, c) in enumerate(where):
        table[b, c] = (16, -1, 2 ** 31 - 1)[k]
    for in_place in (False, True):
        want = PR.step(lens, new, table, ring, [15, 2], T)
        got = _step(lens, new, table, ring, [15, 2], T, in_place)
        _agree(got, want)
        assert int(got[7][0]) == 4
        free = [int(got[6][(got[1][0] + i) % 16]) for i in range(got[1][1])]
        assert all(0 <= p < 16 for p in free) and len(set(free)) == len(free)
        if in_place:
            assert [b for b in range(6) if got[8][b]] == sorted({b for b, _ in where})


def test_long_releases():
    """Requests of many thousand pages finish beside decoding ones, one with a bad id."""
    r = np.random.default_rng(8)
    N, P = 40000, 8200
    lens = np.array([131072, 5, 100000, 64, 131072])
    perm, table, at = r.permutation(N), np.full((5, P), -1, np.int64), 0
    for b in range(5):
        table[b, :-(-lens[b] // 16)] = perm[at:at - (-lens[b] // 16)]
        at += -(-lens[b] // 16)
    ring = np.full(N, -1)
    ring[(N - 3 + np.arange(N - at)) % N] = perm[at:]
    for bad in (False, True):
        if bad:
            table[2, 6000] = N
        for T in (5, 2000):              # the table is wide enough for a cluster in both
            _agree(_step(lens, [-1, 1, -1, 1, -1], table, ring, [N - 3, N - at], T, True),
                   PR.step(lens, [-1, 1, -1, 1, -1], table, ring, [N - 3, N - at], T))


@pytest.mark.parametrize("B,P", [(1, 4096), (1, 4097), (64, 64), (63, 66), (1024, 4), (1024, 5)])
def test_page_step_on_both_sides_of_the_cluster(B, P):
    """A decode step in which a third of the requests finish, with as many table entries as one block takes and with
    more."""
    r = np.random.default_rng(B + P)
    lens = r.integers(0, 16 * P + 1, B)
    N = int(((lens + 15) // 16).sum()) + B
    perm, table, at = r.permutation(N), np.full((B, P), -1, np.int64), 0
    for b in range(B):
        used = -(-int(lens[b]) // 16)
        table[b, :used] = perm[at:at + used]
        at += used
    ring = np.full(N, -1)
    head = int(r.integers(0, N))
    ring[(head + np.arange(N - at)) % N] = perm[at:]
    new = np.where(r.random(B) < 0.34, -1, 1)
    new[0] = -1
    _agree(_step(lens, new, table, ring, [head, N - at], B, True), PR.step(lens, new, table, ring, [head, N - at], B))


@pytest.mark.parametrize("B,P,top,T,seed", [(1, 4, 3, 4, 0), (7, 12, 20, 200, 1), (40, 6, 70, 3000, 2), (300, 20, 25, 8000, 3)])
def test_rejected_drafts_over_many_steps(B, P, top, T, seed):
    """Requests that draft, take some of it back, come and go, also where the pool or a row is too small: every step is the
    definition's, and no page is ever lost or held twice."""
    from kv_cache_computation_gb300 import new_page_pool, page_step
    r = np.random.default_rng(seed)
    N = B * P // 2 + 1
    ring, state = new_page_pool(N)
    lens = torch.zeros(B, dtype=torch.int32).cuda()
    table = torch.zeros((B, P), dtype=torch.int32).cuda()
    ref = [np.zeros(B, np.int64), [0, N], None, None, None, table.cpu().numpy(), ring.cpu().numpy()]
    bits, freed = 0, 0
    for t in range(50):
        new = np.where(r.random(B) < 0.1, -1, r.integers(0, top + 1, B))
        rejected = np.minimum(r.integers(0, top + 1, B) * (r.random(B) < 0.6), ref[0])
        want = PR.step(ref[0], new, ref[5], ref[6], [int(x) for x in ref[1]], T, rejected)
        s = page_step(lens, _i32(new), table, ring, state, max_tokens=T, rejected=_i32(rejected), in_place=t % 2 == 1)
        lens, state = s.lengths, s.free_state
        _agree([x.cpu().numpy() for x in (lens, state, s.starts, s.positions, s.slots, table, ring, s.status)], want[:8])
        freed += sum(PR.pages(int(want[0][b])) < PR.pages(int(ref[0][b])) for b in range(B) if new[b] >= 0)
        bits |= int(want[7][0])
        ref = want
        held = [int(p) for b in range(B) for p in want[5][b, :PR.pages(int(want[0][b]))]]
        free = [int(want[6][(int(want[1][0]) + i) % N]) for i in range(int(want[1][1]))]
        assert sorted(held + free) == list(range(N))
    assert freed and (B == 1 or bits & 3)


def test_rejected_drafts_across_a_page_edge():
    """15 tokens, 3 drafts of which 2 are rejected, one more token: the page that the drafts opened is not lost."""
    from kv_cache_computation_gb300 import new_page_pool, page_step
    ring, state = new_page_pool(8)
    table = torch.zeros((1, 8), dtype=torch.int32).cuda()
    s = page_step(_i32([0]), _i32([15]), table, ring, state, max_tokens=32)
    s = page_step(s.lengths, _i32([3]), table, ring, s.free_state, max_tokens=32)
    s = page_step(s.lengths, _i32([1]), table, ring, s.free_state, max_tokens=32, rejected=_i32([2]))
    assert int(s.lengths) == 17 and int(s.positions[0]) == 16 and int(s.slots[0]) == int(table[0, 1]) * 16
    assert int(s.free_state[1]) == 6
    s = page_step(s.lengths, _i32([0]), table, ring, s.free_state, max_tokens=32, rejected=_i32([17]))
    assert int(s.lengths) == 0 and int(s.free_state[1]) == 8 and int(s.status) == 0


@pytest.mark.parametrize("what,bit", [("more", 4), ("negative", 4), ("ring", 16), ("state", 16), ("page", 4), ("finished", 0),
                                      ("dry", 1), ("row", 2), ("tokens", 8)])
def test_rejected_draft_denials(what, bit):
    lens, new, rejected = [40, 33, 20, 16], [1, 5, 30, 2], [20, 2, 3, 1]
    table = [[0, 1, 2, -1], [3, 4, 5, -1], [6, 7, -1, -1], [8, -1, -1, -1]]
    ring, state, T = np.array([9, 10, 11, 12, 13, 14, 15, -1, -1, -1, -1, -1, -1, -1, -1, -1]), [0, 7], 60
    if what == "more":
        rejected[1] = 34
    elif what == "negative":
        rejected[0] = -1
    elif what == "ring":
        state = [0, 16]
    elif what == "state":
        state = [16, 3]
    elif what == "page":
        table[0][2] = -4
    elif what == "finished":
        new[0], rejected[0] = -1, 999
    elif what == "dry":
        state = [0, 1]
    elif what == "row":
        new[2] = 48
    elif what == "tokens":
        T = 20
    for in_place in (False, True):
        want = PR.step(lens, new, table, ring, state, T, rejected)
        assert int(want[7][0]) & bit == bit and (bit or int(want[7][0]) == 0)
        _agree(_step(lens, new, table, ring, state, T, in_place, rejected=_i32(rejected)), want)


# ---- padded batches through the whole step ---------------------------------------------

class Loop:
    """A decode loop of B slots: lengths, table and pool on the GPU, and what each request holds in float64."""

    def __init__(self, B, nq, pages=60, H=4, Hkv=2, cols=8):
        from kv_cache_computation_gb300 import QkvRotary, QuantKV, new_page_pool
        self.B, self.nq, self.H, self.Hkv = B, nq, H, Hkv
        self.rot = QkvRotary(H, Hkv, base=10000.0)
        self.cache = QuantKV(H, Hkv, num_pages=pages, max_batch=B, max_query=nq)
        self.ring, self.state = new_page_pool(pages)
        self.lens = torch.zeros(B, dtype=torch.int32).cuda()
        self.table = torch.full((B, cols), -1, dtype=torch.int32).cuda()
        self.new = torch.zeros(B, dtype=torch.int32).cuda()
        self.rejected = torch.zeros(B, dtype=torch.int32).cuda()
        self.qkv = torch.zeros((B * nq, (H + 2 * Hkv) * 128), dtype=BF16).cuda()
        self.held = [[] for _ in range(B)]              # (k, v) of each token, as the store holds them

    def prefill(self, counts, seed=1):
        from kv_cache_computation_gb300 import page_step
        T = sum(counts)
        s = page_step(self.lens, _i32(counts), self.table, self.ring, self.state, max_tokens=T, in_place=True)
        assert int(s.status) == 0
        _, _, k, v = self.rot(_randn((T, self.qkv.shape[1]), seed).cuda(), s.positions)
        self.cache.append(k, v, s.slots)
        at = 0
        for b, n in enumerate(counts):
            self._note(b, k[at:at + n], v[at:at + n])
            at += n

    def _note(self, b, k, v):
        self.held[b] += list(zip(R.stored(k.double().cpu().numpy()), R.stored(v.double().cpu().numpy())))

    def step(self, max_tokens=None, with_starts=True):
        from kv_cache_computation_gb300 import page_step
        T = self.B * self.nq if max_tokens is None else max_tokens
        st = page_step(self.lens, self.new, self.table, self.ring, self.state, max_tokens=T, in_place=True,
                       rejected=self.rejected)
        return st, self.cache.decode_step_qkv(self.rot, self.qkv, st.positions, st.slots, self.table, st.lengths,
                                              starts=st.starts if with_starts else None)

    def check(self, out, lse, served):
        """The requests in `served` got their nq tokens: their outputs are those of all their tokens; the others give 0."""
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        for b in range(self.B):
            if b not in served:
                assert (out[b] == 0).all() and np.isneginf(lse[b]).all(), b
                continue
            rows = self.qkv[b * self.nq:(b + 1) * self.nq]
            pos = len(self.held[b]) + torch.arange(self.nq, dtype=torch.int32).cuda()
            _, q, k, v = self.rot(rows, pos)
            self._note(b, k, v)
            K, V = (np.stack(x) for x in zip(*self.held[b]))
            o, l, mag, top = R.attention(q.double().cpu().numpy(), K, V, 1 / np.sqrt(128))
            to, tl = R.attention_tolerance(o, mag, top, l, len(K))
            assert (np.abs(out[b] - o) <= to).all() and (np.abs(lse[b] - l) <= tl).all(), b
        self.check_store()

    def check_store(self):
        """Every request's tokens stand where its table says, and nothing else was written over them."""
        table = self.table.cpu().numpy()
        for b, held in enumerate(self.held):
            if held:
                t = np.arange(len(held))
                k, v = self.cache.gather(_i32(table[b, t // 16] * 16 + t % 16))
                for got, want in zip((k, v), zip(*held)):
                    np.testing.assert_array_equal(got.double().cpu().numpy(), np.stack(want), err_msg=f"request {b}")


@pytest.mark.parametrize("capture", [False, True])
@pytest.mark.parametrize("nq", [1, 3])
def test_idle_and_finished_requests_in_a_decode_batch(nq, capture):
    """A batch of five with an idle slot, a request that has no new token and one that finishes, anywhere in the batch:
    every other request gets its own positions and slots, eager and captured."""
    lp = Loop(5, nq)
    lp.prefill([14, 7, 0, 33, 16])
    if capture:
        keep = [t.clone() for t in (lp.lens, lp.table, lp.ring, lp.state)]
        lp.step()                                           # no new tokens: nothing is stored
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = lp.step()
        for t, o in zip((lp.lens, lp.table, lp.ring, lp.state), keep):
            t.copy_(o)
    # per step: who decodes; -1 finishes
    for t, new in enumerate(([1, 1, 0, 1, 1], [1, -1, 0, 1, 1], [0, 1, 0, -1, 1], [1, 0, 1, 0, 0], [0, 0, 0, 0, 0], [1] * 5,
                             [-1] * 5, [0, 0, 1, 1, 0])):
        lp.new.copy_(_i32(new) * torch.where(_i32(new) > 0, nq, 1))
        lp.qkv.copy_(_randn(tuple(lp.qkv.shape), 40 + t))
        if capture:
            graph.replay()
            st, (out, lse) = res
        else:
            st, (out, lse) = lp.step()
        lp.cache.sync()
        assert int(st.status) == 0
        for b, n in enumerate(new):
            if n < 0:
                lp.held[b] = []
        lp.check(out, lse, [b for b, n in enumerate(new) if n > 0])


def test_denied_requests_in_a_decode_batch():
    """Requests that get no page are left out (their own token is not stored), the others are served; the step's status
    says so, and nothing is left to report."""
    lp = Loop(4, 1, pages=5)
    lp.prefill([16, 3, 32, 15])                             # the pool is empty: 0 and 2 need a page
    lp.new.fill_(1)
    lp.qkv.copy_(_randn(tuple(lp.qkv.shape), 9))
    st, (out, lse) = lp.step()
    lp.cache.sync()
    assert int(st.status) == 1 and st.lengths.tolist() == [16, 4, 32, 16]
    lp.check(out, lse, [1, 3])


@pytest.mark.parametrize("what", ["no_starts", "other_count", "other_table", "late", "garbage"])
def test_tokens_that_are_not_their_rows_are_refused_and_reported(what):
    """A step whose packed tokens cannot be its rows stores nothing under another request's slots: such requests are left
    out and sync reports it."""
    from kv_cache_computation_gb300 import MacError
    lp = Loop(4, 2)
    lp.prefill([5, 17, 30, 9])
    lp.qkv.copy_(_randn(tuple(lp.qkv.shape), 5))
    new, served, T, starts = [2, 2, 2, 2], [0, 1, 2, 3], 8, None
    from kv_cache_computation_gb300 import page_step
    if what == "no_starts":
        new, served = [2, 0, 2, 2], [0]
    elif what == "other_count":
        new, served = [2, 1, 2, 3], [0, 2]
    elif what == "other_table":
        served = [0, 3]
    elif what == "late":
        T, served = 7, [0, 1, 2]
    elif what == "garbage":
        # request 1 is given the packed tokens 0 and 1, which are request 0's
        starts, served = _i32([-2 ** 31, 0, 2, 2 ** 31 - 1, -5]), []
    lp.new.copy_(_i32(new))
    st = page_step(lp.lens, lp.new, lp.table, lp.ring, lp.state, max_tokens=T, in_place=True)
    starts = st.starts if starts is None else starts
    table = lp.table[[0, 2, 1, 3]] if what == "other_table" else lp.table
    if what == "no_starts":
        out, lse = lp.cache.decode_step_qkv(lp.rot, lp.qkv, st.positions, st.slots, table, st.lengths)
    else:
        out, lse = lp.cache.decode_step_qkv(lp.rot, lp.qkv, st.positions, st.slots, table, st.lengths, starts=starts)
    with pytest.raises(MacError, match="not its rows"):
        lp.cache.sync()
    lp.check(out, lse, served)
    lp.cache.sync()


def test_step_without_starts_serves_full_batches():
    lp = Loop(3, 2)
    lp.prefill([5, 17, 30])
    lp.new.fill_(2)
    for t in range(3):
        lp.qkv.copy_(_randn(tuple(lp.qkv.shape), 5 + t))
        st, (out, lse) = lp.step(with_starts=False)
        lp.cache.sync()
        lp.check(out, lse, [0, 1, 2])


def test_step_on_another_stream_and_refusals():
    lp = Loop(3, 1)
    lp.prefill([5, 17, 30])
    lp.new.fill_(1)
    lp.qkv.copy_(_randn(tuple(lp.qkv.shape), 5))
    from kv_cache_computation_gb300 import page_step
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    st = page_step(lp.lens, lp.new, lp.table, lp.ring, lp.state, max_tokens=3, in_place=True, stream=s)
    args = (lp.rot, lp.qkv, st.positions, st.slots, lp.table, st.lengths)
    for kw in (dict(starts=st.starts[:3]), dict(starts=st.starts.long()), dict(starts=st.starts.cpu())):
        with pytest.raises((TypeError, ValueError)):
            lp.cache.decode_step_qkv(*args, **kw)
    for a in ((lp.rot, lp.qkv, st.positions[:2], st.slots[:2], lp.table, st.lengths),
              (lp.rot, lp.qkv, st.positions, st.slots[:2], lp.table, st.lengths),
              (lp.rot, lp.qkv, st.positions.long(), st.slots, lp.table, st.lengths)):
        with pytest.raises((TypeError, ValueError)):
            lp.cache.decode_step_qkv(*a)
    out, lse = lp.cache.decode_step_qkv(*args, starts=st.starts, stream=s)
    s.synchronize()
    lp.cache.sync()
    lp.check(out, lse, [0, 1, 2])


def test_positions_and_slots_of_different_lengths():
    """Only the new tokens' entries are read: either array may be longer."""
    from kv_cache_computation_gb300 import page_step
    lp = Loop(3, 1)
    lp.prefill([5, 17, 30])
    lp.new.fill_(1)
    for t, kw in enumerate((dict(), dict(), dict(starts=True), dict(starts=True))):
        lp.qkv.copy_(_randn(tuple(lp.qkv.shape), 5 + t))
        st = page_step(lp.lens, lp.new, lp.table, lp.ring, lp.state, max_tokens=8, in_place=True)
        pos, slots = (st.positions[:3], st.slots) if t % 2 else (st.positions, st.slots[:3].clone())
        out, lse = lp.cache.decode_step_qkv(lp.rot, lp.qkv, pos, slots, lp.table, st.lengths,
                                            starts=st.starts if kw else None)
        lp.cache.sync()
        lp.check(out, lse, [0, 1, 2])


@pytest.mark.parametrize("capture", [False, True])
def test_drafted_steps_with_rejections_in_a_decode_batch(capture):
    """Four slots that verify three drafted tokens a step and take back up to all of them, one idle, one that finishes and
    starts again: every output is that of the tokens that were kept, and no page is lost."""
    lp = Loop(4, 3, pages=20, cols=10)
    lp.prefill([14, 47, 0, 30])
    if capture:
        keep = [t.clone() for t in (lp.lens, lp.table, lp.ring, lp.state)]
        lp.step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = lp.step()
        for t, o in zip((lp.lens, lp.table, lp.ring, lp.state), keep):
            t.copy_(o)
    r, last = np.random.default_rng(4), [0] * 4
    for t in range(24):
        new = [3, 3 if t % 4 else 0, 3 if t > 5 else 0, -1 if t == 12 else 3]
        back = [int(r.integers(0, n + 1)) if new[b] >= 0 else 0 for b, n in enumerate(last)]
        for b in range(4):
            lp.held[b] = [] if new[b] < 0 else lp.held[b][:len(lp.held[b]) - back[b]]
        lp.new.copy_(_i32(new))
        lp.rejected.copy_(_i32(back))
        lp.qkv.copy_(_randn(tuple(lp.qkv.shape), 70 + t))
        if capture:
            graph.replay()
            st, (out, lse) = res
        else:
            st, (out, lse) = lp.step()
        lp.cache.sync()
        assert int(st.status) == 0
        lp.check(out, lse, [b for b in range(4) if new[b] > 0])
        last = [max(n, 0) for n in new]
        assert st.lengths.tolist() == [len(h) for h in lp.held]
        N, table, ring = 20, lp.table.cpu().numpy(), lp.ring.cpu().numpy()
        head, count = lp.state.tolist()
        held = [int(p) for b in range(4) for p in table[b, :PR.pages(len(lp.held[b]))]]
        assert sorted(held + [int(ring[(head + i) % N]) for i in range(count)]) == list(range(N))

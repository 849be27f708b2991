"""The operators around the decode step on the GPU, against 64-bit restatements
of their definitions (serving_reference.py).  Tolerances are derived there and
in the comments; integers and stored 4-bit values are compared exactly."""
import numpy as np
import pytest
import torch

import serving_reference as R

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF16 = torch.bfloat16


def _randn(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(BF16)


# ---- norm and rotation -------------------------------------------------------

def _check_rope(got, y, what, mag):
    """bf16 output: 2^-8 of the value; fp32 arithmetic: the mean of squares, the inverse root, two products and the
    rotation's two terms, an angle rounded to 2^-24 of half a turn and sine and cosine good to 2^-22: below 2^-19 of
    the pair's magnitude."""
    err = (got.double().cpu() - y).abs()
    tol = 2.0 ** -8 * y.abs() + 2.0 ** -19 * mag
    assert (err <= tol).all(), f"{what}: {(err - tol).max().item():.3g} beyond the bound"


@pytest.mark.parametrize("T,H,Hkv,rotary,inter,norm,pos0", [
    (1, 32, 8, 128, False, True, 0), (1, 1, 1, 128, True, True, 131071), (3, 28, 4, 64, False, True, 7),
    (37, 32, 4, 96, True, True, 1000), (5, 6, 3, 0, False, True, 5), (2, 64, 8, 8, False, False, 2 ** 31 - 3),
    (479, 4, 2, 128, False, True, 100000), (480, 4, 2, 128, False, True, 100000), (901, 5, 5, 40, True, True, 3),
    (1031, 32, 8, 128, False, True, 122880), (2881, 32, 8, 128, False, True, 7), (1203, 8, 4, 112, False, True, 9),
    (1203, 8, 4, 96, True, False, 9),
    (4, 32, 1, 128, False, True, -9)])
def test_norm_rope(T, H, Hkv, rotary, inter, norm, pos0):
    from kv_cache_computation_gb300 import QkvRotary
    wide = _randn((T, (H + 2 * Hkv) * 128 + 24), 1, 3.0)
    qkv = wide.cuda()[:, 8:8 + (H + 2 * Hkv) * 128]             # rows apart, 16-byte aligned
    x = wide[:, 8:8 + (H + 2 * Hkv) * 128].reshape(T, H + 2 * Hkv, 128)
    pos = (pos0 + torch.arange(T)).to(torch.int32)
    wq, wk = (_randn(128, 2), _randn(128, 3)) if norm else (None, None)
    rot = QkvRotary(H, Hkv, rotary_dim=rotary, base=500000.0, interleaved=inter, eps=1e-6)
    w = [None if a is None else a.cuda() for a in (wq, wk)]
    q_pre, q_post, k, v = rot(qkv, pos.cuda(), *w)
    yq, rq = R.norm_rope(x[:, :H], wq, pos, rotary, 500000.0, inter, 1e-6)
    yk, rk = R.norm_rope(x[:, H:H + Hkv], wk, pos, rotary, 500000.0, inter, 1e-6)
    _check_rope(q_pre, yq, "q_pre", yq.abs())
    half = rotary // 2
    for got, y, r, what in ((q_post, yq, rq, "q_post"), (k, yk, rk, "k")):
        mag = y.abs().clone()
        if half:
            a, b = ((slice(0, rotary, 2), slice(1, rotary, 2)) if inter else (slice(0, half), slice(half, rotary)))
            mag[..., a] = mag[..., b] = y[..., a].abs() + y[..., b].abs()
        _check_rope(got, r, what, mag)
    assert torch.equal(v.cpu(), x[:, H + Hkv:])
    # the same from three tensors, without the pre-rotation queries
    parts = [a.contiguous().cuda() for a in (x[:, :H], x[:, H:H + Hkv].reshape(T, -1), x[:, H + Hkv:])]
    none, q2, k2, v2 = rot.split(*parts, pos.cuda(), *w, want_pre=False)
    assert none is None and torch.equal(q2, q_post) and torch.equal(k2, k) and torch.equal(v2, v)


def test_norm_rope_special_rows():
    """A row of zeros stays zero (eps > 0), an infinity or NaN stays in its own row, no token is no work."""
    from kv_cache_computation_gb300 import QkvRotary
    rot = QkvRotary(4, 2)
    x = _randn((3, 8 * 128), 5)
    x[0, :128] = 0
    x[1, 130] = float("inf")
    x[2, 4 * 128 + 5] = float("nan")
    pos = torch.tensor([0, 5, 9], dtype=torch.int32).cuda()
    w = _randn(128, 6).cuda()
    q_pre, q_post, k, v = rot(x.cuda(), pos, w, w)
    assert (q_pre[0, 0] == 0).all() and (q_post[0, 0] == 0).all()
    good = torch.ones(3, 4, dtype=torch.bool)
    good[1, 1] = False
    assert torch.isfinite(q_post.cpu()[good]).all() and not torch.isfinite(q_post[1, 1]).all()
    assert torch.isfinite(k.cpu()[2, 1]).all() and torch.isnan(k[2, 0]).any()
    out = rot(x.cuda()[:0], pos[:0], w, w)
    assert [tuple(t.shape) for t in out] == [(0, 4, 128), (0, 4, 128), (0, 2, 128), (0, 2, 128)]


# ---- page bookkeeping ----------------------------------------------------------

def _pool(B, P, N, seed, max_len):
    r = np.random.default_rng(seed)
    lens = r.integers(0, max_len + 1, B)
    used = (lens + 15) // 16
    perm = r.permutation(N)
    table, at = np.full((B, P), -7, np.int64), 0
    for b in range(B):
        table[b, :used[b]] = perm[at:at + used[b]]
        at += used[b]
    assert at <= N
    head = int(r.integers(0, N))
    ring = np.full(N, -3, np.int64)
    ring[(head + np.arange(N - at)) % N] = perm[at:]
    return lens, table, ring, [head, N - at], r


def _run_step(lens, new, table, ring, state, T, in_place=False, pad=0):
    from kv_cache_computation_gb300 import page_step
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32).cuda()
    wide = torch.full((len(lens), table.shape[1] + pad), -99, dtype=torch.int32).cuda()
    wide[:, :table.shape[1]] = i32(table)
    tab, rng, ln, st = wide[:, :table.shape[1]], i32(ring), i32(lens), i32(state)
    s = page_step(ln, i32(new), tab, rng, st, max_tokens=T, in_place=in_place)
    if in_place:
        assert s.lengths is ln and s.free_state is st
    if pad:
        assert (wide[:, table.shape[1]:] == -99).all()
    return [x.cpu().numpy().astype(np.int64) for x in (s.lengths, s.free_state, s.starts, s.positions, s.slots, tab, rng,
                                                       s.status)]


def _same(got, want):
    for a, b, name in zip(got, want, ("lengths", "free_state", "starts", "positions", "slots", "table", "ring", "status")):
        np.testing.assert_array_equal(a, b, err_msg=name)


@pytest.mark.parametrize("B,P,N,max_len,T,top,seed", [
    (1, 1, 1, 0, 1, 1, 0), (1, 300, 301, 4096, 700, 600, 1), (3, 9, 40, 100, 3, 1, 2), (33, 20, 700, 300, 40, 1, 3),
    (250, 40, 9000, 500, 9000, 60, 4), (1024, 12, 12288, 150, 12000, 20, 5), (1024, 3, 3000, 40, 1024, 1, 6)])
def test_page_step(B, P, N, max_len, T, top, seed):
    lens, table, ring, state, r = _pool(B, P, N, seed, max_len)
    new = r.integers(0, top + 1, B)
    new[r.random(B) < 0.2] = -1 - int(r.integers(0, 5))
    want = R.page_step(lens, new, table, ring, state, T)
    _same(_run_step(lens, new, table, ring, state, T, pad=3), want)
    _same(_run_step(lens, new, table, ring, state, T, in_place=True), want)


@pytest.mark.parametrize("what", ["dry", "row", "tokens", "length", "negative", "state", "double", "page", "ring_page"])
def test_page_step_denials(what):
    """Each way a step can be refused leaves the denied requests as they were, serves the others and sets its bit."""
    lens, table, ring, state, r = _pool(6, 8, 40, 11, 60)
    lens[2], lens[4] = 0, 17
    T = 400
    new = np.array([5, 20, 33, -1, 16, 1])
    if what == "dry":
        state = [state[0], 3]
    elif what == "row":
        new[1] = 500
    elif what == "tokens":
        T = 50
    elif what == "length":
        lens[1] = 8 * 16 + 1
    elif what == "negative":
        lens[1] = -4
    elif what == "state":
        state = [40, 3]
    elif what == "double":
        state = [state[0], 40]
        ring = np.arange(40)
    elif what == "page":
        lens[0], table[0, 0] = 5, 40
    elif what == "ring_page":
        ring[state[0]] = -5
    want = R.page_step(lens, new, table, ring, state, T)
    bit = dict(dry=1, row=2, tokens=8, length=4, negative=4, state=4, double=16, page=4, ring_page=4)[what]
    assert int(want[-1][0]) & bit
    _same(_run_step(lens, new, table, ring, state, T), want)


def test_page_pool_over_many_steps():
    """Requests come, grow and go for 60 steps: no page is ever held twice and none is lost."""
    from kv_cache_computation_gb300 import new_page_pool, page_step
    B, P, N, T = 7, 12, 64, 200
    ring, state = new_page_pool(N)
    lens = torch.zeros(B, dtype=torch.int32).cuda()
    table = torch.zeros((B, P), dtype=torch.int32).cuda()
    r = np.random.default_rng(3)
    ref = [lens.cpu().numpy(), None, None, None, None, table.cpu().numpy(), ring.cpu().numpy(), None]
    rstate = [0, N]
    for t in range(60):
        new = np.where(r.random(B) < 0.15, -1, r.integers(0, 30, B))
        want = R.page_step(ref[0], new, ref[5], ref[6], rstate, T)
        s = page_step(lens, torch.tensor(new, dtype=torch.int32).cuda(), table, ring, state, max_tokens=T)
        lens, state = s.lengths, s.free_state
        _same([x.cpu().numpy() for x in (lens, state, s.starts, s.positions, s.slots, table, ring, s.status)], want)
        ref, rstate = want, [int(x) for x in want[1]]
        held = [int(p) for b in range(B) for p in want[5][b, :-(-int(want[0][b]) // 16)]]
        free = [int(want[6][(rstate[0] + i) % N]) for i in range(rstate[1])]
        assert sorted(held + free) == list(range(N))


# ---- the 4-bit store -------------------------------------------------------------

def _slots(n, pages, seed):
    return torch.from_numpy(np.random.default_rng(seed).permutation(pages * 16)[:n].astype(np.int32))


@pytest.mark.parametrize("T,Hkv,pages,ks,vs", [(1, 1, 1, 1.0, 1.0), (5, 8, 3, 1.0, 4.0), (64, 3, 4, 0.25, 1.0),
                                               (333, 2, 40, 1.0, 2.0 ** -20), (2048, 8, 128, 1.0, 1.0),
                                               (5463, 3, 342, 1.0, 1.0)])
def test_store_round_trip_is_the_format(T, Hkv, pages, ks, vs):
    from kv_cache_computation_gb300 import QuantKV
    cache = QuantKV(Hkv, Hkv, num_pages=pages, k_scale=ks, v_scale=vs)
    k, v = _randn((T, Hkv, 128), 1, 2.0 * ks), _randn((T, Hkv, 128), 2, 0.7 * vs)
    k[0, 0, :16] = torch.linspace(-3, 3, 16).to(BF16) * ks          # ties and equal magnitudes
    k[-1, -1] = torch.cat([torch.tensor([6.0] + [x for x in (.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0) for _ in (0, 1)] + [0.0]),
                           torch.zeros(112)]).to(BF16) * ks
    v[-1, 0] = 0
    v[-1, 0, 3] = 2.0 ** -12 * vs                                    # a scale below the smallest: stored as zeros
    v[0, -1, 16:32] = 30000.0 * vs                                   # saturates at 6 * 448
    slots = _slots(T, pages, 3)
    slots[T // 2] = -1 if T > 1 else slots[0]
    cache.append(k.cuda(), v.cuda(), slots.cuda())
    gk, gv = cache.gather(slots.cuda())
    cache.sync()
    for got, x, scale in ((gk, k, ks), (gv, v, vs)):
        want = R.stored(x.double().numpy(), scale)
        want[slots.numpy() < 0] = 0
        np.testing.assert_array_equal(got.double().cpu().numpy(), want)
    # tokens that were not appended read as zeros
    rest = np.setdiff1d(np.arange(pages * 16), slots.numpy()).astype(np.int32)
    if len(rest):
        gk, gv = cache.gather(torch.from_numpy(rest).cuda())
        assert (gk == 0).all() and (gv == 0).all()


@pytest.mark.parametrize("first,T,pages", [(0, 64, 9), (0, 40, 9), (3, 61, 9), (16, 16, 9), (5, 7, 9), (0, 8208, 514),
                                           (4, 8193, 514), (7, 8195, 514), (0, 8209, 514)])
def test_store_whole_pages(first, T, pages):
    """Runs of consecutive tokens through pages in any order, starting and ending inside a page, beside other tokens of
    the same pages that stay as they are."""
    from kv_cache_computation_gb300 import QuantKV
    Hkv = 2
    cache = QuantKV(Hkv, Hkv, num_pages=pages)
    order = np.random.default_rng(4).permutation(pages)
    every = torch.from_numpy((order[:, None] * 16 + np.arange(16)).reshape(-1).astype(np.int32))
    old = _randn((pages * 16, Hkv, 128), 5), _randn((pages * 16, Hkv, 128), 6)
    cache.append(old[0].cuda(), old[1].cuda(), every.cuda())
    new = _randn((T, Hkv, 128), 7, 3.0), _randn((T, Hkv, 128), 8, 3.0)
    cache.append(new[0].cuda(), new[1].cuda(), every[first:first + T].cuda())
    got = cache.gather(every.cuda())
    for g, o, n in zip(got, old, new):
        want = R.stored(o.double().numpy())
        want[first:first + T] = R.stored(n.double().numpy())
        np.testing.assert_array_equal(g.double().cpu().numpy(), want)


def test_store_strides_nonfinite_and_bad_slots():
    from kv_cache_computation_gb300 import MacError, QuantKV
    cache = QuantKV(4, 2, num_pages=2)
    wide = _randn((6, 2 * 2 * 128), 9)
    wide[1, 5] = float("nan")
    wide[2, 256 + 20] = float("-inf")
    x = wide.cuda()
    k, v = x[:, :256], x[:, 256:]
    slots = torch.tensor([0, 31, 7, 32, -5, 2 ** 31 - 1], dtype=torch.int32)   # two past the store
    cache.append(k, v, slots.cuda())
    gk, gv = cache.gather(slots.cuda())
    with pytest.raises(MacError, match="slot"):
        cache.sync()
    cache.sync()                                                        # reported once
    for got, src in ((gk, wide[:, :256]), (gv, wide[:, 256:])):
        want = R.stored(src.double().numpy().reshape(6, 2, 128))
        want[3:] = 0
        np.testing.assert_array_equal(got.double().cpu().numpy(), want)
    assert torch.isnan(gk[1, 0, :16]).all() and torch.isfinite(gk[1, 0, 16:]).all()
    assert torch.isnan(gv[2, 0, 16:32]).all() and torch.isfinite(gv[2, 1]).all()


def test_store_beyond_32_bit_offsets():
    """A store of 5.5 GB: slots in its last pages are stored, read and attended like any other."""
    from kv_cache_computation_gb300 import QuantKV
    pages, Hkv, n = 300_000, 8, 50
    cache = QuantKV(16, Hkv, num_pages=pages)
    assert cache.sizes["store"] > 5 * 2 ** 30
    table = torch.tensor([[pages - 1, 3, pages - 70_000, pages - 2]], dtype=torch.int32)
    t = torch.arange(n)
    slots = (table[0, t // 16] * 16 + t % 16).to(torch.int32)
    k, v, q = _randn((n, Hkv, 128), 1), _randn((n, Hkv, 128), 2), _randn((1, 16, 128), 3)
    cache.append(k.cuda(), v.cuda(), slots.cuda())
    gk, gv = cache.gather(slots.cuda())
    K, V = R.stored(k.double().numpy()), R.stored(v.double().numpy())
    np.testing.assert_array_equal(gk.double().cpu().numpy(), K)
    np.testing.assert_array_equal(gv.double().cpu().numpy(), V)
    out, lse = cache.attention(q.cuda(), table.cuda(), torch.tensor([n], dtype=torch.int32).cuda())
    cache.sync()
    o, l, mag, top = R.attention(q.double().numpy(), K, V, 1 / np.sqrt(128))
    to, tl = R.attention_tolerance(o, mag, top, l, n)
    assert (np.abs(out.double().cpu().numpy() - o) <= to).all()
    assert (np.abs(lse.double().cpu().numpy() - l) <= tl).all()


# ---- attention over the store -------------------------------------------------------

class Case:
    """A store holding requests of the given lengths in random pages, and what it holds in float64."""

    def __init__(self, lens, H, Hkv, nq, seed=0, scale=0.0, qscale=1.5, spare=3, ks=1.0, vs=1.0):
        from kv_cache_computation_gb300 import QuantKV
        r = np.random.default_rng(seed)
        self.lens, self.H, self.Hkv, self.nq = lens, H, Hkv, nq
        cols = max(1, -(-max(lens) // 16))
        n_pages = sum(-(-n // 16) for n in lens) + spare
        perm = r.permutation(n_pages).astype(np.int32)
        self.table = np.full((len(lens), cols), -1, np.int32)       # never read past a request's pages
        self.cache = QuantKV(H, Hkv, num_pages=n_pages, max_batch=len(lens), max_query=nq, sm_scale=scale, k_scale=ks,
                             v_scale=vs)
        self.scale = scale or 1 / np.sqrt(128)
        # everything starts as NaN: slots past a request's length must have no effect
        nan = torch.full((n_pages * 16, Hkv, 128), float("nan"), dtype=BF16).cuda()
        self.cache.append(nan, nan, torch.arange(n_pages * 16, dtype=torch.int32).cuda())
        self.k, self.v, at = [], [], 0
        for b, n in enumerate(lens):
            p = -(-n // 16)
            self.table[b, :p] = perm[at:at + p]
            at += p
            k, v = _randn((n, Hkv, 128), 100 + b + seed, ks), _randn((n, Hkv, 128), 200 + b + seed, vs)
            t = np.arange(n)
            slots = self.table[b, t // 16] * 16 + t % 16 if n else t
            self.cache.append(k.cuda(), v.cuda(), torch.from_numpy(slots.astype(np.int32)).cuda())
            self.k.append(R.stored(k.double().numpy(), ks))
            self.v.append(R.stored(v.double().numpy(), vs))
        self.q = _randn((len(lens), nq, H, 128), 300 + seed, qscale)
        self.dev = dict(q=self.q.cuda(), page_table=torch.from_numpy(self.table).cuda(),
                        lengths=torch.tensor(lens, dtype=torch.int32).cuda())

    def run(self, **kw):
        out = self.cache.attention(**self.dev, **kw)
        self.cache.sync()
        return out

    def check(self, out, lse, requests=None):
        for b in range(len(self.lens)) if requests is None else requests:
            o, l, mag, top = R.attention(self.q[b].double().numpy(), self.k[b], self.v[b], self.scale)
            to, tl = R.attention_tolerance(o, mag, top, l, self.lens[b])
            go = out[b].double().cpu().numpy().reshape(o.shape)
            assert (np.abs(go - o) <= to).all(), (b, self.lens[b], np.abs(go - o).max(), (np.abs(go - o) - to).max())
            gl = lse[b].double().cpu().numpy().reshape(l.shape)
            empty = np.isneginf(l)
            assert (np.isneginf(gl) == empty).all()
            assert (np.abs(gl[~empty] - l[~empty]) <= tl[~empty]).all(), (b, self.lens[b])


@pytest.mark.parametrize("H,Hkv,nq", [(1, 1, 1), (8, 8, 1), (32, 8, 1), (6, 2, 1), (8, 1, 1), (9, 1, 1), (16, 1, 1),
                                      (28, 2, 1), (17, 1, 1), (32, 1, 1), (24, 8, 4), (4, 4, 8), (12, 4, 3), (2, 1, 16),
                                      (28, 4, 3), (4, 4, 32)])
def test_attention_head_layouts(H, Hkv, nq):
    """Every tile of rows (1 to 32) with lengths that end inside a page, on its edge and inside a pair of pages."""
    c = Case([1, 16, 31, 0, 47, 200, 33], H, Hkv, nq, seed=H + nq)
    c.check(*c.run())


@pytest.mark.parametrize("lens", [[1], [0], [2], [15], [17], [32], [5000], [4096, 1, 0, 777], [0, 0, 0], [33] * 40,
                                  [3] * 300, [1, 3000] * 5])
def test_attention_lengths(lens):
    c = Case(lens, 8, 2, 1, seed=len(lens))
    c.check(*c.run(), requests=range(0, len(lens), max(1, len(lens) // 10)))


def test_attention_many_requests_and_long_one():
    """1024 requests of which one is long: groups that span many blocks beside many that end inside one."""
    lens = [int(x) for x in np.random.default_rng(5).integers(0, 40, 1024)]
    lens[700] = 20000
    c = Case(lens, 4, 2, 1, seed=9)
    out, lse = c.run()
    c.check(out, lse, requests=[0, 1, 2, 699, 700, 701, 1023] + list(range(5, 1000, 90)))


@pytest.mark.parametrize("H,Hkv,nq", [(32, 8, 1), (16, 1, 1), (32, 1, 1), (28, 4, 3)])
def test_attention_long(H, Hkv, nq):
    c = Case([30001], H, Hkv, nq, seed=3)
    c.check(*c.run())


@pytest.mark.parametrize("qscale,scale", [(0.0, 0.0), (1e-30, 0.0), (60.0, 0.0), (3e4, 1e-4), (1.0, 5.0), (1.0, 1e-8)])
def test_attention_score_ranges(qscale, scale):
    """Zero and tiny queries (uniform weights), scores that let one token take all, a growing maximum."""
    c = Case([500, 70], 8, 2, 1, seed=21, qscale=qscale, scale=scale)
    c.check(*c.run())


def test_attention_global_scales():
    c = Case([100, 33], 8, 4, 2, seed=31, ks=2.0 ** -10, vs=2.0 ** 12, qscale=1024.0)
    c.check(*c.run())


def test_attention_rising_scores_move_the_reference():
    """Keys that grow along the query: every unit of tokens passes the running reference."""
    from kv_cache_computation_gb300 import QuantKV
    n, Hkv = 700, 1
    cache = QuantKV(4, Hkv, num_pages=44)
    d = torch.sign(torch.randn(128, generator=torch.Generator().manual_seed(1)))
    k = (torch.linspace(0.01, 8, n)[:, None, None] * d).to(BF16)
    v, q = _randn((n, Hkv, 128), 2), (d * 1.0).to(BF16).expand(1, 4, 128).contiguous()
    slots = torch.arange(n, dtype=torch.int32).cuda()
    cache.append(k.cuda(), v.cuda(), slots)
    out, lse = cache.attention(q.cuda(), torch.arange(44, dtype=torch.int32).cuda()[None], torch.tensor([n]).int().cuda())
    K, V = R.stored(k.double().numpy()), R.stored(v.double().numpy())
    o, l, mag, top = R.attention(q.double().numpy(), K, V, 1 / np.sqrt(128))
    to, tl = R.attention_tolerance(o, mag, top, l, n)
    assert (np.abs(out.double().cpu().numpy() - o) <= to).all()
    assert (np.abs(lse.double().cpu().numpy() - l) <= tl).all()


def test_attention_nonfinite_tokens_stay_in_their_request():
    c = Case([40, 50, 60], 4, 2, 1, seed=41)
    nan = torch.full((1, 2, 128), float("nan"), dtype=BF16).cuda()
    slot = torch.tensor([int(c.table[1, 1]) * 16 + 3], dtype=torch.int32).cuda()     # token 19 of request 1
    c.cache.append(nan, nan, slot)
    out, lse = c.run()
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    c.check(out, lse, requests=[0, 2])


@pytest.mark.parametrize("H,Hkv,nq,n,bad", [
    (2, 1, 4, 40, [(39, 0, 3)]), (8, 2, 3, 34, [(33, 1, 0), (32, 0, 7)]), (4, 1, 4, 18, [(17, 0, 5), (15, 0, 5)]),
    (4, 4, 2, 33, [(32, 2, 1), (31, 3, 2)]), (7, 1, 3, 700, [(699, 0, 6), (698, 0, 2)]), (2, 1, 16, 20, [(19, 0, 4), (6, 0, 0)]),
    (4, 2, 2, 2, [(1, 1, 3)])])
def test_attention_nonfinite_values_of_later_drafts(H, Hkv, nq, n, bad):
    """A drafted token whose values hold an infinity: the queries before it do not see it and stay finite, those from it
    on get NaN in the 16 elements that share its scale, and only there."""
    c = Case([n, 5 + nq], H, Hkv, nq, seed=71)
    for tok, h, block in bad:
        k, v = _randn((1, Hkv, 128), 7), _randn((1, Hkv, 128), 8 + tok)
        v[0, h, 16 * block + 5] = float("inf")
        slot = torch.tensor([int(c.table[0, tok // 16]) * 16 + tok % 16], dtype=torch.int32).cuda()
        c.cache.append(k.cuda(), v.cuda(), slot)
        c.k[0][tok], c.v[0][tok] = R.stored(k.double().numpy())[0], R.stored(v.double().numpy())[0]
    out, lse = c.run()
    c.check(out, lse, requests=[1])
    # the reference with the bad blocks made zero, and where they are seen
    v = c.v[0]
    o, l, mag, top = R.attention(c.q[0].double().numpy(), c.k[0], np.nan_to_num(v), c.scale)
    to, tl = R.attention_tolerance(o, mag, top, l, n)
    seen = np.zeros(o.shape, bool)
    for i in range(nq):
        rows = np.isnan(v[:n - (nq - 1) + i]).any(0)                # [KV head, element]
        seen[i] = np.repeat(rows, H // Hkv, 0)
    assert seen.any() and not seen.all()
    go = out[0].double().cpu().numpy()
    np.testing.assert_array_equal(np.isnan(go), seen)
    assert (np.abs(go - o) <= to)[~seen].all()
    assert (np.abs(lse[0].double().cpu().numpy() - l) <= tl).all()


@pytest.mark.parametrize("H,n", [(4, 7), (4, 3000), (12, 100), (20, 100), (32, 100)])
def test_attention_nonfinite_queries_give_nan_in_their_row(H, n):
    """An infinity in a query leaves no softmax: NaN, also where every score is minus infinity; the group's other rows
    are untouched."""
    c = Case([n], H, 1, 1, seed=81)
    k = _randn((n, 1, 128), 9).abs().clamp(min=0.5)                 # no element rounds to 0
    slots = (torch.from_numpy(c.table[0, np.arange(n) // 16].astype(np.int32)) * 16 + torch.arange(n) % 16).to(torch.int32)
    c.cache.append(k.cuda(), _randn((n, 1, 128), 200 + 81).cuda(), slots.cuda())
    c.k[0] = R.stored(k.double().numpy())
    assert (c.k[0] > 0).all()
    bad = [0, 1, H - 1]
    for row, x in zip(bad, ("-inf", "inf", "nan")):
        c.q[0, 0, row, 77] = float(x)
    c.dev["q"] = c.q.cuda()
    out, lse = c.run()
    assert torch.isnan(out[0, 0, bad]).all() and torch.isnan(lse[0, 0, bad]).all()
    good = [r for r in range(H) if r not in bad]
    q = c.q[0].double().numpy()[:, good]
    o, l, mag, top = R.attention(q, c.k[0], c.v[0], c.scale)
    to, tl = R.attention_tolerance(o, mag, top, l, n)
    assert (np.abs(out[0].double().cpu().numpy()[:, good] - o) <= to).all()
    assert (np.abs(lse[0].double().cpu().numpy()[:, good] - l) <= tl).all()


def test_attention_padded_batch_strided_table_outputs_and_three_dim_q():
    """A padded batch (idle slots of length 0), a table that is a slice of a wider one, given outputs and no lse; the
    rows behind the batch keep what they held."""
    c = Case([70, 0, 9, 0], 8, 2, 1, seed=51)
    wide = torch.full((4, c.table.shape[1] + 5), -1, dtype=torch.int32).cuda()
    wide[:, :c.table.shape[1]] = c.dev["page_table"]
    buf = torch.full((6, 8, 128), 7.0, dtype=BF16).cuda()
    out, lse = c.cache.attention(c.dev["q"][:, 0].contiguous(), wide[:, :c.table.shape[1]], c.dev["lengths"], out=buf[:4])
    c.check(out, lse)
    assert (buf[4:] == 7.0).all() and (out[1] == 0).all() and torch.isneginf(lse[3]).all()
    out2, none = c.cache.attention(c.dev["q"], c.dev["page_table"], c.dev["lengths"], want_lse=False)
    assert none is None and torch.equal(out2[:, 0], out)


def test_attention_reports_bad_pages_and_lengths():
    from kv_cache_computation_gb300 import MacError
    c = Case([40, 50, 60], 4, 2, 1, seed=61)
    good = c.run()
    bad = c.dev["page_table"].clone()
    bad[1, 2] = c.cache.num_pages
    out = c.cache.attention(c.dev["q"], bad, c.dev["lengths"])
    with pytest.raises(MacError, match="page"):
        c.cache.sync()
    for b in (0, 2):
        assert torch.equal(out[0][b], good[0][b])
    for n in (-1, 16 * c.table.shape[1] + 1):
        ln = c.dev["lengths"].clone()
        ln[2] = n
        out = c.cache.attention(c.dev["q"], torch.clamp(c.dev["page_table"], min=0), ln)
        with pytest.raises(MacError, match="length"):
            c.cache.sync()
        c.check(*out, requests=[0, 1])
    c.check(*c.run())


def test_refusals_on_the_gpu():
    from kv_cache_computation_gb300 import MacError, QkvRotary, QuantKV
    c = Case([40, 50], 4, 2, 2, seed=71)
    q, t, n = c.dev["q"], c.dev["page_table"], c.dev["lengths"]
    with pytest.raises(MacError):                                   # more query tokens than the handle was made for
        c.cache.attention(torch.zeros(2, 3, 4, 128, dtype=BF16).cuda(), t, n)
    with pytest.raises(MacError):                                   # more requests
        c.cache.attention(q.repeat(2, 1, 1, 1), t.repeat(2, 1), n.repeat(2))
    for kw in (dict(q=q.float()), dict(q=q[..., :64]), dict(q=q.transpose(1, 2)), dict(page_table=t.long()),
               dict(page_table=t[:1]), dict(page_table=t.t()), dict(lengths=n.long()), dict(lengths=n[:1]),
               dict(lengths=n.cpu()), dict(q=q.cpu()), dict(page_table=t.cpu()), dict(out=q.float())):
        with pytest.raises((TypeError, ValueError)):
            c.cache.attention(**{**c.dev, **kw})
    k = torch.zeros(3, 2, 128, dtype=BF16).cuda()
    s = torch.zeros(3, dtype=torch.int32).cuda()
    for a in ((k, k[:2], s), (k, k, s[:2]), (k.float(), k, s), (k.cpu(), k, s), (k, k, s.long()),
              (k[..., :64], k, s), (k.transpose(0, 1), k, s)):
        with pytest.raises((TypeError, ValueError)):
            c.cache.append(*a)
    with pytest.raises(MacError):                                   # a token stride that is no multiple of 16 bytes
        wide = torch.zeros(3, 2 * 128 + 4, dtype=BF16).cuda()
        c.cache.append(wide[:, :256], k, s)
    with pytest.raises(ValueError):
        c.cache.decode_step_qkv(QkvRotary(8, 2), torch.zeros(2, 8 * 128, dtype=BF16).cuda(), n, n, t, n)
    with pytest.raises(ValueError):                                 # too small a scratch to share
        QuantKV(4, 2, num_pages=1, share=type("Q", (), dict(device=c.cache.device, _scratch=k))())
    c.cache.append(k[:0], k[:0], s[:0])                             # nothing to do is no error
    assert c.cache.gather(s[:0])[0].shape == (0, 2, 128)
    assert c.cache.attention(q[:0], t[:0], n[:0])[0].shape == (0, 2, 4, 128)
    c.check(*c.run())


def test_attention_is_reproducible_and_captured():
    """Two runs agree bit for bit; a captured call serves other lengths, queries and tokens when it is replayed."""
    c = Case([900, 40, 0, 300], 8, 2, 1, seed=81)
    a, b = c.run(), c.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.dev["lengths"].zero_()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.cache.attention(**c.dev)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out, lse = c.cache.attention(**c.dev)
    for lens in ([900, 40, 0, 300], [1, 2, 0, 299], [512, 0, 0, 5]):
        c.dev["lengths"].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        whole = c.lens, c.k, c.v
        c.k, c.v, c.lens = [k[:n] for k, n in zip(c.k, lens)], [v[:n] for v, n in zip(c.v, lens)], lens
        c.check(out, lse)
        c.lens, c.k, c.v = whole


def test_other_streams_and_shared_scratch():
    """Calls on a stream of the caller's, on another layer that shares the scratch, ordered by events."""
    from kv_cache_computation_gb300 import QuantKV
    c = Case([600, 130], 8, 2, 1, seed=91)
    other = QuantKV(8, 2, num_pages=c.cache.num_pages, max_batch=2, share=c.cache)
    every = torch.arange(c.cache.num_pages * 16, dtype=torch.int32).cuda()
    other.append(*c.cache.gather(every), every)         # stored values are fixed points of the format
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        a = c.cache.attention(**c.dev)
        b = other.attention(**c.dev)
    d = c.cache.attention(**c.dev, stream=s)
    s.synchronize()
    c.check(*a)
    assert all(torch.equal(a[i], b[i]) and torch.equal(a[i], d[i]) for i in (0, 1))


# ---- the operators together ---------------------------------------------------------

def _serve(n_query, capture):
    """Six steps of four requests (one finishes and its slot is taken again) from projections to outputs."""
    from kv_cache_computation_gb300 import QkvRotary, QuantKV, new_page_pool, page_step
    B, H, Hkv, P, N = 4, 8, 2, 8, 40
    rot = QkvRotary(H, Hkv, base=10000.0)
    cache = QuantKV(H, Hkv, num_pages=N, max_batch=B, max_query=n_query)
    ring, state = new_page_pool(N)
    lens = torch.zeros(B, dtype=torch.int32).cuda()
    table = torch.zeros((B, P), dtype=torch.int32).cuda()
    w = _randn(128, 1).cuda(), _randn(128, 2).cuda()
    new = torch.tensor([45, 16, 3, 1], dtype=torch.int32).cuda()
    # prefill: packed tokens of uneven requests
    s = page_step(lens, new, table, ring, state, max_tokens=80, in_place=True)
    T = 65
    x = _randn((80, (H + 2 * Hkv) * 128), 3).cuda()
    _, _, k, v = rot(x, s.positions, *w)
    cache.append(k, v, s.slots)                          # the padding's slots are -1
    hist = [[[z.cpu()[int(a):int(b)] for z in (s.positions, k, v)]] for a, b in zip(s.starts[:-1], s.starts[1:])]
    assert int(s.starts[-1]) == T and int(s.status) == 0
    qkv = torch.empty((B * n_query, (H + 2 * Hkv) * 128), dtype=BF16).cuda()
    new.fill_(n_query)

    def step():
        st = page_step(lens, new, table, ring, state, max_tokens=B * n_query, in_place=True)
        return st, cache.decode_step_qkv(rot, qkv, st.positions, st.slots, table, st.lengths, *w)
    run = step
    if capture:
        keep = [t.clone() for t in (lens, table, ring, state)]
        qkv.zero_()
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = step()
        for t, o in zip((lens, table, ring, state), keep):
            t.copy_(o)

        def run():
            graph.replay()
            return res
    for t in range(6):
        if t == 3:                                       # request 2 finishes, a new one takes its slot
            new[2] = -1
            st = page_step(lens, new * torch.tensor([0, 0, 1, 0]).int().cuda(), table, ring, state, max_tokens=1,
                           in_place=True)
            new[2] = n_query
            hist[2] = []
        qkv.copy_(_randn(tuple(qkv.shape), 50 + t))
        st, (out, lse) = run()
        cache.sync()
        assert int(st.status) == 0
        _, q, k, v = rot(qkv, st.positions, *w)          # what the step's own norm and rotation gave
        for b in range(B):
            rows = slice(b * n_query, (b + 1) * n_query)
            hist[b].append([t.cpu()[rows] for t in (st.positions, k, v)])
            pos, kb, vb = (torch.cat(z) for z in zip(*hist[b]))
            assert torch.equal(pos, torch.arange(len(pos), dtype=torch.int32))
            K, V = R.stored(kb.double().numpy()), R.stored(vb.double().numpy())
            o, l, mag, top = R.attention(q.cpu()[rows].double().numpy(), K, V, 1 / np.sqrt(128))
            to, tl = R.attention_tolerance(o, mag, top, l, len(pos))
            assert (np.abs(out[b].double().cpu().numpy() - o) <= to).all()
            assert (np.abs(lse[b].double().cpu().numpy() - l) <= tl).all()


@pytest.mark.parametrize("n_query,capture", [(1, False), (3, False), (1, True)])
def test_serving_steps_together(n_query, capture):
    _serve(n_query, capture)


def test_mac_decode_step_from_a_projection():
    """The MAC step fed by the fused norm and rotation, its pages by page_step, equals the step fed by hand."""
    from kv_cache_computation_gb300 import MacAttention, QkvRotary, new_page_pool, page_step
    B, H, Hkv = 2, 8, 2
    rot = QkvRotary(H, Hkv)
    w = _randn(128, 1).cuda(), _randn(128, 2).cuda()
    ring, state = new_page_pool(64)
    lens, table = torch.zeros(B, dtype=torch.int32).cuda(), torch.zeros((B, 8), dtype=torch.int32).cuda()
    new = torch.tensor([70, 33], dtype=torch.int32).cuda()
    s = page_step(lens, new, table, ring, state, max_tokens=103)
    x = _randn((103, (H + 2 * Hkv) * 128), 3).cuda()
    _, _, k, v = rot(x, s.positions, *w)
    macs = []
    for _ in range(2):
        m = MacAttention(H, Hkv, ring_len=4, band_r=16, max_batch=B, max_ctx=128, num_pages=64)
        for b, (lo, hi) in enumerate(((0, 70), (70, 103))):
            m.set_page_table(b, table[b])
            m.append_kv(b, k[lo:hi], v[lo:hi])
        macs.append(m)
    for t in range(4):
        qkv = _randn((B, (H + 2 * Hkv) * 128), 10).cuda()              # the same queries: later steps hit
        pos = s.lengths + t
        a = macs[0].decode_step_qkv(rot, qkv, pos, *w)
        b = macs[1].decode_step(*rot(qkv, pos, *w))
        for m in macs:
            m.sync()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert macs[0].stats()["hits"] == macs[1].stats()["hits"] > 0
    with pytest.raises(ValueError):
        macs[0].decode_step_qkv(QkvRotary(4, 2), qkv, pos, *w)


def test_mac_decode_step_from_a_projection_on_another_stream():
    """With a stream given, the outputs are made of that stream's memory, so work still queued on the current stream, on
    memory that it has given back, cannot reach them."""
    from kv_cache_computation_gb300 import MacAttention, QkvRotary
    B, H, Hkv = 2, 8, 2
    rot = QkvRotary(H, Hkv)
    qkv, pos = _randn((B, (H + 2 * Hkv) * 128), 3).cuda(), torch.zeros(B, dtype=torch.int32).cuda()
    pages = torch.arange(8, dtype=torch.int32).view(B, 4).cuda()
    got, s = [], torch.cuda.Stream()
    for stream in (None, s):
        m = MacAttention(H, Hkv, ring_len=4, band_r=16, max_batch=B, max_ctx=64, num_pages=8)
        for b in range(B):
            m.set_page_table(b, pages[b])
        m.sync()
        torch.cuda.synchronize()
        got.append(m.decode_step_qkv(rot, qkv, pos, stream=stream))
        torch.cuda.synchronize()
    for x, y in zip(*got):
        assert torch.equal(x, y)
        owner = [seg["stream"] for seg in torch.cuda.memory_snapshot()
                 if seg["address"] <= y.data_ptr() < seg["address"] + seg["total_size"]]
        assert owner == [s.cuda_stream]

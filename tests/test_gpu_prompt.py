"""Prompt attention on the GPU against its definition in 64 bits (torch double).
The tolerances are derived in _tolerance."""
import numpy as np
import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

BF16, F32 = torch.bfloat16, torch.float32


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32).cuda()


def _randn(shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(BF16)


def _reference(q, k, v, lag, scale):
    """One sequence, double: out, lse and the bounds' quantities mag = sum p |v| / sum p, top = max sum |q k| scale."""
    n, H, _ = q.shape
    m, Hkv, _ = k.shape
    G = H // Hkv
    out, mag = torch.zeros((2, n, H, 128), dtype=torch.double, device=q.device)
    lse, top = torch.full((n, H), -np.inf, dtype=torch.double, device=q.device), torch.zeros((n, H), device=q.device).double()
    if n == 0 or m == 0:
        return out, lse, mag, top
    seen = (m - n + 1 - lag + torch.arange(n, device=q.device))[:, None, None]
    kd, vd = k.double(), v.double()
    for h in range(Hkv):
        hs = slice(h * G, (h + 1) * G)
        qd = q[:, hs].double()
        s = torch.einsum("ngd,td->ngt", qd, kd[:, h]) * scale
        hide = torch.arange(m, device=q.device) >= seen
        s = torch.where(hide, -np.inf, s)
        z = torch.logsumexp(s, -1)
        p = torch.exp(s - torch.where(torch.isfinite(z), z, 0.0)[..., None])
        # rows that see a value meet its NaN, the others do not
        clean = torch.nan_to_num(vd[:, h], nan=0.0, posinf=0.0, neginf=0.0)
        o = torch.einsum("ngt,td->ngd", p, clean)
        bad = torch.einsum("ngt,td->ngd", (~hide).double().expand(s.shape), (~torch.isfinite(vd[:, h])).double()) > 0
        out[:, hs] = torch.where(bad, np.nan, o)
        mag[:, hs] = torch.einsum("ngt,td->ngd", p, clean.abs())
        lse[:, hs] = z
        big = torch.einsum("ngd,td->ngt", qd.abs(), kd[:, h].abs()) * scale
        top[:, hs] = torch.where(hide, 0.0, torch.nan_to_num(big)).amax(-1)
    return out, lse, mag, top


def _tolerance(out, mag, top, lse, m, wide):
    """out is rounded to bf16 (2^-8 of it; fp32 2^-24) and each weight to bf16 (2^-8; to hi + lo 2^-16): of mag.  A score
    is a sum of 128 exact products in 8 accumulations of 16, each rounded or cut at 2^-23 of sum |q k|, times an fp32
    scale (2^-24), less the reference in one fused step (2^-24 of at most 2 |score|): within 11 * 2^-23 top; the
    exponential is good to 2^-21.  Weight and normaliser are each off by that.  The sums over m keys take at most
    m / 16 accumulations per row and, between parts, under 64 merges, each 2^-23 of mag; a merge's weight is good to
    2^-21 again."""
    d = 11 * 2.0 ** -23 * top + 2.0 ** -20
    acc = (64 + m / 16) * 2.0 ** -23
    r = 2.0 ** -16 if wide else 2.0 ** -8
    return ((2.0 ** -24 if wide else 2.0 ** -8) * out.abs() + mag * (r + 2 * d + 2 * acc)[..., None] + 1e-30,
            d + acc + 2.0 ** -21 * torch.nan_to_num(lse, neginf=0.0).abs() + 2.0 ** -22)


class Case:
    """Packed sequences [(queries, keys)], with spare rows behind (and between tensors' ends) that hold NaN."""

    def __init__(self, seqs, H, Hkv, lag=0, seed=0, scale=0.0, qscale=1.0, spare=3, wide=False, sliced=False):
        from kv_cache_computation_gb300 import PromptAttention
        self.seqs, self.lag, self.scale, self.wide = seqs, lag, scale or 1 / np.sqrt(128), wide
        self.qs = np.concatenate(([0], np.cumsum([n for n, _ in seqs])))
        self.ks = np.concatenate(([0], np.cumsum([m for _, m in seqs])))
        Tq, Tk = int(self.qs[-1]) + spare, int(self.ks[-1]) + spare
        if sliced:
            x = _randn((Tq, (H + 2 * Hkv) * 128 + 8), seed)
            x[Tq - spare:] = float("nan")
            y = x[:, 8:].unflatten(1, (H + 2 * Hkv, 128))
            self.q, self.k, self.v = y[:, :H], y[:, H:H + Hkv], y[:, H + Hkv:]
        else:
            self.q, self.k, self.v = (_randn((Tq, H, 128), seed, qscale), _randn((Tk, Hkv, 128), seed + 1),
                                      _randn((Tk, Hkv, 128), seed + 2))
            for t, T in ((self.q, Tq), (self.k, Tk), (self.v, Tk)):
                t[T - spare:] = float("nan")
        self.starts, self.k_starts = _i32(self.qs), _i32(self.ks)
        self.attend = PromptAttention(H, Hkv, max_tokens=max(Tq, 1), max_batch=len(seqs), sm_scale=scale)

    def run(self, **kw):
        args = dict(k_starts=self.k_starts, lag=self.lag, out_dtype=F32 if self.wide else BF16)
        return self.attend(self.q, self.k, self.v, self.starts, **{**args, **kw})

    def check(self, out, lse, only=None):
        assert torch.isfinite(self.starts).all()
        for b in range(len(self.seqs)) if only is None else only:
            rows, keys = slice(int(self.qs[b]), int(self.qs[b + 1])), slice(int(self.ks[b]), int(self.ks[b + 1]))
            o, l, mag, top = _reference(self.q[rows], self.k[keys], self.v[keys], self.lag, self.scale)
            to, tl = _tolerance(torch.nan_to_num(o), mag, top, l, self.seqs[b][1], self.wide)
            go, gl = out[rows].double(), lse[rows].double()
            assert torch.equal(torch.isnan(go), torch.isnan(o)), (b, self.seqs[b])
            over = torch.where(torch.isnan(o), 0.0, (go - o).abs() - to)
            assert (over <= 0).all(), (b, self.seqs[b], over.max().item(), over.argmax().item(), (over > 0).sum().item())
            empty = torch.isneginf(l)
            assert torch.equal(torch.isneginf(gl), empty)
            assert (torch.where(empty, 0.0, (gl - l).abs() - tl) <= 0).all(), (b, self.seqs[b])


@pytest.mark.parametrize("n", [1, 16, 17, 64, 127, 128, 129, 255, 256, 257, 1000])
def test_one_prompt(n):
    c = Case([(n, n)], 8, 2)
    c.check(*c.run())
    c.attend.sync()


@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 4), (32, 8), (6, 2), (5, 1), (7, 1), (28, 4), (12, 1), (16, 1), (33, 1),
                                   (32, 1), (64, 1), (100, 1), (128, 1), (256, 2)])
def test_head_layouts(H, Hkv):
    c = Case([(1, 1), (70, 70), (0, 0), (300, 300), (5, 140), (33, 33)], H, Hkv, seed=H)
    c.check(*c.run())


@pytest.mark.parametrize("seqs", [[(0, 0)], [(0, 9), (3, 3)], [(3, 0), (2, 2)], [(4, 4)] * 70, [(1, 500)] * 40, [(9, 5), (3, 2)],
                                  [(1, 1)] * 1024, [(2048, 2048), (1, 1), (777, 777)], [(129, 4000), (64, 64)],
                                  [(40, 7000)], [(1, 20000)], [(3, 9000), (2, 1), (500, 1500)]])
def test_sequences(seqs):
    c = Case(seqs, 8, 2, seed=len(seqs))
    c.check(*c.run(), only=range(0, len(seqs), max(1, len(seqs) // 12)))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("lag", [1, 7, 64, 128, 300, 5000])
def test_lag(lag, wide):
    c = Case([(200, 200), (40, 900), (3, 3), (512, 512)], 8, 2, lag=lag, seed=lag, wide=wide)
    c.check(*c.run())


@pytest.mark.parametrize("H,Hkv,seqs", [(32, 8, [(5000, 5000)]), (4, 1, [(12000, 12000)]), (28, 4, [(1500, 9000), (900, 900)]),
                                        (8, 8, [(3001, 3001)]), (32, 8, [(700, 700)] * 6), (16, 2, [(64, 30000), (4000, 4000)])])
@pytest.mark.parametrize("wide", [False, True])
def test_many_items_per_sm(H, Hkv, seqs, wide):
    """Whole items, the line that is cut and its merge together."""
    c = Case(seqs, H, Hkv, seed=5, wide=wide)
    c.check(*c.run())


@pytest.mark.parametrize("wide", [False, True])
def test_slices_of_a_projection(wide):
    c = Case([(1, 1), (333, 333), (90, 90)], 28, 4, sliced=True, wide=wide)
    out, lse = c.run(k_starts=None)
    c.check(out, lse)
    dense = [t.contiguous() for t in (c.q, c.k, c.v)]
    again = c.attend(*dense, c.starts, out_dtype=F32 if wide else BF16)
    n = int(c.qs[-1])
    assert torch.equal(again[0][:n], out[:n]) and torch.equal(again[1][:n], lse[:n])


@pytest.mark.parametrize("qscale,scale", [(0.0, 0.0), (1e-30, 0.0), (20.0, 0.0), (3e4, 1e-4), (1.0, 5.0), (1.0, 1e-8)])
def test_score_ranges(qscale, scale):
    c = Case([(300, 300), (70, 400)], 8, 2, seed=21, qscale=qscale, scale=scale)
    c.check(*c.run())


def test_rising_scores_move_the_reference():
    """Keys that grow along the queries: every block of keys passes the running reference by far."""
    c = Case([(900, 900)], 4, 1, seed=3)
    d = torch.sign(_randn((128,), 9).float())
    c.k[:900] = (torch.linspace(0.01, 9, 900, device="cuda")[:, None, None] * d).to(BF16)
    c.q[:900] = (d * torch.linspace(0.2, 1.5, 4, device="cuda")[:, None]).to(BF16)
    c.check(*c.run())


@pytest.mark.parametrize("qscale", [2.0 ** 20, 2.0 ** 26, 2.0 ** 30, 1e15, 1e30])
def test_scores_beyond_the_significand(qscale):
    """All weight goes to the row's largest score, where it is further ahead than both scores' errors (and 64 log2 units):
    the output is that key's value, the lse its score."""
    n = 600
    c = Case([(n, n)], 4, 1, seed=17, qscale=qscale)
    out, lse = c.run()
    s = torch.einsum("nhd,td->nht", c.q[:n].double(), c.k[:n, 0].double()) * c.scale
    s = torch.where(torch.arange(n, device="cuda") > torch.arange(n, device="cuda")[:, None, None], -np.inf, s)
    top = torch.einsum("nhd,td->nht", c.q[:n].double().abs(), c.k[:n, 0].double().abs()).amax(-1) * c.scale
    err = 12 * 2.0 ** -23 * top
    two = s.topk(2, -1).values
    clear = (two[..., 0] - two[..., 1] > 2 * err + 64)
    assert clear.sum() > n * 2
    want = c.v[:n, 0].double()[s.argmax(-1)]
    assert torch.isfinite(out[:n]).all() and torch.isfinite(lse[:n]).all()
    assert (((out[:n].double() - want).abs() <= 2.0 ** -7 * want.abs() + 1e-12) | ~clear[..., None]).all()
    assert (((lse[:n].double() - two[..., 0]).abs() <= err + 2.0 ** -21 * two[..., 0].abs()) | ~clear).all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("H,Hkv,seqs,lag", [(8, 2, [(200, 200), (50, 50), (300, 300)], 0), (28, 4, [(130, 400), (9, 9)], 3),
                                            (4, 1, [(5, 9000), (3, 3)], 0), (32, 8, [(2000, 2000), (40, 40)], 0)])
def test_nonfinite_keys_and_values_reach_only_what_sees_them(H, Hkv, seqs, lag, wide):
    """NaN and infinities in single keys and values, and in every token of a neighbouring sequence: rows that do not see
    them are what they would be without, rows that see a bad value have NaN in that element alone, and rows that see a bad
    key are NaN."""
    c = Case(seqs, H, Hkv, lag=lag, seed=31, wide=wide)
    k0, m = int(c.ks[0]), seqs[0][1]
    r = np.random.default_rng(1)
    for t, h, d, x in ((m - 1, 0, 5, "nan"), (m - 2, Hkv - 1, 127, "inf"), (m - 3, 0, 64, "-inf"), (m // 2, 0, 9, "nan"),
                       (m - 40 if m > 40 else 0, Hkv - 1, 63, "inf"), (int(r.integers(0, m)), 0, 100, "nan")):
        c.v[k0 + t, h, d] = float(x)
    last = slice(int(c.ks[-2]), int(c.ks[-1]))
    c.k[last], c.v[last] = float("nan"), float("inf")
    out, lse = c.run()
    c.check(out, lse, only=range(len(seqs) - 1))
    assert torch.isnan(out[int(c.qs[-2]) + lag:int(c.qs[-1])]).all()
    # a key: rows from it on are NaN, those before it are untouched
    bad = m - 7
    c.k[k0 + bad, 0, 3] = float("nan")
    again, alse = c.run()
    n, G = seqs[0][0], H // Hkv
    first = max(bad - (m - n) + lag, 0)                              # the first query that sees it
    assert torch.isnan(again[first:n, :G]).all() and torch.isnan(alse[first:n, :G]).all()
    assert torch.equal(torch.nan_to_num(again[:first].float()), torch.nan_to_num(out[:first].float()))
    assert torch.equal(again[:n, G:].nan_to_num(), out[:n, G:].nan_to_num())


def test_nonfinite_queries_stay_in_their_rows():
    c = Case([(150, 150), (150, 150)], 8, 2, seed=41)
    good = c.run()
    for t, h, x in ((3, 0, "nan"), (77, 5, "inf"), (149, 7, "-inf"), (200, 2, "nan")):
        c.q[t, h, 11] = float(x)
    out, lse = c.run()
    rows = torch.zeros(300, 8, dtype=torch.bool, device="cuda")
    for t, h in ((3, 0), (77, 5), (149, 7), (200, 2)):
        rows[t, h] = True
    assert torch.isnan(out[:300][rows]).all()
    assert torch.equal(out[:300][~rows], good[0][:300][~rows]) and torch.equal(lse[:300][~rows], good[1][:300][~rows])


def test_rows_of_no_sequence_are_left_and_no_lse():
    c = Case([(37, 37), (5, 60)], 8, 2, seed=51, spare=70)
    out, lse = torch.full_like(c.q, 7.0), torch.full(c.q.shape[:2], 7.0, device="cuda")
    got = c.run(out=out, lse=lse)
    assert got[0] is out and (out[42:] == 7.0).all() and (lse[42:] == 7.0).all()
    c.check(out, lse)
    out2, none = c.run(want_lse=False)
    assert none is None and torch.equal(out2[:42], out[:42])
    # starts that leave rows before and between the sequences out
    c.starts, c.k_starts = _i32([2, 37, 42]), _i32([2, 37, 97])
    out.fill_(3.0)
    c.run(out=out)
    assert (out[:2] == 3.0).all() and (out[42:] == 3.0).all() and not (out[2:42] == 3.0).all()


@pytest.mark.parametrize("starts,k_starts,bad", [
    ([0, 50, 40, 110], None, [1]), ([0, -4, 60, 110], None, [0, 1]), ([0, 50, 60, 111], None, [2]), ([5, 50, 60, 110], None, []),
    ([0, 50, 60, 110], [0, 50, 60, 111], [2]), ([0, 50, 60, 110], [0, 50, 40, 110], [1]),
    ([0, 2 ** 31 - 1, 60, 110], None, [0, 1])])
def test_bad_starts_are_reported_and_left_out(starts, k_starts, bad):
    from kv_cache_computation_gb300 import MacError
    c = Case([(50, 50), (10, 10), (50, 50)], 8, 2, seed=61, spare=0)
    good = c.run()
    out = torch.full_like(c.q, 9.0)
    c.attend(c.q, c.k, c.v, _i32(starts), None if k_starts is None else _i32(k_starts), out=out)
    if bad:
        with pytest.raises(MacError, match="starts"):
            c.attend.sync()
    c.attend.sync()
    if 0 not in bad and starts[0] == 0:
        assert torch.equal(out[:40], good[0][:40])
    for b in (2,):
        if b not in bad and starts[2] == 60 and not k_starts:
            assert torch.equal(out[60:], good[0][60:])
        elif b in bad:
            assert (out[60:] == 9.0).all()


def test_starts_that_go_back_again_and_again():
    """Sequences that share nearly all their rows, between others that are left out: more tiles than the call's tokens can
    have.  Nothing is written, it is reported, and the next call is as ever."""
    from kv_cache_computation_gb300 import MacError, PromptAttention
    n, B = 1000, 201
    q, k, v = _randn((n, 8, 128), 5), _randn((n, 2, 128), 6), _randn((n, 2, 128), 7)
    attend = PromptAttention(8, 2, max_tokens=n, max_batch=B)
    out, lse = torch.full_like(q, 9.0), torch.full((n, 8), 9.0, device="cuda")
    attend(q, k, v, _i32([0, n] * 101), out=out, lse=lse)
    with pytest.raises(MacError, match="starts"):
        attend.sync()
    assert (out == 9.0).all() and (lse == 9.0).all()
    one = attend(q, k, v, _i32([0, n]))
    attend.sync()
    o, l, mag, top = _reference(q, k, v, 0, 128 ** -0.5)
    to, tl = _tolerance(o, mag, top, l, n, False)
    assert ((one[0].double() - o).abs() <= to).all() and ((one[1].double() - l).abs() <= tl).all()


def test_reproducible_captured_other_stream_and_shared_scratch():
    """Two runs agree bit for bit; a captured call serves other lengths, tokens and sequences when replayed; objects that
    share a scratch do not disturb one another."""
    from kv_cache_computation_gb300 import PromptAttention
    c = Case([(900, 900), (64, 3000), (0, 0), (333, 333)], 8, 2, seed=81, spare=200)
    a, b = c.run(), c.run()
    n = int(c.qs[-1])
    assert torch.equal(a[0][:n], b[0][:n]) and torch.equal(a[1][:n], b[1][:n])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    d = c.run(stream=s)
    other = PromptAttention(8, 2, max_tokens=5000, max_batch=4, share=c.attend)
    with torch.cuda.stream(s):
        e = other(c.q, c.k, c.v, c.starts, c.k_starts)
        f = c.run()
    s.synchronize()
    for x in (d, e, f):
        assert torch.equal(x[0][:n], a[0][:n]) and torch.equal(x[1][:n], a[1][:n])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out, lse = c.run()
    for seqs in ([(900, 900), (64, 3000), (0, 0), (333, 333)], [(1, 1), (0, 0), (1296, 4000), (3, 5)], [(5, 5)] * 4):
        c.seqs = seqs
        c.qs = np.concatenate(([0], np.cumsum([x for x, _ in seqs])))
        c.ks = np.concatenate(([0], np.cumsum([x for _, x in seqs])))
        c.starts.copy_(_i32(c.qs)), c.k_starts.copy_(_i32(c.ks))
        for t, z in ((c.q, c.qs[-1]), (c.k, c.ks[-1]), (c.v, c.ks[-1])):
            t[:] = _randn(tuple(t.shape), 7 + len(seqs))
            t[int(z):] = float("nan")
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, lse)
    c.attend.sync()


def test_refusals():
    from kv_cache_computation_gb300 import MacError, PromptAttention
    c = Case([(30, 30), (12, 12)], 8, 2, seed=91, spare=0)
    q, k, v, st = c.q, c.k, c.v, c.starts
    good = c.run()
    for args in ((q.float(), k, v, st), (q, k.cpu(), v, st), (q, k, v[:-1], st), (q, k, v, st.long()), (q, k, v, st.cpu()),
                 (q[..., :64], k, v, st), (q, k, v, st[:0]), (q[:-1], k, v, st), (q.transpose(0, 1), k, v, st)):
        with pytest.raises((TypeError, ValueError)):
            c.attend(*args)
    for kw in (dict(out=q.float()), dict(out_dtype=torch.float16), dict(lse=q), dict(k_starts=st[:-1]), dict(out=q[:-1])):
        with pytest.raises((TypeError, ValueError)):
            c.attend(q, k, v, st, **kw)
    with pytest.raises(MacError, match="query tokens"):
        c.attend(q.repeat(2, 1, 1), k, v, st, st)
    with pytest.raises(MacError, match="sequences"):
        c.attend(q, k, v, _i32([0, 1, 2, 3]))
    for lag in (-1, 2 ** 30 + 1):
        with pytest.raises(MacError):
            c.attend(q, k, v, st, lag=lag)
    with pytest.raises(MacError):                                   # tokens that do not start on 16 bytes
        wide = torch.zeros((42, 10 * 128 + 4), dtype=BF16).cuda()
        c.attend(wide[:, :1024], k, v, st)
    with pytest.raises(ValueError):
        PromptAttention(8, 2, max_tokens=1, share=object())
    for kw in (dict(heads=7), dict(heads=258, kv_heads=2), dict(max_tokens=0), dict(max_batch=1025), dict(head_dim=64),
               dict(sm_scale=-1.0)):
        with pytest.raises(MacError):
            PromptAttention(**{**dict(heads=8, kv_heads=2, max_tokens=8), **kw})
    out, lse = c.attend(q[:0], k[:0], v[:0], _i32([0]))             # nothing to do is no error
    assert out.shape == (0, 8, 128) and lse.shape == (0, 8)
    out, lse = c.attend(q, k[:0], v[:0], st, _i32([0, 0, 0]))       # queries without any key
    assert (out == 0).all() and torch.isneginf(lse).all()
    again = c.run()
    assert torch.equal(again[0], good[0])


def test_more_keys_than_levels():
    """Sequences of more blocks than the split has levels to order its items by, beside short ones."""
    c = Case([(40, 300001), (100, 100), (3, 262200), (1, 5), (70, 270000), (0, 9)], 4, 2, seed=77)
    c.check(*c.run())
    c.attend.sync()


@pytest.mark.parametrize("dtype,m,ramp", [(torch.float32, 32768, 0), (torch.float32, 32768, 2), (BF16, 81920, 0), (BF16, 81920, 2)])
def test_rows_over_many_keys_lose_nothing_to_the_order_of_sums(dtype, m, ramp):
    """The tensor cores cut sums off towards 0, which would add up over the hundreds of blocks that an item here has; the sums
    of runs of them are kept apart, and follow the reference where keys that grow (ramp) move it.  A run has 128 products
    of two weights (fp32 rows: 8 blocks) or 4096 (bf16: 512), each at most a step of 2^-23 of the sum, half on average: the
    outputs shrink by at most products 2^-24.  Beside that there are, at random, half a step of the weights (fp32 rows:
    2^-17, bf16: 2^-9), the scores' rounding (2^-21 in the exponent) and, of bf16 outputs, their own 2^-9."""
    from kv_cache_computation_gb300 import PromptAttention
    n, H = 5120, 8
    q, k, v = (_randn((t, H, 128), 300 + i).cuda() for i, t in enumerate((n, m, m)))
    k *= (1 + ramp * torch.arange(m).cuda() / m)[:, None, None].to(BF16)
    attend = PromptAttention(H, H, max_tokens=n)
    o, _ = attend(q, k, v, _i32([0, n]), _i32([0, m]), lag=64, out_dtype=dtype)
    rows = torch.arange(17, n, 640).cuda()
    s = torch.einsum("nhd,mhd->hnm", q[rows].double(), k.double()) / 128 ** 0.5
    seen = (m - n + 1 - 64 + rows)[:, None] > torch.arange(m).cuda()
    want = torch.einsum("hnm,mhd->nhd", s.masked_fill(~seen, float("-inf")).softmax(-1), v.double())
    off = o[rows].double() - want
    shrinks, own = (128 * 2 ** -24, 2 ** -17) if dtype == torch.float32 else (4096 * 2 ** -24, 2 ** -9 + 2 ** -9)
    # A weight's rounding is one for all 128 elements of its row, so where one key has most of the weight the random parts
    # are 64 numbers, one per row and head, within +-own: their mean has a deviation of own / 3^0.5 / 64^0.5 = own / 13.9,
    # and own / 4 is 3.5 of those.
    assert ((off * want).sum() / (want * want).sum()).abs() <= shrinks + own / 4
    assert off.norm() / want.norm() <= shrinks + own + 2 ** -20
    attend.sync()


@pytest.mark.parametrize("dtype,off", [(BF16, 8), (torch.float32, 4), (torch.float32, 12)])
def test_refuses_outputs_off_their_32_bytes(dtype, off):
    """The rows are stored 32 bytes at a time: an out of the caller's that starts elsewhere is refused on the host."""
    from kv_cache_computation_gb300 import MacError
    c = Case([(30, 30), (12, 12)], 8, 2, seed=92, spare=0)
    good = c.attend(c.q, c.k, c.v, c.starts, out_dtype=dtype)[0]
    buf = torch.zeros(good.numel() + 64, dtype=dtype).cuda()
    at = -buf.data_ptr() % 32 // buf.element_size()
    with pytest.raises(MacError):
        c.attend(c.q, c.k, c.v, c.starts, out=buf[at + off:at + off + good.numel()].view(good.shape), out_dtype=dtype)
    torch.cuda.synchronize()
    assert (buf == 0).all()
    at += 32 // buf.element_size()
    out = c.attend(c.q, c.k, c.v, c.starts, out=buf[at:at + good.numel()].view(good.shape), out_dtype=dtype)[0]
    assert torch.equal(out, good)


def test_offsets_beyond_32_bits():
    """Queries, keys and outputs whose byte and element offsets pass 2^32."""
    from kv_cache_computation_gb300 import PromptAttention
    n, far = 200, 600000
    wide = torch.zeros((far + n, 4096), dtype=BF16, device="cuda")        # 2.4e9 elements, 4.9e9 bytes
    wide[far:] = _randn((n, 4096), 3)
    q, k, v = wide[:, :2048], wide[:, 2048:2048 + 1024], wide[:, 2048 + 1024:]
    attend = PromptAttention(16, 8, max_tokens=far + n)
    out = torch.zeros((far + n, 16, 128), dtype=F32, device="cuda")
    attend(q, k, v, _i32([far, far + n]), out=out, out_dtype=F32)
    dense = PromptAttention(16, 8, max_tokens=n)(q[far:].contiguous(), k[far:].contiguous(), v[far:].contiguous(), _i32([0, n]),
                                                 out_dtype=F32)[0]
    attend.sync()
    assert torch.equal(out[far:], dense) and (out[:far] == 0).all() and (dense != 0).any()

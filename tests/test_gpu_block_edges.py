"""Attention over the 8-bit store where it can go wrong beside what
test_gpu_block_kv.py covers: value scales at the two ends of their range in one
request, and far apart beside scores that fp32 holds as whole numbers.  Tolerances: block_reference.attention_tolerance."""
import numpy as np
import pytest
import torch

import block_reference as BR
from test_gpu_block_kv import Case, _i32, _np
from test_gpu_serving_ops import BF16

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("H,nq", [(4, 1), (12, 1), (20, 1), (32, 1), (7, 3)])
@pytest.mark.parametrize("n,at", [(40, 3), (200, 0), (200, 199), (3000, 0), (3000, 1500), (3000, 2990), (60000, 0),
                                  (60000, 31234), (60000, 59990)])
def test_small_values_keep_their_weight_beside_a_huge_one(n, at, H, nq):
    """One token, whose values have the largest scale, leads every other's score by 16 to 24 log2 units; the others' values
    have the smallest.  Together those take up to two fifths of the weight, although each one's product with its value scale is
    2^-136 and less of the first one's."""
    from kv_cache_computation_gb300 import BlockKV
    r = np.random.default_rng(n + at)
    pages = -(-n // 16)
    d = np.sign(r.standard_normal(128))
    k, v = np.zeros((n, 1, 128)), r.standard_normal((n, 1, 128)) * 2.0 ** -56
    k[at, 0], v[at, 0] = d, (1 + 0.5 * r.random(128)) * 2.0 ** 68
    k, v = torch.from_numpy(k).to(BF16), torch.from_numpy(v).to(BF16)
    stored, ev = np.zeros((n, 1, 128)), np.zeros((n, 1), int)
    x = _np(v)
    for p in range(0, n, 16):
        ev[p:p + 16] = e = BR.need(x[p:p + 16])
        stored[p:p + 16] = BR.e4m3(x[p:p + 16] / 2.0 ** e) * 2.0 ** e
    assert set(ev.ravel()) == ({-60, 60} if n > 16 else {60})
    q = torch.from_numpy((1 + 0.5 * np.arange(H) / H)[None, None, :, None] * d * np.ones((1, nq, 1, 1))).to(BF16)
    perm = r.permutation(pages)
    cache = BlockKV(H, 1, num_pages=pages, max_query=nq)
    t = np.arange(n)
    cache.append(k.cuda(), v.cuda(), _i32(perm[t // 16] * 16 + t % 16))
    out, lse = cache.attention(q.cuda(), _i32(perm[None]), _i32([n]))
    o, l, mag, top = BR.attention(_np(q[0]), _np(k), stored, ev, 1 / np.sqrt(128))
    to, tl = BR.attention_tolerance(o, mag, top, l, n)
    assert (np.abs(_np(lse[0]) - l) <= tl).all(), (np.abs(_np(lse[0]) - l) - tl).max()
    assert (np.abs(_np(out[0]) - o) <= to).all()
    cache.sync()


@pytest.mark.parametrize("spread,qscale", [(20.0, 2.0 ** -40), (20.0, 2.0 ** -34), (15.0, 2.0 ** -20), (20.0, 2.0 ** -10),
                                           (8.0, 2.0 ** 4), (8.0, 2.0 ** 60)])
@pytest.mark.parametrize("H,nq,n", [(4, 1, 78), (16, 1, 78), (20, 1, 78), (32, 1, 78), (4, 1, 9000), (32, 1, 3000), (7, 3, 3000)])
def test_scores_beyond_the_significand_and_values_of_any_scale(H, nq, n, spread, qscale):
    """Scores up to 2^100 over values whose scales differ by up to 2^120.  Every output is a mean of the values that its row
    sees, the lse its largest score to the scores' own error, and a row whose largest score is further ahead than both
    scores' errors, 120 for the scales and 64 more (log2) gives that token's value."""
    lens = [n] * (20 if n < 100 else 1) + [5]
    c = Case(lens, H, 1, nq, seed=19, qscale=qscale, spread=spread)
    out, lse = c.run()
    c.cache.sync()
    clear = 0
    for b in range(len(lens)):
        k, v = c.k[b][:, 0], c.v[b][:, 0]
        for i in range(nq):
            seen = lens[b] - (nq - 1) + i
            s = (k[:seen] @ _np(c.q[b, i]).T) * c.scale                                # [tokens, heads]
            err = 14 * 2.0 ** -23 * (np.abs(k[:seen]) @ np.abs(_np(c.q[b, i])).T).max(0) * c.scale
            go, gl = _np(out[b].reshape(nq, H, 128)[i]), _np(lse[b].reshape(nq, H)[i])
            assert np.isfinite(go).all() and np.isfinite(gl).all()
            # weights are rounded to f16 (2^-11 each), outputs to bf16 (2^-8)
            assert (np.abs(go) <= np.abs(v[:seen]).max(0) * (1 + 2.0 ** -7)).all()
            order = np.sort(s, axis=0)
            assert (np.abs(gl - order[-1]) <= err + 2.0 ** -20 * np.abs(gl) + np.log(seen) + 1e-4).all()
            lead = order[-1] - order[-2] > 2 * err + 184 * np.log(2)
            want = v[s.argmax(0)]
            assert (np.abs(go - want) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(want) + 1e-30)[lead].all()
            clear += lead.sum()
    assert clear > 0

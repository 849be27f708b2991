"""Attention over the 8-bit store where it can go wrong beside what
test_gpu_block_kv.py covers: value scales at the two ends of their range in one
request.  Tolerances: block_reference.attention_tolerance."""
import numpy as np
import pytest
import torch

import block_reference as BR
from test_gpu_block_kv import _i32, _np
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

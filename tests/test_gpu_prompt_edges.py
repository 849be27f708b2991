"""Prompt attention where it can go wrong beside what test_gpu_prompt.py covers:
infinities wherever they stand, rows whose every score is minus infinity, large
groups with many items, many short prompts."""
import pytest
import torch

from test_gpu_prompt import BF16, F32, Case, _i32, _randn

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("H,Hkv,m", [(8, 2, 1500), (28, 4, 900), (4, 1, 9000)])
def test_an_infinite_value_gives_nan_wherever_it_stands(H, Hkv, m, wide):
    """Rows that see it have NaN in its element, whether it stands on an edge of theirs or far before, and however the
    prompt is cut into chunks; all other elements are what they are without it."""
    from kv_cache_computation_gb300 import PromptAttention
    q, k, v = _randn((m, H, 128), 1), _randn((m, Hkv, 128), 2), _randn((m, Hkv, 128), 3)
    attend = PromptAttention(H, Hkv, max_tokens=m)
    dtype = F32 if wide else BF16

    def chunks(cuts):
        out = []
        for a, b in zip(cuts, cuts[1:]):
            out.append(attend(q[a:b], k[:b], v[:b], _i32([0, b - a]), _i32([0, b]), out_dtype=dtype)[0])
        attend.sync()
        return torch.cat(out)
    sets = ([0, m], [0, 1, 130, m // 2, m - 1, m], [0, m - 300, m])
    clean = [chunks(c) for c in sets]
    bad = torch.zeros((m, H, 128), dtype=torch.bool, device="cuda")
    G = H // Hkv
    for t, h, d, x in ((0, 0, 3, "inf"), (m // 3, Hkv - 1, 127, "-inf"), (m // 2, 0, 64, "inf"), (m // 2 + 70, 0, 64, "-inf"),
                       (m - 200, 0, 9, "inf"), (m - 2, Hkv - 1, 40, "-inf"), (m - 1, 0, 41, "inf")):
        v[t, h, d] = float(x)
        bad[t:, h * G:(h + 1) * G, d] = True
    for c, want in zip(sets, clean):
        got = chunks(c)
        assert torch.equal(torch.isnan(got), bad) and not torch.isinf(got).any()
        assert torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("H,Hkv,seqs,lag", [(8, 2, [(1, 1), (40, 40), (7, 300)], 0), (28, 4, [(130, 400), (9, 9)], 3),
                                            (4, 1, [(5, 9000), (3, 3)], 0), (32, 8, [(600, 2000), (40, 40)], 64)])
def test_scores_of_minus_infinity_alone_are_no_empty_row(H, Hkv, seqs, lag, wide):
    """A query with an infinity whose scores are all minus infinity: 0 / 0, which is NaN and not the output 0, lse -inf of a
    row that sees nothing.  So is one that sees an infinite key alone.  Rows that see nothing stay as they are."""
    c = Case(seqs, H, Hkv, lag=lag, seed=7, wide=wide)
    G = H // Hkv
    c.k[:, :, 5] = c.k[:, :, 5].abs() + 0.5
    clean, clse = c.run()
    rows = torch.zeros(int(c.qs[-1]), H, dtype=torch.bool, device="cuda")
    empty = torch.zeros_like(rows)
    for b, (n, m) in enumerate(seqs):
        for i in {0, n // 2, n - 1}:
            c.q[int(c.qs[b]) + i, (b + i) % H, 5] = float("-inf")
            rows[int(c.qs[b]) + i, (b + i) % H] = True
        for i in range(n):
            if m - n + i + 1 - lag <= 0:
                empty[int(c.qs[b]) + i] = True
    out, lse = c.run()
    c.attend.sync()
    n = int(c.qs[-1])
    out, lse, clean, clse = out[:n], lse[:n], clean[:n], clse[:n]
    assert torch.isnan(out[rows & ~empty]).all() and torch.isnan(lse[rows & ~empty]).all()
    assert (out[empty] == 0).all() and torch.isneginf(lse[empty]).all()
    good = ~rows & ~empty
    assert torch.equal(out[good], clean[good]) and torch.equal(lse[good], clse[good])
    # a key: the query that sees it alone
    if lag == 0 and seqs[0] == (1, 1):
        c = Case(seqs, H, Hkv, seed=8, wide=wide)
        c.q[0, :, 9] = c.q[0, :, 9].abs() + 0.5
        c.k[0, Hkv - 1, 9] = float("-inf")
        out, lse = c.run()
        assert torch.isnan(out[0, -G:]).all() and torch.isnan(lse[0, -G:]).all()
        assert torch.isfinite(out[0, :-G]).all()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("H,Hkv,seqs", [(32, 1, [(1500, 1500), (3, 700)]), (33, 1, [(900, 1200)]), (64, 1, [(700, 700)] * 2),
                                        (100, 1, [(800, 800), (1, 1)]), (128, 1, [(500, 3000)]), (256, 2, [(400, 900), (33, 33)])])
def test_many_items_of_large_groups(H, Hkv, seqs, wide):
    """Tiles of 4 tokens down to one: whole items, the line that is cut and its merge together."""
    c = Case(seqs, H, Hkv, seed=H, wide=wide)
    c.check(*c.run())
    c.attend.sync()


@pytest.mark.parametrize("H,Hkv,lens", [(32, 8, [16] * 1024), (8, 2, [16] * 300), (8, 2, [64] * 256), (28, 4, [70] * 100),
                                        (16, 1, list(range(1, 140)))])
def test_many_short_prompts(H, Hkv, lens):
    c = Case([(n, n) for n in lens], H, Hkv, seed=len(lens))
    out, lse = c.run()
    step = max(1, len(lens) // 40)
    c.check(out, lse, only=sorted(set(range(0, len(lens), step)) | {len(lens) - 1}))
    n = int(c.qs[-1])
    assert torch.isfinite(out[:n]).all() and torch.isfinite(lse[:n]).all()
    c.attend.sync()

"""Prompt attention where it can go wrong beside what test_gpu_prompt.py covers:
infinities wherever they stand."""
import pytest
import torch

from test_gpu_prompt import BF16, F32, _i32, _randn

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

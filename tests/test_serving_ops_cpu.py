"""The operators around the decode step on a machine without a GPU: refusals of
bad arguments (none of these calls reaches CUDA), sizes, the rotation's table,
and the reference's own formats against torch."""
import ctypes
import math

import numpy as np
import pytest
import torch

import serving_reference as R

P = ctypes.c_void_p(0x10000)          # an aligned address that is never dereferenced
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def native():
    from kv_cache_computation_gb300 import build
    build.build()
    from kv_cache_computation_gb300 import _native
    return _native


def _rope(native, **kw):
    base = dict(heads=32, kv_heads=8, head_dim=128, rotary_dim=128, interleaved=0, eps=1e-6, rope_base=500000.0)
    base.update(kw)
    cfg, out = native.MacRopeConfig(**base), native.MacRope()
    return native.lib().mac_rope_init(ctypes.byref(cfg), ctypes.byref(out)), out


def test_rope_table_holds_turns_per_position(native):
    st, rope = _rope(native, rotary_dim=96, rope_base=10000.0)
    assert st == 0
    for i in range(64):
        want = 10000.0 ** (-2 * i / 96) / (2 * math.pi) if i < 48 else 0.0
        # a double quotient (2^-53, and the power's own 2^-53), rounded to a multiple of 2^-64
        assert abs(rope.turns[i] / 2.0 ** 64 - want) <= 2.0 ** -52 * want + 2.0 ** -65


@pytest.mark.parametrize("bad", [dict(heads=0), dict(heads=30), dict(kv_heads=0), dict(heads=1032), dict(head_dim=64),
                                 dict(rotary_dim=-8), dict(rotary_dim=12), dict(rotary_dim=136), dict(interleaved=2),
                                 dict(eps=-1.0), dict(eps=float("nan")), dict(rope_base=0.5),
                                 dict(rope_base=float("inf"))])
def test_rope_config_refusals(native, bad):
    assert _rope(native, **bad)[0] == -1


def test_norm_rope_refusals(native):
    L = native.lib()
    st, rope = _rope(native)
    good = dict(rope=ctypes.byref(rope), n=1, q=P, qs=4096, k=P, ks=1024, v=P, vs=1024, wq=P, wk=P, pos=P, q_pre=P,
                q_post=P, k_out=P, v_out=P, stream=None)

    def call(**kw):
        return L.mac_qkv_norm_rope(*{**good, **kw}.values())
    for kw in (dict(rope=None), dict(n=-1), dict(q=None), dict(k=None), dict(pos=None), dict(q_post=None),
               dict(k_out=None), dict(v=None), dict(v_out=None), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(wq=ODD),
               dict(wk=ODD), dict(q_pre=ODD), dict(q_post=ODD), dict(k_out=ODD), dict(v_out=ODD),
               dict(pos=ctypes.c_void_p(0x10002)), dict(qs=4095), dict(qs=4100), dict(ks=1016), dict(vs=1020)):
        assert call(**kw) == -1, kw
    assert call(n=0) == 0
    assert L.mac_qkv_norm_rope(ctypes.byref(native.MacRope()), *list(good.values())[1:]) == -1   # never initialised


def test_page_step_refusals(native):
    L = native.lib()
    good = dict(batch=2, tokens=2, pages=8, len_in=P, new=P, len_out=P, table=P, stride=4, cols=4, ring=P, state_in=P,
                state_out=P, starts=P, pos=P, slot=P, status=P, stream=None)
    bad = [dict(batch=0), dict(batch=1025), dict(tokens=0), dict(tokens=(1 << 30) + 1), dict(pages=0),
           dict(pages=1 << 27), dict(cols=0), dict(stride=3), dict(cols=(1 << 26) + 1, stride=1 << 28),
           dict(batch=1024, cols=1 << 21, stride=1 << 21)]
    for name in ("len_in", "new", "len_out", "table", "ring", "state_in", "state_out", "starts", "pos", "slot", "status"):
        bad += [{name: None}, {name: ctypes.c_void_p(0x10002)}]
    for kw in bad:
        assert L.mac_page_step(*{**good, **kw}.values()) == -1, kw


def _quant(native, **kw):
    base = dict(heads=32, kv_heads=8, head_dim=128, page_size=16, num_pages=10, max_batch=4, max_query=2, sm_scale=0.0,
                k_scale=1.0, v_scale=1.0)
    base.update(kw)
    cfg, a, b = native.MacQuantConfig(**base), ctypes.c_size_t(), ctypes.c_size_t()
    return native.lib().mac_quant_query_sizes(ctypes.byref(cfg), ctypes.byref(a), ctypes.byref(b)), a.value, b.value, cfg


def test_quant_store_is_144_bytes_a_token(native):
    st, store, scratch, _ = _quant(native, num_pages=131072 // 16)
    assert st == 0 and store == 131072 * 8 * 144 and scratch > 0


@pytest.mark.parametrize("bad", [dict(heads=0), dict(heads=30), dict(head_dim=64), dict(page_size=32), dict(num_pages=0),
                                 dict(num_pages=1 << 27), dict(max_batch=0), dict(max_batch=1025), dict(max_query=0),
                                 dict(max_query=9), dict(heads=33, kv_heads=1, max_query=1), dict(sm_scale=-1.0),
                                 dict(sm_scale=float("nan")), dict(k_scale=0.0), dict(k_scale=3.0), dict(v_scale=-2.0),
                                 dict(v_scale=float("inf")), dict(k_scale=2.0 ** 60), dict(k_scale=2.0 ** -61)])
def test_quant_config_refusals(native, bad):
    assert _quant(native, **bad)[0] == -1


def test_quant_create_and_null_handles(native):
    L = native.lib()
    st, store, scratch, cfg = _quant(native)
    h = ctypes.c_void_p()
    assert L.mac_quant_create(ctypes.byref(cfg), P, store, P, scratch, None) == -1
    assert L.mac_quant_create(ctypes.byref(cfg), None, store, P, scratch, ctypes.byref(h)) == -1
    assert L.mac_quant_create(ctypes.byref(cfg), P, store, None, scratch, ctypes.byref(h)) == -1
    assert L.mac_quant_create(ctypes.byref(cfg), ODD, store, P, scratch, ctypes.byref(h)) == -2
    assert L.mac_quant_create(ctypes.byref(cfg), P, store - 1, P, scratch, ctypes.byref(h)) == -2
    assert L.mac_quant_create(ctypes.byref(cfg), P, store, P, scratch - 1, ctypes.byref(h)) == -2
    assert L.mac_quant_append(None, 1, P, 1024, P, 1024, P, None) == -1
    assert L.mac_quant_gather(None, 1, P, P, P, None) == -1
    assert L.mac_quant_attention(None, 1, 1, P, P, 1, 1, P, P, None, None) == -1
    assert L.mac_quant_sync(None) == -1 and L.mac_quant_destroy(None) == -1
    assert L.mac_quant_last_error(None) == b""


def test_bindings_refuse_cpu_tensors(native):
    from kv_cache_computation_gb300 import QkvRotary, page_step
    rot = QkvRotary(4, 2)
    with pytest.raises(TypeError, match="CUDA"):
        rot(torch.zeros(1, 8 * 128, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32))
    z = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError, match="CUDA"):
        page_step(z, z, torch.zeros(2, 4, dtype=torch.int32), z, z, max_tokens=2)


def test_reference_formats_against_torch():
    """The reference's grids are the formats': e4m3 against torch's, e2m1 by its seven steps."""
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(R.E4M3, codes)
    x = np.random.default_rng(1).uniform(0, 460, 4000)
    x[::7] = (R.E4M3[:-1] + R.E4M3[1:])[np.arange(len(x[::7])) % 126] / 2          # ties
    want = torch.from_numpy(np.minimum(x, 448.0)).float().to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(R.E4M3[R._nearest_even(x.astype(np.float32).astype(np.float64), R.E4M3)], want)
    ties = {0.25: 0.0, 0.75: 1.0, 1.25: 1.0, 1.75: 2.0, 2.5: 2.0, 3.5: 4.0, 5.0: 4.0, 7.0: 6.0, 100.0: 6.0}
    for a, b in ties.items():
        assert R.E2M1[R._nearest_even(np.array([a]), R.E2M1)][0] == b


def test_store_layout_covers_a_page_once():
    """Where append puts each element of a page (the layout that the kernels share): every nibble of the code areas
    and every scale byte is written by exactly one (token, element), and the attention kernel's fragment index of that
    place names the same token and element."""
    nib, scale = {}, {}
    for tok in range(16):
        for e in range(128):
            j, c, tt = e // 16, tok // 4, tok % 4
            nib.setdefault(2 * (tok * 64 + e // 2) + e % 2, []).append(("k", tok, e))
            i = e % 16 // 2
            byte = 1152 + (i // 4) * 512 + (j * 4 + c) * 16 + tt * 4 + i % 4
            nib.setdefault(2 * byte + e % 2, []).append(("v", tok, e))
            scale.setdefault(1024 + c * 32 + j * 4 + tt, set()).add(("k", tok, j))
            scale.setdefault(2176 + c * 32 + j * 4 + (0, 2, 1, 3)[tt], set()).add(("v", tok, j))
    assert all(len(x) == 1 for x in nib.values()) and all(len(x) == 1 for x in scale.values())
    assert sorted(nib) == list(range(0, 2 * 1024)) + list(range(2 * 1152, 2 * 2176))
    assert sorted(scale) == list(range(1024, 1152)) + list(range(2176, 2304))
    for lane in range(32):
        g, c = lane // 4, lane % 4
        tk = 4 * (g >> 1) + (g & 1)
        for h in range(2):                                       # K scale bytes of the lane's two blocks
            at = 1024 + (g >> 1) * 32 + (2 * c + h) * 4 + (g & 1)
            assert scale[at] == {("k", tk, 2 * c + h)} and scale[at + 2] == {("k", tk + 2, 2 * c + h)}
        for row, tok in ((g, tk), (g + 8, tk + 2)):
            # matrix rows {2c, 2c+1, 2c+8, 2c+9} are tokens 4c .. 4c+3
            assert tok == 4 * (row % 8 // 2) + row % 2 + (2 if row >= 8 else 0)
            for i in range(16):                                  # the thread's 16 K bytes of that token
                for h in range(2):
                    assert nib[2 * (tok * 64 + c * 16 + i) + h] == [("k", tok, 32 * c + 2 * i + h)]
        for w in range(2):
            for tt in range(4):
                for i in range(4):                               # V word tt of load w, byte i: elements of block g
                    for h in range(2):
                        at = 1152 + w * 512 + lane * 16 + tt * 4 + i
                        assert nib[2 * at + h] == [("v", 4 * c + tt, 16 * g + 8 * w + 2 * i + h)]
        # the word of value scales that the lane loads: its block, its four tokens in the order 0, 2, 1, 3
        for k, tt in enumerate((0, 2, 1, 3)):
            assert scale[2176 + c * 32 + g * 4 + k] == {("v", 4 * c + tt, g)}

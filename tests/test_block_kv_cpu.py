"""The 8-bit store on a machine without a GPU: refusals (none of these calls
reaches CUDA), sizes, the layout, and the reference's own format."""
import ctypes

import numpy as np
import pytest
import torch

import block_reference as BR

P = ctypes.c_void_p(0x10000)          # an aligned address that is never dereferenced
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def native():
    from kv_cache_computation_gb300 import build
    build.build()
    from kv_cache_computation_gb300 import _native
    return _native


def _block(native, **kw):
    base = dict(heads=32, kv_heads=8, head_dim=128, page_size=16, num_pages=10, max_batch=4, max_query=2, sm_scale=0.0)
    base.update(kw)
    cfg, a, b = native.MacBlockConfig(**base), ctypes.c_size_t(), ctypes.c_size_t()
    return native.lib().mac_block_query_sizes(ctypes.byref(cfg), ctypes.byref(a), ctypes.byref(b)), a.value, b.value, cfg


def test_store_is_258_bytes_a_token(native):
    st, store, scratch, _ = _block(native, num_pages=131072 // 16)
    assert st == 0 and store == 131072 * 8 * 258
    more = _block(native, num_pages=131072 // 8)[2]
    assert more - scratch == 131072 // 16 * 68


@pytest.mark.parametrize("bad", [dict(heads=0), dict(heads=30), dict(kv_heads=0), dict(head_dim=64), dict(page_size=32),
                                 dict(num_pages=0), dict(num_pages=1 << 27), dict(max_batch=0), dict(max_batch=1025),
                                 dict(max_query=0), dict(max_query=9), dict(heads=33, kv_heads=1, max_query=1),
                                 dict(heads=8192, kv_heads=4096, max_query=1), dict(sm_scale=-1.0),
                                 dict(sm_scale=float("nan")), dict(sm_scale=float("inf"))])
def test_config_refusals(native, bad):
    assert _block(native, **bad)[0] == -1


def test_create_and_null_handles(native):
    L = native.lib()
    st, store, scratch, cfg = _block(native)
    h = ctypes.c_void_p()
    assert L.mac_block_create(ctypes.byref(cfg), P, store, P, scratch, None) == -1
    assert L.mac_block_create(None, P, store, P, scratch, ctypes.byref(h)) == -1
    assert L.mac_block_create(ctypes.byref(cfg), None, store, P, scratch, ctypes.byref(h)) == -1
    assert L.mac_block_create(ctypes.byref(cfg), P, store, None, scratch, ctypes.byref(h)) == -1
    assert L.mac_block_create(ctypes.byref(cfg), ODD, store, P, scratch, ctypes.byref(h)) == -2
    assert L.mac_block_create(ctypes.byref(cfg), P, store - 1, P, scratch, ctypes.byref(h)) == -2
    assert L.mac_block_create(ctypes.byref(cfg), P, store, P, scratch - 1, ctypes.byref(h)) == -2
    assert L.mac_block_append(None, 1, P, 1024, P, 1024, P, None) == -1
    assert L.mac_block_gather(None, 1, P, P, P, None) == -1
    assert L.mac_block_attention(None, 1, 1, P, P, 1, 1, P, P, None, None) == -1
    assert L.mac_block_step_rows(None, 1, 1, 1, P, P, P, P, 1, 1, P, P, P, P, None) == -1
    assert L.mac_block_sync(None) == -1 and L.mac_block_destroy(None) == -1
    assert L.mac_block_last_error(None) == b""


def test_layout_covers_a_page_once():
    """Every code byte of a page belongs to one (token, element), and the attention kernel's lanes find it there."""
    place = {}
    for tok in range(16):
        for e in range(128):
            line = e // 4                                    # the writer's lane
            k = (((tok >> 1 & 1) * 2 + (line >> 2 & 1)) * 512 + ((2 * (tok >> 2) + (tok & 1)) * 4 + (line >> 3)) * 16
                 + (line & 3) * 4 + e % 4)
            v = 2048 + (line & 3) * 512 + ((line >> 2) * 4 + tok // 4) * 16 + 4 * (e % 4) + tok % 4
            place.setdefault(k, []).append(("k", tok, e))
            place.setdefault(v, []).append(("v", tok, e))
    assert sorted(place) == list(range(4096)) and all(len(x) == 1 for x in place.values())
    for lane in range(32):
        g, c = lane // 4, lane % 4
        tk = 4 * (g >> 1) + (g & 1)
        for r in range(2):
            for i in range(2):
                for b in range(16):                          # K: rows g and g + 8 are tokens tk and tk + 2
                    assert place[(r * 2 + i) * 512 + lane * 16 + b] == [("k", tk + 2 * r, 32 * c + 16 * i + b)]
        for i in range(4):
            for b in range(16):                              # V: byte 4 (element) + token of the quad
                assert place[2048 + i * 512 + lane * 16 + b] == [("v", 4 * c + b % 4, 16 * g + 4 * i + b // 4)]


def test_reference_format():
    """The reference's e4m3 against torch's, and its exponents at the borders."""
    x = np.random.default_rng(1).uniform(-447, 447, 5000) * 2.0 ** np.random.default_rng(2).integers(-12, 1, 5000)
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(BR.e4m3(x.astype(np.float32).astype(np.float64)), want)
    assert np.isnan(BR.e4m3(np.array([np.inf, -np.inf, np.nan]))).all() and BR.e4m3(np.array([500.0]))[0] == 448.0
    for top, e in ((448.0, 0), (449.0, 1), (224.0, -1), (225.0, 0), (0.0, -60), (1e30, 60), (np.inf, -60), (7.0, -6)):
        assert BR.need(np.array([top, -top / 3])) == e or (not np.isfinite(top) and BR.need(np.array([top])) == e)

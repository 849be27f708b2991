"""Prompt attention on a machine without a GPU: refusals (none of these calls
reaches CUDA) and sizes."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p(0x10000)          # an aligned address that is never dereferenced
ODD = ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def native():
    from kv_cache_computation_gb300 import build
    build.build()
    from kv_cache_computation_gb300 import _native
    return _native


def _prompt(native, **kw):
    base = dict(heads=32, kv_heads=8, head_dim=128, max_tokens=4096, max_batch=4, sm_scale=0.0)
    base.update(kw)
    cfg, a = native.MacPromptConfig(**base), ctypes.c_size_t()
    return native.lib().mac_prompt_query_sizes(ctypes.byref(cfg), ctypes.byref(a)), a.value, cfg


@pytest.mark.parametrize("bad", [dict(heads=0), dict(heads=30), dict(kv_heads=0), dict(head_dim=64), dict(max_tokens=0),
                                 dict(max_tokens=(1 << 24) + 1), dict(max_batch=0), dict(max_batch=1025),
                                 dict(heads=129, kv_heads=1), dict(heads=4104, kv_heads=8), dict(sm_scale=-1.0),
                                 dict(sm_scale=float("nan")), dict(sm_scale=float("inf"))])
def test_config_refusals(native, bad):
    assert _prompt(native, **bad)[0] == -1


def test_create_and_null_handles(native):
    L = native.lib()
    st, scratch, cfg = _prompt(native)
    assert st == 0 and scratch > 0
    h = ctypes.c_void_p()
    assert L.mac_prompt_create(ctypes.byref(cfg), P, scratch, None) == -1
    assert L.mac_prompt_create(None, P, scratch, ctypes.byref(h)) == -1
    assert L.mac_prompt_create(ctypes.byref(cfg), None, scratch, ctypes.byref(h)) == -1
    assert L.mac_prompt_create(ctypes.byref(cfg), ODD, scratch, ctypes.byref(h)) == -2
    assert L.mac_prompt_create(ctypes.byref(cfg), P, scratch - 1, ctypes.byref(h)) == -2
    assert L.mac_prompt_attention(None, 1, 1, 1, 0, P, 4096, P, 1024, P, 1024, P, None, P, 0, None, None) == -1
    assert L.mac_prompt_sync(None) == -1 and L.mac_prompt_destroy(None) == -1
    assert L.mac_prompt_last_error(None) == b""


def test_bindings_refuse_cpu_tensors(native):
    from kv_cache_computation_gb300.rotary import _rows
    with pytest.raises(TypeError, match="CUDA"):
        _rows(torch.zeros(1, 4, 128, dtype=torch.bfloat16), "q", 4, 128)

"""Refusals of the later entry points around the decode step on a machine
without a GPU (none of these calls reaches CUDA)."""
import ctypes

import pytest

P = ctypes.c_void_p(0x10000)          # an aligned address that is never dereferenced
ODD = ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def native():
    from kv_cache_computation_gb300 import build
    build.build()
    from kv_cache_computation_gb300 import _native
    return _native


def test_page_step_ex_refusals(native):
    L = native.lib()
    good = dict(batch=2, tokens=2, pages=8, len_in=P, new=P, len_out=P, table=P, stride=4, cols=4, ring=P, state_in=P,
                state_out=P, starts=P, pos=P, slot=P, status=P, rejected=None,
                unreleased=None, stream=None)
    bad = [dict(batch=0), dict(batch=1025), dict(tokens=0), dict(tokens=(1 << 30) + 1), dict(pages=0), dict(pages=1 << 27),
           dict(cols=0), dict(stride=3), dict(batch=1024, cols=1 << 21, stride=1 << 21), dict(unreleased=ODD),
           dict(rejected=ODD)]
    for name in ("len_in", "new", "len_out", "table", "ring", "state_in", "state_out", "starts", "pos", "slot", "status"):
        bad += [{name: None}, {name: ODD}]
    for kw in bad:
        assert L.mac_page_step_ex(*{**good, **kw}.values()) == -1, kw


def test_step_rows_refuses_a_null_handle(native):
    assert native.lib().mac_quant_step_rows(None, 1, 1, 1, P, P, P, P, 1, 1, P, P, P, P, None) == -1

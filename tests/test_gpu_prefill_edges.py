"""MacAttention.prefill: what it refuses leaves the request as it was; scales that
are the same; another stream."""
import numpy as np
import pytest
import torch

from test_gpu_prefill import _mac
from test_gpu_prompt import BF16, _randn

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

H, Hkv = 8, 2


def _inputs(n, seed=1):
    return (_randn((n, H, 128), seed), _randn((n, H, 128), seed + 1), _randn((n, Hkv, 128), seed + 2),
            _randn((n, Hkv, 128), seed + 3))


def _off(t):
    """The same tensor 8 bytes off its 16."""
    buf = torch.zeros(t.numel() + 4, dtype=BF16, device="cuda")
    out = buf[4:].view(t.shape)
    out.copy_(t)
    assert out.is_contiguous() and out.data_ptr() % 16 == 8
    return out


@pytest.mark.parametrize("page", [0, 16])
def test_what_prefill_refuses_leaves_the_request_as_it_was(page):
    from kv_cache_computation_gb300 import MacError, PromptAttention
    mac = _mac(H, Hkv, max_ctx=64, page_size=page) if page == 0 else _mac(H, Hkv)
    if page:
        mac.reset_request(0)
        mac.set_page_table(0, torch.tensor([9, 4, 7, 1], dtype=torch.int32).cuda())       # 64 tokens
    prompt = PromptAttention(H, Hkv, max_tokens=100)
    mac.prefill(prompt, 0, *_inputs(20))
    before = mac.read_ring(0)
    assert before["kv_len"] == 20 and before["steps"] == 16

    def refused(err, *args, use=prompt, req=0):
        with pytest.raises(err):
            mac.prefill(use, req, *args)
        now = mac.read_ring(0)
        for key, x in before.items():
            assert np.array_equal(now[key], x), key
    x = _inputs(65, 11)
    refused(MacError, *x)                                            # one token more than the request may hold
    for i in range(4):                                               # tensors that do not start on 16 bytes
        y = list(_inputs(30, 21))
        y[i] = _off(y[i])
        refused(ValueError, *y)
    for req in (-1, 2):
        refused(MacError, *_inputs(30, 31), req=req)
    closed = PromptAttention(H, Hkv, max_tokens=100)
    closed.close()
    refused(MacError, *_inputs(30, 41), use=closed)
    # the request goes on as one that met no refusal
    other = _mac(H, Hkv)
    other.prefill(prompt, 0, *_inputs(20))
    step = _inputs(1, 51)
    a, b = mac.decode_step(*step), other.decode_step(*step)
    mac.sync(), other.sync()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    mac.prefill(prompt, 0, *_inputs(64, 61))                         # as long as the request may be
    assert mac.read_ring(0)["kv_len"] == 64


def test_prefill_takes_the_same_scale_given_or_by_default():
    from kv_cache_computation_gb300 import PromptAttention
    same = 128 ** -0.5
    x = _inputs(40)
    want = _mac(H, Hkv).prefill(PromptAttention(H, Hkv, max_tokens=40), 0, *x)
    for of_mac, of_prompt in ((0.0, same), (same, 0.0), (same, same), (float(np.float32(same)), 0.0)):
        mac = _mac(H, Hkv, sm_scale=of_mac)
        got = mac.prefill(PromptAttention(H, Hkv, max_tokens=40, sm_scale=of_prompt), 0, *x)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for of_mac, of_prompt in ((0.0, 0.1), (0.1, 0.0), (same, 0.0884)):
        with pytest.raises(ValueError, match="scale"):
            _mac(H, Hkv, sm_scale=of_mac).prefill(PromptAttention(H, Hkv, max_tokens=40, sm_scale=of_prompt), 0, *x)


def test_prefill_on_another_stream():
    """Inputs made on that stream, by work that is still under way when the call is made."""
    from kv_cache_computation_gb300 import PromptAttention
    n = 700
    prompt, mac, other = PromptAttention(H, Hkv, max_tokens=n), _mac(H, Hkv), _mac(H, Hkv)
    x = _inputs(n)
    want = mac.prefill(prompt, 1, *x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        y = [torch.zeros_like(t) for t in x]
        big = torch.ones(1 << 28, device="cuda")
        for _ in range(10):
            big.mul_(1.0)
        for a, b in zip(y, x):
            a.copy_(b)
    got = other.prefill(prompt, 1, *y, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    a, b = mac.read_ring(1), other.read_ring(1)
    for key in a:
        assert np.array_equal(a[key], b[key]), key

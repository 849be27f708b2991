"""A prompt into a MAC request: outputs, the stored tokens, the ring's seeds and
the decode steps that reuse them; and a prompt with the 8-bit store behind it."""
import numpy as np
import pytest
import torch

import block_reference as BR
from test_gpu_prompt import BF16, _i32, _randn, _reference, _tolerance

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


def _mac(H, Hkv, **kw):
    from kv_cache_computation_gb300 import MacAttention
    m = MacAttention(H, Hkv, **{**dict(ring_len=16, band_r=32, tau=0.3, max_batch=2, max_ctx=4096, page_size=16), **kw})
    if kw.get("page_size", 16):
        pages = torch.randperm(512, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
        for b in range(2):
            m.set_page_table(b, pages[256 * b:256 * (b + 1)].contiguous())
    return m


@pytest.mark.parametrize("H,Hkv,n,L,r,page", [(8, 2, 300, 16, 32, 16), (32, 8, 1000, 512, 64, 16), (32, 1, 77, 128, 64, 0),
                                              (4, 4, 1, 16, 1, 16), (8, 2, 20, 16, 64, 16), (16, 1, 3000, 32, 128, 0)])
def test_prefill_seeds_the_ring(H, Hkv, n, L, r, page):
    from kv_cache_computation_gb300 import PromptAttention
    mac = _mac(H, Hkv, ring_len=L, band_r=r, page_size=page)
    prompt = PromptAttention(H, Hkv, max_tokens=n)
    qp, q = _randn((n, H, 128), 1), _randn((n, H, 128), 2)
    k, v = _randn((n, Hkv, 128), 3), _randn((n, Hkv, 128), 4)
    for req in (1, 0, 1):                                            # the last one takes an old request's place
        out, lse = mac.prefill(prompt, req, qp, q, k, v)
    prompt.sync()
    o, l, mag, top = _reference(q, k, v, 0, 128 ** -0.5)
    to, tl = _tolerance(o, mag, top, l, n, False)
    assert ((out.double() - o).abs() <= to).all() and ((lse.double() - l).abs() <= tl).all()
    ring = mac.read_ring(1)
    last = min(L, n)
    o, l, mag, top = _reference(q[n - last:], k, v, r, 128 ** -0.5)
    to, tl = _tolerance(o, mag, top, l, n, True)
    assert ring["kv_len"] == n and ring["steps"] == last
    assert list(ring["pos"][:last]) == list(range(n - last + 1, n + 1)) and (ring["pos"][last:] == 0).all()
    got = torch.from_numpy(ring["o"][:, :last]).transpose(0, 1).double().cuda()
    glse = torch.from_numpy(ring["lse"][:, :last]).transpose(0, 1).double().cuda()
    assert ((got - o).abs() <= to).all()
    empty = torch.isneginf(l)
    assert torch.equal(torch.isneginf(glse), empty)
    assert (torch.where(empty, 0.0, (glse - l).abs() - tl) <= 0).all()
    qbits = torch.from_numpy(ring["q"][:, :last].view(np.int16)).transpose(0, 1)
    assert torch.equal(qbits, qp[n - last:].cpu().view(torch.int16))
    mac.sync()


def test_decode_steps_behind_a_prompt_reuse_its_queries():
    """The first decode step's query is close to one of the prompt's: it hits the seeded entry, reads only the band, and
    its output is full attention's to the step's own bound (5e-3 of the largest element) where the query is the same."""
    from kv_cache_computation_gb300 import PromptAttention
    H, Hkv, n = 8, 2, 2000
    mac, prompt = _mac(H, Hkv, ring_len=64, band_r=64), PromptAttention(H, Hkv, max_tokens=n)
    qp, q = _randn((n, H, 128), 1), _randn((n, H, 128), 2)
    k, v = _randn((n, Hkv, 128), 3), _randn((n, Hkv, 128), 4)
    for req in range(2):
        mac.prefill(prompt, req, qp, q, k, v)
    mac.reset_stats()
    back = torch.tensor([5, 40])                                     # the entries that the two requests' queries repeat
    kn, vn = _randn((2, Hkv, 128), 5), _randn((2, Hkv, 128), 6)
    out, lse = mac.decode_step(qp[n - back], q[n - back], kn, vn)
    mac.sync()
    assert mac.stats()["hits"] == 2 * H and mac.stats()["kv_tokens_read"] < 2 * Hkv * 200
    for b in range(2):
        kk, vv = torch.cat((k, kn[b:b + 1])), torch.cat((v, vn[b:b + 1]))
        o, l, _, _ = _reference(q[n - back[b]][None], kk, vv, 0, 128 ** -0.5)
        err = (out[b].double() - o[0]).abs().amax(-1) / o[0].abs().amax(-1)
        assert (err <= 5e-3).all() and ((lse[b].double() - l[0]).abs() <= 1e-4).all()


def test_prefill_refusals():
    from kv_cache_computation_gb300 import MacError, PromptAttention
    mac, prompt = _mac(8, 2, max_ctx=64, page_size=0), PromptAttention(8, 2, max_tokens=100)
    q, k = _randn((70, 8, 128), 1), _randn((70, 2, 128), 2)
    mac.prefill(prompt, 0, q[:20], q[:20], k[:20], k[:20])
    for args in ((PromptAttention(8, 4, max_tokens=100), 0, q, q, k, k), (PromptAttention(8, 2, max_tokens=30), 0, q, q, k, k),
                 (PromptAttention(8, 2, max_tokens=100, sm_scale=0.5), 0, q, q, k, k), (prompt, 0, q[:0], q[:0], k[:0], k[:0]),
                 (prompt, 0, q, q[:5], k, k), (prompt, 0, q, q, k[:5], k), (prompt, 0, q, q, k.float(), k)):
        with pytest.raises((ValueError, TypeError)):
            mac.prefill(*args)
    assert mac.read_ring(0)["kv_len"] == 20                          # nothing was touched
    with pytest.raises(MacError):                                    # longer than the request may be
        mac.prefill(prompt, 0, q, q, k, k)


@pytest.mark.parametrize("H,Hkv", [(8, 2), (28, 4)])
def test_prompts_chunks_and_decode_steps_over_the_8_bit_store(H, Hkv):
    """Prompts from their projections, packed; a second chunk of each behind the stored tokens; then decode steps: every
    output is its definition's over the values that the store holds."""
    from kv_cache_computation_gb300 import BlockKV, PromptAttention, QkvRotary, new_page_pool, page_step
    B, N, P = 3, 120, 40
    rot, cache = QkvRotary(H, Hkv, base=10000.0), BlockKV(H, Hkv, num_pages=N, max_batch=B)
    prompt = PromptAttention(H, Hkv, max_tokens=400, max_batch=B)
    ref = BR.Store(N, Hkv)
    ring, state = new_page_pool(N)
    lens, table = torch.zeros(B, dtype=torch.int32).cuda(), torch.zeros((B, P), dtype=torch.int32).cuda()
    w = _randn((128,), 1), _randn((128,), 2)

    def slots_of(b, n):
        t = np.arange(n)
        return table[b].cpu().numpy()[t // 16] * 16 + t % 16
    for step, new in enumerate(([100, 0, 37], [61, 250, 0], [33, 7, 12])):
        st = page_step(lens, _i32(new), table, ring, state, max_tokens=400, in_place=True)
        assert int(st.status) == 0
        x = _randn((400, (H + 2 * Hkv) * 128), 20 + step)
        _, q, k, v = rot(x, st.positions, *w, want_pre=False)
        cache.append(k, v, st.slots)
        total = [int(z) for z in st.lengths]
        every = [slots_of(b, total[b]) for b in range(B)]
        ref.append(k.double().cpu().numpy(), v.double().cpu().numpy(), st.slots.cpu().numpy())
        # what the chunk attends to: the stored tokens, its own among them
        kk, vv = cache.gather(_i32(np.concatenate(every)))
        k_starts = _i32(np.concatenate(([0], np.cumsum(total))))
        out, lse = prompt(q, kk, vv, st.starts, k_starts)
        prompt.sync(), cache.sync()
        first, kf = st.starts.cpu().numpy(), k_starts.cpu().numpy()
        for b in range(B):
            rows, keys = slice(int(first[b]), int(first[b + 1])), slice(int(kf[b]), int(kf[b + 1]))
            K, V = ref.gather(every[b])
            assert np.array_equal(K, kk[keys].double().cpu().numpy()) and np.array_equal(V, vv[keys].double().cpu().numpy())
            o, l, mag, top = _reference(q[rows], kk[keys], vv[keys], 0, 128 ** -0.5)
            to, tl = _tolerance(o, mag, top, l, total[b], False)
            assert ((out[rows].double() - o).abs() <= to).all() and ((lse[rows].double() - l).abs() <= tl).all()
    for t in range(4):
        st = page_step(lens, _i32([1, 1, 1]), table, ring, state, max_tokens=B, in_place=True)
        qkv = _randn((B, (H + 2 * Hkv) * 128), 70 + t)
        out, lse = cache.decode_step_qkv(rot, qkv, st.positions, st.slots, table, st.lengths, *w, starts=st.starts)
        cache.sync()
        _, q, k, v = rot(qkv, st.positions, *w)
        ref.append(k.double().cpu().numpy(), v.double().cpu().numpy(), st.slots.cpu().numpy())
        # the same rows as one-token prompts over the gathered tokens
        total = [int(z) for z in st.lengths]
        every = [slots_of(b, total[b]) for b in range(B)]
        kk, vv = cache.gather(_i32(np.concatenate(every)))
        pout, plse = prompt(q, kk, vv, _i32(range(B + 1)), _i32(np.concatenate(([0], np.cumsum(total)))))
        for b in range(B):
            K, V = ref.gather(every[b])
            o, l, mag, top = BR.attention(q[b:b + 1].double().cpu().numpy(), K, V, ref.exp[every[b] // 16, 1], 128 ** -0.5)
            to, tl = BR.attention_tolerance(o, mag, top, l, total[b])
            assert (np.abs(out[b].double().cpu().numpy() - o[0]) <= to[0]).all()
            assert (np.abs(lse[b].double().cpu().numpy() - l[0]) <= tl[0]).all()
            o, l, mag, top = _reference(q[b:b + 1], torch.from_numpy(K).cuda(), torch.from_numpy(V).cuda(), 0, 128 ** -0.5)
            to, tl = _tolerance(o, mag, top, l, total[b], False)
            assert ((pout[b].double() - o[0]).abs() <= to[0]).all() and ((plse[b].double() - l[0]).abs() <= tl[0]).all()

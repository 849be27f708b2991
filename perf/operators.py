"""Cases and plain forms of the operators around a decode step with a 4-bit KV cache.

Four operators of a serving loop: the QKV projection's split with per-head
norms and the rotary embedding; the page bookkeeping of a step; the 4-bit
store's append and gather; decode attention over that store.

``own`` selects what :func:`run` calls: the plain torch forms below (False) or
the library's operators (True).

The 4-bit format (both forms and :func:`exact`): 16 consecutive elements of a
head share one scale s = e4m3(max|x| / 6) (round to nearest even, at most 448)
and hold x / s rounded to the nearest e2m1 value (0, 0.5, 1, 1.5, 2, 3, 4, 6
with a sign; ties to the even code; beyond 6 saturates; s = 0 stores zeros).
"""
import math

import numpy as np
import torch

own = False

D = 128          # head dimension
PAGE = 16        # tokens per page
BLOCK = 16       # elements per scale
ROPE_BASE = 500000.0
EPS = 1e-6


def _dev():
    return torch.device("cuda", torch.cuda.current_device())


def _gen(seed, tag):
    g = torch.Generator(device=_dev())
    g.manual_seed((int(seed) * 1000003 + tag) & 0x7FFFFFFFFFFFFFFF)
    return g


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # one token of one request, 32 query heads over 8 KV heads: the latency of a single stream's step
        dict(name="rope_1tok", op="rope", tokens=1, heads=32, kv_heads=8, rotary=128, interleaved=False, norm=True),
        # a batch of 37 decoding requests in a 32-over-4 layer, rotation of half the head in interleaved pairs
        dict(name="rope_37tok_partial", op="rope", tokens=37, heads=32, kv_heads=4, rotary=64, interleaved=True,
             norm=True),
        # a prefill chunk of 32768 tokens
        dict(name="rope_32768tok", op="rope", tokens=32768, heads=32, kv_heads=8, rotary=128, interleaved=False,
             norm=True),
        # a decode step of 32 requests up to 131072 tokens, two of them finished and released
        dict(name="pages_decode_b32", op="pages", batch=32, table=8200, max_len=131072, tokens=32, kind="decode"),
        # a mixed step: 250 requests, prefill chunks of up to 2048 tokens beside decoding ones, some finished
        dict(name="pages_mixed_b250", op="pages", batch=250, table=2100, max_len=32768, tokens=65536, kind="mixed"),
        # the new tokens of 8 decoding requests, into the store and back
        dict(name="store_8tok", op="store", tokens=8, kv_heads=8, kind="decode"),
        # a prefill chunk of 32768 tokens into whole pages, and read back for the prefill's own attention
        dict(name="store_32768tok", op="store", tokens=32768, kv_heads=8, kind="prefill"),
        # one stream at 4096 tokens
        dict(name="attn_b1_4k", op="attn", batch=1, heads=32, kv_heads=8, max_len=4096, ragged=False, queries=1),
        # one stream at 131072 tokens
        dict(name="attn_b1_128k", op="attn", batch=1, heads=32, kv_heads=8, max_len=131072, ragged=False, queries=1),
        # 32 requests of uneven length (an idle slot among them), one KV head under 32 query heads
        dict(name="attn_mqa_b32_ragged", op="attn", batch=32, heads=32, kv_heads=1, max_len=65536, ragged=True,
             queries=1),
        # 4 requests that verify 3 drafted tokens each, 7 query heads to a KV head
        dict(name="attn_b4_draft3", op="attn", batch=4, heads=28, kv_heads=4, max_len=122880, ragged=True, queries=3),
        # 8 requests at 131072 tokens: the largest store
        dict(name="attn_b8_128k", op="attn", batch=8, heads=32, kv_heads=8, max_len=131072, ragged=False, queries=1),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "pages", "store", "attn", "attn"])
    if op == "rope":
        kv = rng.choice([1, 2, 3, 4, 8])
        heads = kv * rng.randint(1, max(1, 32 // kv))
        return dict(op=op, tokens=_log_uniform(rng, 1, 32768), heads=heads, kv_heads=kv,
                    rotary=rng.choice([32, 64, 96, 128]), interleaved=rng.random() < 0.5, norm=rng.random() < 0.8)
    if op == "pages":
        kind = rng.choice(["decode", "mixed", "short"])   # short: the pool runs out within the step
        batch = _log_uniform(rng, 1, 512)
        max_len = _log_uniform(rng, 16, 131072 if batch <= 64 else 16384)
        table = (max_len + 2048 + PAGE - 1) // PAGE + rng.randint(0, 9)
        return dict(op=op, batch=batch, table=table, max_len=max_len,
                    tokens=batch + rng.randint(0, 7) if kind == "decode" else _log_uniform(rng, 2048, 65536), kind=kind)
    if op == "store":
        return dict(op=op, tokens=_log_uniform(rng, 1, 32768), kv_heads=rng.choice([1, 2, 3, 4, 8]),
                    kind=rng.choice(["decode", "prefill"]))
    kv = rng.choice([1, 2, 4, 8])
    queries = rng.choice([1, 1, 1, 2, 4])
    group = rng.randint(1, 32 // queries)
    batch = _log_uniform(rng, 1, 32)
    # KV tokens over all heads, and rows against them: at most the largest case's
    most = min(131072, (1 << 23) // (batch * kv), (1 << 25) // (batch * kv * group * queries))
    return dict(op=op, batch=batch, heads=group * kv, kv_heads=kv, max_len=_log_uniform(rng, 1, most),
                ragged=rng.random() < 0.6, queries=queries)


# ---- inputs ----------------------------------------------------------------

def _rope_inputs(case, seed):
    d, T, H, Hkv = _dev(), case["tokens"], case["heads"], case["kv_heads"]
    g = _gen(seed, 1)
    qkv = torch.randn((T, (H + 2 * Hkv) * D), generator=g, device=d).to(torch.bfloat16)
    pos = torch.randint(0, 131072, (1,), generator=g, device=d) + torch.arange(T, device=d)
    wq = (1 + 0.1 * torch.randn(D, generator=g, device=d)).to(torch.bfloat16)
    wk = (1 + 0.1 * torch.randn(D, generator=g, device=d)).to(torch.bfloat16)
    return dict(qkv=qkv, pos=pos.to(torch.int32), wq=wq if case["norm"] else None, wk=wk if case["norm"] else None)


def _pages_inputs(case, seed):
    """A consistent page pool in the middle of its life (host arrays)."""
    r = np.random.default_rng([int(seed) & 0x7FFFFFFF, 2])
    B, P = case["batch"], case["table"]
    lens = r.integers(0, case["max_len"] + 1, B)
    if case["kind"] == "decode":
        new = np.ones(B, np.int64)
    else:
        new = np.where(r.random(B) < 0.25, r.integers(1, 2049, B), 1)
        while new.sum() > case["tokens"]:                  # the step's token budget
            new[int(new.argmax())] = 1 if new.max() > 1 else 0
    new[r.random(B) < 1 / 16] = -1                         # finished: released
    used = (lens + PAGE - 1) // PAGE
    spare = int(np.maximum((lens + np.maximum(new, 0) + PAGE - 1) // PAGE - used, 0).sum())
    spare = spare // 2 if case["kind"] == "short" else spare + 64
    N = B * ((case["max_len"] + PAGE - 1) // PAGE + 129) + 1
    perm = r.permutation(N).astype(np.int32)
    table = np.full((B, P), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :used[b]] = perm[at:at + used[b]]
        at += int(used[b])
    head = int(r.integers(0, N))
    ring = np.full(N, -1, np.int32)
    free = perm[at:at + spare]                             # the rest is held elsewhere
    ring[(head + np.arange(len(free))) % N] = free
    return dict(lengths=lens.astype(np.int32), new=new.astype(np.int32), table=table, ring=ring,
                state=np.array([head, len(free)], np.int32))


def _store_slots(case, seed, g):
    T = case["tokens"]
    d = _dev()
    if case["kind"] == "prefill":                          # whole requests, pages in random order
        pages = (T + PAGE - 1) // PAGE
        perm = torch.randperm(pages + 8, generator=g, device=d)[:pages]
        t = torch.arange(T, device=d)
        return (perm[t // PAGE] * PAGE + t % PAGE).to(torch.int32), pages + 8
    pages = T + 8                                          # one token of each request, anywhere in its page
    perm = torch.randperm(pages, generator=g, device=d)[:T]
    off = torch.randint(0, PAGE, (T,), generator=g, device=d)
    return (perm * PAGE + off).to(torch.int32), pages


def _kv(T, Hkv, g, scale):
    x = torch.randn((T, Hkv, D), generator=g, device=_dev())
    return (x * scale).to(torch.bfloat16)


def _store_inputs(case, seed):
    g = _gen(seed, 3)
    T, Hkv = case["tokens"], case["kv_heads"]
    scale = 0.5 * 4 ** torch.rand((2, Hkv, D), generator=g, device=_dev())
    slots, pages = _store_slots(case, seed, g)
    return dict(k=_kv(T, Hkv, g, scale[0]), v=_kv(T, Hkv, g, scale[1]), slots=slots, pages=pages)


def _attn_lengths(case, seed):
    r = np.random.default_rng([int(seed) & 0x7FFFFFFF, 4])
    B, n = case["batch"], case["max_len"]
    if not case["ragged"]:
        return [n] * B
    lens = r.integers(0, n + 1, B)
    lens[int(r.integers(0, B))] = n
    if B > 4:
        lens[int((lens.argmax() + 1) % B)] = 0             # an idle slot of the batch
    return [int(x) for x in lens]


def _attn_inputs(case, seed):
    """Lengths, page table, queries, and a function that yields request b's (k, v) in order."""
    g = _gen(seed, 5)
    d, Hkv = _dev(), case["kv_heads"]
    lens = _attn_lengths(case, seed)
    pages = [(n + PAGE - 1) // PAGE for n in lens]
    total = sum(pages) + 8
    perm = torch.randperm(total, generator=g, device=d)
    table = torch.zeros((len(lens), max(max(pages), 1)), dtype=torch.int32, device=d)
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = perm[at:at + p].to(torch.int32)
        at += p
    q = 1.5 * torch.randn((case["batch"], case["queries"], case["heads"], D), generator=g, device=d)
    scale = 0.5 * 4 ** torch.rand((2, Hkv, D), generator=g, device=d)

    def kv():
        for b, n in enumerate(lens):
            if n:
                yield b, n, _kv(n, Hkv, g, scale[0]), _kv(n, Hkv, g, scale[1])
    return lens, table, total, q.to(torch.bfloat16), kv


def _slots_of(table, b, n):
    t = torch.arange(n, device=table.device)
    return table[b, t // PAGE].to(torch.int64) * PAGE + t % PAGE


def prepare(case, seed):
    op = case["op"]
    st = dict(case)
    if op == "rope":
        st.update(_rope_inputs(case, seed))
        if own:
            import kv_cache_computation_gb300 as kvc
            st["rot"] = kvc.QkvRotary(case["heads"], case["kv_heads"], rotary_dim=case["rotary"], base=ROPE_BASE,
                                      interleaved=case["interleaved"], eps=EPS)
    elif op == "pages":
        st.update({k: torch.from_numpy(v).to(_dev()) for k, v in _pages_inputs(case, seed).items()})
    elif op == "store":
        st.update(_store_inputs(case, seed))
        if own:
            import kv_cache_computation_gb300 as kvc
            st["cache"] = kvc.QuantKV(case["kv_heads"], case["kv_heads"], num_pages=st["pages"], max_batch=1)
        else:
            st["store"] = _plain_store(st["pages"], case["kv_heads"])
    else:
        lens, table, pages, q, kv = _attn_inputs(case, seed)
        st.update(lens=lens, table=table, q=q, lengths=torch.tensor(lens, dtype=torch.int32, device=_dev()))
        if own:
            import kv_cache_computation_gb300 as kvc
            st["cache"] = kvc.QuantKV(case["heads"], case["kv_heads"], num_pages=pages, max_batch=case["batch"],
                                      max_query=case["queries"])
            for b, n, k, v in kv():
                st["cache"].append(k, v, _slots_of(table, b, n).to(torch.int32))
        else:
            st["store"] = _plain_store(pages, case["kv_heads"])
            for b, n, k, v in kv():
                _plain_append(st["store"], k, v, _slots_of(table, b, n))
    return st


# ---- plain forms -------------------------------------------------------------

_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _plain_store(pages, Hkv):
    """Codes (two to a byte) and scales of K and V by slot; the last slot takes what has none."""
    n, d = pages * PAGE + 1, _dev()
    return [(torch.zeros((n, Hkv, D // 2), dtype=torch.uint8, device=d),
             torch.zeros((n, Hkv, D // BLOCK), dtype=torch.float8_e4m3fn, device=d)) for _ in range(2)]


def _plain_quantise(x):
    xb = x.float().reshape(*x.shape[:-1], D // BLOCK, BLOCK)
    s = (xb.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.float()[..., None]
    y = torch.where(sf > 0, xb.abs() / torch.where(sf > 0, sf, torch.ones_like(sf)), torch.zeros_like(xb))
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    code = (code + 8 * (xb < 0)).to(torch.uint8).reshape(x.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), s


def _plain_dequantise(codes, scales):
    table = torch.tensor(_LEVELS + tuple(-v for v in _LEVELS), dtype=torch.float32, device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).to(torch.int32)
    x = table[c].reshape(*codes.shape[:-1], D // BLOCK, BLOCK)
    return (x * scales.float()[..., None]).reshape(*codes.shape[:-1], D)


def _plain_append(store, k, v, slots):
    idx = torch.where(slots < 0, store[0][0].shape[0] - 1, slots.to(torch.int64))
    for (codes, scales), x in zip(store, (k, v)):
        c, s = _plain_quantise(x)
        codes[idx] = c
        scales.view(torch.uint8)[idx] = s.view(torch.uint8)


def _plain_gather(store, slots):
    idx = slots.to(torch.int64)
    return [_plain_dequantise(codes[idx], scales.view(torch.uint8)[idx].view(torch.float8_e4m3fn))
            for codes, scales in store]


def _plain_rope(st):
    H, Hkv, r = st["heads"], st["kv_heads"], st["rotary"]
    x = st["qkv"].float().reshape(-1, H + 2 * Hkv, D)
    half = r // 2
    freq = ROPE_BASE ** (-2.0 * torch.arange(half, device=x.device, dtype=torch.float64) / r)
    ang = st["pos"].double()[:, None] * freq
    cos, sin = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]

    def norm(y, w):
        if w is None:
            return y
        return y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()

    def rotate(y):
        a, b = (y[..., 0:r:2], y[..., 1:r:2]) if st["interleaved"] else (y[..., :half], y[..., half:r])
        ra, rb = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack((ra, rb), -1).flatten(-2) if st["interleaved"] else torch.cat((ra, rb), -1)
        return torch.cat((turned, y[..., r:]), -1)

    q, k = norm(x[:, :H], st["wq"]), norm(x[:, H:H + Hkv], st["wk"])
    return [y.to(torch.bfloat16) for y in (q, rotate(q), rotate(k), x[:, H + Hkv:])]


def _plain_pages(st):
    lens, new, table, ring, state = (st[k] for k in ("lengths", "new", "table", "ring", "state"))
    T, (B, P), N = st["tokens"], st["table"].shape, st["ring"].shape[0]
    len64, n = lens.long(), new.long().clamp(min=0)
    ends = n.cumsum(0)
    begin = ends - n
    before, after = (len64 + PAGE - 1) // PAGE, (len64 + n + PAGE - 1) // PAGE
    long_, late = after > P, ends > T
    can = (new >= 0) & ~long_ & ~late
    need = torch.where(can, after - before, torch.zeros_like(n))
    cum = need.cumsum(0)
    head, count = state[0].long(), state[1].long()
    dry = can & (need > 0) & (cum > count)
    ok = can & ~dry
    popped = torch.where(ok & (need > 0), cum, torch.zeros_like(cum)).max()
    first = cum - need
    # block table: the new pages' columns take the ring's ids
    col = torch.arange(P, device=table.device)[None]
    fresh = ok[:, None] & (col >= before[:, None]) & (col < after[:, None])
    source = ring[(head + first[:, None] + (col - before[:, None]).clamp(min=0)) % N]
    table.copy_(torch.where(fresh, source, table))
    # released requests' pages go to the ring's end
    rel = torch.where(new < 0, before, torch.zeros_like(before))
    rel_first = rel.cumsum(0) - rel
    back = (new < 0)[:, None] & (col < before[:, None])
    where = (head + count + rel_first[:, None] + col) % N
    padded = torch.cat((ring, ring[:1]))
    padded.scatter_(0, torch.where(back, where, N).flatten(), table.flatten())
    ring.copy_(padded[:N])
    new_len = torch.where(new < 0, 0, torch.where(ok, len64 + n, len64)).to(torch.int32)
    new_state = torch.stack(((head + popped) % N, count - popped + rel.sum())).to(torch.int32)
    starts = torch.cat((begin, ends[-1:])).clamp(max=T).to(torch.int32)
    # slot map of the packed new tokens
    t = torch.arange(T, device=table.device)
    req = torch.searchsorted(ends, t, right=True).clamp(max=B - 1)
    live = t < ends[-1]
    pos = torch.where(live, len64[req] + t - begin[req], 0)
    page = table[req, (pos // PAGE).clamp(max=P - 1)].long()
    slots = torch.where(live & ok[req], page * PAGE + pos % PAGE, -1).to(torch.int32)
    status = (dry.any() * 1 + (long_ & (new >= 0)).any() * 2 + (late & (new >= 0) & ~long_).any() * 8).to(torch.int32)
    return [new_len, new_state, starts, pos.to(torch.int32), slots, table, ring, status.reshape(1)]


def _plain_attn(st):
    B, nq, H, Hkv = st["batch"], st["queries"], st["heads"], st["kv_heads"]
    G = H // Hkv
    out = torch.zeros((B, nq, H, D), dtype=torch.float32, device=st["q"].device)
    lse = torch.full((B, nq, H), -math.inf, dtype=torch.float32, device=st["q"].device)
    for b, n in enumerate(st["lens"]):
        if n == 0:
            continue
        k, v = _plain_gather(st["store"], _slots_of(st["table"], b, n))
        k, v = k.transpose(0, 1), v.transpose(0, 1)                                    # [Hkv, n, D]
        q = st["q"][b].float().reshape(nq, Hkv, G, D).transpose(0, 1).reshape(Hkv, nq * G, D)
        s = torch.matmul(q, k.transpose(1, 2)) * (1.0 / math.sqrt(D))                  # [Hkv, nq G, n]
        seen = n - nq + 1 + torch.arange(nq, device=q.device).repeat_interleave(G)     # tokens of each row
        s = s.masked_fill(torch.arange(n, device=q.device) >= seen[:, None], -math.inf)
        m = s.amax(-1, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        p = torch.exp(s - m)
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
        out[b] = o.reshape(Hkv, nq, G, D).transpose(0, 1).reshape(nq, H, D)
        lse[b] = (m + torch.log(total)).reshape(Hkv, nq, G).transpose(0, 1).reshape(nq, H)
    return [out.to(torch.bfloat16), lse]


def run(st):
    op = st["op"]
    if not own:
        if op == "rope":
            return _plain_rope(st)
        if op == "pages":
            return _plain_pages(st)
        if op == "store":
            _plain_append(st["store"], st["k"], st["v"], st["slots"])
            return [x.to(torch.bfloat16) for x in _plain_gather(st["store"], st["slots"])]
        return _plain_attn(st)
    import kv_cache_computation_gb300 as kvc
    if op == "rope":
        return list(st["rot"](st["qkv"], st["pos"], st["wq"], st["wk"]))
    if op == "pages":
        p = kvc.page_step(st["lengths"], st["new"], st["table"], st["ring"], st["state"], max_tokens=st["tokens"])
        return [p.lengths, p.free_state, p.starts, p.positions, p.slots, st["table"], st["ring"], p.status]
    if op == "store":
        st["cache"].append(st["k"], st["v"], st["slots"])
        return list(st["cache"].gather(st["slots"]))
    return list(st["cache"].attention(st["q"], st["table"], st["lengths"]))


# ---- work ----------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "rope":
        T, H, Hkv = case["tokens"], case["heads"], case["kv_heads"]
        rows_in, rows_out = H + 2 * Hkv, 2 * H + 2 * Hkv
        return {"bytes": T * ((rows_in + rows_out) * D * 2 + 4), "flops": T * (H + Hkv) * D * 8}
    if op == "pages":
        B, T = case["batch"], case["tokens"]
        return {"bytes": B * 12 + 4 * (B + 1) + T * 8 + (T // PAGE + B) * 8, "flops": T * 4 + B * 16}
    if op == "store":
        n = case["tokens"] * case["kv_heads"]
        return {"bytes": 2 * n * (512 + 144) + 8 * case["tokens"], "flops": n * 2 * D * 4}
    n = sum(_attn_lengths(case, 0)) if not case["ragged"] else case["batch"] * (case["max_len"] + 1) // 2
    rows = case["queries"] * case["heads"]
    return {"bytes": n * case["kv_heads"] * 144 + case["batch"] * rows * (2 * D * 2 + 4) + n // PAGE * 4,
            "flops": 4 * D * rows * n}


# ---- exact ---------------------------------------------------------------------

def _exact_stored(x):
    """The values that the 4-bit store holds for x (any shape [..., 128]), in 64 bits."""
    d = x.double().reshape(-1, BLOCK)
    want = d.abs().max(dim=1).values / 6.0
    # e4m3 by its grid: 2^e steps of 1/8 from 2^-6 up, 2^-9 below
    e = torch.floor(torch.log2(want.clamp(min=2.0 ** -6)))
    e = torch.where(torch.exp2(e) > want.clamp(min=2.0 ** -6), e - 1, e)
    step = torch.exp2(e - 3)
    s = (torch.round(want / step) * step).clamp(max=448.0)          # torch.round: ties to even
    q = torch.where(s[:, None] > 0, d.abs() / torch.where(s > 0, s, torch.ones_like(s))[:, None], torch.zeros_like(d))
    # e2m1 by its grid: steps of 0.5 below 2, 1 from 2, 2 from 4; at most 6
    grid = torch.where(q < 2, 0.5, torch.where(q < 4, 1.0, 2.0)).to(torch.float64)
    m = (torch.round(q / grid) * grid).clamp(max=6.0)
    return (torch.sign(d) * m * s[:, None]).reshape(x.shape)


def _exact_rope(case, seed):
    i = _rope_inputs(case, seed)
    H, Hkv, r, T = case["heads"], case["kv_heads"], case["rotary"], case["tokens"]
    x = i["qkv"].view(T, H + 2 * Hkv, D)
    out = [torch.empty((T, h, D), dtype=torch.float64, device="cpu") for h in (H, H, Hkv, Hkv)]
    j = torch.arange(r // 2, device=x.device, dtype=torch.float64)
    inv = torch.exp(j * (-2.0 / r) * math.log(ROPE_BASE))
    for t in range(0, T, 2048):
        y = x[t:t + 2048].double()
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                           i["pos"][t:t + 2048].double().outer(inv))[:, None]
        rows = [y[:, :H], y[:, H:H + Hkv]]
        if case["norm"]:
            rows = [a / torch.sqrt(a.square().mean(-1, keepdim=True) + EPS) * w.double()
                    for a, w in zip(rows, (i["wq"], i["wk"]))]
        done = []
        for a in rows:
            head = a[..., :r].unflatten(-1, (r // 2, 2) if case["interleaved"] else (2, r // 2))
            if not case["interleaved"]:
                head = head.transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(head.contiguous()) * turn)
            if not case["interleaved"]:
                z = z.transpose(-1, -2)
            done.append(torch.cat((z.flatten(-2), a[..., r:]), -1))
        for o, a in zip(out, (rows[0], done[0], done[1], y[:, H + Hkv:])):
            o[t:t + 2048] = a.cpu()
    return out


def _exact_pages(case, seed):
    i = _pages_inputs(case, seed)
    T, B, P, N = case["tokens"], case["batch"], case["table"], len(i["ring"])
    lens, new, table, ring = i["lengths"].astype(np.int64), i["new"], i["table"], i["ring"]
    head, count = (int(x) for x in i["state"])
    starts, pos, slots = np.zeros(B + 1, np.int64), np.zeros(T, np.int64), np.full(T, -1, np.int64)
    out_len, status, at, want, popped, freed = lens.copy(), 0, 0, 0, 0, []
    for b in range(B):
        n, old = int(new[b]), int(lens[b])
        have = -(-old // PAGE)
        if n < 0:
            freed.extend(table[b, :have].tolist())
            out_len[b] = 0
            n = 0
        else:
            more = -(-(old + n) // PAGE) - have
            if have + more > P:
                status |= 2
            elif at + n > T:
                status |= 8
            else:
                want += more
                if more and want > count:
                    status |= 1
                else:
                    for c in range(more):
                        table[b, have + c] = ring[(head + want - more + c) % N]
                    popped = max(popped, want if more else 0)
                    out_len[b] = old + n
                    p = old + np.arange(n)
                    slots[at:at + n] = table[b, p // PAGE].astype(np.int64) * PAGE + p % PAGE
            stop = min(at + n, T)
            pos[at:stop] = old + np.arange(max(stop - at, 0))
        at = at + n
        starts[b + 1] = min(at, T)
    for c, page in enumerate(freed):
        ring[(head + count + c) % N] = page
    state = np.array([(head + popped) % N, count - popped + len(freed)])
    return [torch.from_numpy(np.asarray(x).astype(np.int32))
            for x in (out_len, state, starts, pos, slots, table, ring, np.array([status]))]


def _exact_attn(case, seed):
    if sum(_attn_lengths(case, seed)) * case["queries"] * case["heads"] > 1 << 26:     # more than some seconds
        return None
    lens, table, pages, q, kv = _attn_inputs(case, seed)
    B, nq, H, Hkv = case["batch"], case["queries"], case["heads"], case["kv_heads"]
    G = H // Hkv
    out = torch.zeros((B, nq, H, D), dtype=torch.float64, device=q.device)
    lse = torch.full((B, nq, H), -math.inf, dtype=torch.float64, device=q.device)
    for b, n, k, v in kv():
        for h in range(Hkv):
            kh, vh = _exact_stored(k[:, h]), _exact_stored(v[:, h])
            for i in range(nq):
                seen = n - nq + 1 + i
                if seen <= 0:
                    continue
                s = kh[:seen] @ q[b, i, h * G:(h + 1) * G].double().t() / math.sqrt(D)      # [seen, G]
                z = torch.logsumexp(s, 0)
                lse[b, i, h * G:(h + 1) * G] = z
                out[b, i, h * G:(h + 1) * G] = torch.exp(s - z).t() @ vh[:seen]
    return [out, lse]


def exact(case, seed):
    op = case["op"]
    if op == "rope":
        return _exact_rope(case, seed)
    if op == "pages":
        return _exact_pages(case, seed)
    if op == "store":
        i = _store_inputs(case, seed)
        return [_exact_stored(i["k"]), _exact_stored(i["v"])]
    return _exact_attn(case, seed)

"""Cases and plain forms of prompt attention and of decode attention with an 8-bit KV cache.

Three operators of a serving loop: causal attention over whole prompts, packed
behind one another (with the summaries that seed the decode step's rings); the
8-bit store's append and gather; decode attention over that store.

``own`` selects what :func:`run` calls: the plain torch forms below (False) or
the library's operators (True).

The 8-bit format (both forms and :func:`exact`): the 16 tokens of a page share,
per KV head and for keys and values apart, a scale 2^e, and an element x is held
as e4m3(x / 2^e) (round to nearest even, at most 448).  A token needs the
smallest e in -60 .. 60 whose 448 * 2^e is at least its largest element.  A
call that stores the first slot of a page starts the page anew: e is the largest
that its tokens need.  Otherwise e is the larger of that and the page's old e,
and where it grows, the page's other slots are rounded again at the new scale.
"""
import math

import numpy as np
import torch

own = False

D = 128          # head dimension
PAGE = 16        # tokens per page
E_MIN, E_MAX = -60, 60


def _dev():
    return torch.device("cuda", torch.cuda.current_device())


def _gen(seed, tag):
    g = torch.Generator(device=_dev())
    g.manual_seed((int(seed) * 1000003 + tag) & 0x7FFFFFFFFFFFFFFF)
    return g


# ---- cases -----------------------------------------------------------------
# lens: one entry per request, tokens; for prompts "new+before" where the new
# tokens' queries come behind keys that are there already.

def listed():
    return [
        # a short question: the latency of a first token
        dict(name="prompt_b1_16", op="prompt", heads=32, kv_heads=8, lens="16", lag=0, summaries=False, sliced=False),
        # a batch of prompts that arrived together, packed: chat turns, documents, an empty one, one of a single token
        dict(name="prompt_b24_ragged", op="prompt", heads=32, kv_heads=8,
             lens="4096,17,801,2500,1,130,64,1999,0,333,1024,75,4001,256,90,1280,611,2048,29,128,3500,450,7,1700",
             lag=0, summaries=False, sliced=False),
        # odd lengths, 7 query heads to a KV head, read in place from one QKV projection
        dict(name="prompt_28h_sliced", op="prompt", heads=28, kv_heads=4, lens="1,2047,333,1201,6001", lag=0,
             summaries=False, sliced=True),
        # chunked prefill: 2048 and 509 new tokens behind longer contexts
        dict(name="prompt_chunk", op="prompt", heads=32, kv_heads=8, lens="2048+30720,509+8191", lag=0, summaries=False,
             sliced=False),
        # one whole prompt of 32768 tokens: the largest
        dict(name="prompt_b1_32k", op="prompt", heads=32, kv_heads=8, lens="32768", lag=0, summaries=False, sliced=False),
        # ring seeds: the summaries, 64 tokens back, of a prompt's last 512 queries
        dict(name="prompt_seeds_512", op="prompt", heads=32, kv_heads=8, lens="512+32256", lag=64, summaries=True,
             sliced=False),
        # the new tokens of 8 decoding requests, behind others in their pages, and the pages read back
        dict(name="block_store_8tok", op="store", tokens=8, kv_heads=8, kind="decode"),
        # a prefill chunk of 32768 tokens into whole pages, and back
        dict(name="block_store_32768tok", op="store", tokens=32768, kv_heads=8, kind="prefill"),
        # one stream at 4096 tokens
        dict(name="block_attn_b1_4k", op="attn", heads=32, kv_heads=8, lens="4096", queries=1),
        # 32 requests of uneven length (an idle slot among them), one KV head under 32 query heads
        dict(name="block_attn_mqa_b32", op="attn", heads=32, kv_heads=1,
             lens="65536,1200,31000,0,54321,777,16,40000,8191,25000,60001,3333,47000,12345,29,36000,"
                  "58000,19999,5,44444,22222,50001,9000,33333,61000,15000,1,27777,39000,48,20480,57000", queries=1),
        # 4 requests that verify 3 drafted tokens each, 7 query heads to a KV head
        dict(name="block_attn_b4_draft3", op="attn", heads=28, kv_heads=4, lens="122880,30011,77777,2", queries=3),
        # 8 requests at 131072 tokens: the largest store
        dict(name="block_attn_b8_128k", op="attn", heads=32, kv_heads=8, lens=",".join(["131072"] * 8), queries=1),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "store", "attn", "attn"])
    if op == "store":
        return dict(op=op, tokens=_log_uniform(rng, 1, 32768), kv_heads=rng.choice([1, 2, 3, 4, 8]),
                    kind=rng.choice(["decode", "prefill", "chunk"]))
    kv = rng.choice([1, 2, 3, 4, 8])
    if op == "attn":
        queries = rng.choice([1, 1, 1, 2, 4])
        group = rng.randint(1, 32 // queries)
        batch = _log_uniform(rng, 1, 48)
        # KV tokens over all heads, and rows against them: at most the largest case's
        most = min(131072, (1 << 23) // (batch * kv), (1 << 25) // (batch * kv * group * queries))
        lens = [rng.randint(0, most) if rng.random() < 0.7 else _log_uniform(rng, 1, most) for _ in range(batch)]
        return dict(op=op, heads=group * kv, kv_heads=kv, lens=",".join(map(str, lens)), queries=queries)
    group = rng.choice([1, 2, 4, 8, rng.randint(1, 16)])
    heads = kv * group
    kind = rng.choice(["whole", "whole", "chunk", "seeds"])
    batch = 1 if kind == "seeds" else _log_uniform(rng, 1, 40)
    lens, pairs, room = [], 0, 65536
    for _ in range(batch):
        n = _log_uniform(rng, 1, 16384) if rng.random() < 0.95 else 0
        before = _log_uniform(rng, 1, 49152) if kind == "chunk" and rng.random() < 0.8 else 0
        if kind == "seeds":
            n, before = _log_uniform(rng, 16, 2048), _log_uniform(rng, 1, 60000)
        n = min(n, max(room, 0))
        before = min(before, max(room - n, 0))
        if (pairs + n * (n + before)) * heads > 1 << 33:   # a quarter of the largest case's
            continue
        pairs += n * (n + before)
        room -= n + before
        lens.append(f"{n}+{before}" if before else str(n))
    return dict(op=op, heads=heads, kv_heads=kv, lens=",".join(lens or ["1"]),
                lag=rng.choice([32, 64, 128]) if kind == "seeds" else 0, summaries=kind == "seeds",
                sliced=kind == "whole" and rng.random() < 0.4)


def _lens(case):
    """[(new tokens, tokens before them)] of each request."""
    out = []
    for part in case["lens"].split(","):
        n, _, before = part.partition("+")
        out.append((int(n), int(before or 0)))
    return out


# ---- inputs ----------------------------------------------------------------

def _channel_scale(Hkv, g):
    """Per-channel scales of keys and values, log-uniform in 1/2 .. 2."""
    return 0.5 * 4 ** torch.rand((2, Hkv, D), generator=g, device=_dev())


def _kv(T, Hkv, g, scale):
    return (torch.randn((T, Hkv, D), generator=g, device=_dev()) * scale).to(torch.bfloat16)


def _prompt_inputs(case, seed):
    g, d = _gen(seed, 11), _dev()
    H, Hkv = case["heads"], case["kv_heads"]
    lens = _lens(case)
    Tq, Tk = sum(n for n, _ in lens), sum(n + b for n, b in lens)
    scale = _channel_scale(Hkv, g)
    if case["sliced"]:                                     # no tokens before: Tq == Tk
        qkv = torch.randn((Tq, H + 2 * Hkv, D), generator=g, device=d)
        qkv[:, H:H + Hkv] *= scale[0]
        qkv[:, H + Hkv:] *= scale[1]
        qkv = qkv.to(torch.bfloat16)
        q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    else:
        q = torch.randn((Tq, H, D), generator=g, device=d).to(torch.bfloat16)
        k, v = _kv(Tk, Hkv, g, scale[0]), _kv(Tk, Hkv, g, scale[1])
    edge = lambda x: torch.from_numpy(np.concatenate(([0], np.cumsum(x))).astype(np.int32)).to(d)
    return dict(q=q, k=k, v=v, starts=edge([n for n, _ in lens]), k_starts=edge([n + b for n, b in lens]))


def _store_inputs(case, seed):
    """Tokens that are in the pages already and the call's own, each with its slots."""
    g, d = _gen(seed, 13), _dev()
    T, Hkv = case["tokens"], case["kv_heads"]
    shape = np.random.default_rng([T, Hkv, 14])            # how full the pages are goes with the case
    if case["kind"] == "decode":                           # one token of each request, at any place in its page
        fill = shape.integers(0, PAGE, T)
        pages = T
        old_slot = np.concatenate([b * PAGE + np.arange(f) for b, f in enumerate(fill)] + [np.zeros(0, np.int64)])
        new_slot = np.arange(T) * PAGE + fill
    else:                                                  # whole pages from the first slot, or from inside one
        fill = np.array([int(shape.integers(1, PAGE)) if case["kind"] == "chunk" else 0])
        pages = -(-(T + int(fill[0])) // PAGE)
        old_slot, new_slot = np.arange(fill[0]), fill[0] + np.arange(T)
    perm = np.random.default_rng([int(seed) & 0x7FFFFFFF, 14]).permutation(pages + 8)
    move = lambda s: torch.from_numpy((perm[s // PAGE] * PAGE + s % PAGE).astype(np.int32)).to(d)
    scale = _channel_scale(Hkv, g)
    size = lambda n: torch.exp(0.5 * torch.randn((n, 1, 1), generator=g, device=d))      # tokens differ in size
    tok = lambda n, s: (torch.randn((n, Hkv, D), generator=g, device=d) * s * size(n)).to(torch.bfloat16)
    return dict(old_k=tok(len(old_slot), scale[0]), old_v=tok(len(old_slot), scale[1]), k=tok(T, scale[0]),
                v=tok(T, scale[1]), old_slots=move(old_slot), slots=move(new_slot), pages=pages + 8,
                read=move(np.concatenate((old_slot, new_slot)).astype(np.int64)))


def _attn_inputs(case, seed):
    """Lengths, page table, queries, and a function that yields request b's (b, n, k, v) in order."""
    g, d, Hkv = _gen(seed, 15), _dev(), case["kv_heads"]
    lens = [n for n, _ in _lens(case)]
    pages = [-(-n // PAGE) for n in lens]
    total = sum(pages) + 8
    perm = torch.randperm(total, generator=g, device=d)
    table = torch.zeros((len(lens), max(max(pages), 1)), dtype=torch.int32, device=d)
    at = 0
    for b, p in enumerate(pages):
        table[b, :p] = perm[at:at + p].to(torch.int32)
        at += p
    q = 1.5 * torch.randn((len(lens), case["queries"], case["heads"], D), generator=g, device=d)
    scale = _channel_scale(Hkv, g)

    def kv():
        for b, n in enumerate(lens):
            if n:
                yield b, n, _kv(n, Hkv, g, scale[0]), _kv(n, Hkv, g, scale[1])
    return lens, table, total, q.to(torch.bfloat16), kv


def _slots_of(table, b, n):
    t = torch.arange(n, device=table.device)
    return (table[b, t // PAGE].to(torch.int64) * PAGE + t % PAGE).to(torch.int32)


def prepare(case, seed):
    op, st = case["op"], dict(case)
    if own:
        import kv_cache_computation_gb300 as kvc
    if op == "prompt":
        st.update(_prompt_inputs(case, seed))
        if own:
            st["prompt"] = kvc.PromptAttention(case["heads"], case["kv_heads"], max_tokens=max(st["q"].shape[0], 1),
                                               max_batch=st["starts"].numel() - 1)
    elif op == "store":
        st.update(_store_inputs(case, seed))
        if own:
            st["cache"] = kvc.BlockKV(case["kv_heads"], case["kv_heads"], num_pages=st["pages"], max_batch=1)
            st["cache"].append(st["old_k"], st["old_v"], st["old_slots"])
        else:
            st["store"] = _plain_store(st["pages"], case["kv_heads"])
            _plain_append(st["store"], st["old_k"], st["old_v"], st["old_slots"])
    else:
        lens, table, pages, q, kv = _attn_inputs(case, seed)
        st.update(lengths=lens, table=table, q=q, lens_dev=torch.tensor(lens, dtype=torch.int32, device=_dev()))
        if own:
            st["cache"] = kvc.BlockKV(case["heads"], case["kv_heads"], num_pages=pages, max_batch=len(lens),
                                      max_query=case["queries"])
            for b, n, k, v in kv():
                st["cache"].append(k, v, _slots_of(table, b, n))
        else:
            st["store"] = _plain_store(pages, case["kv_heads"])
            for b, n, k, v in kv():
                _plain_append(st["store"], k, v, _slots_of(table, b, n))
    return st


# ---- plain forms -------------------------------------------------------------

def _plain_store(pages, Hkv):
    """Codes by page and offset and exponents by page, of keys and of values."""
    d = _dev()
    return [dict(codes=torch.zeros((pages, PAGE, Hkv, D), dtype=torch.float8_e4m3fn, device=d),
                 exp=torch.full((pages, Hkv), E_MIN, dtype=torch.int32, device=d)) for _ in range(2)]


def _two_to(e):
    return torch.ldexp(torch.ones((), device=e.device), e)


def _plain_append(store, k, v, slots):
    if k.shape[0] == 0:
        return
    page, off = torch.div(slots, PAGE, rounding_mode="floor").long(), (slots % PAGE).long()
    touched = torch.unique(page)
    first = torch.zeros(store[0]["exp"].shape[0], dtype=torch.bool, device=k.device)
    first[page[off == 0]] = True
    for s, x in zip(store, (k, v)):
        x = x.float()
        m, e = torch.frexp(x.abs().amax(-1))                               # max = m 2^e, m in [1/2, 1); 448 = 7/8 2^9
        need = torch.where(m > 0.875, e - 8, e - 9)
        need = torch.where(m == 0, E_MIN, need).clamp(E_MIN, E_MAX).to(torch.int32)
        old = s["exp"]
        new = torch.where(first[:, None], E_MIN, old).scatter_reduce(0, page[:, None].expand_as(need), need, "amax")
        shift = (old[touched] - new[touched]).clamp(max=0)[:, None, :, None]
        s["codes"].view(torch.uint8)[touched] = (s["codes"].view(torch.uint8)[touched].view(torch.float8_e4m3fn).float()
                                                 * _two_to(shift)).to(torch.float8_e4m3fn).view(torch.uint8)
        y = (x * _two_to(-new[page])[..., None]).clamp(-448.0, 448.0)
        s["codes"].view(torch.uint8)[page, off] = y.to(torch.float8_e4m3fn).view(torch.uint8)
        s["exp"] = new


def _plain_gather(store, slots):
    page, off = torch.div(slots, PAGE, rounding_mode="floor").long(), (slots % PAGE).long()
    return [s["codes"].view(torch.uint8)[page, off].view(torch.float8_e4m3fn).float() * _two_to(s["exp"][page])[..., None]
            for s in store]


def _plain_rows(q, k, v, seen):
    """Attention of rows q [Hkv, R, D] over k, v [Hkv, n, D], row r seeing the first seen[r] keys; fp32."""
    s = torch.matmul(q, k.transpose(1, 2)) * (1.0 / math.sqrt(D))
    s = s.masked_fill(torch.arange(k.shape[1], device=q.device) >= seen[:, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o, (m + torch.log(total)).squeeze(-1)


def _plain_prompt(st):
    H, Hkv = st["heads"], st["kv_heads"]
    G, q, lens = H // Hkv, st["q"], _lens(st)
    out = torch.zeros((q.shape[0], H, D), dtype=torch.float32, device=q.device)
    lse = torch.full((q.shape[0], H), -math.inf, dtype=torch.float32, device=q.device)
    qa = ka = 0
    for n, before in lens:
        m = n + before
        k = st["k"][ka:ka + m].float().transpose(0, 1)                                    # [Hkv, m, D]
        v = st["v"][ka:ka + m].float().transpose(0, 1)
        for i0 in range(0, n, 1024):                                                      # rows i0 .. i1 of the new tokens
            i1 = min(i0 + 1024, n)
            top = before + i1 - st["lag"]
            if top <= 0:
                continue
            rows = q[qa + i0:qa + i1].float().reshape(i1 - i0, Hkv, G, D).transpose(0, 1).reshape(Hkv, (i1 - i0) * G, D)
            seen = (before + 1 - st["lag"] + torch.arange(i0, i1, device=q.device)).repeat_interleave(G)
            o, l = _plain_rows(rows, k[:, :top], v[:, :top], seen)
            out[qa + i0:qa + i1] = o.reshape(Hkv, i1 - i0, G, D).transpose(0, 1).reshape(i1 - i0, H, D)
            lse[qa + i0:qa + i1] = l.reshape(Hkv, i1 - i0, G).transpose(0, 1).reshape(i1 - i0, H)
        qa += n
        ka += m
    return [out if st["summaries"] else out.to(torch.bfloat16), lse]


def _plain_attn(st):
    B, nq, H, Hkv = len(st["lengths"]), st["queries"], st["heads"], st["kv_heads"]
    G = H // Hkv
    out = torch.zeros((B, nq, H, D), dtype=torch.float32, device=st["q"].device)
    lse = torch.full((B, nq, H), -math.inf, dtype=torch.float32, device=st["q"].device)
    for b, n in enumerate(st["lengths"]):
        if n == 0:
            continue
        k, v = [x.transpose(0, 1) for x in _plain_gather(st["store"], _slots_of(st["table"], b, n))]
        q = st["q"][b].float().reshape(nq, Hkv, G, D).transpose(0, 1).reshape(Hkv, nq * G, D)
        seen = n - nq + 1 + torch.arange(nq, device=q.device).repeat_interleave(G)
        o, l = _plain_rows(q, k, v, seen)
        out[b] = o.reshape(Hkv, nq, G, D).transpose(0, 1).reshape(nq, H, D)
        lse[b] = l.reshape(Hkv, nq, G).transpose(0, 1).reshape(nq, H)
    return [out.to(torch.bfloat16), lse]


def run(st):
    op = st["op"]
    if not own:
        if op == "prompt":
            return _plain_prompt(st)
        if op == "store":
            _plain_append(st["store"], st["k"], st["v"], st["slots"])
            return [x.to(torch.bfloat16) for x in _plain_gather(st["store"], st["read"])]
        return _plain_attn(st)
    if op == "prompt":
        return list(st["prompt"](st["q"], st["k"], st["v"], st["starts"], st["k_starts"], lag=st["lag"],
                                 out_dtype=torch.float32 if st["summaries"] else torch.bfloat16))
    if op == "store":
        st["cache"].append(st["k"], st["v"], st["slots"])
        return list(st["cache"].gather(st["read"]))
    return list(st["cache"].attention(st["q"], st["table"], st["lens_dev"]))


# ---- work ----------------------------------------------------------------------

def _pairs(case):
    """Query-key pairs that are seen, per head."""
    total = 0
    for n, before in _lens(case):
        lo = before + 1 - case["lag"]                      # keys the first row sees, one more for each row behind it
        skip = min(max(-lo, 0), n)
        total += sum(range(lo + skip, lo + n)) if n < 64 else (n - skip) * (2 * lo + skip + n - 1) // 2
    return total


def work(case):
    op = case["op"]
    if op == "prompt":
        H, Hkv, lens = case["heads"], case["kv_heads"], _lens(case)
        Tq, Tk = sum(n for n, _ in lens), sum(n + b for n, b in lens)
        return {"bytes": Tq * H * (D * 2 + D * (4 if case["summaries"] else 2) + 4) + Tk * Hkv * D * 4,
                "flops": 4 * D * H * _pairs(case)}
    if op == "store":
        n, Hkv = case["tokens"], case["kv_heads"]
        read = n + {"decode": n * 15 // 2, "chunk": 8, "prefill": 0}[case["kind"]]
        return {"bytes": Hkv * (n * (512 + 256) + read * (256 + 512)) + 8 * n, "flops": Hkv * (n + read) * 2 * D * 4}
    n = sum(a for a, _ in _lens(case))
    rows = case["queries"] * case["heads"]
    return {"bytes": n * case["kv_heads"] * 256 + n // PAGE * (case["kv_heads"] * 2 + 4) +
            len(_lens(case)) * rows * (2 * D * 2 + 4), "flops": 4 * D * rows * n}


# ---- exact ---------------------------------------------------------------------

def _e4m3(y):
    """The nearest e4m3 value of y (64 bits, ties to even, at most 448)."""
    e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    e = torch.where(torch.exp2(e) > y.abs().clamp(min=2.0 ** -6), e - 1, e)
    step = torch.exp2(e - 3)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0)


def _exact_exponent(top):
    """The smallest e in E_MIN .. E_MAX with top <= 448 2^e."""
    e = torch.ceil(torch.log2((top / 448.0).clamp(min=2.0 ** -140)))
    e = torch.where(448.0 * torch.exp2(e - 1) >= top, e - 1, e)
    e = torch.where(448.0 * torch.exp2(e) < top, e + 1, e)
    return e.clamp(E_MIN, E_MAX)


def _exact_pages(x):
    """Tokens x [n, Hkv, D] stored from the first slot of a page on: the values held, in 64 bits."""
    n, Hkv, _ = x.shape
    out = torch.empty((n, Hkv, D), dtype=torch.float64, device=x.device)
    for i in range(0, n, 4096):                            # whole pages at a time
        y = x[i:i + 4096].double()
        pad = -len(y) % PAGE
        z = torch.cat((y, y.new_zeros((pad, Hkv, D)))).reshape(-1, PAGE, Hkv, D)
        s = torch.exp2(_exact_exponent(z.abs().amax(dim=(1, 3))))[:, None, :, None]
        out[i:i + 4096] = (_e4m3(z / s) * s).reshape(-1, Hkv, D)[:len(y)]
    return out


def _exact_store(case, seed):
    i = _store_inputs(case, seed)
    page = lambda s: torch.div(s.long(), PAGE, rounding_mode="floor")
    op, np_ = page(i["old_slots"]), page(i["slots"])
    fresh = set((i["slots"][i["slots"] % PAGE == 0].long() // PAGE).tolist())
    assert not fresh.intersection(op.tolist())             # a page that starts anew held nothing here
    res = []
    for old, new in ((i["old_k"], i["k"]), (i["old_v"], i["v"])):
        need = _exact_exponent(new.double().abs().amax(-1))                       # [T, Hkv]
        e1 = torch.full((i["pages"], case["kv_heads"]), float(E_MIN), dtype=torch.float64, device=new.device)
        if len(old):
            was = _exact_exponent(old.double().abs().amax(-1))
            e1 = e1.scatter_reduce(0, op[:, None].expand_as(was), was, "amax")
        e2 = e1.scatter_reduce(0, np_[:, None].expand_as(need), need, "amax")
        parts = []
        if len(old):
            s1, s2 = torch.exp2(e1[op])[..., None], torch.exp2(e2[op])[..., None]
            parts.append(_e4m3(_e4m3(old.double() / s1) * s1 / s2) * s2)
        s2 = torch.exp2(e2[np_])[..., None]
        parts.append(_e4m3(new.double() / s2) * s2)
        res.append(torch.cat(parts))
    return res


def _exact_head(q, k, v, lo):
    """Rows q [n, G, D] (row i sees the first lo + i of the keys) over one head's k, v, in 64 bits, a block of rows at a
    time: (out [n, G, D], lse [n, G])."""
    n, G, _ = q.shape
    out = torch.zeros((n, G, D), dtype=torch.float64, device=q.device)
    lse = torch.full((n, G), -math.inf, dtype=torch.float64, device=q.device)
    step = max(1, (1 << 26) // max(1, G * k.shape[0]))
    for i in range(max(0, 1 - lo), n, step):
        j = min(i + step, n)
        s = torch.einsum("rgd,td->rgt", q[i:j].double(), k[:lo + j - 1].double()) / math.sqrt(D)
        row = torch.arange(lo + i, lo + j, device=q.device)[:, None, None]
        s = torch.where(torch.arange(lo + j - 1, device=q.device) < row, s, -math.inf)
        z = torch.logsumexp(s, -1)
        lse[i:j] = z
        out[i:j] = torch.einsum("rgt,td->rgd", torch.exp(s - z[..., None]), v[:lo + j - 1].double())
    return out, lse


def _exact_prompt(case, seed):
    H, Hkv = case["heads"], case["kv_heads"]
    if 4 * D * H * _pairs(case) > 4e12:                    # more than some seconds
        return None
    i, G = _prompt_inputs(case, seed), H // Hkv
    out = torch.zeros((i["q"].shape[0], H, D), dtype=torch.float64, device=_dev())
    lse = torch.full((i["q"].shape[0], H), -math.inf, dtype=torch.float64, device=_dev())
    qa = ka = 0
    for n, before in _lens(case):
        for h in range(Hkv if n else 0):
            head = slice(h * G, (h + 1) * G)
            out[qa:qa + n, head], lse[qa:qa + n, head] = _exact_head(
                i["q"][qa:qa + n, head], i["k"][ka:ka + n + before, h], i["v"][ka:ka + n + before, h],
                before + 1 - case["lag"])
        qa += n
        ka += n + before
    return [out, lse]


def _exact_attn(case, seed):
    H, Hkv, nq = case["heads"], case["kv_heads"], case["queries"]
    G = H // Hkv
    if sum(n for n, _ in _lens(case)) * nq * H > 1 << 26:  # more than some seconds
        return None
    lens, table, pages, q, kv = _attn_inputs(case, seed)
    out = torch.zeros((len(lens), nq, H, D), dtype=torch.float64, device=q.device)
    lse = torch.full((len(lens), nq, H), -math.inf, dtype=torch.float64, device=q.device)
    for b, n, k, v in kv():
        k, v = _exact_pages(k), _exact_pages(v)
        for h in range(Hkv):
            head = slice(h * G, (h + 1) * G)
            out[b, :, head], lse[b, :, head] = _exact_head(q[b, :, head], k[:, h], v[:, h], n - nq + 1)
    return [out, lse]


def exact(case, seed):
    op = case["op"]
    if op == "prompt":
        return _exact_prompt(case, seed)
    return _exact_store(case, seed) if op == "store" else _exact_attn(case, seed)

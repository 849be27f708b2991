"""A paged KV store of 4 bits per value and decode attention over it (the
mac_quant_* calls of include/mac.h)."""
from __future__ import annotations

import ctypes

import torch

from . import _native as N
from .attention import _dev, _on, _out, _stream_ptr, _table
from .rotary import _rows


def _check(fn, status, handle=None):
    if status != N.MAC_OK:
        detail = (N.lib().mac_quant_last_error(handle) or b"").decode() if handle is not None and handle.value else ""
        raise N.MacError(fn, status, detail)


def quant_query_sizes(cfg: N.MacQuantConfig):
    """(store_bytes, scratch_bytes) for a configuration (host only)."""
    store, scratch = ctypes.c_size_t(), ctypes.c_size_t()
    _check("mac_quant_query_sizes",
           N.lib().mac_quant_query_sizes(ctypes.byref(cfg), ctypes.byref(store), ctypes.byref(scratch)))
    return store.value, scratch.value


class QuantKV:
    """One attention layer's 4-bit paged KV store on the current CUDA device.

    append stores post-RoPE keys and values at slots (page * 16 + offset, as
    page_step makes them), gather reads them back, attention decodes over the
    pages of a page table.  max_query new tokens per request and call at most
    (heads / kv_heads * max_query <= 32).  Calls on one object must be ordered
    with one another (they share its scratch); layers whose calls are ordered
    may share scratch: pass another QuantKV as `share` (sync of either then
    reports what the calls of both met).
    """

    def __init__(self, heads, kv_heads, num_pages, head_dim=128, page_size=16, max_batch=1, max_query=1, sm_scale=0.0,
                 k_scale=1.0, v_scale=1.0, device=None, share=None):
        self.cfg = N.MacQuantConfig(heads, kv_heads, head_dim, page_size, num_pages, max_batch, max_query, float(sm_scale),
                                    float(k_scale), float(v_scale))
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.num_pages, self.page_size, self.max_batch, self.max_query = num_pages, page_size, max_batch, max_query
        device = torch.device("cuda" if device is None else device)
        self.device = torch.device("cuda", torch.cuda.current_device()) if device.index is None else device
        self._h = ctypes.c_void_p()
        store, scratch = quant_query_sizes(self.cfg)
        self.sizes = dict(store=store, scratch=scratch)
        with torch.cuda.device(self.device):
            self._store = torch.empty(store, dtype=torch.uint8, device=self.device)
            if share is not None:
                if share.device != self.device or share._scratch.numel() < scratch:
                    raise ValueError("share must be a QuantKV on the same device with as large a scratch")
                self._scratch = share._scratch
            else:
                self._scratch = torch.empty(scratch, dtype=torch.uint8, device=self.device)
            h = ctypes.c_void_p()
            _check("mac_quant_create",
                   N.lib().mac_quant_create(ctypes.byref(self.cfg), self._store.data_ptr(), store, self._scratch.data_ptr(),
                                            scratch, ctypes.byref(h)))
        self._h = h

    # -- lifetime -----------------------------------------------------------
    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            N.lib().mac_quant_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- store --------------------------------------------------------------
    def append(self, k, v, slots, stream=None):
        """Store bf16 k, v [tokens, kv_heads, 128] (tokens may stand apart) at slots int32 [tokens]; negative: skipped."""
        n = k.shape[0]
        if v.shape[0] != n:
            raise ValueError("k and v must hold the same tokens")
        if k.device != self.device or v.device != self.device:
            raise ValueError(f"k and v must be on {self.device}")
        kp, ks = _rows(k, "k", self.kv_heads, self.head_dim)
        vp, vs = _rows(v, "v", self.kv_heads, self.head_dim)
        s = _dev(slots, "slots", torch.int32, (n,), self.device)
        with _on(self.device, stream):
            _check("mac_quant_append", N.lib().mac_quant_append(self._h, n, kp, ks, vp, vs, s,
                                                                _stream_ptr(stream, self.device)), self._h)

    def gather(self, slots, stream=None):
        """The stored k, v bf16 [tokens, kv_heads, 128] at slots int32 [tokens]; zeros where negative."""
        n = slots.shape[0]
        s = _dev(slots, "slots", torch.int32, (n,), self.device)
        shape = (n, self.kv_heads, self.head_dim)
        with _on(self.device, stream):
            k, v = _out(shape, self.device), _out(shape, self.device)
            _check("mac_quant_gather", N.lib().mac_quant_gather(self._h, n, s, k.data_ptr(), v.data_ptr(),
                                                                _stream_ptr(stream, self.device)), self._h)
        return k, v

    # -- attention ------------------------------------------------------------
    def attention(self, q, page_table, lengths, out=None, lse=None, want_lse=True, stream=None):
        """Decode attention: q bf16 [batch, heads, 128] or [batch, n_query, heads, 128] over the tokens that
        page_table int32 [batch, columns] and lengths int32 [batch] name; query i of n sees the first
        length - (n - 1) + i tokens.  Returns (out, lse) of q's shape (lse without the last axis)."""
        B = q.shape[0]
        if q.dim() not in (3, 4):
            raise ValueError("q must be [batch, heads, 128] or [batch, n_query, heads, 128]")
        nq = q.shape[1] if q.dim() == 4 else 1
        shape = tuple(q.shape[:-2]) + (self.heads, self.head_dim)
        qp = _dev(q, "q", torch.bfloat16, shape, self.device)
        table, row, cols = _table(page_table, B, self.device)
        lp = _dev(lengths, "lengths", torch.int32, (B,), self.device)
        with _on(self.device, stream):
            if out is None:
                out = _out(shape, self.device)
            if lse is None and want_lse:
                lse = _out(shape[:-1], self.device, torch.float32)
            _check("mac_quant_attention",
                   N.lib().mac_quant_attention(self._h, B, nq, qp, table, row, cols, lp,
                                               _dev(out, "out", torch.bfloat16, shape, self.device),
                                               None if lse is None else _dev(lse, "lse", torch.float32, shape[:-1],
                                                                             self.device),
                                               _stream_ptr(stream, self.device)), self._h)
        return out, lse

    def decode_step_qkv(self, rotary, qkv, positions, slots, page_table, lengths, q_weight=None, k_weight=None,
                        stream=None, starts=None):
        """One layer's step from its QKV projection: norm and rotation, append, attention.

        qkv [batch * n_query, (heads + 2 kv_heads) * 128]: row b * n_query + i is request b's i-th new token;
        positions, slots, lengths (the tokens after the step) and starts as page_step gives them.  Without
        starts every request must have n_query new tokens; with them, a request without any (an idle or
        finished one of a padded batch), or one that page_step denied, is left out: nothing of its rows is
        stored, its out is 0 and its lse -inf.  So is a request with another number of new tokens, or whose
        slots are not those of its own row of page_table, which sync() then reports.  Returns (out, lse).
        """
        B = lengths.shape[0]
        if B == 0 or qkv.shape[0] % B:
            raise ValueError("qkv must hold the same number of new tokens for every request")
        if rotary.heads != self.heads or rotary.kv_heads != self.kv_heads:
            raise ValueError("rotary was made for other heads")
        n = qkv.shape[0]
        # what the attention would refuse, before anything is stored
        if not 1 <= n // B <= self.max_query or B > self.max_batch:
            raise ValueError(f"{n // B} query tokens for each of {B} requests; the handle was made for up to "
                             f"{self.max_query} of {self.max_batch}")
        table, row, cols = _table(page_table, B, self.device)
        if cols < 1 or row < cols:
            raise ValueError("page_table must have a column, and rows that do not overlap")
        packed = min(positions.numel(), slots.numel())
        if starts is None and packed < n:
            raise ValueError(f"positions and slots must hold the {n} new tokens, got {packed}")
        lp = _dev(lengths, "lengths", torch.int32, (B,), self.device)
        pp = _dev(positions, "positions", torch.int32, (positions.numel(),), self.device)
        sp = _dev(slots, "slots", torch.int32, (slots.numel(),), self.device)
        first = None if starts is None else _dev(starts, "starts", torch.int32, (B + 1,), self.device)
        with _on(self.device, stream):
            rows = _out((2 * n + B,), self.device, torch.int32)
            pos, slot, lens = rows[:n], rows[n:2 * n], rows[2 * n:]
            _check("mac_quant_step_rows",
                   N.lib().mac_quant_step_rows(self._h, B, n // B, packed, first, pp, sp, table, row, cols, lp,
                                               pos.data_ptr(), slot.data_ptr(), lens.data_ptr(),
                                               _stream_ptr(stream, self.device)), self._h)
        _, q, k, v = rotary(qkv, pos, q_weight, k_weight, want_pre=False, stream=stream)
        self.append(k, v, slot, stream=stream)
        return self.attention(q.view(B, n // B, self.heads, self.head_dim), page_table, lens, stream=stream)

    def sync(self):
        """Wait for the device; raises MacError if its checks met a bad slot, page, length or row since the last call."""
        with _on(self.device, None):
            _check("mac_quant_sync", N.lib().mac_quant_sync(self._h), self._h)

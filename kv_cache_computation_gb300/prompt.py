"""Causal attention of whole prompts (the mac_prompt_* calls of include/mac.h)."""
from __future__ import annotations

import ctypes

import torch

from . import _native as N
from .attention import _dev, _on, _out, _stream_ptr
from .rotary import _rows


def _check(fn, status, handle=None):
    if status != N.MAC_OK:
        detail = (N.lib().mac_prompt_last_error(handle) or b"").decode() if handle is not None and handle.value else ""
        raise N.MacError(fn, status, detail)


def prompt_query_sizes(cfg: N.MacPromptConfig):
    """scratch_bytes for a configuration (host only)."""
    scratch = ctypes.c_size_t()
    _check("mac_prompt_query_sizes", N.lib().mac_prompt_query_sizes(ctypes.byref(cfg), ctypes.byref(scratch)))
    return scratch.value


class PromptAttention:
    """Causal attention of prompts packed behind one another, on the current CUDA device.

    attend(q, k, v, starts) -> (out, lse): q bf16 [tokens, heads, 128], k and v
    bf16 [keys, kv_heads, 128], post-RoPE (tokens may stand apart, so slices of a
    projection are read in place).  Sequence b's queries are rows starts[b] ..
    starts[b + 1] - 1 of q and its keys rows k_starts[b] .. of k and v (starts
    and k_starts int32 [batch + 1] on the GPU; k_starts None: the same rows), and
    its queries are the last of its tokens: query i of n over m keys sees the
    first m - n + i + 1 - lag of them.  So a chunk of a prompt comes behind the
    keys of what was there before, and with lag = r the rows are the summaries
    AS_{1:pos-r} that MacAttention.seed_ring takes.  A query that sees nothing
    gives out 0, lse -inf.  Rows of q that belong to no sequence are not written.

    max_tokens query tokens and max_batch sequences per call.  Calls on one
    object must be ordered with one another (they share its scratch, 101 MB
    whatever the sizes); objects whose calls are ordered may share scratch: pass
    another as `share`.
    """

    def __init__(self, heads, kv_heads, max_tokens, max_batch=1, head_dim=128, sm_scale=0.0, device=None, share=None):
        self.cfg = N.MacPromptConfig(heads, kv_heads, head_dim, max_tokens, max_batch, float(sm_scale))
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.max_tokens, self.max_batch = max_tokens, max_batch
        device = torch.device("cuda" if device is None else device)
        self.device = torch.device("cuda", torch.cuda.current_device()) if device.index is None else device
        self._h = ctypes.c_void_p()
        scratch = prompt_query_sizes(self.cfg)
        self.sizes = dict(scratch=scratch)
        with torch.cuda.device(self.device):
            if share is not None:
                if not isinstance(share, PromptAttention) or share.device != self.device or share._scratch.numel() < scratch:
                    raise ValueError("share must be a PromptAttention on the same device")
                self._scratch = share._scratch
            else:
                self._scratch = torch.empty(scratch, dtype=torch.uint8, device=self.device)
            h = ctypes.c_void_p()
            _check("mac_prompt_create",
                   N.lib().mac_prompt_create(ctypes.byref(self.cfg), self._scratch.data_ptr(), scratch, ctypes.byref(h)))
        self._h = h

    # -- lifetime -----------------------------------------------------------
    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            N.lib().mac_prompt_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- attention ------------------------------------------------------------
    def __call__(self, q, k, v, starts, k_starts=None, lag=0, out=None, lse=None, want_lse=True, out_dtype=torch.bfloat16,
                 stream=None):
        """out [tokens, heads, 128] (out_dtype: bfloat16 or float32) and lse float32 [tokens, heads] (natural log); an out
        of the caller's starts on a multiple of 32 bytes.  The outputs carry no gradient."""
        dev, n, m = self.device, q.shape[0], k.shape[0]
        if v.shape[0] != m:
            raise ValueError("k and v must hold the same tokens")
        if q.device != dev or k.device != dev or v.device != dev:
            raise ValueError(f"q, k and v must be on {dev}")
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("out_dtype must be torch.bfloat16 or torch.float32")
        if k_starts is None and n != m:
            raise ValueError("without k_starts, q and k must hold the same tokens")
        qp, qs = _rows(q, "q", self.heads, self.head_dim)
        kp, ks = _rows(k, "k", self.kv_heads, self.head_dim)
        vp, vs = _rows(v, "v", self.kv_heads, self.head_dim)
        B = starts.numel() - 1
        if B < 0:
            raise ValueError("starts must hold batch + 1 entries")
        sp = _dev(starts, "starts", torch.int32, (B + 1,), dev)
        kst = None if k_starts is None else _dev(k_starts, "k_starts", torch.int32, (B + 1,), dev)
        shape = (n, self.heads, self.head_dim)
        op = None if out is None else _dev(out, "out", out_dtype, shape, dev)
        lp = None if lse is None else _dev(lse, "lse", torch.float32, shape[:-1], dev)
        with _on(dev, stream):
            if out is None:
                out = _out(shape, dev, out_dtype)
                op = out.data_ptr()
            if lse is None and want_lse:
                lse = _out(shape[:-1], dev, torch.float32)
                lp = lse.data_ptr()
            status = N.lib().mac_prompt_attention(self._h, B, n, m, lag, qp, qs, kp, ks, vp, vs, sp, kst, op,
                                                  int(out_dtype == torch.float32), lp, _stream_ptr(stream, dev))
        if status:
            _check("mac_prompt_attention", status, self._h)
        return out, lse

    def sync(self):
        """Wait for the device; raises MacError if its checks met a bad sequence since the last call."""
        with _on(self.device, None):
            _check("mac_prompt_sync", N.lib().mac_prompt_sync(self._h), self._h)

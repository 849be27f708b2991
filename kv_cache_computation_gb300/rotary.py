"""Per-head norms, rotary embedding and split of a QKV projection
(mac_qkv_norm_rope of include/mac.h)."""
from __future__ import annotations

import ctypes

import torch

from . import _native as N
from .attention import _check, _dev, _on, _stream_ptr


def _rows(t, name, heads, head_dim):
    """(pointer, stride) of a bf16 tensor [tokens, heads * head_dim] or [tokens,
    heads, head_dim] whose tokens may stand apart but whose heads are dense."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    shape, stride = t.shape, t.stride()
    if len(shape) == 3:
        ok = shape[1:] == (heads, head_dim) and stride[2] == 1 and (heads == 1 or stride[1] == head_dim)
    else:
        ok = len(shape) == 2 and shape[1] == heads * head_dim and stride[1] == 1
    if not ok and t.numel():
        raise ValueError(f"{name} must be [tokens, {heads} x {head_dim}] with dense tokens, got shape {tuple(shape)}, "
                         f"strides {stride}")
    # a single token's stride is never used; torch may report anything for it
    return t.data_ptr(), stride[0] if shape[0] > 1 else heads * head_dim


class QkvRotary:
    """The norm and rotation between a layer's QKV projection and its attention.

    rot(qkv, positions, q_weight, k_weight) -> (q_pre, q_post, k, v): the
    queries before and after the rotation (the decode step's q_pre and q_post),
    the rotated keys and the values, all bf16 and dense.  qkv is [tokens,
    (heads + 2 kv_heads) * 128] bf16 (rows may stand apart), positions int32
    [tokens] on the same GPU, the weights bf16 [128] or None for no norm.

    The outputs carry no gradient.  rotary_dim: the first elements of a head
    that are rotated (a multiple of 8); interleaved: pairs (2i, 2i+1) instead of (i, i + rotary_dim/2).
    """

    def __init__(self, heads, kv_heads, head_dim=128, rotary_dim=128, base=500000.0, interleaved=False, eps=1e-6):
        cfg = N.MacRopeConfig(heads, kv_heads, head_dim, rotary_dim, int(interleaved), float(eps), float(base))
        self._rope = N.MacRope()
        _check("mac_rope_init", N.lib().mac_rope_init(ctypes.byref(cfg), ctypes.byref(self._rope)))
        self._ref = ctypes.byref(self._rope)
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self._all = heads + 2 * kv_heads
        self._k_at, self._v_at = 2 * heads * head_dim, 2 * (heads + kv_heads) * head_dim     # bytes into a token's row

    def __call__(self, qkv, positions, q_weight=None, k_weight=None, want_pre=True, stream=None):
        at, stride = _rows(qkv, "qkv", self._all, self.head_dim)
        return self._run(qkv, at, stride, at + self._k_at, stride, at + self._v_at, stride, positions, q_weight, k_weight,
                         want_pre, stream)

    def split(self, q, k, v, positions, q_weight=None, k_weight=None, want_pre=True, stream=None):
        """The same from separate projections q [tokens, heads * 128], k and v [tokens, kv_heads * 128]."""
        T = q.shape[0]
        if k.shape[0] != T or v.shape[0] != T:
            raise ValueError("q, k and v must hold the same tokens")
        if k.device != q.device or v.device != q.device:
            raise ValueError("q, k and v must be on one device")
        qp, qs = _rows(q, "q", self.heads, self.head_dim)
        kp, ks = _rows(k, "k", self.kv_heads, self.head_dim)
        vp, vs = _rows(v, "v", self.kv_heads, self.head_dim)
        return self._run(q, qp, qs, kp, ks, vp, vs, positions, q_weight, k_weight, want_pre, stream)

    def _run(self, like, q, qs, k, ks, v, vs, positions, q_weight, k_weight, want_pre, stream):
        T, device, d = like.shape[0], like.device, self.head_dim
        pos = _dev(positions, "positions", torch.int32, (T,), device)
        wq = None if q_weight is None else _dev(q_weight, "q_weight", torch.bfloat16, (d,), device)
        wk = None if k_weight is None else _dev(k_weight, "k_weight", torch.bfloat16, (d,), device)
        qshape, kshape = (T, self.heads, d), (T, self.kv_heads, d)
        with _on(device, stream):
            new = like.new_empty
            q_post, k_out, v_out = new(qshape), new(kshape), new(kshape)
            q_pre = new(qshape) if want_pre else None
            status = N.lib().mac_qkv_norm_rope(self._ref, T, q, qs, k, ks, v, vs, wq, wk, pos,
                                               None if q_pre is None else q_pre.data_ptr(), q_post.data_ptr(),
                                               k_out.data_ptr(), v_out.data_ptr(), _stream_ptr(stream, device))
        if status:
            _check("mac_qkv_norm_rope", status)
        return q_pre, q_post, k_out, v_out

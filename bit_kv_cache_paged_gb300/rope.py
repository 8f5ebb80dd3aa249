"""Rotary positions of query and key rows (oscar_rope_*), with PyTorch tensors."""
from __future__ import annotations

import ctypes

import torch

from . import binding as B
from .pool import HEAD_DIM, _need, _on_current_device, _raw_stream

SCALING = {"none": 0, "linear": 1, "base": 2, "ramp": 3}
_BF16 = torch.bfloat16


def _rows(t, n, name):
    """Row stride (elements) of bf16 [n, heads, 128] whose tokens may be apart (a slice of packed qkv rows)."""
    # the checks as one expression: a decode step calls this for every layer, and its launches are short
    if type(t) is torch.Tensor and t.dtype is _BF16 and t.dim() == 3:
        tokens, heads, dim = t.shape
        s0, s1, s2 = t.stride()
        if tokens == n and heads > 0 and dim == HEAD_DIM and s2 == 1 and (s1 == HEAD_DIM or heads == 1) and _on_current_device(t):
            return s0 if n > 1 else heads * HEAD_DIM
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != _BF16:
        raise TypeError(f"{name} must be {_BF16}, got {t.dtype}")
    if t.dim() != 3 or t.shape[0] != n or t.shape[1] < 1 or t.shape[2] != HEAD_DIM:
        raise ValueError(f"{name} must have shape ({n}, heads, {HEAD_DIM}), got {tuple(t.shape)}")
    if not _on_current_device(t):
        raise ValueError(f"{name} must be on the current CUDA device")
    if t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != HEAD_DIM):
        raise ValueError(f"{name}: heads of a token must be contiguous")
    return t.stride(0) if n > 1 else t.shape[1] * HEAD_DIM


class Rope:
    """Rotary positions of one configuration: pairs (j, j + rot_dim/2), or neighbours when interleaved, of the
    first rot_dim dims; scaling "none", "linear", "base" or "ramp" by `factor` for long contexts ("ramp" between
    the pairs that turn beta_fast and beta_slow times in original_len positions); amplitude None takes the
    scaling's own."""

    def __init__(self, rot_dim=HEAD_DIM, interleaved=False, base=10000.0, scaling="none", factor=1.0, original_len=0,
                 beta_fast=32.0, beta_slow=1.0, amplitude=None):
        if scaling not in SCALING:
            raise ValueError(f"scaling must be one of {sorted(SCALING)}, got {scaling!r}")
        self.cfg = B.OscarRopeConfig(rot_dim, 1 if interleaved else 0, SCALING[scaling], original_len, base, factor,
                                     beta_fast, beta_slow, 0.0 if amplitude is None else amplitude)
        self.table = B.oscar_rope_init(self.cfg)
        self._ref = ctypes.byref(self.table)

    def apply(self, q, k, positions, q_out=None, k_out=None):
        """Rotate bf16 q [n, Hq, 128] and k [n, Hkv, 128] (None: q alone) at int32 positions [n] in one launch.
        Rows may be strided by token. Returns (q_out, k_out), new contiguous tensors unless given (q_out=q
        rotates in place)."""
        n = q.shape[0] if isinstance(q, torch.Tensor) and q.dim() == 3 else -1
        qs = _rows(q, n, "q")
        hq = q.shape[1]
        if q_out is None:
            q_out, qos = torch.empty((n, hq, HEAD_DIM), dtype=_BF16, device=q.device), hq * HEAD_DIM
        else:
            qos = _rows(q_out, n, "q_out")
            if q_out.shape != q.shape:
                raise ValueError(f"q_out must have shape {tuple(q.shape)}, got {tuple(q_out.shape)}")
        if k is None:
            if k_out is not None:
                raise ValueError("k_out without k")
            hk = ks = kos = 0
            kp = kop = None
        else:
            ks, hk = _rows(k, n, "k"), k.shape[1]
            if k_out is None:
                k_out, kos = torch.empty((n, hk, HEAD_DIM), dtype=_BF16, device=k.device), hk * HEAD_DIM
            else:
                kos = _rows(k_out, n, "k_out")
                if k_out.shape != k.shape:
                    raise ValueError(f"k_out must have shape {tuple(k.shape)}, got {tuple(k_out.shape)}")
            kp, kop = k.data_ptr(), k_out.data_ptr()
        _need(positions, torch.int32, (n,), "positions")
        if positions.get_device() != q.get_device():
            raise ValueError("positions must be on the device of q")
        B._check("oscar_rope_apply", B.lib().oscar_rope_apply(self._ref, n, positions.data_ptr(), hq, q.data_ptr(), qs,
                                                              q_out.data_ptr(), qos, hk, kp, ks, kop, kos, _raw_stream()))
        return q_out, k_out

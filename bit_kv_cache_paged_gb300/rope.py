"""Rotary positions of query and key rows (oscar_rope_*), with PyTorch tensors."""
from __future__ import annotations

import torch

from . import binding as B
from .pool import HEAD_DIM, _need, _stream

SCALING = {"none": 0, "linear": 1, "base": 2, "ramp": 3}


def _rows(t, n, name):
    """Row stride (elements) of bf16 [n, heads, 128] whose tokens may be apart (a slice of packed qkv rows)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() != 3 or t.shape[0] != n or t.shape[1] < 1 or t.shape[2] != HEAD_DIM:
        raise ValueError(f"{name} must have shape ({n}, heads, {HEAD_DIM}), got {tuple(t.shape)}")
    if not t.is_cuda or t.device.index != torch.cuda.current_device():
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

    def apply(self, q, k, positions, q_out=None, k_out=None):
        """Rotate bf16 q [n, Hq, 128] and k [n, Hkv, 128] (None: q alone) at int32 positions [n] in one launch.
        Rows may be strided by token. Returns (q_out, k_out), new contiguous tensors unless given (q_out=q
        rotates in place)."""
        n = q.shape[0] if isinstance(q, torch.Tensor) and q.dim() == 3 else -1
        args = []
        for x, y, name in ((q, q_out, "q"), (k, k_out, "k")):
            if x is None and name == "k":
                if y is not None:
                    raise ValueError("k_out without k")
                args += [0, None, 0, None, 0]
                continue
            xs = _rows(x, n, name)
            if y is None:
                y = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
            ys = _rows(y, n, name + "_out")
            if y.shape != x.shape:
                raise ValueError(f"{name}_out must have shape {tuple(x.shape)}, got {tuple(y.shape)}")
            args += [x.shape[1], x, xs, y, ys]
        _need(positions, torch.int32, (n,), "positions")
        B.oscar_rope_apply(self.table, n, positions, *args, _stream())
        return args[3], args[8]

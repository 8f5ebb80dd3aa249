"""Attention in 64 bits with a bound on the error of a whole output row, narrow enough that a lost block of keys shows.

A row's error is bounded in the 2-norm, which a rotation keeps. With p the softmax weights and A = sum_s p_s |v_s| of a part of
the keys, in the basis where its weights meet its values:
  2^-8 |o|             the output's rounding to bf16
  w |A|                weights (and values) of the part rounded by w: 2^-8 for bf16 weights; 2^-9 for fp16 weights, twice where
                       a stored weight is scaled, fp16 values (2^-11 each) and the two limbs of the un-rotation (2^-16)
  sum_s p_s d_s (|v_s| + |o|)   scores off by d_s: sum_i |q_i k_si| 2^-17 / sqrt(128) for fp32 additions of exact products, and
                       where q R_K and k^ are rounded to fp16 six standard deviations of 128 products with two independent
                       roundings, each even over 2^-11 either way (2^-11 / sqrt(3)), and 2^-16 for the limbs of R_K.
Queries point at three keys each (`pointed`), which draw most of the attention: outputs are then of the size of a value."""
import math

import torch

E = 128
BF16_WEIGHTS, INT2_WEIGHTS = 2.0 ** -8, 2.0 ** -9 + 2.0 ** -16


def pointed(g, keys, rows, plain=None):
    """[len(rows), E] bf16 queries, each the sum of the three keys [n, E] that rows names, dims outside `plain` left out."""
    assert 0 <= int(rows.min()) and int(rows.max()) < len(keys)
    q = 0.9 * keys[rows].double().sum(1)
    if plain is not None:
        q = q * plain
    return (q + 0.1 * torch.randn(q.shape, generator=g, device=q.device, dtype=torch.float64)).bfloat16()


def reference(parts, seen=None):
    """parts: (q in the part's basis [r, E], k [n, E], v [n, E], back [E, E] or None: the values' way to the output, INT2 or not);
    seen [r, all n] bool. Returns (o [r, E], bound [r]) in 64 bits; rows that see nothing are zero."""
    s, d, sizes = [], [], []
    for q, k, v, back, int2 in parts:
        q, k = q.double(), k.double()
        s.append(q @ k.T / math.sqrt(E))
        e = (q.abs() @ k.abs().T) * (2.0 ** -16 if int2 else 2.0 ** -17)
        if int2:
            e = e + 6 * math.sqrt(2 / 3) * 2.0 ** -11 * ((q * q) @ (k * k).T).sqrt()
        d.append(e / math.sqrt(E))
        sizes.append(len(k))
    s, d = torch.cat(s, -1), torch.cat(d, -1)
    if seen is not None:
        s = s.masked_fill(~seen, -math.inf)
    p = torch.softmax(s, -1).nan_to_num(0.0)
    o = 0
    bound = 0
    for pp, dd, (_, _, v, back, int2) in zip(p.split(sizes, -1), d.split(sizes, -1), parts):
        v = v.double()
        x = pp @ v
        o = o + (x if back is None else x @ back)
        bound = bound + (INT2_WEIGHTS if int2 else BF16_WEIGHTS) * (pp @ v.abs()).norm(dim=-1) + (pp * dd) @ v.norm(dim=-1)
    bound = bound + o.norm(dim=-1) * (2.0 ** -8 + (p * d).sum(-1)) + 1e-6
    return o, bound


def check_rows(got, o, bound, what=""):
    r = (got.double() - o).norm(dim=-1) / bound
    assert (r <= 1).all(), f"{what}: {int((~(r <= 1)).sum())} of {r.numel()} rows off, worst {r.max():.3g} bounds"

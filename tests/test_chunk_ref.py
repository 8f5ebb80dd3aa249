"""The row bound of chunk_ref on the CPU: the roundings that a kernel is allowed pass, mistakes of a kernel's kind do not."""
import math

import pytest
import torch

import oracle as O
from chunk_ref import E, check_rows, pointed, reference

ROWS = 40


def quantised(x, group):
    """Codes restored with fp16 scale and zero: [n, E]."""
    t = x.view(len(x), E // group, group)
    lo, hi = 0.9 * t.amin(-1, keepdim=True), 0.9 * t.amax(-1, keepdim=True)
    s, z = ((hi - lo) / 3).half().double(), lo.half().double()
    return (((t - z) / s).round().clamp(0, 3) * s + z).reshape(len(x), E)


def case(n, group, seed):
    """A cache of n INT2 tokens and 320 BF16 ones with strong channels, rotations, and queries that point at keys everywhere."""
    g = torch.Generator().manual_seed(seed)
    gain = torch.ones(E, dtype=torch.float64)
    gain[5] = 8
    k, v = ((torch.randn((n + 320, E), generator=g, dtype=torch.float64) * gain).bfloat16().double() for _ in "kv")
    rk, rv = (torch.from_numpy(O.rotation_matrix(torch.linalg.qr(torch.randn((E, E), generator=g, dtype=torch.float64))[0].float().numpy())) for _ in "kv")
    at = torch.randint(0, n + 320, (ROWS, 3), generator=g)
    at[0], at[1], at[2] = torch.tensor([3, 77, 127]), torch.tensor([n - 1, n - 9, n - 30]), torch.tensor([n + 1, n + 319, n + 64])
    q = pointed(g, k, at, plain=(gain == 1).double()).double()
    return q, quantised(k[:n] @ rk, group), quantised(v[:n] @ rv, group), k[n:], v[n:], rk, rv


def parts(q, kh, vh, kb, vb, rk, rv):
    return [(q @ rk, kh, vh, rv.T, True), (q, kb, vb, None, False)]


def as_a_kernel(q, kh, vh, kb, vb, rk, rv):
    """The roundings of a chunk kernel: fp16 rotated queries, values and weights, bf16 weights, bf16 outputs."""
    qh = q @ rk
    top = qh.abs().amax(-1, keepdim=True)
    qh = (qh / top).half().double() * top
    s = torch.cat([qh @ kh.half().double().T, q @ kb.T], -1) / math.sqrt(E)
    w = torch.exp(s - s.amax(-1, keepdim=True) + 1.3)  # under a maximum that is not this row's last
    n = len(kh)
    o = w[:, :n].half().double() @ vh.half().double() @ rv.T + w[:, n:].bfloat16().double() @ vb
    return (o / w.sum(-1, keepdim=True)).bfloat16()


@pytest.mark.parametrize("group", [128, 32])
@pytest.mark.parametrize("n", [64, 1000, 3900, 9000])
def test_allowed_roundings_pass_and_mistakes_do_not(n, group):
    c = case(n, group, n + group)
    o, bound = reference(parts(*c))
    check_rows(o.bfloat16(), o, bound, "rounded")
    check_rows(as_a_kernel(*c), o, bound, "kernel's roundings")
    assert (bound <= 0.06 * o.norm(dim=-1)).all()
    q, kh, vh, kb, vb, rk, rv = c
    eye = torch.eye(E, dtype=torch.float64)
    wrong = {
        "nothing": torch.zeros_like(o),
        "values x 0.8": reference(parts(q, kh, 0.8 * vh, kb, vb, rk, rv))[0],
        "no un-rotation": reference(parts(q, kh, vh, kb, vb, rk, eye))[0],
        "no rotation": reference(parts(q, kh, vh, kb, vb, eye, rv))[0],
        "first block left out": reference(parts(q, kh[128:], vh[128:], kb, vb, rk, rv))[0],
        "last page left out": reference(parts(q, kh[:-64], vh[:-64], kb, vb, rk, rv))[0],
        "BF16 keys left out": reference(parts(q, kh, vh, kb[:0], vb[:0], rk, rv))[0],
        "values of the next token": reference(parts(q, kh, vh.roll(1, 0), kb, vb, rk, rv))[0],
        "a half block twice": reference(parts(q, torch.cat([kh, kh[64:128] if n > 64 else kh]), torch.cat([vh, vh[64:128] if n > 64 else vh]), kb, vb, rk, rv))[0],
        "another scale of scores": reference(parts(1.05 * q, kh, vh, kb, vb, rk, rv))[0],
        "sums not scaled": o * 1.1,
    }
    for what, x in wrong.items():
        with pytest.raises(AssertionError):
            check_rows(x, o, bound, what)

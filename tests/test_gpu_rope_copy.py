"""Rotary positions against a 64-bit rotation, and page copies bit for bit.

Tolerance of a rotated value: the bf16 rounding, half a step (2^-8 relative), and the fp32 arithmetic before it: cos and
sin within 2^-22 (angle 2^-24 of half a turn, sincospif a few ulp) times |u| + |v|, doubled."""
import math

import numpy as np
import pytest
import torch

from bit_kv_cache_paged_gb300 import Rope, bf16_copy_pages
from bit_kv_cache_paged_gb300 import binding as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


def rotated(x, pos, w, amp, rot, inter):
    """(value, tolerance) in 64 bits."""
    ang = pos.double()[:, None] * w
    c, s = amp * ang.cos()[:, None], amp * ang.sin()[:, None]
    x = x.double()
    y, m = x.clone(), torch.zeros_like(x)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    u, v = x[..., a], x[..., b]
    y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    m[..., a] = m[..., b] = amp * (u.abs() + v.abs())
    return y, 2.0 ** -8 * y.abs() + 2.0 ** -21 * m + 2.0 ** -134


@pytest.mark.parametrize("n", [1, 2, 37])
@pytest.mark.parametrize("hq,hkv", [(1, 0), (4, 1), (33, 8)])
@pytest.mark.parametrize("rot,inter", [(16, False), (48, True), (112, False), (128, False), (128, True)])
def test_rope_against_64_bits(n, hq, hkv, rot, inter):
    g = torch.Generator(device="cuda").manual_seed(n * 1000 + hq * 10 + rot)
    packed = torch.randn((n, hq + hkv + 3, 128), generator=g, device="cuda").bfloat16()  # a packed row, other columns around
    q, k = packed[:, 1:1 + hq], packed[:, 2 + hq:2 + hq + hkv] if hkv else None
    pos = torch.randint(-1000, 2 ** 31 - 1, (n,), generator=g, device="cuda").int()
    pos[0] = 0 if n > 1 else pos[0]
    r = Rope(rot_dim=rot, interleaved=inter, base=1e6, scaling="ramp", factor=4.0, original_len=32768)
    w = torch.tensor([float(r.table.turns[j]) for j in range(rot // 2)], dtype=torch.float64, device="cuda") * 2.0 ** -64
    # the angle in 64 bits from the table's exact turns (far positions would lose it in p * w otherwise)
    turns = [[(int(p) * int(r.table.turns[j])) % 2 ** 64 / 2.0 ** 64 for j in range(rot // 2)] for p in pos.tolist()]
    ang = torch.tensor(turns, dtype=torch.float64, device="cuda") * 2 * math.pi
    assert w.max() < 0.16
    yq, yk = r.apply(q, k, pos)
    for x, y in ((q, yq), (k, yk)):
        if x is None:
            assert y is None
            continue
        ref, tol = rotated(x, torch.ones_like(pos), ang, r.table.amplitude, rot, inter)
        assert y.is_contiguous()
        assert ((y.double() - ref).abs() <= tol).all()
        assert torch.equal(y[..., rot:], x[..., rot:])
    # in place, inside the packed rows: the same values, nothing around them touched
    keep = packed.clone()
    r.apply(q, k, pos, q_out=q, k_out=k)
    assert torch.equal(q, yq) and (k is None or torch.equal(k, yk))
    mask = torch.ones(packed.shape[1], dtype=torch.bool)
    mask[1:1 + hq] = False
    mask[2 + hq:2 + hq + hkv] = False
    assert torch.equal(packed[:, mask.cuda()], keep[:, mask.cuda()])


def test_rope_keeps_the_angle_of_far_positions():
    # positions p and p + 1 a million tokens in differ by one turn of w: scores depend on distance alone
    r = Rope(base=10000.0)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((1, 1, 128), generator=g, device="cuda").bfloat16().expand(4, 1, 128).contiguous()
    y, _ = r.apply(x, None, torch.tensor([5, 17, 1000005, 1000017], device="cuda", dtype=torch.int32))
    y = y[:, 0].double()
    # |x|^2 of products of two bf16 roundings (2^-8 each): 2 * 2^-8 * |x|^2
    assert abs((y[0] @ y[1] - y[2] @ y[3]).item()) <= 4 * 2.0 ** -8 * (y[0] @ y[0]).item()


def test_rope_of_nothing_and_special_values():
    r = Rope(rot_dim=64)
    q = torch.empty((0, 4, 128), dtype=torch.bfloat16, device="cuda")
    y, _ = r.apply(q, None, torch.empty(0, dtype=torch.int32, device="cuda"))
    assert y.shape == q.shape
    x = torch.zeros((1, 1, 128), dtype=torch.bfloat16, device="cuda")
    x[0, 0, 70], x[0, 0, 3] = math.nan, math.inf
    y, _ = r.apply(x, None, torch.tensor([1], device="cuda", dtype=torch.int32))
    assert y[0, 0, 70].isnan() and not y[0, 0, 3].isfinite() and not y[0, 0, 35].isfinite()
    assert y[0, 0, [0, 1, 2, 4, 36, 64, 127]].isfinite().all()


def test_rope_under_capture_follows_positions():
    r = Rope()
    q = torch.randn((8, 4, 128), device="cuda").bfloat16()
    pos, out = torch.arange(8, device="cuda", dtype=torch.int32), torch.empty_like(q)
    r.apply(q, None, pos, q_out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.apply(q, None, pos, q_out=out)
    pos += 1000
    graph.replay()
    want, _ = r.apply(q, None, pos)
    assert torch.equal(out, want)


@pytest.mark.parametrize("layers,pages,hkv,moves", [(1, 2, 1, 1), (1, 9, 3, 4), (5, 40, 2, 13), (2, 2500, 1, 1200)])
def test_copy_pages_bit_for_bit(layers, pages, hkv, moves):
    g = torch.Generator(device="cuda").manual_seed(pages)
    k, v = (torch.randint(-2 ** 15, 2 ** 15, (layers, pages, hkv, 64, 128), generator=g, device="cuda").short().view(torch.bfloat16)
            for _ in range(2))
    perm = np.random.default_rng(pages).permutation(pages)
    dst = perm[:moves]
    src = np.random.default_rng(1).choice(perm[moves:], moves)  # a page may go to several places
    want = []
    for x in (k, v):
        y = x.view(torch.int16).clone()
        y[:, torch.from_numpy(dst).cuda()] = y[:, torch.from_numpy(src).cuda()]
        want.append(y)
    bf16_copy_pages(k, v, src.tolist(), dst.tolist())
    assert torch.equal(k.view(torch.int16), want[0]) and torch.equal(v.view(torch.int16), want[1])
    if layers == 1:  # the same through pages without a layer axis: nothing changes any more
        bf16_copy_pages(k[0], v[0], src.tolist(), dst.tolist())
        assert torch.equal(k.view(torch.int16), want[0])


def test_copy_pages_on_another_stream_and_in_a_graph():
    k = torch.randn((6, 2, 64, 128), device="cuda").bfloat16()
    v = torch.randn((6, 2, 64, 128), device="cuda").bfloat16()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bf16_copy_pages(k, v, [0, 0], [5, 3])
    k[0] += 1
    graph.replay()
    assert torch.equal(k[5], k[0]) and torch.equal(v[3], v[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        bf16_copy_pages(k, v, [1], [2])
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(k[2], k[1]) and torch.equal(v[2], v[1])


def test_copy_pages_past_32_bit_offsets():
    pages = 2 * (2 ** 32 // 16384) // 2 + 5  # one KV head: past 4 GB of K
    k = torch.zeros((pages, 1, 64, 128), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[-1], v[-1] = 3.0, 4.0
    bf16_copy_pages(k, v, [pages - 1], [pages - 3])
    assert (k[-3] == 3).all() and (v[-3] == 4).all() and k[:-3].count_nonzero() == 0
    with pytest.raises(B.OscarError):
        bf16_copy_pages(k, v, [pages], [0])

"""Refusals of the rotary, chunk-attention and page-copy entry points: bad arguments come back as status codes
before anything is launched (no GPU is needed; the addresses are never followed)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from bit_kv_cache_paged_gb300 import Rope, bf16_copy_pages
from bit_kv_cache_paged_gb300 import binding as B
from bit_kv_cache_paged_gb300 import build as BLD
from bit_kv_cache_paged_gb300.pool import Pool

A = 1 << 20  # an address with every alignment the calls ask for


@pytest.fixture(scope="module", autouse=True)
def built():
    BLD.build()


def refused(f, *a, status=B.OSCAR_EINVAL):
    with pytest.raises(B.OscarError) as e:
        f(*a)
    assert e.value.status == status


# ---------------------------------------------------------------- rotary positions
@pytest.mark.parametrize("bad", [dict(rot_dim=0), dict(rot_dim=8), dict(rot_dim=24), dict(rot_dim=144), dict(base=1.0),
                                 dict(base=math.inf), dict(base=math.nan), dict(factor=0.5, scaling="linear"),
                                 dict(factor=2.0), dict(factor=math.nan, scaling="linear"),
                                 dict(scaling="ramp", factor=2.0), dict(scaling="ramp", factor=2.0, original_len=100, beta_slow=0.0),
                                 dict(scaling="ramp", factor=2.0, original_len=100, beta_fast=0.5),
                                 dict(scaling="base", base=1e300, factor=1e300), dict(amplitude=-1.0), dict(amplitude=math.inf)])
def test_rope_configurations_refused(bad):
    refused(lambda: Rope(**bad))


def test_rope_unknown_scaling():
    with pytest.raises(ValueError):
        Rope(scaling="cubic")


@pytest.mark.parametrize("rot,inter", [(16, False), (64, True), (128, False)])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 4.0), ("base", 2.0), ("ramp", 8.0)])
def test_rope_table_is_the_frequency_in_turns(rot, inter, scaling, factor):
    r = Rope(rot_dim=rot, interleaved=inter, base=500000.0, scaling=scaling, factor=factor, original_len=4096)
    j = np.arange(rot // 2)
    base = 500000.0 * (factor ** (rot / (rot - 2)) if scaling == "base" else 1.0)
    w = base ** (-2.0 * j / rot)
    if scaling == "linear":
        w = w / factor
    if scaling == "ramp":
        at = [rot * math.log(4096 / (t * 2 * math.pi)) / (2 * math.log(base)) for t in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        t = np.clip((j - lo) / max(hi - lo, 0.001), 0, 1)
        w = w / factor * t + w * (1 - t)
    got = np.array([float(r.table.turns[i]) for i in j]) * 2.0 ** -64 * 2 * math.pi
    # the table holds whole units of 2^-64 of a turn: up to one unit (2 pi 2^-64 rad a position) below w, and a few
    # roundings of 64-bit arithmetic
    np.testing.assert_allclose(got, w, rtol=1e-14, atol=2 * math.pi * 2.0 ** -64)
    assert r.table.amplitude == np.float32(0.1 * math.log(factor) + 1 if scaling == "ramp" else 1)


def test_rope_apply_refused():
    t = Rope().table
    n, ok = 4, dict(positions=A, hq=2, q=A, qs=256, qo=2 * A, qos=256, hk=1, k=3 * A, ks=128, ko=4 * A, kos=128)

    def call(rope=t, n=n, **kw):
        a = dict(ok, **kw)
        B.oscar_rope_apply(rope, n, a["positions"], a["hq"], a["q"], a["qs"], a["qo"], a["qos"], a["hk"], a["k"], a["ks"],
                           a["ko"], a["kos"], None)

    for bad in (dict(n=-1), dict(positions=None), dict(positions=A + 2), dict(hq=-1), dict(q=None), dict(qo=None), dict(q=A + 8),
                dict(qo=2 * A + 2), dict(qs=128), dict(qs=260), dict(qos=128), dict(kos=-128), dict(hk=2), dict(hk=0),
                dict(hq=0, q=None, qo=None, hk=0, k=None, ko=None), dict(hq=0), dict(qo=A + 512), dict(qo=A, qos=512),
                dict(q=A, qs=512, qo=A + 256, qos=512), dict(ko=3 * A + 256)):
        refused(lambda bad=bad: call(**bad))
    bent = B.OscarRope(rot_dim=20, interleaved=0, amplitude=1.0)
    refused(lambda: call(rope=bent))
    call(n=0)  # nothing to do


def test_rope_python_checks():
    r = Rope()
    q = torch.zeros((3, 2, 128), dtype=torch.bfloat16)
    pos = torch.zeros(3, dtype=torch.int32)
    for args in ((q, None, pos), (q.float(), None, pos), (q[:, 0], None, pos)):  # host tensors, type, shape
        with pytest.raises((TypeError, ValueError)):
            r.apply(*args)


# ---------------------------------------------------------------- page copies
def test_copy_pages_refused():
    def call(hkv=2, layers=1, stride=0, k=A, v=2 * A, total=10, src=(1,), dst=(2,)):
        B.oscar_bf16_copy_pages(hkv, layers, stride, k, v, total, list(src), list(dst), None)

    for bad in (dict(hkv=0), dict(layers=0), dict(k=None), dict(v=None), dict(k=A + 8), dict(total=0), dict(src=(10,)), dict(src=(-1,)),
                dict(dst=(10,)), dict(dst=(-1,)), dict(src=(1,), dst=(1,)), dict(src=(1, 2), dst=(3, 3)),
                dict(src=(1, 2), dst=(2, 3)), dict(src=(1, 2), dst=(3,)), dict(layers=2, stride=10 * 2 * 16384 - 16),
                dict(layers=2, stride=10 * 2 * 16384 + 8)):
        refused(lambda bad=bad: call(**bad))
    call(src=(), dst=())
    with pytest.raises((TypeError, ValueError)):
        bf16_copy_pages(torch.zeros(4, 1, 64, 128, dtype=torch.bfloat16), torch.zeros(4, 1, 64, 128, dtype=torch.bfloat16), [0], [1])
    with pytest.raises(ValueError):
        bf16_copy_pages(torch.zeros(4, 128), torch.zeros(4, 128), [0], [1])


# ---------------------------------------------------------------- chunk attention
def test_bf16_chunk_refused():
    nb = B.oscar_bf16_chunk_workspace_bytes(8, 2, 3, 100)
    assert nb > 0
    for shape in ((8, 3, 1, 1), (24, 8, 1, 1), (8, 0, 1, 1), (64, 2, 1, 1), (8, 2, 0, 1), (8, 2, 1, -1)):
        assert B.oscar_bf16_chunk_workspace_bytes(*shape) == 0

    def call(hq=8, hkv=2, seqs=3, tokens=100, k=A, v=A, total=50, table=A, width=20, lens=A, cu=A, q=A, stride=1024, ws=A, ws_bytes=nb,
             out=A, err=A):
        B.oscar_bf16_chunk(hq, hkv, seqs, tokens, k, v, total, table, width, lens, cu, q, stride, ws, ws_bytes, out, err, None)

    for bad in (dict(hq=24, hkv=8), dict(hkv=0), dict(seqs=0), dict(tokens=-1), dict(k=None), dict(v=None), dict(k=A + 4),
                dict(v=A + 8), dict(total=0), dict(table=None), dict(width=0), dict(width=2 ** 31 - 1), dict(lens=None), dict(cu=None),
                dict(q=None), dict(q=A + 2), dict(stride=1023), dict(stride=1016), dict(ws=None), dict(ws=A + 8),
                dict(ws_bytes=nb - 1), dict(out=None), dict(out=A + 4), dict(err=None), dict(table=A + 2), dict(lens=A + 1), dict(cu=A + 2), dict(err=A + 2)):
        refused(lambda bad=bad: call(**bad))
    call(tokens=0)


def test_pool_chunk_refused_outside_a_device_step():
    p = Pool(2, 8, 2, max_seqs=2, max_seq_len=1000, max_int2_pages=20, host_only=True)
    assert B.oscar_chunk_workspace_bytes(None) == 0 and B.oscar_chunk_workspace_bytes(p.handle) == 0
    a = (A, A, A, A, A, None)
    refused(B.oscar_chunk_attend, None, 0, *a)
    refused(B.oscar_chunk_attend, p.handle, 2, *a)
    refused(B.oscar_chunk_attend, p.handle, -1, *a)
    refused(B.oscar_chunk_attend, p.handle, 0, *a, status=B.OSCAR_ESTATE)
    p.seq_add(0)
    p.step_begin([0], [5])
    refused(B.oscar_chunk_attend, p.handle, 0, *a)  # a host-only pool computes nothing
    with pytest.raises((TypeError, ValueError)):
        p.chunk_attend(0, torch.zeros(5, 8, 128, dtype=torch.bfloat16), None, None)


def test_structures_match_the_header():
    assert ctypes.sizeof(B.OscarRope) == 16 + 64 * 8 and ctypes.sizeof(B.OscarRopeConfig) == 16 + 5 * 8


def test_bf16_chunk_positions_stay_in_32_bits():
    nb = B.oscar_bf16_chunk_workspace_bytes(8, 2, 3, 100)
    for width in ((2 ** 31 - 1 - 4096) // 64 + 1, 2 ** 25):
        refused(B.oscar_bf16_chunk, 8, 2, 3, 100, A, A, 50, A, width, A, A, A, 1024, A, nb, A, A, None)


def test_copy_pages_ids_past_32_bits():
    for src, dst in (([2 ** 32 + 1], [2]), ([1], [2 ** 31])):
        with pytest.raises(OverflowError):
            B.oscar_bf16_copy_pages(2, 1, 0, A, 2 * A, 10, src, dst, None)

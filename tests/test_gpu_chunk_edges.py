"""Calls of chunk attention that stand at an edge: infinite keys, outputs on a 16-byte boundary alone, a process's first call
inside a capture, and the operators one after another as a server of the BF16 cache runs them."""
import math
import os
import subprocess
import sys

import pytest
import torch

from bit_kv_cache_paged_gb300 import Rope, bf16_chunk_attend, bf16_copy_pages
from bit_kv_cache_paged_gb300 import binding as B
from chunk_ref import check_rows, reference
from test_gpu_chunk import E, Mixed, Pages, built, check, softmax64  # noqa: F401

pytestmark = pytest.mark.gpu


def infinite(q, k, v, seen, out):
    """Rows that see a score of +inf (or a NaN) are NaN, a score of -inf has no weight, the others are as ever."""
    o, tol = softmax64(q, [(q, k.nan_to_num(nan=0, posinf=0, neginf=0), v, v.abs(), 2.0 ** -17)], seen)
    s = q.double() @ k.double().T
    with_inf = (((s == math.inf) | s.isnan()) & seen[:, None]).any(-1)
    gone = ((s == -math.inf) & seen[:, None]).any(-1)
    assert with_inf.any() and gone.any() and out[with_inf].isnan().all()
    at = ~(with_inf | gone)
    check(out[at], o[at], tol[at], "rows without it")
    at = gone & ~with_inf
    dead = (k.isinf()).any(-1)
    o, tol = softmax64(q, [(q, k.nan_to_num(posinf=0, neginf=0), v, v.abs(), 2.0 ** -17)], seen & ~dead[None])
    check(out[at], o[at], tol[at], "rows that lose a key")


@pytest.mark.parametrize("special", [math.inf, -math.inf])
@pytest.mark.parametrize("at", [0, 60, 120, 199])  # of the cache, the chunk, its last token
def test_bf16_an_infinite_key(special, at):
    c = Pages([200, 90], 1, seed=21)
    new = [150, 90]
    q = torch.randn((240, 4, E), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    q[149, 0, 17], q[149, 1, 17] = 1, -1  # both signs, where the last token alone sees the key
    good = c.attend(q, new)
    c.rows[0][0][at, 0, 17] = special
    c.put(c.k, 0, c.rows[0][0])
    out = c.attend(q, new)
    assert torch.equal(out[150:], good[150:]) and torch.equal(out[:max(0, at - 50)], good[:max(0, at - 50)])
    seen = torch.arange(200, device="cuda")[None] <= 50 + torch.arange(150, device="cuda")[:, None]
    infinite(q[:150], c.rows[0][0][:, 0], c.rows[0][1][:, 0], seen, out[:150])


def apart(t, n):
    """A copy of t's shape that starts 16 but not 32 bytes into a buffer of marks."""
    buf = torch.full((n + 24,), 7.0, dtype=torch.bfloat16, device="cuda")
    x = buf[8:8 + n].view(t.shape)
    assert x.data_ptr() % 32 == 16
    return buf, x


def test_outputs_16_bytes_in():
    c = Pages([300, 2000, 40], 2, seed=5)
    new = [300, 7, 20]
    q = torch.randn((327, 8, E), device="cuda").bfloat16()
    want = c.attend(q, new)
    buf, out = apart(want, want.numel())
    assert torch.equal(c.attend(q, new, out=out), want) and (buf[:8] == 7).all() and (buf[-16:] == 7).all()
    for hkv, ctx, steps in ((2, 1500, (1, 9, 400)), (8, 5400, (1,))):  # expanded in the kernel, tiles; the decode kernels
        m = Mixed(hq=4 * hkv, hkv=hkv, seed=6, max_seqs=1)
        m.add(0)
        m.pool.step_begin([0], [ctx])
        kv = m.new_rows(ctx)
        m.pool.append_and_demote(0, kv[0][0], kv[1][0])
        for n in steps:
            m.pool.step_begin([0], [n])
            k, v = (x[0] for x in m.new_rows(n))
            q = torch.randn((n, 4 * hkv, E), device="cuda").bfloat16()
            want = m.pool.chunk_attend(0, q, k, v)
            buf, out = apart(want, want.numel())
            assert torch.equal(m.pool.chunk_attend(0, q, k, v, out=out), want) and (buf[:8] == 7).all() and (buf[-16:] == 7).all()
            m.pool.append_and_demote(0, k, v)
        m.pool.check()


FIRST = """
import sys
sys.path[:0] = [%r, %r]
import torch
from test_gpu_chunk import E, Mixed, Pages
from bit_kv_cache_paged_gb300 import Rope, bf16_copy_pages
which = sys.argv[1]
g = torch.Generator(device="cuda").manual_seed(1)
graph = torch.cuda.CUDAGraph()
if which == "rope":
    x, pos = torch.randn((9, 4, E), generator=g, device="cuda").bfloat16(), torch.arange(9, device="cuda").int()
    call = lambda: Rope().apply(x, None, pos)[0]
elif which == "copy":
    k, v = (torch.randn((6, 1, 64, E), generator=g, device="cuda").bfloat16() for _ in "kv")
    def call():
        bf16_copy_pages(k, v, [0], [5])
        return k
elif which == "bf16":
    c = Pages([500, 900], 2, seed=9)
    q = torch.randn((6, 8, E), generator=g, device="cuda").bfloat16()
    cu, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 2, 6], [500, 900]))
    from bit_kv_cache_paged_gb300 import bf16_chunk_attend
    call = lambda: bf16_chunk_attend(q, c.k, c.v, c.table, lens, cu, c.err)
else:
    hkv, ctx, n = {"dequant": (2, 900, 9), "tiles": (1, 900, 400), "single": (8, 5400, 1)}[which]
    m = Mixed(hq=4 * hkv, hkv=hkv, max_seqs=1)
    m.add(0)
    m.pool.step_begin([0], [ctx])
    kv = m.new_rows(ctx)
    m.pool.append_and_demote(0, kv[0][0], kv[1][0])
    m.pool.step_begin([0], [n])
    k, v = (x[0] for x in m.new_rows(n))
    q = torch.randn((n, 4 * hkv, E), generator=g, device="cuda").bfloat16()
    call = lambda: m.pool.chunk_attend(0, q, k, v)
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    got = call()
graph.replay()
torch.cuda.synchronize()
assert torch.equal(got, call()) and got.isfinite().all() and got.abs().max() > 0
print("the same")
"""


@pytest.mark.parametrize("which", ["rope", "copy", "bf16", "dequant", "tiles", "single"])
def test_first_call_of_a_process_inside_a_capture(which):
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", FIRST % (os.path.dirname(here), here), which], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("the same"), r.stdout + r.stderr


def test_bf16_rotary_packed_rows_chunks_and_a_fork():
    """Rotated rows into pages, a prompt in chunks, the fork of its last page, then different tokens on both sides."""
    hq, hkv, pages = 8, 2, 12
    g = torch.Generator(device="cuda").manual_seed(2)
    st = torch.cuda.current_stream().cuda_stream
    k, v = (torch.full((pages, hkv, 64, E), math.nan, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    err, rope = torch.zeros(1, dtype=torch.int32, device="cuda"), Rope(base=5e5)
    table = torch.tensor([[3, 7, 0, 9, 11], [3, 7, 0, 1, 5]], dtype=torch.int32, device="cuda")  # the fork shares three full pages
    rows = [[torch.zeros((0, hkv, E), dtype=torch.bfloat16, device="cuda") for _ in "kv"] for _ in range(2)]

    def feed(seqs, n):
        raw = [torch.randn((n, hq + 2 * hkv, E), generator=g, device="cuda").bfloat16() for _ in seqs]
        qs = []
        for i, x in zip(seqs, raw):
            at = len(rows[i][0])
            q, kk = rope.apply(x[:, :hq], x[:, hq:hq + hkv], torch.arange(at, at + n, device="cuda").int())
            new = [kk, x[:, hq + hkv:].contiguous()]
            for y, p in zip(new, (k, v)):
                B.oscar_bf16_pack(y, n, at, hkv, table[i], pages, p, err, st)
            rows[i] = [torch.cat([a, b]) for a, b in zip(rows[i], new)]
            qs.append(q)
        q = torch.cat(qs)
        out = bf16_chunk_attend(q, k, v, table[seqs].contiguous(), torch.tensor([len(rows[i][0]) for i in seqs], dtype=torch.int32, device="cuda"),
                                torch.arange(len(seqs) + 1, device="cuda", dtype=torch.int32) * n, err)
        assert int(err) == 0
        for j, i in enumerate(seqs):
            L = len(rows[i][0])
            for h in range(hkv):
                x = q[j * n:j * n + n, h * 4:h * 4 + 4].reshape(-1, E)
                t = torch.arange(n * 4, device="cuda")[:, None] // 4
                o, bound = reference([(x, rows[i][0][:, h], rows[i][1][:, h], None, False)], torch.arange(L, device="cuda")[None] <= L - n + t)
                check_rows(out[j * n:j * n + n, h * 4:h * 4 + 4].reshape(-1, E), o, bound, f"seq {i}")
    feed([0], 130)
    feed([0], 70)  # 200: three pages and 8 rows of a fourth
    bf16_copy_pages(k, v, [9], [1])
    rows[1] = [x.clone() for x in rows[0]]
    feed([0, 1], 5)
    feed([1], 60)
    feed([0, 1], 1)


@pytest.mark.parametrize("ctx,new", [(0, 200), (900, 9), (900, 200), (900, 400)])
def test_pool_later_tokens_leave_the_bits_of_earlier_ones(ctx, new):
    """Keys of later tokens that outgrow every maximum, in all places of a warp's rows."""
    m = Mixed(hq=8, hkv=2, seed=8, max_seqs=1)
    m.add(0)
    if ctx:
        m.pool.step_begin([0], [ctx])
        kv = m.new_rows(ctx)
        m.pool.append_and_demote(0, kv[0][0], kv[1][0])
    m.pool.step_begin([0], [new])
    k, v = (x[0] for x in m.new_rows(new))
    q = torch.randn((new, 8, E), generator=m.g, device="cuda").bfloat16()
    good = m.pool.chunk_attend(0, q, k, v)
    for at in sorted({new - 1, new - 2, new - 7, new // 2, new // 2 + 3} & set(range(new))):
        loud = k.clone()
        loud[at] *= 30
        out = m.pool.chunk_attend(0, q, loud, v)
        assert torch.equal(out[:at], good[:at]) and not torch.equal(out[at], good[at])
    m.pool.check()

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

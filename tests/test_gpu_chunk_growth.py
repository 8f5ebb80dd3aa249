"""Chunk attention where later keys outgrow the maximum of earlier ones, against softmax attention in 64 bits.

The kernels renew a row's maximum only where a block's weights outgrow it, so scores are chosen here: key s has the level
l_s (a power of two of its weight) up to small differences, along one of the stairs below. The caches hold exact numbers, so
that nothing but the weights and the output is rounded: the rotations are the permutation H H P, queries are multiples of
2^-5, INT2 rows z + code / 4 with z a multiple of 2^-6.

Tolerance of an output value o = sum_s p_s v_s, with A = sum_s p_s |v_s| over the BF16 and the INT2 keys apart:
  2^-8 |o|      the output's own rounding
  2^-8 A_bf16   weights rounded to bf16
  2^-10 A_int2  weights rounded to fp16, twice where a stored weight is scaled by a new maximum (2^-11 each), and the two bf16
                limbs of the un-rotation (2^-16)
  2 d A         scores off by d = sum_i |q_i k_si| 2^-17 / sqrt(128) (fp32 additions of exact products), weighted by p
  2^-24 sum_s |v_s|   fp16 weights below 2^-14 of a maximum of at least 1 are off by 2^-25"""
import math

import numpy as np
import pytest
import torch

import oracle as O
from bit_kv_cache_paged_gb300 import Pool
from test_gpu_chunk import E, Pages, built  # noqa: F401

pytestmark = pytest.mark.gpu
NAT = math.log(2) * math.sqrt(E)  # a power of two of the weight in units of q . k


def ramp(j):
    """Up by 1.5 every 32 keys: the last few steps all count, and renewals fall on every column of a block."""
    return 1.5 * (j // 32)


def jumps(slot):
    """Up by 22 at one slot of every block of 128; the keys behind it count a 2^-5 each."""
    def level(j):
        b, s = j // 128, j % 128
        top = 22.0 * (b + (s >= slot))
        return top - 5.0 * (s != slot)
    return level


def bumps(j):
    """Up by 9 for 20 keys of every 32, then by 16 for one key: what lies before the renewal counts as much as the key."""
    s = j % 32
    return 2.0 * (j // 32) + np.where(s < 10, 0.0, np.where(s < 30, 9.0, np.where(s == 30, 14.5, 0.0)))


STAIRS = {"ramp": ramp, "slot 0": jumps(0), "slot 40": jumps(40), "slot 100": jumps(100), "bumps": bumps,
          "down": lambda j: -ramp(j)}


def queries(g, *shape):
    return ((1 + 0.25 * torch.randn(shape, generator=g, device="cuda")).clamp(-1, 3) * 32).round().div(32).bfloat16()


def key_rows(levels, shape, g):
    """bf16 keys whose product with a query of mean 1 has the level: [n, *shape, E]."""
    z = torch.from_numpy(np.asarray(levels, np.float64) * NAT / E).cuda()
    x = z.view(-1, *[1] * len(shape), 1) + torch.randint(0, 4, (len(levels), *shape, E), generator=g, device="cuda") / 4
    return x.bfloat16()


def expected(q, keys, seen):
    """(o, tolerance) for q [t, hg, E] and keys: a list of (q in the keys' basis, k, v, v rotated back by |R|, weight error)."""
    s = torch.cat([qb @ k.T for qb, k, _, _, _ in keys], -1) / math.sqrt(E)
    d = torch.cat([qb.abs() @ k.abs().T for qb, k, _, _, _ in keys], -1) * 2.0 ** -17 / math.sqrt(E)
    s = s.masked_fill(~seen[:, None], -math.inf)
    p = torch.softmax(s, -1)
    o = p @ torch.cat([x[2] for x in keys])
    mag = torch.cat([x[3] for x in keys])
    eps = torch.cat([torch.full((len(x[1]),), x[4], dtype=torch.float64, device="cuda") for x in keys])
    tol = 2.0 ** -8 * o.abs() + (p * (eps + d)) @ mag + (p * d).sum(-1, keepdim=True) * o.abs() + 2.0 ** -24 * mag.sum(0)
    return o, tol


def check(got, o, tol, what):
    r = (got.double() - o).abs() / tol
    assert (r <= 1).all(), f"{what}: {int((~(r <= 1)).sum())} of {r.numel()} off, worst {r.max():.3g} tolerances"


@pytest.mark.parametrize("stairs", STAIRS)
@pytest.mark.parametrize("seqs,length,new,hq,hkv", [(1, 1000, 5, 4, 1), (1, 1500, 700, 32, 8), (20, 900, 70, 32, 8), (6, 700, 257, 16, 16), (3, 777, 1, 16, 1)])
def test_bf16(stairs, seqs, length, new, hq, hkv):
    g = torch.Generator(device="cuda").manual_seed(length)
    c = Pages([length + 3 * i for i in range(seqs)], hkv, seed=length)
    for i, n in enumerate(c.lens):
        k = key_rows(STAIRS[stairs](np.arange(n)), (hkv,), g)
        c.rows[i] = [k, c.rows[i][1]]
        c.put(c.k, i, k)
    q = queries(g, seqs * new, hq, E)
    out = c.attend(q, [new] * seqs)
    assert int(c.err) == 0
    hg = hq // hkv
    for i, n in enumerate(c.lens):
        seen = torch.arange(n, device="cuda")[None] <= n - new + torch.arange(new, device="cuda")[:, None]
        for h in range(hkv):
            k, v = (x[:, h].double() for x in c.rows[i])
            at = (slice(i * new, i * new + new), slice(h * hg, h * hg + hg))
            check(out[at], *expected(q[at].double(), [(q[at].double(), k, v, v.abs(), 2.0 ** -8)], seen), f"seq {i} head {h}")


class Stairs:
    """A pool of sequences of the same length, whose INT2 histories climb the stairs; BF16 keys (sink, recent, new) lie at
    the history's end, or above it by `over` from the first token on."""

    def __init__(self, level, seqs, hist, hq, hkv, over, seed):
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.hq, self.hkv, self.seqs, self.hist = hq, hkv, seqs, hist
        u = torch.from_numpy(np.broadcast_to(O.hadamard(E).astype(np.float32), (1, hkv, E, E)).copy()).cuda()
        self.R = torch.from_numpy(O.rotation_matrix(u[0, 0].cpu().numpy())).cuda()
        clip = torch.full((1, hkv), 0.9, device="cuda")
        L = self.L = 64 + hist + 256
        self.pool = Pool(1, hq, hkv, max_seqs=seqs, max_seq_len=L + 2000, max_int2_pages=seqs * (L // 64 + 40), U_k=u, U_v=u, clip_k=clip, clip_v=clip)
        self.top = float(np.max(level(np.arange(hist))))
        self.over = over
        for i in range(seqs):
            self.pool.seq_add(i)
        self.pool.step_begin(range(seqs), [L] * seqs)
        # what the sink and the ring hold, one behind the other; the history's rows are replaced below
        self.k, self.v = self.rows(seqs * L)
        if over:
            self.k.view(seqs, L, hkv, E)[:, 0] = key_rows([self.top + over], (hkv,), g)
        self.pool.append_and_demote(0, self.k, self.v)
        self.codes = {}
        z = torch.from_numpy(np.asarray(level(np.arange(hist)), np.float64) * NAT / E).mul(64).round().div(64).half().cuda()
        for i in range(seqs):
            for h in range(hkv):
                ck, cv = (torch.randint(0, 256, (hist, 32), generator=g, device="cuda").byte() for _ in "kv")
                szk = torch.stack([torch.full_like(z, 0.25), z], -1)[:, None].contiguous()
                szv = torch.stack([torch.full_like(z, 0.5), -torch.randint(1, 9, (hist,), generator=g, device="cuda").half() / 4], -1)[:, None].contiguous()
                self.pool.debug_write_int2(i, 0, h, 64, ck, szk, cv, szv)
                self.codes[i, h] = ck, szk, cv, szv

    def rows(self, n):
        lv = self.top + self.over * 0.5 - 4 + 3 * np.sin(np.arange(n))
        return key_rows(lv, (self.hkv,), self.g), torch.randn((n, self.hkv, E), generator=self.g, device="cuda").bfloat16()

    def held(self, i, h):
        ck, szk, cv, szv = self.codes[i, h]
        out = []
        for c, sz in ((ck, szk), (cv, szv)):
            code = torch.stack([(c >> (2 * j)) & 3 for j in range(4)], -1).reshape(-1, E).double()
            out.append(code * sz[:, 0, :1].double() + sz[:, 0, 1:].double())
        at = torch.cat([torch.arange(64), torch.arange(64 + self.hist, self.L)]).cuda() + i * self.L
        return self.k[at, h].double(), self.v[at, h].double(), out

    def chunk(self, new, launches):
        T, hg = sum(new), self.hq // self.hkv
        kn, vn = self.rows(T)
        q = queries(self.g, T, self.hq, E)
        self.pool.step_begin(range(self.seqs), new)
        before = self.pool.launch_count()
        out = self.pool.chunk_attend(0, q, kn, vn)
        assert self.pool.launch_count() - before == launches
        self.pool.check()
        r = 0
        for i, n in enumerate(new):
            for h in range(self.hkv):
                kb, vb, (kh, vh) = self.held(i, h)
                k, v = torch.cat([kb, kn[r:r + n, h].double()]), torch.cat([vb, vn[r:r + n, h].double()])
                qh = q[r:r + n, h * hg:h * hg + hg].double()
                seen = torch.cat([torch.arange(len(k), device="cuda")[None] <= len(kb) + torch.arange(n, device="cuda")[:, None],
                                  torch.ones((n, self.hist), dtype=torch.bool, device="cuda")], -1)
                keys = [(qh, k, v, v.abs(), 2.0 ** -8), (qh @ self.R, kh, vh @ self.R.T, vh.abs() @ self.R.abs().T, 2.0 ** -10)]
                check(out[r:r + n, h * hg:h * hg + hg], *expected(qh, keys, seen), f"seq {i} head {h}")
            r += n


# chunk kernel and join: 2 launches; with the histories as tiles 4; single tokens over long histories 5
@pytest.mark.parametrize("stairs", STAIRS)
@pytest.mark.parametrize("over", [0, 25])
@pytest.mark.parametrize("seqs,hist,hq,hkv,new,launches", [
    (1, 700, 4, 1, 9, 2), (1, 650, 8, 1, 40, 2), (12, 700, 32, 8, 100, 2),      # codes expanded in the kernel: parts, whole items
    (1, 700, 4, 1, 330, 4), (4, 650, 32, 8, 330, 4), (3, 577, 64, 8, 200, 4),   # tiles
    (8, 705, 32, 8, 1, 5)])
def test_pool(stairs, over, seqs, hist, hq, hkv, new, launches):
    Stairs(STAIRS[stairs], seqs, hist, hq, hkv, over, seed=hist + new).chunk([new] * seqs, launches)

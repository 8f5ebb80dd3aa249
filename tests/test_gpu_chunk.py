"""Chunk attention over the BF16 pages and over the mixed pool, against softmax attention in 64 bits.

Tolerance of an output value o = sum_s p_s v_s (sum_s p_s = 1), A = sum_s p_s |v_s|, from the roundings alone:
  2^-8 |o|     the output's own rounding to bf16 (half a step)
  2^-8 A       the softmax weights rounded to bf16 for the value product
  2^-10 A      fp16 values and weights of the INT2 part (2^-11 each), exp2 and fp32 sums far below
  2 d A        scores off by d: every weight is off by the factor e^(2d) at most
with d = max_s (sum_i |q_i k_si|) / sqrt(128) * c, c = 2^-17 for 128 fp32 additions of exact products (BF16 keys), and
2^-10 + 2^-17 for the INT2 keys (q_rot and k^ in fp16, 2^-11 each)."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from bit_kv_cache_paged_gb300 import Pool, Rope, bf16_chunk_attend
from bit_kv_cache_paged_gb300 import binding as B

pytestmark = pytest.mark.gpu
E = 128
TOK = np.arange(64)[:, None]
SWZ = torch.from_numpy(((np.arange(E)[None, :] // 8) ^ (TOK % 8)) * 8 + np.arange(E)[None, :] % 8)  # dim -> place in its page row


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


def softmax64(q, parts, seen):
    """q [t, hg, E]; parts: (q basis [t, hg, E], k [n, E], v [n, E], |v| [n, E], c); seen [t, all n] bool, or None for all.
    Returns (o, tolerance) [t, hg, E] in 64 bits; rows that see nothing are zero."""
    s = torch.cat([qb.double() @ k.double().T for qb, k, _, _, _ in parts], -1) / math.sqrt(E)
    d = torch.cat([(qb.double().abs() @ k.double().abs().T) * c for qb, k, _, _, c in parts], -1) / math.sqrt(E)
    if seen is not None:
        s = s.masked_fill(~seen[:, None], -math.inf)
        d = d.masked_fill(~seen[:, None], 0)
    m = s.amax(-1, keepdim=True) if s.shape[-1] else s.new_full((*s.shape[:2], 1), -math.inf)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-300)
    o = p @ torch.cat([x[2].double() for x in parts])
    a = p @ torch.cat([x[3].double() for x in parts])
    d = d.amax(-1, keepdim=True) if d.shape[-1] else d.new_zeros((*d.shape[:2], 1))
    return o, 2.0 ** -8 * o.abs() + (2.0 ** -8 + 2.0 ** -10 + 2 * d) * a + 1e-6


def check(got, o, tol, what):
    bad = ~((got.double() - o).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {((got.double() - o).abs() / tol).max():.3g} tolerances"


# ------------------------------------------------------------------------------------------------ BF16 pages
class Pages:
    """A BF16 cache of random rows in shuffled pages; the slots past each length hold NaN, the table's other entries -1."""

    def __init__(self, lens, hkv, seed=0, extra=0, gain=1.0, poison=True):
        g = torch.Generator(device="cuda").manual_seed(seed)
        need = [-(-n // 64) for n in lens]
        self.total, self.width, self.hkv, self.lens = sum(need) + 1, max(need + [1]) + extra, hkv, list(lens)
        perm = np.random.default_rng(seed).permutation(self.total - 1)
        self.pt = np.full((len(lens), self.width), -1, np.int32)
        shape = (self.total, hkv, 64, E)
        self.k, self.v = (torch.full(shape, math.nan if poison else 0.0, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        self.rows = []
        at = 0
        for i, n in enumerate(lens):
            self.pt[i, :need[i]] = perm[at:at + need[i]]
            at += need[i]
            kv = [(torch.randn((n, hkv, E), generator=g, device="cuda") * gain).bfloat16() for _ in range(2)]
            self.rows.append(kv)
            for x, pages in zip(kv, (self.k, self.v)):
                self.put(pages, i, x)
        self.table = torch.from_numpy(self.pt).cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def put(self, pages, i, x):
        p = np.arange(len(x))
        ids, t = torch.from_numpy(self.pt[i, p // 64]).long().cuda(), torch.from_numpy(p % 64).cuda()
        where = SWZ.cuda()[t]  # [n, E]
        pages[ids[:, None, None], torch.arange(self.hkv, device="cuda")[None, :, None], t[:, None, None], where[:, None, :]] = x

    def attend(self, q, new, **kw):
        cu = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
        lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        return bf16_chunk_attend(q, self.k, self.v, self.table, lens, cu, self.err, **kw)

    def check(self, q, new, out, what=""):
        hg, r = q.shape[1] // self.hkv, 0
        for i, n in enumerate(new):
            pos = self.lens[i] - n + torch.arange(n, device="cuda")
            seen = torch.arange(self.lens[i], device="cuda")[None, :] <= pos[:, None]
            for h in range(self.hkv):
                k, v = (x[:, h] for x in self.rows[i])
                qh = q[r:r + n, h * hg:(h + 1) * hg]
                check(out[r:r + n, h * hg:(h + 1) * hg], *softmax64(qh, [(qh, k, v, v.abs(), 2.0 ** -17)], seen), f"{what} seq {i} head {h}")
            r += n


MIX = [(1, 1), (5, 5), (64, 1), (65, 65), (64, 64), (300, 300), (1001, 1), (200, 70), (5, 0), (0, 0), (2100, 3), (777, 129), (128, 128)]


@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (8, 2), (8, 1), (32, 2)])
def test_bf16_ragged_batch(hq, hkv):
    c = Pages([a for a, _ in MIX], hkv, seed=hq, extra=2)
    new = [b for _, b in MIX]
    T = sum(new)
    g = torch.Generator(device="cuda").manual_seed(7)
    rows = torch.randn((T + 9, hq + 2, E), generator=g, device="cuda").bfloat16()
    q = rows[:, 1:1 + hq]  # tokens apart, and rows behind the last sequence
    out = torch.full((T + 9, hq, E), 77.0, dtype=torch.bfloat16, device="cuda")
    c.attend(q, new, out=out)
    assert (out[T:] == 77).all()  # left as they were
    c.check(q, new, out)
    assert int(c.err) == 0
    again = c.attend(q.contiguous(), new)
    assert torch.equal(again[:T], out[:T])  # the same bits whatever the strides, and run to run


@pytest.mark.parametrize("length,new", [(1, 1), (4096, 1), (9000, 2), (9000, 33), (5000, 1100), (3001, 3001)])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (8, 1)])
def test_bf16_one_long_sequence(length, new, hq, hkv):
    c = Pages([length], hkv, seed=length, gain=2.0)
    q = torch.randn((new, hq, E), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    c.check(q, [new], c.attend(q, [new]))


def test_bf16_rows_that_see_nothing_are_zero():
    c = Pages([3, 0, 100], 2, seed=5)
    new = [10, 4, 130]  # more rows than tokens: the first ones have no position
    q = torch.randn((144, 8, E), device="cuda").bfloat16()
    out = c.attend(q, new)
    c.check(q, new, out)
    assert (out[:7] == 0).all() and (out[10:14] == 0).all() and (out[14:44] == 0).all()
    assert out[7:10].abs().amax(-1).min() > 0


def test_bf16_single_tokens_equal_the_decode():
    lens = [1, 63, 64, 65, 700, 2049]
    c = Pages(lens, 2, seed=11, poison=False)
    q = torch.randn((len(lens), 8, E), generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
    out = c.attend(q, [1] * len(lens))
    c.check(q, [1] * len(lens), out)
    nb = B.oscar_bf16_partials_bytes(8, 2, len(lens), max(lens))
    part, dec = torch.empty(nb, dtype=torch.uint8, device="cuda"), torch.empty((len(lens), 8, E), device="cuda")
    B.oscar_bf16_decode(8, 2, len(lens), max(lens), c.k, c.v, c.total, c.table, c.width,
                        torch.tensor(lens, dtype=torch.int32, device="cuda"), q, part, nb, dec, c.err,
                        torch.cuda.current_stream().cuda_stream)
    c.check(q, [1] * len(lens), dec.bfloat16(), "decode")


@pytest.mark.parametrize("special", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("which", [0, 1])
def test_bf16_a_bad_row_reaches_only_the_tokens_that_see_it(special, which):
    lens, new = [200, 90], [150, 90]
    c = Pages(lens, 1, seed=21)
    q = torch.randn((240, 4, E), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    good = c.attend(q, new)
    c.rows[0][which][120, 0, 17] = special  # token 120: row 70 of the chunk
    c.put((c.k, c.v)[which], 0, c.rows[0][which])
    out = c.attend(q, new)
    assert torch.equal(out[:70], good[:70]) and torch.equal(out[150:], good[150:])
    hit = out[70:150]
    if which == 1:  # a value: its dim alone
        dims = torch.arange(E, device="cuda") != 17
        c.rows[0][1][120, 0, 17] = 0
        ref = c.rows[0]
        pos = 50 + torch.arange(150, device="cuda")
        seen = torch.arange(200, device="cuda")[None, :] <= pos[:, None]
        o, tol = softmax64(q[:150], [(q[:150], ref[0][:, 0], ref[1][:, 0], ref[1][:, 0].abs(), 2.0 ** -17)], seen)
        check(hit[..., dims], o[70:][..., dims], tol[70:][..., dims], "other dims")
        if math.isnan(special):
            assert hit[..., 17].isnan().all()
        else:
            assert (hit[..., 17] == special).all()
    elif math.isnan(special):
        assert hit.isnan().all()


def test_bf16_pages_past_32_bit_offsets():
    hkv, total = 8, 33000  # 128 KB a page: past 4 GB of K
    k = torch.zeros((total, hkv, 64, E), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    c = Pages([200], hkv, seed=4)
    far = torch.tensor([total - 1, total - 9, 3, total - 2], dtype=torch.int32, device="cuda")
    k[far.long()], v[far.long()] = c.k[c.table[0].long()], c.v[c.table[0].long()]
    q = torch.randn((5, 32, E), device="cuda").bfloat16()
    cu, lens = torch.tensor([0, 5], dtype=torch.int32, device="cuda"), torch.tensor([200], dtype=torch.int32, device="cuda")
    out = bf16_chunk_attend(q, k, v, far[None].contiguous(), lens, cu, c.err)
    c.check(q, [5], out)


def test_bf16_bad_page_is_reported_and_not_followed():
    c = Pages([300, 300], 2, seed=8, poison=False)
    q = torch.randn((8, 8, E), device="cuda").bfloat16()
    good = c.attend(q, [4, 4])
    for bad in (-1, c.total, 2 ** 31 - 1):
        c.table[1, 2] = bad
        out = c.attend(q, [4, 4])
        assert int(c.err) & B.DEVERR_PAGE
        c.err.zero_()
        assert torch.equal(out[:4], good[:4])
    c.table[1, 2] = int(c.pt[1, 2])
    c.lens[1] = 64 * c.width + 1  # longer than its table row
    c.attend(q, [4, 4])
    assert int(c.err) & B.DEVERR_PAGE


def test_bf16_under_capture_follows_lengths():
    c = Pages([500, 900], 2, seed=9)
    q = torch.randn((6, 8, E), device="cuda").bfloat16()
    cu = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    lens = torch.tensor([500, 900], dtype=torch.int32, device="cuda")
    ws = [torch.empty(B.oscar_bf16_chunk_workspace_bytes(8, 2, 2, 6), dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty_like(q) for _ in range(2)]
    bf16_chunk_attend(q, c.k, c.v, c.table, lens, cu, c.err, workspace=ws[0], out=outs[0])
    graphs = []
    for w, o in zip(ws, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            bf16_chunk_attend(q, c.k, c.v, c.table, lens, cu, c.err, workspace=w, out=o)
    for l0, l1, a in ((500, 900, 2), (77, 640, 5), (128, 3, 0)):
        lens.copy_(torch.tensor([l0, l1]))
        cu.copy_(torch.tensor([0, a, 6]))
        for o in outs:
            o.fill_(5)
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for s, gr in zip(streams, graphs):  # two replays at once, each with its own workspace
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        short = Pages.__new__(Pages)
        short.lens, short.hkv, short.rows = [l0, l1], 2, [[x[:n] for x in r] for r, n in zip(c.rows, (l0, l1))]
        short.check(q, [a, 6 - a], outs[0])
        assert torch.equal(outs[0], outs[1])


# ------------------------------------------------------------------------------------------------ the mixed pool
class Mixed:
    """A pool filled with random rows (strong channels in K and V), and 64-bit references from what it holds."""

    def __init__(self, layers=1, hq=8, hkv=2, group=128, absorbed=False, lloyd=None, max_seqs=16, max_len=6000, seed=0):
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.layers, self.hq, self.hkv, self.group, self.absorbed, self.lloyd = layers, hq, hkv, group, absorbed, lloyd
        u = [torch.linalg.qr(torch.randn((layers, hkv, E, E), generator=g, device="cuda", dtype=torch.float64))[0].float().contiguous() for _ in "kv"]
        self.R = [torch.from_numpy(np.stack([[O.rotation_matrix(x[l, h].cpu().numpy()) for h in range(hkv)] for l in range(layers)])).cuda() for x in u]
        clip = torch.full((layers, hkv), 0.9, device="cuda")
        self.pool = Pool(layers, hq, hkv, max_seqs=max_seqs, max_seq_len=max_len, max_int2_pages=max_seqs * (max_len // 64), U_k=u[0], U_v=u[1],
                         clip_k=clip, clip_v=clip, group_size=group, v_rot_absorbed=absorbed, lloyd_max=lloyd is not None)
        if lloyd is not None:
            self.pool.set_codebook(np.broadcast_to(np.asarray(lloyd, np.float32), (layers, hkv, 2)))
        self.gain = torch.ones((2, hkv, E), device="cuda")
        self.gain[:, :, 5] = 8.0
        self.rows = {}  # seq -> [K, V] of [layers, n, hkv, E]

    def add(self, seq, share_from=-1, shared=0):
        self.pool.seq_add(seq, share_from, shared)
        self.rows[seq] = [x[:, :shared].clone() for x in self.rows[share_from]] if shared else \
            [torch.zeros((self.layers, 0, self.hkv, E), dtype=torch.bfloat16, device="cuda") for _ in "kv"]

    def new_rows(self, n):
        return [(torch.randn((self.layers, n, self.hkv, E), generator=self.g, device="cuda") * self.gain[kv]).bfloat16() for kv in (0, 1)]

    def held(self, seq, layer, h):
        """The cache of a sequence as BF16 rows (k, v) and dequantised INT2 rows (rotated k^, v^)."""
        L, F, _ = self.pool.seq_info(seq)
        k, v = (x[layer, :, h].double() for x in self.rows[seq])
        at = torch.tensor([p for p in range(L) if p < 64 or p >= F], dtype=torch.long, device="cuda")
        hist = []
        if F > 64:
            ck, szk, cv, szv = self.pool.debug_read_int2(seq, layer, h, 64, F - 64)
            for c, sz, a in ((ck, szk, 0), (cv, szv, 1)):
                codes = torch.stack([(c >> (2 * i)) & 3 for i in range(4)], -1).reshape(-1, E).long()
                lv = torch.tensor([0, 1, 2, 3] if self.lloyd is None else [0, self.lloyd[a], 3 - self.lloyd[a], 3], dtype=torch.float64, device="cuda")[codes]
                hist.append((lv.view(-1, E // self.group, self.group) * sz[..., :1].double() + sz[..., 1:].double()).reshape(-1, E))
        return k[at], v[at], hist

    def chunk(self, ids, n_new, layers=None, q=None, kv=None, append=True):
        """step_begin, chunk attention of every layer against the reference, then the append."""
        T, hg = sum(n_new), self.hq // self.hkv
        kn, vn = self.new_rows(T) if kv is None else kv
        q = torch.randn((self.layers, T, self.hq, E), generator=self.g, device="cuda").bfloat16() if q is None else q
        held = {(s, l, h): self.held(s, l, h) for s, n in zip(ids, n_new) if n for l in range(self.layers) for h in range(self.hkv)}
        self.pool.step_begin(ids, n_new)
        outs = []
        for l in range(self.layers):
            out = self.pool.chunk_attend(l, q[l], kn[l], vn[l])
            again = self.pool.chunk_attend(l, q[l], kn[l], vn[l])
            assert torch.equal(out, again)
            outs.append(out)
            if append and T:
                self.pool.append_and_demote(l, kn[l], vn[l])
                with pytest.raises(B.OscarError) as e:
                    self.pool.chunk_attend(l, q[l], kn[l], vn[l])
                assert e.value.status == B.OSCAR_ESTATE
        self.pool.check()
        for l in range(self.layers):
            r = 0
            for s, n in zip(ids, n_new):
                for h in range(self.hkv) if n else ():
                    kb, vb, hist = held[s, l, h]
                    k, v = torch.cat([kb, kn[l, r:r + n, h].double()]), torch.cat([vb, vn[l, r:r + n, h].double()])
                    qh = q[l, r:r + n, h * hg:(h + 1) * hg].double()
                    parts = [(qh, k, v, v.abs(), 2.0 ** -17)]
                    seen = [torch.arange(len(k), device="cuda")[None, :] <= len(kb) + torch.arange(n, device="cuda")[:, None]]
                    if hist:
                        kh, vh = hist
                        Rv = torch.eye(E, dtype=torch.float64, device="cuda") if self.absorbed else self.R[1][l, h]
                        parts.append((qh @ self.R[0][l, h], kh, vh @ Rv.T, vh.abs() @ Rv.abs().T, 2.0 ** -10 + 2.0 ** -17))
                        seen.append(torch.ones((n, len(kh)), dtype=torch.bool, device="cuda"))
                    check(outs[l][r:r + n, h * hg:(h + 1) * hg], *softmax64(qh, parts, torch.cat(seen, -1)), f"seq {s} layer {l} head {h}")
                r += n
        if append:
            r = 0
            for s, n in zip(ids, n_new):
                self.rows[s] = [torch.cat([x, y[:, r:r + n]], 1) for x, y in zip(self.rows[s], (kn, vn))]
                r += n
        return outs


@pytest.mark.parametrize("group,absorbed,lloyd,hq", [(128, False, None, 8), (32, False, None, 8), (128, True, None, 16), (32, True, None, 8),
                                                     (128, False, (1.17, 0.82), 8), (32, False, (0.7, 1.3), 16)])
def test_pool_ragged_chunks(group, absorbed, lloyd, hq):
    m = Mixed(layers=2, hq=hq, group=group, absorbed=absorbed, lloyd=lloyd, seed=group + hq)
    ctx = [0, 1, 63, 64, 65, 319, 320, 321, 384, 400, 1000, 2500]
    ids = list(range(len(ctx)))
    for i in ids:
        m.add(i)
    m.pool.step_begin(ids, ctx)
    kv = m.new_rows(sum(ctx))
    for l in range(2):
        m.pool.append_and_demote(l, kv[0][l], kv[1][l])
    r = 0
    for i, n in zip(ids, ctx):
        m.rows[i] = [x[:, r:r + n] for x in kv]
        r += n
    m.chunk(ids, [1, 3, 1, 70, 1, 2, 1, 5, 130, 0, 400, 33])
    m.chunk(ids[::-1], [1] * len(ids))  # single tokens, another order
    m.chunk([10, 0, 4], [0, 260, 129])


@pytest.mark.parametrize("group,absorbed,lloyd,hq", [(128, False, None, 32), (32, False, None, 64), (128, True, None, 64), (32, True, (1.2, 0.8), 32),
                                                     (128, False, (0.9, 1.3), 64)])
def test_pool_single_tokens_over_long_histories(group, absorbed, lloyd, hq):
    """Single tokens whose histories together are long take another path than chunks; alone, and beside chunks."""
    m = Mixed(hq=hq, hkv=8, group=group, absorbed=absorbed, lloyd=lloyd, seed=group + hq, max_seqs=8, max_len=4096)
    ctx = [3500, 0, 400, 3904, 63, 2000, 1000, 330]
    ids = list(range(8))
    for i in ids:
        m.add(i)
    m.pool.step_begin(ids, ctx)
    kv = m.new_rows(sum(ctx))
    m.pool.append_and_demote(0, kv[0][0], kv[1][0])
    r = 0
    for i, n in zip(ids, ctx):
        m.rows[i] = [x[:, r:r + n] for x in kv]
        r += n
    launches = m.pool.launch_count()
    m.chunk(ids, [1] * 8)
    assert m.pool.launch_count() - launches > 6  # the decode kernels ran: a chunk is two launches a call
    m.chunk([3, 5, 1, 0], [1, 7, 1, 1])
    m.chunk([2, 0, 3, 6], [0, 1, 1, 130])


@pytest.mark.parametrize("group,absorbed,lloyd,hq", [(128, False, None, 4), (32, False, None, 8), (128, True, None, 8), (32, True, (1.2, 0.8), 4),
                                                     (128, False, (0.9, 1.3), 8)])
def test_pool_long_chunks_over_histories(group, absorbed, lloyd, hq):
    """Chunks long enough for their histories to be expanded beforehand, several sequences and one without a history."""
    m = Mixed(hq=hq, hkv=1, group=group, absorbed=absorbed, lloyd=lloyd, seed=group + hq, max_seqs=5, max_len=6000)
    ctx = [1500, 0, 385, 2049, 320]
    for i in range(5):
        m.add(i)
    m.pool.step_begin(range(5), ctx)
    kv = m.new_rows(sum(ctx))
    m.pool.append_and_demote(0, kv[0][0], kv[1][0])
    r = 0
    for i, n in enumerate(ctx):
        m.rows[i] = [x[:, r:r + n] for x in kv]
        r += n
    m.pool.step_begin(range(5), [0] * 5)
    launches = m.pool.launch_count()
    m.chunk([4, 3, 1, 0, 2], [600, 701, 900, 1025, 0])
    assert m.pool.launch_count() - launches > 8  # two calls of four launches, and the append
    m.chunk([0, 2, 3], [555, 513, 1])


def test_pool_single_tokens_bad_value_and_bad_page():
    m = Mixed(hq=32, hkv=8, seed=22, max_seqs=4, max_len=4096)
    for i in range(4):
        m.add(i)
    m.pool.step_begin([0, 1, 2, 3], [3500, 3000, 2500, 3800])
    kv = m.new_rows(12800)
    m.pool.append_and_demote(0, kv[0][0], kv[1][0])
    m.pool.step_begin([0, 1, 2, 3], [1, 1, 1, 1])
    kn, vn = m.new_rows(4)
    q = torch.randn((4, 32, E), generator=m.g, device="cuda").bfloat16()
    good = m.pool.chunk_attend(0, q, kn[0], vn[0])
    vn[0, 1, 0, 9], kn[0, 2, 3, 5] = math.inf, math.nan
    out = m.pool.chunk_attend(0, q, kn[0], vn[0])
    assert torch.equal(out[[0, 3]], good[[0, 3]]) and torch.equal(out[1, 4:], good[1, 4:])
    assert (out[1, :4, 9] == math.inf).all() and out[1, :4, :9].isfinite().all()
    assert out[2, 12:16].isnan().all() and torch.equal(out[2, :12], good[2, :12])
    m.pool.check()
    st = torch.cuda.current_stream().cuda_stream
    B.oscar_debug_set_page_entry(m.pool.handle, 3, 7, m.pool.cfg.max_int2_pages, st)
    out = m.pool.chunk_attend(0, q, kn[0], vn[0])
    with pytest.raises(B.OscarError) as e:
        m.pool.check()
    assert e.value.detail & B.DEVERR_PAGE and torch.equal(out[0], good[0])


def test_pool_first_prefill_and_decode_afterwards():
    """rotary positions, chunks from the first token on, and a decode step at the end, as a server runs them."""
    m = Mixed(hq=8, hkv=2, seed=3)
    m.add(0)
    m.add(1)
    rope = Rope(base=1e6)
    for step, n_new in enumerate(([40, 1], [300, 7], [513, 0], [1, 1], [2, 64])):
        T = sum(n_new)
        L = [m.rows[i][0].shape[1] for i in (0, 1)]
        pos = torch.cat([L[i] + torch.arange(n_new[i]) for i in (0, 1)]).int().cuda()
        raw = torch.randn((T, 8 + 2 * 2, E), generator=m.g, device="cuda").bfloat16()  # packed projection rows
        q, k = rope.apply(raw[:, :8], raw[:, 8:10], pos)
        m.chunk([0, 1], n_new, q=q[None], kv=(k[None], raw[:, 10:].contiguous()[None]))
    m.pool.step_begin([0, 1], [1, 1])
    kn, vn = m.new_rows(2)
    m.pool.append_and_demote(0, kn[0], vn[0])
    q = torch.randn((2, 8, E), generator=m.g, device="cuda").bfloat16()
    out = m.pool.attend(0, q)
    m.pool.check()
    for i in (0, 1):
        m.rows[i] = [torch.cat([x, y[:, i:i + 1]], 1) for x, y in zip(m.rows[i], (kn, vn))]
        for h in range(2):
            kb, vb, hist = m.held(i, 0, h)
            qh = q[i:i + 1, 4 * h:4 * h + 4].double()
            parts = [(qh, kb, vb, vb.abs(), 2.0 ** -17)]
            if hist:
                parts.append((qh @ m.R[0][0, h], hist[0], hist[1] @ m.R[1][0, h].T, hist[1].abs() @ m.R[1][0, h].abs().T, 2.0 ** -10))
            check(out[i:i + 1, 4 * h:4 * h + 4].bfloat16(), *softmax64(qh, parts, None), f"decode {i}")


def test_pool_shared_prefix():
    m = Mixed(seed=6)
    m.add(0)
    m.chunk([0], [1500])
    m.add(1, 0, 64 + 64 * 10)
    m.chunk([1, 0], [5, 1])   # the sharer's recent window starts empty
    m.chunk([0, 1], [2, 300])


@pytest.mark.parametrize("ctx,new", [(5000, 1), (5000, 8), (3000, 1500), (0, 2000)])
@pytest.mark.parametrize("hq,hkv,group", [(4, 1, 128), (32, 8, 128), (8, 1, 32)])
def test_pool_one_long_sequence(ctx, new, hq, hkv, group):
    m = Mixed(hq=hq, hkv=hkv, group=group, max_seqs=1, seed=ctx + new)
    m.add(0)
    if ctx:
        kv = m.new_rows(ctx)
        m.pool.step_begin([0], [ctx])
        m.pool.append_and_demote(0, kv[0][0], kv[1][0])
        m.rows[0] = kv
    m.chunk([0], [new])


def test_pool_values_of_another_sequence_and_later_tokens_stay_apart():
    m = Mixed(hq=4, hkv=1, seed=12)
    for i in (0, 1):
        m.add(i)
    m.pool.step_begin([0, 1], [70, 90])
    kn, vn = m.new_rows(160)
    q = torch.randn((160, 4, E), generator=m.g, device="cuda").bfloat16()
    good = m.pool.chunk_attend(0, q, kn[0], vn[0])
    vn[0, 30, 0, 9], kn[0, 100, 0, 3] = math.nan, math.nan
    out = m.pool.chunk_attend(0, q, kn[0], vn[0])
    assert torch.equal(out[:30], good[:30]) and torch.equal(out[70:100], good[70:100])
    assert out[30:70, :, 9].isnan().all() and out[100:].isnan().all()
    keep = torch.arange(E, device="cuda") != 9
    check(out[30:70][..., keep], good[30:70][..., keep].double(), 2.0 ** -7 * good[30:70][..., keep].abs().double() + 1e-2, "other dims")


def test_pool_bad_page_is_reported():
    m = Mixed(hq=4, hkv=1, seed=13, max_seqs=2)
    for i in (0, 1):
        m.add(i)
    m.chunk([0, 1], [900, 900])
    st = torch.cuda.current_stream().cuda_stream
    m.pool.step_begin([0, 1], [3, 3])
    kn, vn = m.new_rows(6)
    q = torch.randn((6, 4, E), generator=m.g, device="cuda").bfloat16()
    good = m.pool.chunk_attend(0, q, kn[0], vn[0])
    for bad in (-1, m.pool.cfg.max_int2_pages, 2 ** 31 - 1):
        B.oscar_debug_set_page_entry(m.pool.handle, 1, 2, bad, st)
        out = m.pool.chunk_attend(0, q, kn[0], vn[0])
        with pytest.raises(B.OscarError) as e:
            m.pool.check()
        assert e.value.detail & B.DEVERR_PAGE
        assert torch.equal(out[:3], good[:3])
        B.oscar_debug_restore_page_table(m.pool.handle, 1, st)
    assert torch.equal(m.pool.chunk_attend(0, q, kn[0], vn[0]), good)
    m.pool.check()


@pytest.mark.parametrize("group", [128, 32])
def test_pool_history_with_chosen_contents(group):
    """Codes, scales and zeros written back as they were read change nothing, and chosen ones are what the chunk sees:
    zero scales, large ones, all codes alike."""
    m = Mixed(hq=8, hkv=2, group=group, seed=15)
    m.add(0)
    m.chunk([0], [1000])
    n = m.pool.seq_info(0)[1] - 64
    g = torch.Generator(device="cuda").manual_seed(16)
    for h in (0, 1):
        c = m.pool.debug_read_int2(0, 0, h, 64, n)
        m.pool.debug_write_int2(0, 0, h, 64, *c)
        assert all(torch.equal(a, b) for a, b in zip(c, m.pool.debug_read_int2(0, 0, h, 64, n)))
        for a in (0, 2):
            c[a][:] = torch.randint(0, 256, c[a].shape, generator=g, device="cuda").byte()
        c[0][5:70], c[2][300:330] = 255, 0
        for a in (1, 3):
            c[a][:] = torch.randn(c[a].shape, generator=g, device="cuda").half()
            c[a][10:20, :, 0] = 0  # constant rows
        c[3][40], c[1][50] = 500.0, 0.0
        m.pool.debug_write_int2(0, 0, h, 64, *c)
        assert all(torch.equal(a, b) for a, b in zip(c, m.pool.debug_read_int2(0, 0, h, 64, n)))
    with pytest.raises(B.OscarError):
        m.pool.debug_write_int2(0, 0, 0, 65, *c)
    m.chunk([0], [9])


def test_pool_chunk_on_a_stream_and_in_graphs():
    m = Mixed(hq=8, hkv=2, seed=14)
    m.add(0)
    m.chunk([0], [700])
    m.pool.step_begin([0], [20])
    kn, vn = m.new_rows(20)
    q = torch.randn((20, 8, E), generator=m.g, device="cuda").bfloat16()
    want = m.pool.chunk_attend(0, q, kn[0], vn[0])
    outs = [torch.empty_like(want) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in outs]
    for gr, o in zip(graphs, outs):
        with torch.cuda.graph(gr):
            m.pool.chunk_attend(0, q, kn[0], vn[0], out=o)
    streams = [torch.cuda.Stream() for _ in outs]
    for s, gr in zip(streams, graphs):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    with torch.cuda.stream(streams[0]):
        got = m.pool.chunk_attend(0, q, kn[0], vn[0])
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    m.pool.check()


def test_pool_long_single_tokens_on_streams_and_in_graphs():
    """The decode kernels' path runs on two branches outside a capture and on one inside; the outputs are the same bits."""
    m = Mixed(hq=32, hkv=8, seed=15, max_seqs=8, max_len=4096)
    ctx = [3900, 3000, 2500, 3900, 3500, 3333]
    ids = list(range(len(ctx)))
    for i in ids:
        m.add(i)
    m.pool.step_begin(ids, ctx)
    kv = m.new_rows(sum(ctx))
    m.pool.append_and_demote(0, kv[0][0], kv[1][0])
    m.pool.step_begin(ids, [1] * len(ids))
    kn, vn = (x[0] for x in m.new_rows(len(ids)))
    q = torch.randn((len(ids), 32, E), generator=m.g, device="cuda").bfloat16()
    launches = m.pool.launch_count()
    want = m.pool.chunk_attend(0, q, kn, vn)
    assert m.pool.launch_count() - launches > 4  # of them a chunk alone has at most four
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for k in range(12):
        with torch.cuda.stream(streams[k % 3]):
            got.append(m.pool.chunk_attend(0, q, kn, vn))
    out = torch.empty_like(want)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        m.pool.chunk_attend(0, q, kn, vn, out=out)
        m.pool.chunk_attend(0, q, kn, vn, out=out)
    gr.replay()
    gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in got + [out])
    m.pool.check()


def test_buffers_elsewhere_are_refused():
    c = Pages([100], 2)
    q = torch.randn((5, 8, E), device="cuda").bfloat16()
    nb = B.oscar_bf16_chunk_workspace_bytes(8, 2, 1, 5)
    with pytest.raises(ValueError):
        c.attend(q, [5], workspace=torch.empty(nb, dtype=torch.uint8))
    with pytest.raises(ValueError):
        c.attend(q, [5], workspace=torch.empty(2 * nb, dtype=torch.uint8, device="cuda")[::2])
    with pytest.raises(B.OscarError):
        c.attend(q, [5], workspace=torch.empty(nb - 1, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        Rope().apply(q, None, torch.arange(5, dtype=torch.int32))


def test_bf16_many_sequences():
    r = np.random.default_rng(5)
    lens = r.integers(0, 200, 700).tolist()
    new = [int(r.integers(0, min(n, 9) + 1)) for n in lens]
    c = Pages(lens, 1, seed=31)
    q = torch.randn((sum(new), 4, E), generator=torch.Generator(device="cuda").manual_seed(31), device="cuda").bfloat16()
    c.check(q, new, c.attend(q, new))
    assert int(c.err) == 0


@pytest.mark.parametrize("most", [1, 4, 330])
def test_pool_many_sequences(most):
    """More sequences than a block has threads, on each of the paths: single tokens beside others, chunks, long chunks."""
    n = 290
    m = Mixed(hq=4, hkv=1, seed=32, max_seqs=n, max_len=1100)
    r = np.random.default_rng(most)
    ctx = r.integers(400, 700, n).tolist()
    ids = r.permutation(n).tolist()
    for i in range(n):
        m.add(i)
    m.pool.step_begin(ids, ctx)
    kv = m.new_rows(sum(ctx))
    m.pool.append_and_demote(0, kv[0][0], kv[1][0])
    at = np.concatenate([[0], np.cumsum(ctx)])
    for j, i in enumerate(ids):
        m.rows[i] = [x[:, at[j]:at[j + 1]] for x in kv]
    new = [1 if most == 1 and j % 5 else 300 if most == 330 and j % 3 else int(r.integers(0, most + 1)) for j in range(n)]
    m.chunk(ids[::-1], new, append=False)


def test_pool_bad_page_of_a_long_chunk_is_reported():
    m = Mixed(hq=8, hkv=1, seed=33, max_seqs=2)
    for i in (0, 1):
        m.add(i)
    m.chunk([0, 1], [900, 900])
    st = torch.cuda.current_stream().cuda_stream
    m.pool.step_begin([0, 1], [400, 300])
    kn, vn = m.new_rows(700)
    q = torch.randn((700, 8, E), generator=m.g, device="cuda").bfloat16()
    good = m.pool.chunk_attend(0, q, kn[0], vn[0])
    for bad in (-1, m.pool.cfg.max_int2_pages):
        B.oscar_debug_set_page_entry(m.pool.handle, 1, 2, bad, st)
        out = m.pool.chunk_attend(0, q, kn[0], vn[0])
        with pytest.raises(B.OscarError) as e:
            m.pool.check()
        assert e.value.detail & B.DEVERR_PAGE
        assert torch.equal(out[:400], good[:400])
        B.oscar_debug_restore_page_table(m.pool.handle, 1, st)
    assert torch.equal(m.pool.chunk_attend(0, q, kn[0], vn[0]), good)
    m.pool.check()

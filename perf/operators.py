"""The chunked-prefill operators of the KV caches and what is measured of them.

Four operators, with E = head_dim = 128 everywhere and query head h reading KV head h / (Hq / Hkv):

* rope: rotary positions of q and k rows before they enter a cache. For frequency j and position p the angle is
  p * w_j and the pair (x_a, x_b) becomes A * (x_a cos - x_b sin, x_b cos + x_a sin); pairs are (j, j + r/2) or
  (2j, 2j + 1) of the first r dims, the others are copied. Long contexts scale w_j and the amplitude A.
* bf16 chunk: attention of the last n_i tokens of every sequence over its BF16 pages, causal inside the chunk.
* pool chunk: the same over the mixed cache: history in rotated INT2 (k^ = code * s + z, compared with q R_K, values
  un-rotated by R_V^T), sink and recent rows in BF16, the chunk's own rows as they come.
* copy pages: pages of the BF16 cache copied to other pages of it (fork of a tail page, compaction), all layers.
"""
import math

import numpy as np
import torch

own = False

E = 128
PAGE = 64
SINK = 64
RECENT = 256


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # decode step of 32 sequences, one token each: a call whose latency counts
        dict(name="rope_step_b32", op="rope", tokens=32, hq=32, hkv=8, rot=128, inter=False, scaling="none", factor=1.0,
             base=1000000.0, far=100000, packed=True),
        # prefill of 8192 tokens out of a packed qkv projection, frequencies ramped for a long context
        dict(name="rope_prefill_8k", op="rope", tokens=8192, hq=64, hkv=8, rot=128, inter=False, scaling="ramp", factor=4.0,
             base=1000000.0, far=131072, packed=True),
        # interleaved pairs in half of the head, an odd number of tokens, positions interpolated
        dict(name="rope_interleaved_4097", op="rope", tokens=4097, hq=16, hkv=4, rot=64, inter=True, scaling="linear", factor=2.0,
             base=10000.0, far=40000, packed=False),
        # verification of 4 drafted tokens in each of 16 ragged sequences
        dict(name="bf16_verify_b16", op="bf16", seqs=16, least=4, most=4, ctx_least=1000, ctx_most=32768, hq=32, hkv=8),
        # first prefill of one sequence
        dict(name="bf16_prefill_8k", op="bf16", seqs=1, least=8192, most=8192, ctx_least=0, ctx_most=0, hq=32, hkv=8),
        # a chunk of a long prompt: 1024 tokens after 64K
        dict(name="bf16_chunk_1k_after_64k", op="bf16", seqs=1, least=1024, most=1024, ctx_least=65536, ctx_most=65536, hq=64, hkv=8),
        # a mixed serving batch: single tokens beside odd chunks
        dict(name="bf16_ragged_b12", op="bf16", seqs=12, least=1, most=257, ctx_least=0, ctx_most=8192, hq=32, hkv=8),
        # single tokens over a long INT2 history
        dict(name="pool_single_b8_32k", op="pool", seqs=8, least=1, most=1, ctx_least=32768, ctx_most=32768, hq=32, hkv=8, group=128),
        # a chunk of a long prompt: 2048 tokens after 30000
        dict(name="pool_chunk_2k_after_30k", op="pool", seqs=1, least=2048, most=2048, ctx_least=30000, ctx_most=30000, hq=32, hkv=8,
             group=128),
        # a mixed serving batch with groups of 32 and eight query heads a KV head
        dict(name="pool_ragged_b10_g32", op="pool", seqs=10, least=1, most=300, ctx_least=0, ctx_most=6000, hq=64, hkv=8, group=32),
        # one sequence forked: its last page of one layer
        dict(name="copy_1_page", op="copy", pages=64, moves=1, hkv=8, layers=1),
        # 32 sequences forked: the last page of each, all 36 layers
        dict(name="copy_32_pages_36_layers", op="copy", pages=80, moves=32, hkv=8, layers=36),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["rope", "bf16", "bf16", "pool", "pool", "copy"])
    if op == "rope":
        hkv = rng.choice([1, 2, 4, 8])
        return dict(op=op, tokens=_log(rng, 1, 8000), hq=hkv * rng.choice([1, 4, 8]), hkv=hkv, rot=16 * rng.randint(1, 8),
                    inter=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "base", "ramp"]), factor=rng.choice([2.0, 4.0, 8.0]),
                    base=rng.choice([10000.0, 500000.0, 1000000.0]), far=_log(rng, 64, 1000000), packed=rng.random() < 0.5)
    if op == "copy":
        pages = _log(rng, 8, 100)
        return dict(op=op, pages=pages, moves=rng.randint(1, pages // 2), hkv=rng.choice([1, 2, 4, 8]), layers=rng.randint(1, 20))
    seqs = _log(rng, 1, 16)
    hkv = rng.choice([1, 2, 4, 8])
    most = _log(rng, 1, 2000 // seqs + 1)
    ctx = _log(rng, 1, 32000 if seqs < 4 else 12000)
    case = dict(op=op, seqs=seqs, least=rng.choice([1, most]), most=most, ctx_least=rng.choice([0, ctx // 2, ctx]), ctx_most=ctx,
                hq=hkv * rng.choice([4, 8]), hkv=hkv)
    if op == "pool":
        case["group"] = rng.choice([32, 128])
    return case


def _lengths(case):
    """(new tokens, cached tokens) of every sequence: a function of the case alone, so that all seeds share the work."""
    r = np.random.RandomState(case["seqs"] * 1009 + case["most"] * 31 + case["ctx_most"])
    new = r.randint(case["least"], case["most"] + 1, case["seqs"])
    ctx = r.randint(case["ctx_least"], case["ctx_most"] + 1, case["seqs"])
    new[0], ctx[0] = case["most"], case["ctx_most"]
    return new.astype(np.int64), ctx.astype(np.int64)


def work(case):
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * (case["hq"] + case["hkv"])
        return {"bytes": n * E * 2 * 2 + case["tokens"] * 4, "flops": n * case["rot"] * 3}
    if op == "copy":
        return {"bytes": case["moves"] * case["layers"] * case["hkv"] * PAGE * E * 2 * 2 * 2, "flops": 0}
    new, ctx = _lengths(case)
    seen = int((new * ctx + new * (new + 1) // 2).sum())
    rows = int(new.sum())
    data = rows * case["hq"] * E * 2 * 2
    flops = 4 * E * case["hq"] * seen
    if op == "bf16":
        data += int((new + ctx).sum()) * case["hkv"] * 512
    else:
        front = np.maximum(SINK, ctx - RECENT)
        hist = int((front - SINK).sum())
        data += hist * case["hkv"] * (72 if case["group"] == 128 else 96) + int((new + ctx).sum() - hist) * case["hkv"] * 512
        if hist:
            flops += 2 * 2 * E * E * case["hq"] * rows
    return {"bytes": data, "flops": flops}


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed, salt=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + salt)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _frequencies(case):
    """w_j of the case's pairs (float64) and the amplitude."""
    half = case["rot"] // 2
    j = np.arange(half, dtype=np.float64)
    f, base = case["factor"], case["base"]
    if case["scaling"] == "base":
        base = base * f ** (case["rot"] / max(1, case["rot"] - 2))
    w = base ** (-2.0 * j / case["rot"])
    if case["scaling"] == "linear":
        return w / f, 1.0
    if case["scaling"] == "ramp":
        at = lambda turns: case["rot"] * math.log(32768 / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), case["rot"] - 1)
        ramp = np.clip((j - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        return w / f * ramp + w * (1.0 - ramp), 0.1 * math.log(f) + 1.0
    return w, 1.0


def _hadamard_basis(g, heads):
    """Random orthogonal U [heads][E][E] and R = U H P: H the orthonormal Walsh-Hadamard matrix, P the bit reversal."""
    u = torch.linalg.qr(torch.randn((heads, E, E), generator=g, device="cuda", dtype=torch.float64))[0].float().contiguous()
    i = torch.arange(E, device="cuda")
    par = i[:, None] & i[None, :]
    par = sum((par >> b) & 1 for b in range(7)) & 1
    had = (1.0 - 2.0 * par.double()) / math.sqrt(E)
    rev = sum(((i >> b) & 1) << (6 - b) for b in range(7))
    r = torch.empty((heads, E, E), dtype=torch.float64, device="cuda")
    r[:, :, rev] = u.double() @ had
    return u, r


def _quantised(x, r, group, clip):
    """(code, s, z) of bf16 rows x [..., heads, E] in the rotated basis: s and z fp16 a group, codes 0..3."""
    t = torch.einsum("...he,hef->...hf", x.double(), r).float()
    t = t.reshape(*t.shape[:-1], E // group, group)
    lo, hi = clip * t.amin(-1, keepdim=True), clip * t.amax(-1, keepdim=True)
    s, z = ((hi - lo) / 3.0).half(), lo.half()
    u = torch.where(s == 0, torch.zeros_like(t), (t - z.float()) / s.float())
    return torch.round(u).clamp(0, 3).to(torch.uint8), s, z


def prepare(case, seed):
    op = case["op"]
    g = _gen(seed)
    st = {"case": case, "op": op}
    if op == "rope":
        n, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        if case["packed"]:  # q, k and v of a token in one row, as a fused projection leaves them
            rows = _normal(g, n, hq + 2 * hkv, E).bfloat16()
            st["q"], st["k"] = rows[:, :hq], rows[:, hq:hq + hkv]
        else:
            st["q"], st["k"] = _normal(g, n, hq, E).bfloat16(), _normal(g, n, hkv, E).bfloat16()
        first = torch.randint(0, max(1, case["far"] - n), (1,), generator=g, device="cuda")
        st["pos"] = (first + torch.arange(n, device="cuda")).int()
        if n <= 64:  # a decode step: every token at a position of its own
            st["pos"] = torch.randint(0, case["far"], (n,), generator=g, device="cuda").int()
        w, amp = _frequencies(case)
        st["w"], st["amp"] = torch.from_numpy(w).cuda(), amp
        if own:
            from bit_kv_cache_paged_gb300 import Rope
            st["rope"] = Rope(rot_dim=case["rot"], interleaved=case["inter"], base=case["base"], scaling=case["scaling"],
                              factor=case["factor"] if case["scaling"] != "none" else 1.0, original_len=32768)
        return st
    if op == "copy":
        shape = (case["layers"], case["pages"], case["hkv"], PAGE, E)
        st["k"], st["v"] = _normal(g, *shape).bfloat16(), _normal(g, *shape).bfloat16()
        perm = np.random.RandomState(seed % (1 << 31)).permutation(case["pages"])
        st["src"], st["dst"] = perm[:case["moves"]].tolist(), perm[case["moves"]:2 * case["moves"]].tolist()
        st["src_d"], st["dst_d"] = torch.tensor(st["src"], device="cuda"), torch.tensor(st["dst"], device="cuda")
        return st
    new, ctx = _lengths(case)
    n, hq, hkv, rows = len(new), case["hq"], case["hkv"], int(new.sum())
    st["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)])).int().cuda()
    st["q"] = _normal(g, rows, hq, E).bfloat16()
    st["most_new"], st["most_len"] = int(new.max()), int((new + ctx).max())
    if op == "bf16":
        lens = new + ctx
        st["lengths"] = torch.from_numpy(lens).int().cuda()
        need = -(-lens // PAGE)
        total, st["max_pages"] = int(need.sum()), int(need.max())
        st["k"], st["v"] = (_normal(g, total, hkv, PAGE, E).bfloat16() for _ in range(2))
        perm = np.random.RandomState(seed % (1 << 31)).permutation(total).astype(np.int32)
        table = np.zeros((n, st["max_pages"]), np.int32)
        table[np.arange(st["max_pages"])[None, :] < need[:, None]] = perm
        st["table"] = torch.from_numpy(table).cuda()
        st["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if own:
            from bit_kv_cache_paged_gb300 import binding
            nb = binding.oscar_bf16_chunk_workspace_bytes(hq, hkv, n, rows)
            st["workspace"] = torch.empty(nb, dtype=torch.uint8, device="cuda")
        return st
    # the mixed cache: keys and values with a few strong channels a head, as the rotation is there to spread
    group, clip = case["group"], 0.9
    most = int(ctx.max())
    gain = torch.ones((2, hkv, E), device="cuda")
    gain.scatter_(2, torch.rand((2, hkv, E), generator=g, device="cuda").topk(4, -1)[1], 10.0)
    hist = [(_normal(g, n, most, hkv, E) * gain[kv]).bfloat16() for kv in (0, 1)]
    st["k_new"], st["v_new"] = ((_normal(g, rows, hkv, E) * gain[kv]).bfloat16() for kv in (0, 1))
    (uk, rk), (uv, rv) = _hadamard_basis(g, hkv), _hadamard_basis(g, hkv)
    st["rk"], st["rv"] = rk.float(), rv.float()
    st["ctx"] = torch.from_numpy(ctx).cuda()
    st["front"] = torch.from_numpy(np.maximum(SINK, ctx - RECENT)).cuda()
    st["kq"] = _quantised(hist[0], rk, group, clip) if most > SINK + RECENT else None
    st["vq"] = _quantised(hist[1], rv, group, clip) if most > SINK + RECENT else None
    # BF16 rows of the cache: the sink's positions, then the recent ones
    pos = torch.arange(SINK + RECENT, device="cuda")[None, :].expand(n, -1)
    pos = torch.where(pos < SINK, pos, pos - SINK + st["front"][:, None])
    st["bf_live"] = pos < st["ctx"][:, None]
    at = torch.where(st["bf_live"], pos, torch.zeros_like(pos))
    seq = torch.arange(n, device="cuda")[:, None]
    st["bf"] = [h[seq, at] if most else h.new_zeros((n, SINK + RECENT, hkv, E)) for h in hist]
    if own:
        from bit_kv_cache_paged_gb300 import Pool
        pages = int((-(-np.maximum(0, ctx + new - RECENT) // PAGE)).sum()) + n
        pool = Pool(1, hq, hkv, max_seqs=n, max_seq_len=int((ctx + new).max()) + PAGE, max_int2_pages=pages, U_k=uk[None].contiguous(),
                    U_v=uv[None].contiguous(), clip_k=torch.full((1, hkv), clip, device="cuda"),
                    clip_v=torch.full((1, hkv), clip, device="cuda"), group_size=group)
        ids = list(range(n))
        for i in ids:
            pool.seq_add(i)
        pool.step_begin(ids, [int(x) for x in ctx])
        if ctx.sum():
            pool.append_and_demote(0, *(torch.cat([h[i, :int(ctx[i])] for i in ids]).contiguous() for h in hist))
        # the pool's own demote rounds a few codes and scales in a million the other way: the history given is what counts
        for i in ids:
            front = int(st["front"][i])
            for h in range(hkv) if front > SINK else ():
                hist_i = []
                for c, sc, z in (st["kq"], st["vq"]):
                    c = c[i, SINK:front, h].reshape(front - SINK, 32, 4).int()
                    hist_i.append((c << (2 * torch.arange(4, device="cuda"))).sum(-1).to(torch.uint8).contiguous())
                    hist_i.append(torch.stack([sc[i, SINK:front, h, :, 0], z[i, SINK:front, h, :, 0]], -1).contiguous())
                pool.debug_write_int2(i, 0, h, SINK, *hist_i)
        pool.step_begin(ids, [int(x) for x in new])
        st["pool"] = pool
    return st


# ------------------------------------------------------------------------------------------------ one pass
def _turned(x, pos, w, amp, rot, inter):
    a = pos.double()[:, None] * w
    c, s = (amp * a.cos()).float()[:, None, :], (amp * a.sin()).float()[:, None, :]
    x = x.float()
    y = x.clone()
    if inter:
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = u * c - v * s, v * c + u * s
    else:
        u, v = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = u * c - v * s, v * c + u * s
    return y.bfloat16()


def _padded(st, rows):
    """Rows [tokens, heads, E] of the batch as [sequences, most new tokens, heads, E], where each row goes, and which are there."""
    cu = st["cu"].long()
    n = cu[1:] - cu[:-1]
    t = torch.arange(st["most_new"], device="cuda")[None, :]
    there = t < n[:, None]
    at = torch.where(there, cu[:-1, None] + t, torch.zeros_like(t))
    return rows[at], there, n


def _attend(parts, mask):
    """softmax(q k^T / sqrt(E)) v over the keys of all parts (q [n, t, heads, E], k and v [n, l, kv heads, E]) under mask [n, t, all l]:
    a list of each part's share of the output, zero for rows that see no key."""
    n, t, hq, _ = parts[0][0].shape
    hkv = parts[0][1].shape[2]
    heads = lambda q: q.reshape(n, t, hkv, hq // hkv, E).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, E)  # noqa: E731
    s = torch.cat([heads(q) @ k.permute(0, 2, 3, 1) for q, k, _ in parts], -1).view(n, hkv, hq // hkv, t, -1).mul_(1.0 / math.sqrt(E))
    s.masked_fill_(~mask[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    s.sub_(torch.where(m == -math.inf, torch.zeros_like(m), m)).exp_()
    total = s.sum(-1, keepdim=True)
    s.div_(torch.where(total == 0, torch.ones_like(total), total))
    shares = s.view(n, hkv, -1, s.shape[-1]).split([k.shape[1] for _, k, _ in parts], -1)
    return [(p @ v.permute(0, 2, 1, 3)).view(n, hkv, hq // hkv, t, E).permute(0, 3, 1, 2, 4).reshape(n, t, hq, E)
            for p, (_, _, v) in zip(shares, parts)]


def _page_rows(pages, table):
    """Rows [sequences, positions, kv heads, E] in fp32 of swizzled pages [pages, kv heads, 64, E]: chunk c of token t lies at c ^ (t & 7)."""
    t = torch.arange(PAGE, device="cuda")[:, None]
    at = torch.arange(16, device="cuda")[None, :] ^ (t & 7)
    rows = pages.view(*pages.shape[:-1], 16, 8)[:, :, t, at].reshape(pages.shape)[table.long()]
    return rows.permute(0, 1, 3, 2, 4).reshape(table.shape[0], -1, pages.shape[1], E).float()


def run(state):
    st, op, case = state, state["op"], state["case"]
    if op == "rope":
        if own:
            return st["rope"].apply(st["q"], st["k"], st["pos"])
        return tuple(_turned(x, st["pos"], st["w"], st["amp"], case["rot"], case["inter"]) for x in (st["q"], st["k"]))
    if op == "copy":
        if own:
            from bit_kv_cache_paged_gb300 import bf16_copy_pages
            bf16_copy_pages(st["k"], st["v"], st["src"], st["dst"])
        else:
            st["k"][:, st["dst_d"]] = st["k"][:, st["src_d"]]
            st["v"][:, st["dst_d"]] = st["v"][:, st["src_d"]]
        return st["k"], st["v"]
    if op == "bf16":
        if own:
            from bit_kv_cache_paged_gb300 import bf16_chunk_attend
            return bf16_chunk_attend(st["q"], st["k"], st["v"], st["table"], st["lengths"], st["cu"], st["err"], workspace=st["workspace"])
        q, there, n = _padded(st, st["q"])
        k, v = _page_rows(st["k"], st["table"]), _page_rows(st["v"], st["table"])
        pos = st["lengths"].long()[:, None] - n[:, None] + torch.arange(st["most_new"], device="cuda")
        mask = torch.arange(k.shape[1], device="cuda")[None, None, :] <= pos[:, :, None]
        return _attend([(q.float(), k, v)], mask & there[:, :, None])[0][there].bfloat16()
    if own:
        return st["pool"].chunk_attend(0, st["q"], st["k_new"], st["v_new"])
    # keys: the BF16 rows of the cache and the chunk, and the INT2 history in its rotated basis
    q, there, n = _padded(st, st["q"])
    kn, vn = _padded(st, st["k_new"])[0].float(), _padded(st, st["v_new"])[0].float()
    q, t = q.float(), torch.arange(st["most_new"], device="cuda")
    mask = [st["bf_live"][:, None, :].expand(-1, len(t), -1), (t[None, :] <= t[:, None])[None] & there[:, None, :]]
    parts = [(q, torch.cat([st["bf"][0].float(), kn], 1), torch.cat([st["bf"][1].float(), vn], 1))]
    if st["kq"] is not None:
        kh, vh = ((c.float() * s.float() + z.float()).flatten(-2) for c, s, z in (st["kq"], st["vq"]))
        p = torch.arange(kh.shape[1], device="cuda")[None, :]
        mask.append(((p >= SINK) & (p < st["front"][:, None]))[:, None, :].expand(-1, len(t), -1))
        grouped = q.unflatten(2, (case["hkv"], -1))
        parts.append((torch.einsum("nthge,hef->nthgf", grouped, st["rk"]).flatten(2, 3), kh, vh))
    o = _attend(parts, torch.cat(mask, -1) & there[:, :, None])
    if len(o) > 1:
        o[0] = o[0] + torch.einsum("nthgf,hef->nthge", o[1].unflatten(2, (case["hkv"], -1)), st["rv"]).flatten(2, 3)
    return o[0][there].bfloat16()


# ------------------------------------------------------------------------------------------------ in 64 bits
def _softmax64(scores):
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "rope":
        # as a rotation of complex numbers
        w, amp = _frequencies(case)
        turn = torch.polar(torch.full((1, 1, 1), amp, dtype=torch.float64, device="cuda"),
                           (st["pos"].double()[:, None, None] * torch.from_numpy(w).cuda()))
        out, rot = [], case["rot"]
        for x in (st["q"], st["k"]):
            y = x.double().clone()
            pairs = y[..., :rot].unflatten(-1, (-1, 2)) if case["inter"] else y[..., :rot].unflatten(-1, (2, -1)).transpose(-1, -2)
            z = torch.view_as_real(torch.complex(pairs[..., 0].contiguous(), pairs[..., 1].contiguous()) * turn)
            y[..., :rot] = z.flatten(-2) if case["inter"] else z.transpose(-1, -2).flatten(-2)
            out.append(y)
        return tuple(out)
    if op == "copy":
        out = []
        for x in (st["k"], st["v"]):
            of = np.arange(case["pages"])
            of[st["dst"]] = st["src"]
            out.append(x.index_select(1, torch.from_numpy(of).cuda()).double())
        return tuple(out)
    new, ctx = _lengths(case)
    hq, hkv = case["hq"], case["hkv"]
    if 4 * E * hq * float((new * (ctx + new)).sum()) * (2 if op == "pool" else 1) > 8e12:  # over about 20 seconds in 64 bits
        return None
    hg, cu, scale = hq // hkv, np.concatenate([[0], np.cumsum(new)]), 1.0 / math.sqrt(E)
    out = torch.zeros((int(cu[-1]), hq, E), dtype=torch.float64, device="cuda")
    tok, chunk = np.arange(PAGE)[:, None], np.arange(E)[None, :]
    stored = torch.from_numpy(((chunk // 8) ^ (tok % 8)) * 8 + chunk % 8).cuda()  # dim -> stored place, by token of the page
    for i in range(len(new)):
        t = int(new[i])
        for h in range(hkv):
            q = st["q"][int(cu[i]):int(cu[i + 1]), h * hg:(h + 1) * hg].double().reshape(t * hg, E)
            mine = torch.arange(t, device="cuda").repeat_interleave(hg)[:, None]
            if op == "bf16":
                ids = st["table"][i, :-(-int(ctx[i] + t) // PAGE)].long()
                k, v = (x[ids, h].gather(-1, stored.expand(len(ids), -1, -1)).double().flatten(0, 1) for x in (st["k"], st["v"]))
                s = q @ k.T * scale
                s = s.masked_fill(torch.arange(len(k), device="cuda")[None, :] > mine + int(ctx[i]), -math.inf)
                o = _softmax64(s) @ v
            else:
                here = st["bf_live"][i]
                k, v = (torch.cat([b[i, here, h], x[int(cu[i]):int(cu[i + 1]), h]]).double() for b, x in zip(st["bf"], (st["k_new"], st["v_new"])))
                s = q @ k.T * scale
                s = s.masked_fill(torch.arange(len(k), device="cuda")[None, :] > mine + int(here.sum()), -math.inf)
                front = int(st["front"][i])
                if front > SINK:
                    kh, vh = (torch.addcmul(z.double(), c.double(), sc.double()).flatten(-2)
                              for c, sc, z in ([y[i, SINK:front, h] for y in x] for x in (st["kq"], st["vq"])))
                    p = _softmax64(torch.cat([q @ st["rk"][h].double() @ kh.T * scale, s], -1))
                    o = p[:, :front - SINK] @ vh @ st["rv"][h].double().T + p[:, front - SINK:] @ v
                else:
                    o = _softmax64(s) @ v
            out[int(cu[i]):int(cu[i + 1]), h * hg:(h + 1) * hg] = o.view(t, hg, E)
    return out

"""Chunk attention over both caches within a narrow row bound (chunk_ref): queries point at keys of the whole cache, so that
every block of it matters to some row."""
import pytest
import torch

from bit_kv_cache_paged_gb300 import binding as B
from chunk_ref import check_rows, pointed, reference
from test_gpu_chunk import E, Mixed, Pages, built  # noqa: F401

pytestmark = pytest.mark.gpu


def targets(g, rows, n, hist):
    """Three of n cached positions a row; the first rows take the ends of the history [64, 64 + hist) and of the cache."""
    at = torch.randint(0, n, (rows, 3), generator=g, device="cuda")
    ends = [[0, n - 1, n // 2]]
    if hist:
        ends += [[64, 64 + hist - 1, 64 + min(127, hist - 1)], [64 + hist - 1 - min(hist - 1, 63), 63, 64 + min(128, hist - 1)]]
    e = torch.tensor(ends, device="cuda")[:rows]
    at[:len(e)] = e
    return at


class Pointed(Mixed):
    """A Mixed pool whose queries point at cached keys."""

    def fill(self, ctx):
        for i in range(len(ctx)):
            self.add(i)
        self.pool.step_begin(range(len(ctx)), ctx)
        kv = self.new_rows(sum(ctx))
        for l in range(self.layers):
            self.pool.append_and_demote(l, kv[0][l], kv[1][l])
        r = 0
        for i, n in enumerate(ctx):
            self.rows[i] = [x[:, r:r + n] for x in kv]
            r += n
        return self

    def chunk(self, ids, n_new, launches, least=0):
        """One step: chunk attention against the reference, the append. least: launches of a call with the least workspace."""
        T, hg = sum(n_new), self.hq // self.hkv
        kn, vn = self.new_rows(T)
        cached = [self.pool.seq_info(s) for s in ids]
        assert all(self.rows[s][0].shape[1] == L for s, (L, _, _) in zip(ids, cached))
        held = {(s, l, h): self.held(s, l, h) for s, n in zip(ids, n_new) if n for l in range(self.layers) for h in range(self.hkv)}
        q = torch.empty((self.layers, T, self.hq, E), dtype=torch.bfloat16, device="cuda")
        for l in range(self.layers):
            r = 0
            for s, n, (L, F, _) in zip(ids, n_new, cached):
                for h in range(self.hkv) if n else ():
                    keys = torch.cat([self.rows[s][0][l, :, h], kn[l, r:r + n, h]]).double()
                    at = targets(self.g, n * hg, L, max(0, F - 64)) if L else torch.full((n * hg, 3), 0, device="cuda")
                    x = pointed(self.g, keys, at, plain=(self.gain[0, h] == 1).double())
                    q[l, r:r + n, h * hg:h * hg + hg] = x.view(n, hg, E)
                r += n
        self.pool.step_begin(ids, n_new)
        outs = []
        for l in range(self.layers):
            both = []
            for count in (launches, least) if least else (launches,):
                before = self.pool.launch_count()
                ws = torch.empty(B.oscar_chunk_workspace_min_bytes(self.pool.handle), dtype=torch.uint8, device="cuda") if both else None
                both.append(self.pool.chunk_attend(l, q[l], kn[l], vn[l], workspace=ws))
                assert self.pool.launch_count() - before == count
            outs.append(both)
            self.pool.append_and_demote(l, kn[l], vn[l])
        self.pool.check()
        r = 0
        for s, n in zip(ids, n_new):
            self.rows[s] = [torch.cat([x, y[:, r:r + n]], 1) for x, y in zip(self.rows[s], (kn, vn))]
            r += n
        for l in range(self.layers):
            r = 0
            for s, n in zip(ids, n_new):
                for h in range(self.hkv) if n else ():
                    kb, vb, hist = held[s, l, h]
                    k, v = torch.cat([kb, kn[l, r:r + n, h].double()]), torch.cat([vb, vn[l, r:r + n, h].double()])
                    x = q[l, r:r + n, h * hg:h * hg + hg].reshape(-1, E).double()
                    t = torch.arange(n * hg, device="cuda")[:, None] // hg
                    parts, seen = [(x, k, v, None, False)], [torch.arange(len(k), device="cuda")[None] <= len(kb) + t]
                    if hist:
                        parts.append((x @ self.R[0][l, h], hist[0], hist[1], None if self.absorbed else self.R[1][l, h].T, True))
                        seen.append(torch.ones((n * hg, len(hist[0])), dtype=torch.bool, device="cuda"))
                    o, bound = reference(parts, torch.cat(seen, -1))
                    for out in outs[l]:
                        check_rows(out[r:r + n, h * hg:h * hg + hg].reshape(-1, E), o, bound, f"seq {s} layer {l} head {h}")
                r += n


FORMS = [dict(group=128), dict(group=32), dict(group=128, absorbed=True), dict(group=32, absorbed=True, lloyd=(1.2, 0.8)),
         dict(group=128, lloyd=(0.9, 1.3))]
IDS = ["128", "32", "128 absorbed", "32 absorbed lloyd", "128 lloyd"]


@pytest.mark.parametrize("form", FORMS, ids=IDS)
@pytest.mark.parametrize("hq,hkv", [(8, 2), (8, 1)])
def test_pool_codes_expanded_in_the_kernel(form, hq, hkv):
    m = Pointed(layers=2, hq=hq, hkv=hkv, seed=40, **form).fill([0, 63, 64, 321, 385, 400, 1000, 2500, 5500])
    m.chunk([8, 7, 6, 5, 4, 3, 2, 1, 0], [3, 1, 70, 0, 2, 130, 5, 1, 40], 2)
    m.chunk([8], [1], 2)


@pytest.mark.parametrize("form", FORMS, ids=IDS)
@pytest.mark.parametrize("hq,hkv", [(32, 8), (64, 8)])
def test_pool_single_tokens(form, hq, hkv):
    m = Pointed(hq=hq, hkv=hkv, seed=41, **form).fill([3500, 0, 400, 5904, 63, 2000, 1000, 330])
    m.chunk(list(range(8)), [1] * 8, 5)
    m.chunk([3, 6, 0, 5], [1, 9, 1, 1], 7)  # beside a chunk


@pytest.mark.parametrize("form", FORMS, ids=IDS)
@pytest.mark.parametrize("hq", [4, 8])
def test_pool_tiles(form, hq):
    m = Pointed(hq=hq, hkv=1, seed=42, **form).fill([1500, 0, 385, 5049, 320])
    m.chunk([4, 3, 1, 0, 2], [600, 701, 900, 425, 0], 4, least=2)


@pytest.mark.parametrize("form", FORMS, ids=IDS)
def test_pool_whole_items(form):
    """More items than SMs: each is one block's, its key blocks one after another."""
    m = Pointed(hq=32, hkv=8, seed=43, **form).fill([1300, 900, 1111, 700, 450, 1600, 800, 1000, 1200, 640])
    m.chunk(list(range(10)), [100, 64, 65, 128, 80, 2, 90, 70, 1, 77], 2)
    m.chunk(list(range(0, 10, 2)), [300, 385, 333, 400, 320], 4)


def test_pool_single_tokens_beside_tiles():
    """Both kinds in one call: nine launches, the single tokens left out of the tiles and of the chunk kernel's work."""
    m = Pointed(hq=32, hkv=8, seed=44).fill([3500, 1500, 400, 5904])
    m.chunk([0, 1, 2, 3], [1, 500, 1, 1], 9, least=7)
    m.chunk([0, 1, 2, 3], [330, 500, 0, 1], 9)


@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (32, 8), (8, 1), (16, 1)])
def test_bf16(hq, hkv):
    lens, new = [65, 300, 1001, 200, 2100, 777, 9000, 128], [65, 128, 1, 70, 3, 129, 40, 0]
    c = Pages(lens, hkv, seed=hq)
    g = torch.Generator(device="cuda").manual_seed(hq)
    q, hg, r = torch.empty((sum(new), hq, E), dtype=torch.bfloat16, device="cuda"), hq // hkv, 0
    for i, (n, L) in enumerate(zip(new, lens)):
        for h in range(hkv) if n else ():
            q[r:r + n, h * hg:h * hg + hg] = pointed(g, c.rows[i][0][:, h], targets(g, n * hg, max(1, L - n), 0)).view(n, hg, E)
        r += n
    out = c.attend(q, new)
    assert int(c.err) == 0
    r = 0
    for i, (n, L) in enumerate(zip(new, lens)):
        for h in range(hkv) if n else ():
            k, v = (x[:, h].double() for x in c.rows[i])
            x = q[r:r + n, h * hg:h * hg + hg].reshape(-1, E)
            t = torch.arange(n * hg, device="cuda")[:, None] // hg
            o, bound = reference([(x, k, v, None, False)], torch.arange(L, device="cuda")[None] <= L - n + t)
            check_rows(out[r:r + n, h * hg:h * hg + hg].reshape(-1, E), o, bound, f"seq {i} head {h}")
        r += n

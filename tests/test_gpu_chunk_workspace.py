"""The scratch of a chunk over the pool: how much a step needs, and what happens with less."""
import pytest
import torch

from bit_kv_cache_paged_gb300 import binding as B
from test_gpu_chunk import E, Mixed, built  # noqa: F401

pytestmark = pytest.mark.gpu


def step(m, new):
    """A step of new tokens a sequence: (q, k, v) for it."""
    m.pool.step_begin(range(len(new)), new)
    k, v = (x[0] for x in m.new_rows(sum(new)))
    return torch.randn((sum(new), m.hq, E), generator=m.g, device="cuda").bfloat16(), k, v


def filled(hq, hkv, ctx, **kw):
    m = Mixed(hq=hq, hkv=hkv, max_seqs=len(ctx), **kw)
    for i in range(len(ctx)):
        m.add(i)
    m.pool.step_begin(range(len(ctx)), ctx)
    k, v = m.new_rows(sum(ctx))
    m.pool.append_and_demote(0, k[0], v[0])
    return m


def attend(m, q, k, v, ws, out, nbytes=None):
    B.oscar_chunk_attend(m.pool.handle, 0, q, k, v, ws, out, torch.cuda.current_stream().cuda_stream, nbytes)


def refused(f, *a):
    with pytest.raises(B.OscarError) as e:
        f(*a)
    assert e.value.status == B.OSCAR_EINVAL


# a chunk whose codes the kernel expands, one with tiles, single tokens through the decode kernels, all together
@pytest.mark.parametrize("hq,hkv,ctx,new", [(8, 2, [700], [9]), (4, 1, [1500], [600]), (32, 8, [3500, 3000], [1, 1]),
                                            (32, 8, [3500, 3000, 1000], [1, 1, 400])])
def test_a_call_stays_within_its_workspace_and_refuses_a_smaller_one(hq, hkv, ctx, new):
    m = filled(hq, hkv, ctx)
    q, k, v = step(m, new)
    need = B.oscar_chunk_workspace_bytes(m.pool.handle)
    want = m.pool.chunk_attend(0, q, k, v)
    out = torch.full_like(want, 3.0)
    for at in (0, 16):  # 256-byte aligned and not
        buf = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        attend(m, q, k, v, buf[at:at + need], out)
        assert torch.equal(out, want) and (buf[at + need:] == 0xA5).all() and (buf[:at] == 0xA5).all()
    out.fill_(3.0)
    launches = m.pool.launch_count()
    refused(attend, m, q, k, v, torch.empty(15, dtype=torch.uint8, device="cuda"), out)
    refused(attend, m, q, k, v, buf.data_ptr(), out)  # an address without a size
    refused(attend, m, q, k, v, buf.data_ptr(), out, 0)
    assert m.pool.launch_count() == launches and (out == 3).all()
    m.pool.check()


def test_a_buffer_kept_from_a_shorter_step_is_not_overrun():
    m = filled(32, 8, [3500, 3000])
    step(m, [1, 1])
    need = B.oscar_chunk_workspace_bytes(m.pool.handle)
    buf = torch.full((64 << 20,), 0xA5, dtype=torch.uint8, device="cuda")
    for new in ([2, 2], [1, 2], [400, 400]):  # parts of a chunk; beside the decode kernels' partials; tiles
        q, k, v = step(m, new)
        assert B.oscar_chunk_workspace_bytes(m.pool.handle) > need
        want = m.pool.chunk_attend(0, q, k, v)
        out = torch.zeros_like(want)
        try:
            attend(m, q, k, v, buf[:need], out)
        except B.OscarError as e:
            assert e.status == B.OSCAR_EINVAL and (out == 0).all()
        else:
            torch.testing.assert_close(out, want, atol=2e-2, rtol=2e-2)
        torch.cuda.synchronize()
        assert (buf[need:] == 0xA5).all()


def test_tiles_are_left_out_where_they_do_not_fit(monkeypatch):
    m = filled(8, 2, [2000, 900])
    q, k, v = step(m, [330, 400])
    most, least = B.oscar_chunk_workspace_bytes(m.pool.handle), B.oscar_chunk_workspace_min_bytes(m.pool.handle)
    assert least + 10 * 2 * 65536 < most  # 2000 - 320 and 900 - 320 tokens of history: 14 + 5 blocks of 2 heads
    before = m.pool.launch_count()
    want = m.pool.chunk_attend(0, q, k, v)
    assert m.pool.launch_count() - before == 4  # with the tiles' two kernels
    buf = torch.full((most + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(want)
    for size in (most - 1, least):
        before = m.pool.launch_count()
        assert m.pool.chunk_attend(0, q, k, v, out=out, workspace=buf[:size]) is out
        assert m.pool.launch_count() - before == 2
        assert (buf[size:] == 0xA5).all()
        # the same codes and fp16 values; maxima are renewed by 32 scores in place of 128, which moves where a weight rounds:
        # fp16 weights by 2^-11 in one and twice that in the other, on rotated values of about 1 (1.5 * 2^-10, times sum |R_V|
        # = 9 a dim); bf16 weights by 2^-8 in both, on values of about 0.8 times their channel's gain; two outputs' roundings
        tol = 2.0 ** -7 * want.double().abs() + 1.5 * 2.0 ** -10 * 9 + 2.0 ** -7 * 0.8 * m.gain[1].double().repeat_interleave(4, 0)
        assert ((out.double() - want.double()).abs() <= tol).all()
    refused(lambda: m.pool.chunk_attend(0, q, k, v, workspace=buf[:least - 1]))
    empty = torch.empty

    def short(*a, **kw):  # an allocator that has the least left, but no more
        if a and isinstance(a[0], int) and a[0] > least:
            raise torch.cuda.OutOfMemoryError
        return empty(*a, **kw)
    small = m.pool.chunk_attend(0, q, k, v, workspace=buf[:least])
    monkeypatch.setattr(torch, "empty", short)
    before = m.pool.launch_count()
    got = m.pool.chunk_attend(0, q, k, v)
    assert m.pool.launch_count() - before == 2 and torch.equal(got, small)
    m.pool.check()


def test_workspace_argument_is_checked():
    m = filled(8, 2, [700])
    q, k, v = step(m, [9])
    n = B.oscar_chunk_workspace_bytes(m.pool.handle)
    for bad in (torch.empty(n, dtype=torch.uint8), torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            m.pool.chunk_attend(0, q, k, v, workspace=bad)
    for bad in (torch.empty(n, dtype=torch.int8, device="cuda"), 1 << 20):
        with pytest.raises(TypeError):
            m.pool.chunk_attend(0, q, k, v, workspace=bad)
    refused(lambda: m.pool.chunk_attend(0, q, k, v, workspace=torch.empty(n + 8, dtype=torch.uint8, device="cuda")[8:]))  # alignment


def test_tiles_stay_within_their_limit():
    """Histories whose tiles would take more than 4 GB (64 KB per block of 128 tokens and KV head) are expanded in the kernel;
    plans alone, nothing is computed."""
    m = Mixed(hq=32, hkv=8, max_seqs=2, max_len=1100000)
    for i in (0, 1):
        m.add(i)
    limit = 4 << 30
    for length, tiles in ((1000000, True), (1048576 + 320 - 200, True), (1048576 + 320 + 200, False)):
        m.pool.step_begin([0], [length - m.pool.seq_info(0)[0]])
        m.pool.step_begin([0], [400])  # seven pairs of tiles
        most, least = B.oscar_chunk_workspace_bytes(m.pool.handle), B.oscar_chunk_workspace_min_bytes(m.pool.handle)
        assert (most > least) == tiles and most - least <= limit
        assert not tiles or most - least > 0.9 * limit
        m.pool.seq_remove(0)
        m.pool.seq_add(0)

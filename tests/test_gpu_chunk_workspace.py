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

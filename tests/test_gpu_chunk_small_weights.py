"""Chunk attention over INT2 histories in which one key draws nearly all the attention and the others share the rest evenly:
weights far below the maximum still count, however they add up.

One key of value 0 and level 0; the others have value 1 and the level -x, so an output is the others' share of the attention
and has to be right in its own size. Levels around 2^-25 are where an fp16 weight under a maximum of 1 would vanish or be
rounded up to 2^-24.

Tolerance of an output o: 2^-8 o for its own rounding, 2^-10 o for fp16 weights (2^-11, twice where stored weights are scaled) and
the un-rotation, d o for scores off by d = sum_i |q_i k_si| 2^-17 / sqrt(128); and 2^-29 a key, half a step of the smallest fp16
number where the largest weight is 2^4."""
import math

import pytest
import torch

from test_gpu_chunk import E, built  # noqa: F401
from test_gpu_chunk_growth import NAT, Stairs

pytestmark = pytest.mark.gpu


class Spike(Stairs):
    def __init__(self, level, seqs, hist, hq, hkv, at):
        super().__init__(lambda j: j * 0.0, seqs, hist, hq, hkv, over=-400, seed=3)  # BF16 keys are out of sight
        z = torch.full((hist,), round(level * NAT / E * 512) / 512, device="cuda").half()
        z[at] = 0
        one = torch.ones(hist, device="cuda").half()
        one[at] = 0
        zero, code = torch.zeros_like(z), torch.zeros((hist, 32), dtype=torch.uint8, device="cuda")
        for i, h in self.codes:
            szk, szv = (torch.stack([zero, x], -1)[:, None].contiguous() for x in (z, one))
            self.pool.debug_write_int2(i, 0, h, 64, code, szk, code, szv)
        self.z = z.double()

    def share(self, new, launches):
        T = sum(new)
        q = torch.ones((T, self.hq, E), dtype=torch.bfloat16, device="cuda")
        kn, vn = self.rows(T)
        self.pool.step_begin(range(self.seqs), new)
        before = self.pool.launch_count()
        out = self.pool.chunk_attend(0, q, kn, vn)
        assert self.pool.launch_count() - before == launches
        self.pool.check()
        w = torch.exp(self.z * E / math.sqrt(E))
        o = ((w.sum() - 1) / w.sum()).item()
        d = E * self.z.abs().max().item() * 2.0 ** -17 / math.sqrt(E)
        err = (out.double() - o).abs().max().item()
        tol = (2.0 ** -8 + 2.0 ** -10 + d) * o + len(w) * 2.0 ** -29
        assert err <= tol, f"share {o:.4g}, off by {err:.3g}, {err / tol:.3g} tolerances"


@pytest.mark.parametrize("level", [-20, -24.3, -25.2, -27])
@pytest.mark.parametrize("seqs,hist,hq,hkv,new,launches", [(2, 700, 32, 8, 100, 2), (12, 700, 32, 8, 100, 2), (4, 650, 32, 8, 330, 4), (1, 5000, 4, 1, 330, 4)])
def test_the_others_share(level, seqs, hist, hq, hkv, new, launches):
    for at in (0, 45):
        Spike(level, seqs, hist, hq, hkv, at).share([new] * seqs, launches)


def test_the_others_share_of_a_long_history():
    Spike(-25.2, 1, 131072, 4, 1, 0).share([400], 4)

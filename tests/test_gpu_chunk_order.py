"""GPU checks of what the rows' threads and the tensor core do to the outputs in
turn: accumulators that every step rescales, and values that are weighed one by
one in first and later steps, several items to a CTA."""
import math

import pytest
import torch

from tests.chunk_ref import BF16, F16, Chunk

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


def stairs(s, rise):
    """Scores that rise by `rise` from one tile of 128 positions to the next, values that
    fall by as much: every tile weighs the same in the end, whatever was rescaled before."""
    g = torch.Generator().manual_seed(9)
    s.q.copy_(torch.where(s.q.isnan(), s.q, torch.ones_like(s.q)))
    for b in range(s.B):
        n = int(s.pos[b]) + s.n[b]
        for t in range(n):
            at = (int(s.table[b, t // s.bs]), t % s.bs)
            k = (rise * (t // 128) + torch.randn((s.Hkv, 1), generator=g)) / (s.D * s.scale) * torch.ones(s.D)
            s.block(at[0], 0)[:, at[1]] = k.to(s.dtype)
            s.block(at[0], 1)[:, at[1]] *= math.exp(rise * ((n - 1) // 128 - t // 128))


@pytest.mark.parametrize("rise", [1.0, 6.0, 9.0])      # the maximum is taken anew past a growth of 2^8 = e^5.5
@pytest.mark.parametrize("D,bs", [(64, 16), (128, 16), (64, 3), (32, 16)])
def test_every_tile_weighs_the_same_after_all_rescaling(rise, D, bs):
    s = Chunk(dtype=BF16, D=D, bs=bs, B=3, T=130, H=4, Hkv=2, pos=[500, 0, 771], counts=[130, 130, 1])
    stairs(s, rise)
    s.check(s.call())


@pytest.mark.parametrize("window", [0, 200])
@pytest.mark.parametrize("dtype,D,H", [(BF16, 64, 8), (F16, 64, 8), (BF16, 128, 8), (BF16, 64, 64)])
def test_values_that_are_not_finite_in_many_short_items(dtype, D, H, window):
    """More items than CTAs, some with one step, an odd value in the first or the last."""
    B = 60
    s = Chunk(dtype=dtype, D=D, B=B, T=9, H=H, Hkv=8, bs=16, window=window,
              pos=[(b * 97) % 400 for b in range(B)], counts=[1 + b % 9 for b in range(B)])
    for b in range(0, B, 2):
        for t in ((int(s.pos[b]) + s.n[b] - 1) if b % 4 else int(s.pos[b]),):
            s.block(int(s.table[b, t // 16]), 1)[b % 8, t % 16, b % D] = (math.inf, -math.inf, math.nan)[b % 3]
    s.check(s.call())

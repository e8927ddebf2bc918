"""GPU checks of how 16-bit weights enter the second product: in two parts for
few rows and in the differential form, else in one, and then normalised by
what they were rounded to.  Keys are such that scores hold no rounding but the
scale's: what is left is the weights'."""
import math

import pytest
import torch

from tests.chunk_ref import BF16, F16, F32, Chunk, half_step

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


def fill(s, keys, values):
    """Every query row is (1, 1, 0, ...), key t (keys[t], 0, ...), so that its score is their
    sum in full (scale 1); value t is values[t] [D] for every kv head."""
    q = torch.zeros(s.D, dtype=s.dtype)
    q[:2] = 1
    s.q.copy_(torch.where(s.q.isnan(), s.q, q))
    for b in range(s.B):
        for t in range(int(s.pos[b]) + s.n[b]):
            blk, slot = int(s.table[b, t // s.bs]), t % s.bs
            s.block(blk, 0)[:, slot] = 0
            s.block(blk, 0)[:, slot, :2] = keys[t].to(s.dtype)
            s.block(blk, 1)[:, slot] = values[t].to(s.dtype)


# (single tokens, speculative ones, 128 rows; blocks in boxes and on mma.sync)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("T,H,Hkv", [(1, 8, 1), (1, 4, 4), (4, 8, 2), (16, 8, 1), (128, 2, 2)])
@pytest.mark.parametrize("D,bs", [(64, 16), (128, 16), (128, 3), (32, 16), (256, 16), (64, 1)])
def test_values_that_all_but_cancel_keep_their_bits_in_calls_of_few_rows(D, bs, T, H, Hkv, dtype):
    """Neighbouring positions weigh almost alike and hold opposite values.  Each weight off
    by the square of half a step (2^-16; 2^-22, or 2^-25 of the largest), the exponent by 4
    roundings of fp32, 2^-22 for the exponential, 2 roundings a position for the sums of
    both."""
    s = Chunk(dtype=dtype, D=D, bs=bs, B=2, T=T, H=H, Hkv=Hkv, pos=[31, 0], scale=1.0)
    g = torch.Generator().manual_seed(4)
    n = 31 + T
    keys = torch.stack((-torch.rand(n, generator=g) * 3, torch.rand(n, generator=g) / 64), -1).to(dtype)
    keys[1::2, 0] = keys[:n // 2 * 2:2, 0]
    values = (torch.where(torch.rand(n, D, generator=g) < 0.5, 1.0, 1.25)).to(dtype)
    values[1::2] = -values[:n // 2 * 2:2]
    fill(s, keys, values)
    out = s.call().cpu().double()
    u = 2.0 ** -24
    x = keys.double().sum(-1)
    for b in range(2):
        for t in range(s.n[b]):
            m = int(s.pos[b]) + t + 1
            w = (x[:m] - x[:m].max()).exp()
            a = w / w.sum()
            want, av = a @ values[:m].double(), a @ values[:m].double().abs()
            tol = av * (2 * (4 * u * float(x[:m].abs().max()) + 2.0 ** -22) + half_step(dtype) ** 2 + 2 * (m + 8) * 2 * u)
            if dtype == F16:
                tol = tol + 2.0 ** -25 * values[:m].double().abs().sum(0) / w.sum()
            tol = tol + half_step(dtype) * (want.abs() + tol)
            off = ((out[b, t] - want).abs() / tol).max()
            assert off <= 1, f"sequence {b}, token {t}: {float(off):.2f} of the bound"


@pytest.mark.parametrize("dtype,step", [(F16, 2.0 ** -11), (BF16, 2.0 ** -8)])
@pytest.mark.parametrize("D,bs", [(64, 16), (128, 16), (128, 3), (32, 16), (256, 16)])
@pytest.mark.parametrize("T,H,Hkv", [(1, 4, 4), (140, 4, 2)])
@pytest.mark.parametrize("window", [0, 200])
def test_equal_values_come_back_as_they_are(window, T, H, Hkv, D, bs, dtype, step):
    """All weights but one are just under the middle between a half and the next element:
    rounding takes the same 0.9 of half a step from each, and the sum must know of it.
    What is left, some roundings of fp32 a position, is far below half a step."""
    s = Chunk(dtype=dtype, D=D, bs=bs, B=2, T=T, H=H, Hkv=Hkv, pos=[300, 180], scale=1.0, window=window)
    n = 300 + T
    want = math.log(0.5 * (1 + 0.9 * step))
    first = float(torch.tensor(want).to(dtype))
    keys = torch.tensor([first, want - first]).repeat(n, 1).to(dtype)
    w = keys[1].double().sum().exp()
    assert abs(w / 0.5 - 1 - 0.9 * step) < 0.05 * step and float(w.to(dtype)) == 0.5
    keys[::50] = 0                                # of every window one position of weight 1
    fill(s, keys, torch.ones(n, D))
    out = s.call().cpu()
    for b in range(2):
        assert (out[b] == 1).all(), f"sequence {b}: {float(out[b].float().min())} to {float(out[b].float().max())}"


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_values_that_all_but_cancel_in_the_differential_form(dtype):
    """Both maps the same and lambda 1: the maps' two sums are the same sums."""
    s = Chunk(dtype=dtype, D=128, B=2, T=3, H=4, Hkv=2, pos=[700, 5], diff=True, norm=False, out_scale=1.0)
    q = s.q[..., :64].clone()
    s.q[..., 64:] = q
    for b in range(2):
        for j in range(-(-(int(s.pos[b]) + s.n[b]) // s.bs)):
            k = s.block(int(s.table[b, j]), 0)
            k[..., 64:] = k[..., :64].clone()
    s.lam.fill_(1.0)
    out = s.call()
    for b in range(2):
        n = s.n[b]
        v = s.rows(b, 1, int(s.pos[b]) + n).double().abs().amax()
        # two divisions and a product of sums that agree to the bit, 3 roundings of them
        assert float(out[b, :n].abs().max()) <= float(v) * 3 * 2.0 ** -24 * 2

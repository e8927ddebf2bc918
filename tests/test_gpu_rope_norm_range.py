"""GPU checks of the norm of paged_kv_append_rope near both ends of what the sum
of a row's squares may be, against the 64-bit restatement with the bound of any
other row, and of what the header says of rows past them."""
import pytest
import torch

from tests import fp4_ref as ref
from tests.test_gpu_rope_append import BF16, F16, F32, Step

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("dtype,magnitude,eps", [
    (BF16, 1e18, 1e-6), (F32, 1e18, 0.0), (F32, 1e-12, 0.0), (F32, 3e-19, 0.0), (F32, 2.0 ** -55, 2.0 ** -110),
    (F32, 1e-25, 1e-6), (BF16, 1e-25, 1e-6), (F16, 6e3, 0.0), (F16, 1e-6, 0.0)])
def test_rows_near_the_ends(dtype, magnitude, eps, fp4):
    s = Step(T=5, counts=[5, 1, 3], H=6, Hkv=2, D=64 if dtype == F16 else 128, dtype=dtype, norm=True, fp4=fp4, eps=eps,
             magnitude=magnitude, seed=31)
    out = s.gpu()
    torch.cuda.synchronize()
    s.check(*out)


@pytest.mark.parametrize("T", [2, 300])
@pytest.mark.parametrize("dtype,fp4", [(BF16, False), (F32, False), (BF16, True)])
def test_rows_whose_squares_pass_binary32_are_zeros(dtype, fp4, T):
    """One head of queries and one of keys of each token; the heads beside them are as ever."""
    s = Step(B=4, T=T, counts=[2, 1, 0, 2], H=8, Hkv=4, dtype=dtype, norm=True, fp4=fp4, seed=32)
    s.q, s.k, s.v = s.q.clone(), s.k.clone(), s.v.contiguous()
    s.q[:, :, 5] *= 1e20
    s.k[:, :, 2] *= 1e20
    q_out, pool, scales = (x.cpu() for x in s.gpu())
    torch.cuda.synchronize()
    for b in range(s.B):
        n = int(s.counts[b])
        pos = s.pos[b] + torch.arange(n)
        y = ref.turn(s.q[b, :n], s.qw, s.cs, pos, s.R, s.pairs, s.eps, torch.float64)
        tol = ref.turn_bound(s.q[b, :n], s.qw, s.cs, pos, s.R, s.pairs, s.eps) * (1 + 2.0 ** -7) + ref.half_step(y, dtype)
        near = [h for h in range(s.H) if h != 5]
        assert ((q_out[b, :n].double() - y).abs() <= tol)[:, near].all() and not q_out[b, :n, 5].any()
        blk, slot = s.table[b, pos // s.bs].long(), pos % s.bs
        assert not (pool if fp4 else pool.view(dtype))[blk, 0, 2, slot].any()
        assert not fp4 or not scales[blk, 0, 2, slot].any()

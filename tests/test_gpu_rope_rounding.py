"""GPU checks that the rotation of paged_kv_append_rope and its 4-bit form is the
stated formula operation by operation: fp32 queries and keys bit for bit, each
product and each sum rounded by itself."""
import pytest
import torch

from tests import fp4_ref as ref
from tests.test_gpu_rope_append import F32, Step, bits

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("D,R,pairs,fp4", [(16, 16, False, False), (64, 64, False, False), (128, 128, False, False),
                                           (128, 48, False, False), (128, 128, True, False), (64, 16, True, False),
                                           (64, 64, False, True), (128, 48, False, True), (256, 256, False, True),
                                           (128, 112, True, True)])
@pytest.mark.parametrize("T", [1, 300])
def test_rotation_is_rounded_operation_by_operation(D, R, pairs, fp4, T):
    s = Step(B=8, T=T, counts=[min(T, n) for n in (9, 1, 3, 40, 5, 2, 1, 4)], pos=[0, 3, 300, 7, 1900, 1, 200, 14], H=6, Hkv=2,
             D=D, R=R, pairs=pairs, dtype=F32, fp4=fp4, seed=D + R)
    q_out, pool, scales = s.gpu()
    torch.cuda.synchronize()
    q_out, pool, scales = q_out.cpu(), pool.cpu(), scales.cpu()
    for b in range(s.B):
        n = int(s.counts[b])
        pos = s.pos[b] + torch.arange(n)
        q, k = (ref.turn(x[b, :n], None, s.cs, pos, R, pairs, 0.0, torch.float32) for x in (s.q, s.k))
        assert torch.equal(bits(q_out[b, :n]), bits(q))
        blk, slot = s.table[b, pos // s.bs].long(), pos % s.bs
        if fp4:
            codes, sc = ref.quantise(k, 1.0)
            assert torch.equal(pool[blk, 0, :, slot], codes) and torch.equal(scales[blk, 0, :, slot], sc)
        else:
            assert torch.equal(pool[blk, 0, :, slot], bits(k).view(n, s.Hkv, -1))

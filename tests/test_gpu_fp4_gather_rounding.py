"""GPU check of how paged_kv_gather_fp4 rounds: the product with a factor that is
no power of two in binary32, then to the dtype, at factors whose product lies
beside the middle between two values of the dtype and binary32's is that
middle."""
import pytest
import torch

import pagedattention_decode_paged_gb300 as pa
from tests import fp4_ref as ref
from tests.test_gpu_fp4 import BF16, F16, F32, Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


def factors(dtype):
    """fp32 factors g for which 1.5 g or 3.5 g in binary32 is half a step of dtype above 1, and is not in 64 bits."""
    found = []
    mid = torch.tensor(1 + torch.finfo(dtype).eps / 2, dtype=torch.float64)
    for c in (1.5, 3.5, 1.75):
        near = (mid / c).float()
        for step in range(-3, 4):
            g = (near.view(torch.int32) + step).view(torch.float32)
            if (c * g).double() == mid and c * g.double() != mid:
                found.append(float(g))
    return found


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_the_product_is_rounded_to_binary32_first(dtype):
    gs = factors(dtype) if dtype != F32 else [0.1, 1.1]
    assert gs
    for g in gs:
        c = Cache(lens=[40, 7], H=3, Hkv=3, D=128, dtype=dtype, k_scale=g, v_scale=g, seed=81).to_gpu()
        k, v = (torch.zeros((2, 40, 3, 128), dtype=dtype, device="cuda") for _ in range(2))
        i32 = dict(dtype=torch.int32, device="cuda")
        pa.paged_kv_gather_fp4(k, v, c.flat, c.flat[c.g["pool"].stride(1):], c.g["scales"], c.g["table"],
                               torch.zeros(2, **i32), c.g["lens"], k_scale=g, v_scale=g, **c.kw)
        for b, n in enumerate((40, 7)):
            x = ref.cached_rows(c.pool, c.scales, c.table[b], c.bs, 0, n, (1.0, 1.0)).transpose(1, 2).float()
            want = (x * torch.tensor(g, dtype=torch.float32)).to(dtype)
            assert torch.equal(k[b, :n].cpu(), want[0]) and torch.equal(v[b, :n].cpu(), want[1])

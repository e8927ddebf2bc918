"""GPU checks of the number of sequences that the 4-bit decode takes in one
call: what the header promises is accepted and right, more is refused."""
import pytest
import torch

import pagedattention_decode_paged_gb300 as pa
from tests.test_gpu_fp4 import BF16, F16, F32, Cache, held_to

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("group", [1, 4, 8, 16])
@pytest.mark.parametrize("D,most", [(64, 8000), (128, 8000), (256, 2000)])
def test_sequences_that_always_fit(D, most, group, dtype):
    for bs in (16, 24):
        size = dict(num_heads=2 * group, num_kv_heads=2, head_dim=D, block_size=bs, max_blocks_per_seq=4, num_blocks=8,
                    block_stride=2 * 2 * bs * D // 2, dtype=dtype)
        assert pa.paged_attention_fp4_workspace(pa.make_shape(batch=most, **size)) > 0
        assert pa.paged_attention_fp4_workspace(pa.make_shape(batch=30000, **size)) == 0
        assert pa.paged_attention_fp4_workspace(pa.make_shape(batch=1 << 26, **size)) == 0


@pytest.mark.parametrize("D,dtype,H,B", [(64, F16, 4, 8000), (128, BF16, 1, 8000), (256, BF16, 1, 2000), (256, F32, 2, 2000)])
def test_as_many_sequences_as_promised(D, dtype, H, B):
    c = Cache(lens=[(i * 7) % 5 if i % 100 else 40 for i in range(B)], H=H, Hkv=1, D=D, dtype=dtype, seed=71).to_gpu()
    held_to(c.decode(), c.reference())


def test_more_sequences_are_refused():
    B, D = 30000, 128
    q = torch.zeros((B, 1, D), dtype=BF16, device="cuda")
    pool, scales = (torch.zeros((1, 2, 1, 16, n), dtype=torch.uint8, device="cuda") for n in (D // 2, D // 16))
    table, lens = torch.zeros((B, 1), dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    kw = dict(num_kv_heads=1, block_size=16, num_blocks=1, block_stride=pool.stride(0))
    with pytest.raises(pa.PagedAttnError) as e:
        pa.fp4_workspace_for(q, table, **kw)
    assert e.value.status == pa.PA_ERR_UNSUPPORTED
    flat = pool.view(-1)
    with pytest.raises(pa.PagedAttnError) as e:
        pa.paged_attention_decode_fp4(torch.empty_like(q), q, flat, flat[pool.stride(1):], scales, table, lens, 0.1,
                                      torch.zeros(1 << 24, dtype=torch.uint8, device="cuda"), **kw)
    assert e.value.status == pa.PA_ERR_UNSUPPORTED

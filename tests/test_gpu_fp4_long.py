"""GPU checks that no token of a long context is lost or taken twice where the
4-bit decode cuts items between CTAs: every score is the same, one token of each
32 has a value, each tile in an element of its own, so that an output is a
count of tokens over the length; and that the workspace's counters, those of
both levels of merging, are left at zero."""
import pytest
import torch

import pagedattention_decode_paged_gb300 as pa
from tests.test_gpu_fp4 import BF16, F16, F32, Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


def markers(c, shift):
    """Keys of zero; values of one in one token of each tile of 32, at element
    (tile + shift) % D for the tokens of kv head 0, further on for the others.
    Returns how many markers each output element counts, [B][Hkv][D]."""
    live = c.scales != 0x7F
    c.scales[:, 0] = torch.where(live[:, 0], 0, 0x7F).to(torch.uint8)
    c.scales[:, 1] = torch.where(live[:, 1], 0x38, 0x7F).to(torch.uint8)
    c.pool[:, 1] = torch.where(live[:, 1].repeat_interleave(8, -1), 0, 0xFF).to(torch.uint8)
    count = torch.zeros(c.B, c.Hkv, c.D, dtype=torch.float64)
    for b in range(c.B):
        n = int(c.lens[b])
        tile = torch.arange(-(-n // 32))
        tok = torch.minimum(tile * 32 + (tile * 7 + shift) % 32, torch.tensor(n - 1))
        blk, slot = c.table[b, tok // c.bs].long(), tok % c.bs
        for h in range(c.Hkv):
            d = (tile + shift + 5 * h) % c.D
            c.pool[blk, 1, h, slot, d // 2] = torch.where(d % 2 == 0, 0x02, 0x20).to(torch.uint8)
            count[b, h].index_add_(0, d, torch.ones(len(d), dtype=torch.float64))
    return count


@pytest.mark.parametrize("lens,H,Hkv,dtype,D,bs", [
    ([40000], 8, 1, BF16, 128, 16),              # one item over every CTA: two levels of merging
    ([39999], 16, 1, F16, 128, 32),
    ([40001], 2, 1, F32, 128, 16),
    ([30011], 12, 1, F32, 64, 16),               # two column tiles
    ([20000], 4, 1, BF16, 256, 16),
    ([9001], 8, 1, BF16, 64, 24),                # rows looked up one by one
    ([25000, 13001], 16, 2, BF16, 128, 16),      # several items over many CTAs each
    ([5000, 3, 0, 7777, 640], 8, 8, F16, 128, 16),
    ([31, 32, 33, 4097], 4, 4, F32, 256, 16)])
def test_every_tile_counts_once(lens, H, Hkv, dtype, D, bs):
    for shift in (0, 77):
        c = Cache(lens=lens, H=H, Hkv=Hkv, D=D, bs=bs, dtype=dtype, seed=51)
        count = markers(c, shift)
        c.to_gpu()
        got = c.decode().double().cpu().view(c.B, Hkv, H // Hkv, D)
        # Equal weights, exact in fp16, and whole sums below 2^24: exact up to the quotient
        # (two roundings and a product's) and the last rounding.
        want = (count / c.lens.clamp(min=1)[:, None, None])[:, :, None].expand_as(got)
        tol = want * (torch.finfo(dtype).eps / 2 + 4 * 2.0 ** -24)
        assert ((got - want).abs() <= tol).all()
        assert not counters(c).any()


def counters(c):
    """Everything behind the records in the workspace: the counters of groups and of items."""
    n = pa.paged_attention_fp4_workspace(pa.decode_shape(c.g["q"], c.g["table"], num_kv_heads=c.Hkv, **c.kw))
    heads = 16 if c.D <= 128 and c.H // c.Hkv * (2 if c.dtype == F32 else 1) > 8 else 8
    heads //= 2 if c.dtype == F32 else 1
    items = c.B * c.Hkv * -(-(c.H // c.Hkv) // heads)
    ctas = min(192, torch.cuda.get_device_properties(0).multi_processor_count)
    assert n == ctas * (4 * (16 * 128 + 2 * 16) * 4 + 2 * 4) + 4 * items
    return c.ws[n - 4 * items - 8 * ctas:n]

"""GPU checks of sequences whose counts or positions are out of range among valid ones:
what is written, what is reported, and that their rows' zeros are spread over the GPU."""
import pytest
import torch

import pagedattention_decode_paged_gb300 as pa
from tests.chunk_ref import BF16, F16, F32, Chunk

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


# fp32, mma.sync, tcgen05 in boxes and row by row; batches that a warp sums over and others
@pytest.mark.parametrize("dtype,D,bs,T", [(F32, 16, 16, 5), (F32, 64, 16, 5), (BF16, 32, 16, 5), (F16, 256, 8, 5),
                                          (BF16, 128, 16, 5), (F16, 64, 16, 5), (BF16, 64, 3, 150)])
@pytest.mark.parametrize("B", [1, 3, 128, 129, 700])
def test_zeros_and_reports(B, dtype, D, bs, T):
    g = torch.Generator().manual_seed(B)
    cnt = torch.randint(0, min(T, 5) + 1, (B,), generator=g).tolist()
    cnt[-1] = T
    s = Chunk(dtype=dtype, D=D, bs=bs, B=B, T=T, H=2, Hkv=1, counts=cnt,
              pos=torch.randint(0, 60, (B,), generator=g).tolist())
    for what in ("none", "lengths", "positions", "both", "last"):
        counts, pos = s.counts.clone(), s.pos.clone()
        zero, skip, err_want = [], [], 0
        for b in range(B):
            kind = (b * 7 + 3) % 5 if what != "last" else 4
            if kind == 0 and what in ("lengths", "both"):
                counts[b] = (-1, T + 1, 2 ** 31 - 1, -2 ** 31)[b % 4]
                skip.append(b)
                err_want |= pa.DEVERR_BAD_LEN
            if (kind == 1 and what in ("positions", "both")) or (what == "last" and b == B - 1):
                pos[b] = (-1, s.MB * bs - s.n[b] + 1, 2 ** 31 - 1, -2 ** 31)[b % 4]
                zero.append(b)
                err_want |= pa.DEVERR_BAD_POS
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = s.call(positions=pos, counts=counts, err=err)
        assert int(err.item()) == err_want
        got = out.cpu()
        for b in zero:
            assert not got[b, :s.n[b]].any() and torch.equal(got[b, s.n[b]:], s.out[b, s.n[b]:])
        s.check(out, zero=zero, skip=skip)


@pytest.mark.parametrize("D,dtype", [(128, BF16), (64, F32), (256, F16)])
def test_the_zeros_of_a_long_prompt_take_a_fill_s_time(D, dtype):
    """A prompt of 16384 tokens with positions out of range beside a single token that is
    attended to as ever.  By one CTA in 2-byte stores the zeros alone take a hundred times
    the fill."""
    B, T, H, Hkv, bs = 2, 16384, 64, 8, 16
    per = 2 * Hkv * bs * D
    pool = torch.randn(8 * per, device="cuda").to(dtype)
    q = torch.randn((B, 1, H, D), device="cuda").to(dtype).expand(B, T, H, D).contiguous()
    out = torch.ones((B, T, H, D), dtype=dtype, device="cuda")
    table = torch.arange(4, dtype=torch.int32, device="cuda").repeat(B, 1)
    pos = torch.tensor([2 ** 30, 9], dtype=torch.int32, device="cuda")
    cnt = torch.tensor([T, 1], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(num_kv_heads=Hkv, block_size=bs, num_blocks=8, block_stride=per)
    ws = pa.chunk_workspace_for(q, table, **kw)

    def best(f):
        times = []
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            f()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    fill = best(lambda: out[0].zero_())
    out.fill_(1)
    call = best(lambda: pa.paged_attention_chunk(out, q, pool, pool[Hkv * bs * D:], table, pos, D ** -0.5, ws, counts=cnt,
                                                 err_word=err, **kw))
    assert int(err.item()) == pa.DEVERR_BAD_POS
    assert not out[0].any() and (out[1, 1:] == 1).all()
    k, v = (pool.view(8, 2, Hkv, bs, D)[0, i, :, :10].double() for i in (0, 1))
    a = torch.softmax(torch.einsum("hgd,hld->hgl", q[1, 0].double().view(Hkv, -1, D), k) * D ** -0.5, -1)
    want = torch.einsum("hgl,hld->hgd", a, v).view(H, D)
    # weights and the result rounded to the type at most, and fp32's roundings of 10 positions and D products
    assert ((out[1, 0].double() - want).abs() <= torch.finfo(dtype).eps * 4 + 2.0 ** -12).all()
    assert call < 10 * fill + 0.2, f"{call} ms, a fill {fill} ms"

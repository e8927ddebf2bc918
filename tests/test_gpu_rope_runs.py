"""GPU checks of paged_kv_append_rope and its 4-bit forms beyond those of
tests/test_gpu_rope_append.py: batches of so many tokens that a warp takes full
runs of rows (8 iterations of queries, 4 of keys with their values; fp32 half of
that) and shorter last ones; single tokens of every type; the plain 4-bit append
in each of its forms, with counts and device errors, byte for byte."""
import pytest
import torch

import pagedattention_decode_paged_gb300 as pa
from tests import fp4_ref as ref
from tests.test_gpu_rope_append import BF16, F16, F32, Step

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


def held(**kw):
    s = Step(**kw)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = s.gpu(err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    s.check(*out)


# Iterations of 32 lanes over the heads (D/8 lanes a row): queries, keys.
FULL = [(16, 8, 128), (18, 10, 128), (30, 11, 128), (9, 5, 256), (15, 6, 256), (36, 17, 64), (64, 8, 128), (5, 4, 256)]


@pytest.mark.parametrize("H,Hkv,D", FULL)
@pytest.mark.parametrize("dtype,fp4,R,pairs", [
    (BF16, False, None, False), (F16, False, None, True), (F32, False, None, False),
    (BF16, True, None, False), (F16, True, None, True), (F16, True, 48, False), (F32, True, None, False), (BF16, True, 0, False)])
def test_full_runs_of_rows(H, Hkv, D, dtype, fp4, R, pairs):
    """2400 tokens of a padded batch, few of them valid: more than 12 warps of
    one iteration each for every SM, so runs are as long as they get."""
    if D == 256 and dtype == F32 and not fp4:
        H, Hkv, D = 2 * H, 2 * Hkv, 128     # fp32 rows end at 128, two of them side by side
    held(B=8, T=300, counts=[9, 0, 3, 1, 5, 0, 2, 4], pos=[0, 3, 30, 0, 7, 1, 200, 14], H=H, Hkv=Hkv, D=D, R=R, pairs=pairs,
         dtype=dtype, fp4=fp4, norm=H % 2 == 0, seed=H + D)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dtype,D,fp4", [(F16, 128, False), (F32, 64, False), (F16, 32, False), (F16, 64, True), (F32, 128, True),
                                         (F32, 256, True)])
@pytest.mark.parametrize("B", [1, 5, 300])
def test_single_tokens_of_every_type(B, dtype, D, fp4, norm):
    held(B=B, dtype=dtype, D=D, fp4=fp4, norm=norm, pos=[(7 * b) % 83 for b in range(B)], H=6, Hkv=3, seed=B)


class Plain:
    """One paged_kv_append_fp4 over buffers of random bytes."""

    def __init__(self, *, B, T, Hkv, D, bs, dtype, pos, counts=None, g=(1.0, 1.0), seed=0):
        gen = torch.Generator().manual_seed(seed)
        self.B, self.T, self.bs, self.g = B, T, bs, g
        self.pos, self.counts = pos, counts
        self.MB = -(-(max(pos) + T) // bs) + 1
        self.NB = B * self.MB + 2
        self.table = torch.randperm(self.NB, generator=gen)[:B * self.MB].view(B, self.MB).to(torch.int32)
        self.k, self.v = (torch.randn((B, T, Hkv, D), generator=gen).to(dtype) for _ in range(2))
        self.pool = torch.randint(0, 256, (self.NB, 2, Hkv, bs, D // 2), generator=gen, dtype=torch.uint8)
        self.scales = torch.randint(0, 256, (self.NB, 2, Hkv, bs, D // 16), generator=gen, dtype=torch.uint8)

    def check(self, k, v, lost=(), bits=0, counts="own"):
        """The call with new rows k, v; every byte after it.  lost: sequences, or
        (sequence, block) pairs, that are not written."""
        i32 = dict(dtype=torch.int32, device="cuda")
        pool, scales, err = self.pool.cuda(), self.scales.cuda(), torch.zeros(1, **i32)
        cnt = self.counts if isinstance(counts, str) else counts
        pa.paged_kv_append_fp4(k.cuda(), v.cuda(), pool.view(-1), pool.view(-1)[pool.stride(1):], scales, self.table.cuda(),
                               torch.tensor(self.pos, **i32), counts=None if cnt is None else torch.tensor(cnt, **i32),
                               k_scale=self.g[0], v_scale=self.g[1], block_size=self.bs, num_blocks=self.NB,
                               block_stride=pool.stride(0), err_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == bits
        want, want_scales = self.pool.clone(), self.scales.clone()
        for half, x in ((0, self.k), (1, self.v)):
            codes, sc = ref.quantise(x.float(), self.g[half])
            for b in range(self.B):
                for t in range(0 if b in lost else self.T if cnt is None else cnt[b]):
                    j, slot = (self.pos[b] + t) // self.bs, (self.pos[b] + t) % self.bs
                    if (b, j) not in lost:
                        blk = int(self.table[b, j])
                        want[blk, half, :, slot], want_scales[blk, half, :, slot] = codes[b, t], sc[b, t]
        assert torch.equal(scales.cpu(), want_scales) and torch.equal(pool.cpu(), want)


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("D,Hkv,bs", [(64, 3, 16), (128, 8, 24), (256, 5, 1)])
def test_plain_fp4_append(dtype, D, Hkv, bs):
    """Single tokens, [B][Hkv][D] and [B][1][Hkv][D]; padded batches with counts,
    whole and sliced from a packed projection; many tokens."""
    one = Plain(B=4, T=1, Hkv=Hkv, D=D, bs=bs, dtype=dtype, pos=[0, 17, 3, 40], g=(0.5, 3.0), seed=D)
    one.check(one.k[:, 0], one.v[:, 0])
    one.check(one.k, one.v)
    some = Plain(B=4, T=21, Hkv=Hkv, D=D, bs=bs, dtype=dtype, pos=[5, 0, 30, 2], counts=[21, 0, 7, 1], seed=D + 1)
    some.check(some.k, some.v)
    some.check(some.k, some.v, counts=None)
    packed = torch.cat((some.k, some.v, some.k), 2).cuda()
    some.check(packed[:, :, :Hkv], packed[:, :, Hkv:2 * Hkv])
    many = Plain(B=7, T=300, Hkv=Hkv, D=D, bs=bs, dtype=dtype, pos=[0] * 7, counts=[3, 300, 1, 0, 2, 9, 40], seed=D + 2)
    many.check(many.k, many.v)


@pytest.mark.parametrize("T", [6, 400])
def test_plain_fp4_append_errors(T):
    s = Plain(B=6, T=T, Hkv=4, D=128, bs=4, dtype=F16, pos=[0, 2, 1, 5, 0, 3], counts=[6, 6, 0, 6, 5, 6], seed=61)
    s.table[0, 1], s.table[5, 0] = -1, s.NB
    s.pos[3] = s.MB * s.bs - 5               # runs past the table row
    s.counts[4] = T + 1
    s.pos[1] = -1
    s.check(s.k, s.v, lost={(0, 1), (5, 0), 1, 3, 4}, bits=pa.DEVERR_BAD_LEN | pa.DEVERR_BAD_POS | pa.DEVERR_BAD_BLOCK)

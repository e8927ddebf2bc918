"""GPU checks of paged_kv_append_rope_axes: bit for bit against
paged_kv_append_rope where the axes agree, and against the 64-bit restatement of
tests/fp4_ref.py, pair by pair, where they do not."""
import pytest
import torch

import pagedattention_decode_paged_gb300 as pa
from tests import fp4_ref as ref

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


class Rows:
    def __init__(self, *, B=3, T=5, H=4, Hkv=2, D=64, R=None, bs=8, dtype=BF16, pairs=False, norm=True, sections=None,
                 cyclic=False, counts=None, pos=(0, 7, 30), most=60, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.B, self.T, self.H, self.Hkv, self.D, self.bs, self.dtype, self.pairs = B, T, H, Hkv, D, bs, dtype, pairs
        self.R = D if R is None else R
        half = self.R // 2
        self.axis = pa.rope_axes(sections or (half // 4, half // 2, half - half // 4 - half // 2), cyclic)
        A = max(3, max(self.axis) + 1)
        self.pos = torch.tensor(pos[:B], dtype=torch.int32)
        self.counts = torch.tensor(counts if counts is not None else [T] * B, dtype=torch.int32)
        self.MB = -(-(int(self.pos.max()) + T) // bs) + 1
        self.NB = B * self.MB + 2
        self.table = torch.randperm(self.NB, generator=g)[:B * self.MB].view(B, self.MB).int()
        qkv = torch.randn((B, T, H + 2 * Hkv, D), generator=g).to(dtype)
        self.q, self.k, self.v = qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]
        self.qkv = qkv
        self.qw, self.kw = ((1 + 0.2 * torch.randn(D, generator=g)).to(dtype) if norm else None for _ in range(2))
        self.most = most
        self.cs = pa.rope_table(most, self.R)
        self.axis_pos = torch.randint(0, most, (A, B, T), generator=g, dtype=torch.int32)
        es = torch.empty(0, dtype=dtype).element_size()
        self.pool = torch.randint(0, 256, (self.NB, 2, Hkv, bs, D * es), generator=g, dtype=torch.uint8).view(dtype)
        self.q_out = torch.randint(0, 256, (B, T, H, D * es), generator=g, dtype=torch.uint8).view(dtype)

    def call(self, err=None, axis_pos=None, plain=False, table=None, positions=None):
        qkv = self.qkv.cuda()
        q, k, v = qkv[:, :, :self.H], qkv[:, :, self.H:self.H + self.Hkv], qkv[:, :, self.H + self.Hkv:]
        pool, q_out = self.pool.cuda(), self.q_out.cuda()
        flat = pool.view(-1)
        kw = dict(counts=self.counts.cuda(), interleaved=self.pairs, q_norm=self.qw.cuda() if self.qw is not None else None,
                  k_norm=self.kw.cuda() if self.kw is not None else None, block_size=self.bs, num_blocks=self.NB,
                  block_stride=pool.stride(0), err_word=err)
        table = (self.table if table is None else table).cuda()
        pos = (self.pos if positions is None else positions).cuda()
        head = (q_out, q, k, v, flat, flat[pool.stride(1):], table, pos)
        if plain:
            pa.paged_kv_append_rope(*head, self.cs.cuda(), **kw)
        else:
            ap = (self.axis_pos if axis_pos is None else axis_pos).cuda()
            pa.paged_kv_append_rope_axes(*head, ap, self.cs.cuda(), self.axis, **kw)
        torch.cuda.synchronize()
        return q_out.cpu(), pool.cpu()

    def table_of(self, b, t):
        """A cos_sin row [1][R] with each pair's own cosine and sine."""
        i = torch.arange(self.R // 2)
        p = self.axis_pos[torch.tensor(list(self.axis)), b, t].long()
        return torch.cat((self.cs[p, i], self.cs[p, self.R // 2 + i]))[None]

    def check(self, q_out, pool, skip=()):
        u8 = torch.uint8
        want_q, want_pool = self.q_out.clone(), self.pool.clone()
        for b in range(self.B):
            for t in range(int(self.counts[b])):
                p = int(self.pos[b]) + t
                blk, slot = int(self.table[b, p // self.bs]), p % self.bs
                if (b, t) in skip:
                    want_q[b, t] = 0
                    continue
                args = (self.table_of(b, t), torch.zeros(1, dtype=torch.long), self.R, self.pairs, 1e-6)
                for x, w, got in ((self.q[b, t:t + 1], self.qw, q_out[b, t]), (self.k[b, t:t + 1], self.kw, pool[blk, 0, :, slot])):
                    y = ref.turn(x, w, *args, torch.float64)
                    tol = ref.turn_bound(x, w, *args) * (1 + 2.0 ** -7) + ref.half_step(y, self.dtype)
                    assert ((got.double() - y[0]).abs() <= tol[0]).all(), f"token {t} of sequence {b}"
                want_q[b, t] = q_out[b, t]
                want_pool[blk, 0, :, slot] = pool[blk, 0, :, slot]
                want_pool[blk, 1, :, slot] = self.v[b, t]
        assert torch.equal(q_out.view(u8), want_q.view(u8)), "rows of q_out that are not the call's were written"
        assert torch.equal(pool.view(u8), want_pool.view(u8)), "the pool differs"


def run(**over):
    s = Rows(**over)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    s.check(*s.call(err))
    assert int(err.item()) == 0


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dtype,D", [(F32, 16), (F32, 32), (F32, 64), (F32, 128), (F16, 32), (BF16, 64), (F16, 128), (BF16, 256)])
def test_types_and_head_sizes(dtype, D, pairs, norm):
    run(dtype=dtype, D=D, pairs=pairs, norm=norm)


@pytest.mark.parametrize("cyclic", [False, True])
@pytest.mark.parametrize("sections", [(32, 0, 0), (0, 32), (1, 30, 1), (8, 8, 8, 8), (11, 11, 10), (31, 0, 1), (0, 0, 0, 32)])
def test_sections(sections, cyclic):
    run(sections=sections, cyclic=cyclic)
    run(sections=sections, cyclic=cyclic, pairs=True, dtype=F32)


@pytest.mark.parametrize("R", [16, 32, 48, 96, 128])
@pytest.mark.parametrize("dtype", [F32, F16])
def test_rotated_parts(R, dtype):
    for pairs in (False, True):
        run(R=R, D=128, dtype=dtype, pairs=pairs, cyclic=True)


@pytest.mark.parametrize("counts", [(0, 0, 0), (1, 0, 5), (5, 5, 5), (2, 3, 4)])
def test_counts(counts):
    run(counts=list(counts))


@pytest.mark.parametrize("T,H,Hkv", [(1, 64, 8), (1, 1, 1), (130, 32, 8), (33, 5, 5), (7, 40, 40)])
def test_runs_of_rows(T, H, Hkv):
    run(T=T, H=H, Hkv=Hkv, D=128, B=2, pos=(3, 0), dtype=BF16)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dtype,D,R", [(F32, 64, 64), (BF16, 128, 64), (F16, 256, 256)])
def test_equal_axes_are_the_plain_rotation_bit_for_bit(dtype, D, R, pairs):
    s = Rows(dtype=dtype, D=D, R=R, pairs=pairs, most=60)
    same = (s.pos[:, None] + torch.arange(s.T, dtype=torch.int32)).expand(3, s.B, s.T).contiguous()
    got, want = s.call(axis_pos=same), s.call(plain=True)
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_axis_positions_out_of_range_are_one_tokens_error():
    s = Rows(T=6)
    bad = s.axis_pos.clone()
    bad[0, 0, 2], bad[1, 1, 5], bad[2, 2, 0] = -1, s.most, 2 ** 31 - 1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = s.call(err, axis_pos=bad)
    assert int(err.item()) == pa.DEVERR_BAD_POS
    s.check(*out, skip={(0, 2), (1, 5), (2, 0)})


def test_padding_has_no_axis_positions():
    s = Rows(T=6, counts=[2, 0, 6])
    pad = s.axis_pos.clone()
    pad[:, 0, 2:], pad[:, 1] = -5, 2 ** 31 - 1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = s.call(err, axis_pos=pad)
    assert int(err.item()) == 0
    s.check(*out)


def test_cache_positions_may_pass_the_table_of_cosines():
    run(pos=(100, 500, 61), most=20)


def test_bad_counts_positions_and_blocks():
    s = Rows(T=4)
    pos, table = s.pos.clone(), s.table.clone()
    pos[0] = s.MB * s.bs - 3
    table[2, int(s.pos[2]) // s.bs] = -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out, pool = s.call(err, positions=pos, table=table)
    assert int(err.item()) == pa.DEVERR_BAD_POS | pa.DEVERR_BAD_BLOCK
    assert not q_out[0].any()
    s2 = Rows(T=4)
    s2.counts = torch.tensor([-1, 4, 5], dtype=torch.int32)
    err.zero_()
    q_out, pool = s2.call(err)
    assert int(err.item()) == pa.DEVERR_BAD_LEN
    assert torch.equal(q_out[0].view(torch.uint8), s2.q_out[0].view(torch.uint8))
    assert torch.equal(q_out[2].view(torch.uint8), s2.q_out[2].view(torch.uint8))


def test_captured_call_keeps_its_axes():
    """pair_axis is read before the call returns; positions when it runs."""
    s = Rows(T=3)
    qkv, pool, q_out = s.qkv.cuda(), s.pool.cuda(), s.q_out.cuda()
    q, k, v = qkv[:, :, :s.H], qkv[:, :, s.H:s.H + s.Hkv], qkv[:, :, s.H + s.Hkv:]
    flat, ap, cs = pool.view(-1), torch.zeros_like(s.axis_pos).cuda(), s.cs.cuda()
    table, pos, cnt, qw, kw = s.table.cuda(), s.pos.cuda(), s.counts.cuda(), s.qw.cuda(), s.kw.cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        axis = bytearray(s.axis)
        pa.paged_kv_append_rope_axes(q_out, q, k, v, flat, flat[pool.stride(1):], table, pos, ap, cs, axis, counts=cnt,
                                     q_norm=qw, k_norm=kw, block_size=s.bs, num_blocks=s.NB, block_stride=pool.stride(0))
        axis[:] = bytes(len(axis))
    ap.copy_(s.axis_pos)
    graph.replay()
    torch.cuda.synchronize()
    s.check(q_out.cpu(), pool.cpu())

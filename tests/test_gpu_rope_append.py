"""GPU checks of paged_kv_append_rope and its 4-bit forms against the plain
restatements of tests/fp4_ref.py: queries and keys within a bound counted from
their roundings, values bit for bit, 4-bit codes byte for byte where the
stated binary32 order decides them, everything else in the buffers untouched,
and the device-side errors."""
import math

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


def bits(t):
    return t.contiguous().view(torch.uint8)


class Step:
    """Inputs of one append: a packed projection output, a table over shuffled
    blocks, positions and counts; buffers filled with patterns that show a
    stray write."""

    def __init__(self, *, B=3, T=1, H=4, Hkv=2, D=128, bs=16, dtype=BF16, pos=None, counts=None, R=None, pairs=False,
                 norm=False, fp4=False, packed=True, seed=0, eps=1e-6, k_scale=1.0, v_scale=1.0, magnitude=1.0):
        g = torch.Generator().manual_seed(seed)
        self.B, self.T, self.H, self.Hkv, self.D, self.bs, self.dtype = B, T, H, Hkv, D, bs, dtype
        self.fp4, self.pairs, self.eps, self.kg, self.vg = fp4, pairs, eps, k_scale, v_scale
        self.R = D if R is None else R
        self.pos = torch.tensor(pos if pos is not None else [7 * b for b in range(B)], dtype=torch.int32)
        self.counts = torch.tensor(counts, dtype=torch.int32) if counts is not None else None
        held = [int(p) + (int(self.counts[b]) if counts is not None else T) for b, p in enumerate(self.pos)]
        nblk = [max(0, -(-h // bs)) for h in held]
        self.MB = max(max(nblk), 1) + 1
        self.NB = sum(nblk) + 3
        perm = torch.randperm(self.NB, generator=g).to(torch.int32)
        self.table = torch.full((B, self.MB), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(nblk):
            self.table[b, :n] = perm[at:at + n]
            at += n
        qkv = (torch.randn((B, T, H + 2 * Hkv, D), generator=g) * magnitude).to(dtype)
        self.q, self.k, self.v = qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]
        if not packed:
            self.q, self.k, self.v = (t.contiguous() for t in (self.q, self.k, self.v))
        self.qw, self.kw = ((1 + 0.2 * torch.randn(D, generator=g)).to(dtype) if norm else None for _ in range(2))
        self.cs = pa.rope_table(max(held) + 1, self.R) if self.R else None
        es = torch.empty(0, dtype=dtype).element_size()
        row = D // 2 if fp4 else D * es
        self.pool = torch.randint(0, 256, (self.NB, 2, Hkv, bs, row), generator=g, dtype=torch.uint8)
        self.scales = torch.randint(0, 256, (self.NB, 2, Hkv, bs, D // 16), generator=g, dtype=torch.uint8)
        self.q_out = torch.randint(0, 256, (B, T, H, D * es), generator=g, dtype=torch.uint8).view(dtype)

    def gpu(self, *, with_q=True, in_place=False, err=None, device="cuda", prepare=False, table=None, positions=None,
            counts="own", cos_sin="own", stream=None):
        """One call; returns (q_out, pool, scales) on the device."""
        d = device
        qkv = torch.cat((self.q, self.k, self.v), 2).to(d) if not self.q.is_contiguous() else None
        if qkv is not None:
            q, k, v = qkv[:, :, :self.H], qkv[:, :, self.H:self.H + self.Hkv], qkv[:, :, self.H + self.Hkv:]
        else:
            q, k, v = self.q.to(d), self.k.to(d), self.v.to(d)
        q_out = q if in_place else self.q_out.to(d)
        pool, scales = self.pool.to(d), self.scales.to(d)
        view = pool if self.fp4 else pool.view(self.dtype)
        flat = view.view(-1)
        table = (self.table if table is None else table).to(d)
        pos = (self.pos if positions is None else positions).to(d)
        cnt = self.counts if isinstance(counts, str) else counts
        cnt = cnt.to(d) if cnt is not None else None
        cs = self.cs if isinstance(cos_sin, str) else cos_sin
        more = dict(counts=cnt, interleaved=self.pairs, eps=self.eps, block_size=self.bs, num_blocks=self.NB,
                    block_stride=view.stride(0), err_word=err, prepare=prepare, stream=stream,
                    q_norm=self.qw.to(d) if self.qw is not None else None,
                    k_norm=self.kw.to(d) if self.kw is not None else None)
        self.keep = (q, k, v, table, pos, cnt, more)
        head = (q_out if with_q else None, q if with_q else None, k, v, flat, flat[view.stride(1):])
        cs = cs.to(d) if cs is not None else None
        if self.fp4:
            call = pa.paged_kv_append_rope_fp4(*head, scales, table, pos, cs, k_scale=self.kg, v_scale=self.vg, **more)
        else:
            call = pa.paged_kv_append_rope(*head, table, pos, cs, **more)
        self.keep += (cs,)
        return (q_out, pool, scales) + ((call,) if prepare else ())

    def check(self, q_out, pool, scales, *, with_q=True, skip=(), skip_kv=(), zero_q=()):
        """Every byte of the three buffers.  skip: sequences of which nothing is
        written; skip_kv: (sequence, token) whose cache rows are not; zero_q:
        sequences whose queries are zeros."""
        u = 2.0 ** -24
        pool, scales = pool.cpu(), scales.cpu()
        want_pool, want_scales = self.pool.clone(), self.scales.clone()
        want_q = self.q_out.clone()
        got_q = q_out.cpu().view(self.B, self.T, self.H, self.D)
        for b in range(self.B):
            n = self.T if self.counts is None else int(self.counts[b])
            if b in skip or n == 0:
                continue
            pos = self.pos[b] + torch.arange(n)
            args = (self.cs, pos, self.R, self.pairs, self.eps)
            if with_q:
                if b in zero_q:
                    assert not got_q[b, :n].any()
                else:
                    y = ref.turn(self.q[b, :n], self.qw, *args, torch.float64)
                    tol = ref.turn_bound(self.q[b, :n], self.qw, *args) * (1 + 2.0 ** -7) + ref.half_step(y, self.dtype)
                    off = (got_q[b, :n].double() - y).abs()
                    assert (off <= tol).all(), f"queries of sequence {b}: {float((off / tol).max()):.2f} of the bound"
                want_q[b, :n] = got_q[b, :n]
            if b in zero_q:
                continue
            k64 = ref.turn(self.k[b, :n], self.kw, *args, torch.float64)
            k32 = ref.turn(self.k[b, :n], self.kw, *args, torch.float32)
            kb = ref.turn_bound(self.k[b, :n], self.kw, *args)
            codes = {0: ref.quantise(k32, self.kg), 1: ref.quantise(self.v[b, :n].float(), self.vg)} if self.fp4 else None
            for t in range(n):
                if (b, t) in skip_kv:
                    continue
                blk, slot = int(self.table[b, int(pos[t]) // self.bs]), int(pos[t]) % self.bs
                if not self.fp4:
                    got = pool.view(self.dtype)[blk, 0, :, slot]
                    tol = kb[t] * (1 + 2.0 ** -7) + ref.half_step(k64[t], self.dtype)
                    assert ((got.double() - k64[t]).abs() <= tol).all(), f"keys of ({b}, {t})"
                    want_pool[blk, 0, :, slot] = pool[blk, 0, :, slot]
                    want_pool[blk, 1, :, slot] = bits(self.v[b, t]).view(self.Hkv, -1)
                    continue
                for half in (0, 1):
                    want_pool[blk, half, :, slot], want_scales[blk, half, :, slot] = codes[half][0][t], codes[half][1][t]
                if self.kw is not None:
                    self.check_normed(k64[t], kb[t], pool[blk, 0, :, slot], scales[blk, 0, :, slot])
                    want_pool[blk, 0, :, slot], want_scales[blk, 0, :, slot] = pool[blk, 0, :, slot], scales[blk, 0, :, slot]
        assert torch.equal(pool, want_pool), "the pools differ"
        if self.fp4:
            assert torch.equal(scales, want_scales), "the scales differ"
        if with_q:
            assert torch.equal(bits(got_q), bits(want_q)), "rows of q_out that are not the call's were written"

    def check_normed(self, y, bound, codes, scales):
        """Normed keys: a root rounded the other way may move a value across a
        code border, so scale and codes are each held to half a step, widened
        by the value's own bound."""
        G, e = y.unflatten(-1, (-1, 16)), bound.unflatten(-1, (-1, 16))
        s = ref.E4M3[scales.long()]
        a = G.abs().amax(-1) / (6 * self.kg)
        # half a step of E4M3: 2^-4 of the value, 2^-10 below its normal range
        assert ((s - a.clamp(max=448.0)).abs() <= (a * 2.0 ** -4).clamp(min=2.0 ** -10) + e.amax(-1)).all()
        c = ref.E2M1[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()].unflatten(-1, (-1, 16))
        t = (s * self.kg)[..., None]
        z = (G / t.clamp(min=1e-300)).abs()
        step = torch.where(z < 2, 0.25, torch.where(z < 4, 0.5, 1.0))
        off = torch.where(t > 0, (c - G / t.clamp(min=1e-300)).abs(), c.abs())
        assert (off <= torch.where(t > 0, step + e / t.clamp(min=1e-300) + 2.0 ** -20, 0.0)).all()


def run(**over):
    with_q, in_place = over.pop("with_q", True), over.pop("in_place", False)
    s = Step(**over)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = s.gpu(err=err, with_q=with_q, in_place=in_place)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    s.check(*out, with_q=with_q)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("D,dtype,fp4", [(16, F32, False), (32, F32, False), (64, F32, False), (128, F32, False),
                                         (32, F16, False), (64, BF16, False), (128, F16, False), (256, BF16, False),
                                         (64, F32, True), (128, BF16, True), (256, F16, True), (256, F32, True)])
def test_types_and_head_sizes(D, dtype, fp4, norm):
    run(D=D, dtype=dtype, fp4=fp4, norm=norm, T=5, counts=[5, 0, 3], pos=[0, 4, 30], seed=D)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("R,pairs", [(0, False), (16, False), (16, True), (48, False), (64, True), (112, True), (128, True)])
def test_rotated_parts_of_a_head(R, pairs, fp4):
    run(R=R, pairs=pairs, fp4=fp4, norm=R == 48, T=3, seed=R)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("H,Hkv,D", [(1, 1, 128), (1, 1, 64), (3, 1, 64), (7, 7, 128), (64, 8, 128), (5, 5, 256),
                                     (40, 2, 64)])
def test_head_counts(H, Hkv, D, fp4):
    """From several tokens of a CTA side by side to several passes per token."""
    run(H=H, Hkv=Hkv, D=D, fp4=fp4, B=2, T=37, counts=[37, 20], pos=[3, 100], norm=H == 7, seed=H)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("bs", [1, 3, 8, 24, 128])
def test_block_sizes(bs, fp4):
    run(bs=bs, fp4=fp4, T=70, counts=[70, 1, 69], pos=[0, 23, 5], seed=bs)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("B", [1, 2, 300])
def test_single_tokens_packed_rows_and_in_place_queries(B, fp4):
    run(B=B, fp4=fp4, packed=False, in_place=True, pos=[(11 * b) % 97 for b in range(B)], seed=B)
    run(B=B, fp4=fp4, packed=True, pos=[(5 * b) % 61 for b in range(B)], with_q=False, seed=B)


def test_far_positions_and_factors():
    run(pos=[131071, 0, 65536], T=2, seed=1)
    for g in (0.0625, 3.0, 1e-6, 1e6):
        run(fp4=True, T=2, k_scale=g, v_scale=1 / g, magnitude=0.3, seed=2)


def test_quantising_append_edges():
    """Ties of codes and scales, saturation, infinities and NaN, zero groups:
    byte for byte (no rotation: the values are the inputs)."""
    s = Step(B=2, T=40, H=1, Hkv=2, D=64, dtype=F32, R=0, fp4=True, seed=4)
    k = torch.randn(2, 40, 2, 64, generator=torch.Generator().manual_seed(5))
    grid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    k[0, 0] = torch.cat((grid, -grid)).repeat(8).view(2, 64)
    k[0, 1] = k[0, 0] * 2.0 ** -9
    k[0, 2] = k[0, 0] * 448
    k[0, 3] = 1e30
    k[0, 4] = 0.0
    k[0, 5, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 1.0])
    k[0, 6] = math.nan
    k[0, 7] = 1e-30
    mids = (ref.E4M3[1:127] + ref.E4M3[0:126]) / 2            # ties between neighbouring scales, times 6
    k[1, :31] = 0.0
    k[1, :31, 0, ::16] = (6 * mids[:124]).float().view(31, 4)
    s.k, s.v = k, -k.flip(1)
    s.q = torch.zeros(2, 40, 1, 64)
    out = s.gpu()
    torch.cuda.synchronize()
    s.check(*out)


def test_wholly_masked_groups_of_bf16_extremes():
    s = Step(B=1, T=4, H=2, Hkv=2, D=128, fp4=True, R=0, seed=9)
    lowest = torch.finfo(BF16).min
    s.k = torch.full((1, 4, 2, 128), lowest, dtype=BF16)
    s.v = torch.full((1, 4, 2, 128), torch.finfo(BF16).tiny, dtype=BF16)
    s.q = torch.zeros(1, 4, 2, 128, dtype=BF16)
    out = s.gpu()
    torch.cuda.synchronize()
    s.check(*out)


@pytest.mark.parametrize("fp4", [False, True])
def test_device_errors(fp4):
    s = Step(B=6, T=4, counts=[4, 5, 4, -1, 3, 4], pos=[0, 3, 8, 2, 1, 40], H=4, Hkv=2, fp4=fp4, norm=True, eps=0.0, seed=7)
    s.table[0, 0] = s.NB                       # a block past the pool: keys and values of its 4 tokens are lost
    s.table[4, 0] = -1
    s.pos[5] = s.MB * s.bs - 3                 # runs past the table row
    s.cs = pa.rope_table(11, 128)              # sequence 2 ends at position 11: past the table of cosines
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = s.gpu(err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == pa.DEVERR_BAD_LEN | pa.DEVERR_BAD_POS | pa.DEVERR_BAD_BLOCK
    lost = {(0, t) for t in range(4)} | {(4, t) for t in range(3)}
    s.check(*out, skip={1, 3}, zero_q={2, 5}, skip_kv=lost)
    # a negative position; and no err_word to write to
    s2 = Step(B=2, T=2, pos=[0, 4], fp4=fp4, seed=8)
    s2.pos[1] = -1
    out = s2.gpu()
    torch.cuda.synchronize()
    s2.check(*out, zero_q={1})


def test_offsets_past_32_bits():
    """Blocks far into pools of more than 4 GB, written and read back."""
    D, Hkv, bs, NB = 128, 8, 16, 1 << 18       # 2 x 8 x 16 x 64 bytes a block: 4 GB of codes, 512 MB of scales
    pool = torch.empty((NB + 8, 2, Hkv, bs, D // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((NB + 8, 2, Hkv, bs, D // 16), dtype=torch.uint8, device="cuda")
    table = torch.tensor([[NB + 7, 0], [NB + 3, NB // 2 + 1]], dtype=torch.int32, device="cuda")
    k = torch.randn(2, 32, Hkv, D, dtype=BF16, device="cuda")
    v = torch.randn(2, 32, Hkv, D, dtype=BF16, device="cuda")
    flat = pool.view(-1)
    kw = dict(block_size=bs, num_blocks=NB + 8, block_stride=pool.stride(0))
    start = torch.zeros(2, dtype=torch.int32, device="cuda")
    pa.paged_kv_append_fp4(k, v, flat, flat[pool.stride(1):], scales, table, start, **kw)
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    pa.paged_kv_gather_fp4(ko, vo, flat, flat[pool.stride(1):], scales, table, start, **kw)
    torch.cuda.synchronize()
    for got, x in ((ko, k), (vo, v)):
        want = ref.dequantise(*ref.quantise(x.cpu().float(), 1.0), 1.0)
        assert torch.equal(got.cpu().double(), want)       # at most 6 significant bits: bf16 holds them
    # and attended to, against the same rows in a small pool
    q = torch.randn(2, 2 * Hkv, D, dtype=BF16, device="cuda")
    lens = torch.tensor([32, 19], dtype=torch.int32, device="cuda")
    ids = table.flatten().long()
    near, near_scales = pool[ids].contiguous(), scales[ids].contiguous()
    outs = []
    for p, sc, tb in ((pool, scales, table), (near, near_scales, torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2))):
        kw = dict(num_kv_heads=Hkv, block_size=bs, num_blocks=p.shape[0], block_stride=p.stride(0))
        outs.append(torch.empty_like(q))
        pa.paged_attention_decode_fp4(outs[-1], q, p.view(-1), p.view(-1)[p.stride(1):], sc, tb, lens, D ** -0.5,
                                      pa.fp4_workspace_for(q, tb, **kw), **kw)
    torch.cuda.synchronize()
    assert torch.equal(*outs) and torch.isfinite(outs[0]).all()


@pytest.mark.parametrize("fp4", [False, True])
def test_side_stream_prepared_call_and_graph(fp4):
    s = Step(T=6, counts=[6, 2, 5], fp4=fp4, seed=11)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        q_out, pool, scales, call = s.gpu(prepare=True)
        call()
    stream.synchronize()
    s.check(q_out, pool, scales)
    # captured once, replayed with other positions in the same buffers
    with torch.cuda.stream(stream):
        q_out, pool, scales, call = s.gpu(prepare=True)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        call()
    s.keep[4].copy_(torch.tensor([1, 9, 0], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    s.pos = torch.tensor([1, 9, 0], dtype=torch.int32)
    s.check(q_out, pool, scales)


def test_matches_the_plain_append_without_norm_and_rotation():
    """Nothing to do to the keys: the pools are those of paged_kv_append_tokens."""
    s = Step(T=9, counts=[9, 4, 0], R=0, packed=False, seed=12)
    _, pool, _ = s.gpu()
    other = s.pool.cuda()
    flat = other.view(BF16).view(-1)
    stride = other.view(BF16).stride()
    pa.paged_kv_append_tokens(s.k.cuda(), s.v.cuda(), flat, flat[stride[1]:], s.table.cuda(), s.pos.cuda(),
                              s.counts.cuda(), block_size=s.bs, num_blocks=s.NB, block_stride=stride[0])
    torch.cuda.synchronize()
    assert torch.equal(pool, other)


@pytest.mark.parametrize("g", [1.0, 0.37, 5.3e-7, 1.9e11, 2.0 ** -64, 2.0 ** 64])
def test_quotients_beside_every_border(g):
    """Keys a few steps of binary32 from t * (border between two codes), group
    maxima of values as close to 6 g * (border between two scales): codes and
    scales are those of IEEE division, byte for byte."""
    rng = torch.Generator().manual_seed(21)
    T, Hkv, D, bs = 2048, 4, 64, 16

    def steps(x):
        """x moved by -3..3 steps of binary32."""
        return (x.view(torch.int32) + torch.randint(-3, 4, x.shape, generator=rng, dtype=torch.int32)).view(torch.float32)

    shape = (1, T, Hkv, D // 16)
    val = ref.E4M3[torch.randint(1, 127, shape, generator=rng)].float()
    t = (val * torch.tensor(g, dtype=torch.float32))[..., None]
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])[torch.randint(0, 7, (*shape, 16), generator=rng)]
    k = steps(border * t)
    k[..., 0] = (6 * torch.tensor(g, dtype=torch.float32) * val)
    k = (k * (torch.randint(0, 2, k.shape, generator=rng) * 2 - 1)).flatten(-2)
    mids = ((ref.E4M3[1:127] + ref.E4M3[0:126]) / 2).float()[torch.randint(0, 126, shape, generator=rng)]
    v = torch.randn((*shape, 16), generator=rng).clamp(-1, 1) * 0.5 * mids[..., None] * g
    v[..., 5] = steps(6 * torch.tensor(g, dtype=torch.float32) * mids)
    v = v.flatten(-2)
    NB = T // bs
    pool = torch.zeros((NB, 2, Hkv, bs, D // 2), dtype=torch.uint8, device="cuda")
    scales = torch.zeros((NB, 2, Hkv, bs, D // 16), dtype=torch.uint8, device="cuda")
    table = torch.arange(NB, dtype=torch.int32, device="cuda").view(1, NB)
    flat = pool.view(-1)
    pa.paged_kv_append_fp4(k.cuda(), v.cuda(), flat, flat[pool.stride(1):], scales, table,
                           torch.zeros(1, dtype=torch.int32, device="cuda"), k_scale=g, v_scale=g, block_size=bs,
                           num_blocks=NB, block_stride=pool.stride(0))
    torch.cuda.synchronize()
    for half, x in ((0, k), (1, v)):
        codes, sc = ref.quantise(x[0], g)
        rows = lambda y: y[:, half].transpose(1, 2).reshape(T, Hkv, -1).cpu()
        assert torch.equal(rows(scales), sc)
        assert torch.equal(rows(pool), codes)


def test_positions_of_empty_sequences_are_checked():
    """As in paged_kv_append_tokens, a position is checked whatever the count."""
    for fp4 in (False, True):
        s = Step(B=2, T=3, counts=[0, 2], fp4=fp4, seed=13)
        s.pos[0] = -1
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = s.gpu(err=err)
        torch.cuda.synchronize()
        assert int(err.item()) == pa.DEVERR_BAD_POS
        s.check(*out)


def test_two_appends_at_once_on_two_streams():
    """Different sequences of one cache, on two streams, many times over."""
    a, b = Step(B=2, T=40, fp4=True, seed=14), Step(B=2, T=40, fp4=True, seed=15)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for s, stream in zip((a, b), streams):
        with torch.cuda.stream(stream):
            outs.append(s.gpu(prepare=True))
    torch.cuda.synchronize()
    for _ in range(20):
        for out, stream in zip(outs, streams):
            out[3]()
    torch.cuda.synchronize()
    for s, out in zip((a, b), outs):
        s.check(*out[:3])


def test_nothing_to_append_is_a_no_op():
    """No tokens, or no sequences: accepted, and nothing is written."""
    for kw in (dict(B=3, T=0), dict(B=2, T=4, counts=[0, 0])):
        for fp4 in (False, True):
            s = Step(fp4=fp4, seed=16, **kw)
            out = s.gpu()
            torch.cuda.synchronize()
            s.check(*out)

"""GPU checks of the 4-bit cache's gather and decode attention against the
plain 64-bit restatement of tests/fp4_ref.py, with tolerances counted there
from the kernel's roundings; poisoned slots outside the attended tokens; work
split over many CTAs; repeatability, graphs, streams and shared workspaces."""
import math

import pytest
import torch

import pagedattention_decode_paged_gb300 as pa
from tests import fp4_ref as ref

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
LENS = [0, 1, 15, 16, 17, 31, 33, 64, 100, 257]


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


class Cache:
    """A cache of random codes and scales over shuffled blocks; every slot that
    no sequence holds has NaN scales (0x7F) and codes of all ones."""

    def __init__(self, *, lens, H=4, Hkv=4, D=128, bs=16, dtype=BF16, seed=0, k_scale=1.0, v_scale=1.0, poison=True,
                 q_magnitude=1.0, flat_scores=False):
        g = torch.Generator().manual_seed(seed)
        self.B, self.H, self.Hkv, self.D, self.bs, self.dtype = len(lens), H, Hkv, D, bs, dtype
        self.kg, self.vg = k_scale, v_scale
        self.lens = torch.tensor(lens, dtype=torch.int32)
        nblk = [-(-n // bs) for n in lens]
        self.MB, self.NB = max(max(nblk), 1) + 1, sum(nblk) + 3
        perm = torch.randperm(self.NB, generator=g).to(torch.int32)
        self.table = torch.full((self.B, self.MB), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(nblk):
            self.table[b, :n] = perm[at:at + n]
            at += n
        x = torch.randn((self.NB, 2, Hkv, bs, D), generator=g)
        self.pool, self.scales = ref.quantise(x / (32 if flat_scores else 1), 1.0)
        if poison:
            held = torch.zeros(self.NB, bs, dtype=torch.bool)
            for b, n in enumerate(lens):
                for j in range(nblk[b]):
                    held[int(self.table[b, j]), :max(0, min(bs, n - j * bs))] = True
            self.scales.masked_fill_(~held[:, None, None, :, None], 0x7F)
            self.pool.masked_fill_(~held[:, None, None, :, None], 0xFF)
        self.q = (torch.randn((self.B, H, D), generator=g) * q_magnitude).to(dtype)
        self.scale = 1.0 / math.sqrt(D)

    def to_gpu(self):
        self.g = {n: getattr(self, n).cuda() for n in ("pool", "scales", "table", "q", "lens")}
        self.kw = dict(block_size=self.bs, num_blocks=self.NB, block_stride=self.g["pool"].stride(0))
        self.ws = pa.fp4_workspace_for(self.g["q"], self.g["table"], num_kv_heads=self.Hkv, **self.kw)
        self.flat = self.g["pool"].view(-1)
        return self

    def decode(self, *, window=0, err=None, lens=None, out=None, ws=None, table=None, **more):
        out = torch.full_like(self.g["q"], math.nan) if out is None else out
        call = pa.paged_attention_decode_fp4(out, self.g["q"], self.flat, self.flat[self.g["pool"].stride(1):],
                                             self.g["scales"], self.g["table"] if table is None else table,
                                             self.g["lens"] if lens is None else lens, self.scale,
                                             self.ws if ws is None else ws, k_scale=self.kg, v_scale=self.vg,
                                             window=window, num_kv_heads=self.Hkv, err_word=err, **more, **self.kw)
        return (out, call) if more.get("prepare") else out

    def reference(self, window=0, lens=None):
        return ref.decode64(self.q, self.pool, self.scales, self.table, self.lens if lens is None else lens, self.bs,
                            self.scale, window, self.kg, self.vg)

    def counters(self):
        """The workspace's item counters, at its end: all zero between calls."""
        n = pa.paged_attention_fp4_workspace(pa.decode_shape(self.g["q"], self.g["table"], num_kv_heads=self.Hkv, **self.kw))
        heads = 16 if self.D <= 128 and self.H // self.Hkv * (2 if self.dtype == F32 else 1) > 8 else 8
        heads //= 2 if self.dtype == F32 else 1
        units = -(-(self.H // self.Hkv) // heads)
        return self.ws[n - 4 * self.B * self.Hkv * units:n]


def held_to(got, want, what=""):
    out, tol = want
    off = (got.double().cpu() - out).abs()
    assert torch.isfinite(got).all(), f"{what}: non-finite outputs"
    assert (off <= tol).all(), f"{what}: {float((off / tol.clamp(min=1e-300)).max()):.2f} of the bound"


def run(window=0, **kw):
    c = Cache(**kw).to_gpu()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = c.decode(window=window, err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    held_to(out, c.reference(window))
    assert not c.counters().any()
    return c, out


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
def test_decode_types_and_head_sizes(dtype, D):
    run(lens=LENS, D=D, dtype=dtype, seed=D)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64), (F16, 256)])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (6, 2), (8, 2), (16, 2), (18, 2), (12, 1), (16, 1), (40, 2), (64, 8), (7, 7)])
def test_decode_head_groups(H, Hkv, dtype, D):
    """One, partly filled, two and several column tiles per kv head."""
    run(lens=[33, 0, 100, 257], H=H, Hkv=Hkv, D=D, dtype=dtype, seed=H)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bs", [1, 3, 8, 24, 32, 128])
def test_decode_block_sizes(bs, D):
    run(lens=LENS, H=4, Hkv=2, D=D, bs=bs, seed=bs)


@pytest.mark.parametrize("window", [1, 5, 15, 16, 17, 64, 100, 1000, 2 ** 31 - 1])
def test_decode_windows(window):
    run(lens=LENS, H=6, Hkv=2, window=window, seed=window % 97)


@pytest.mark.parametrize("lens,H,Hkv,dtype,D", [
    ([5000], 8, 8, F16, 128),          # a few CTAs an item
    ([40000], 8, 1, BF16, 128),        # one item over every CTA: two levels of merging
    ([40000], 2, 1, F32, 64),
    ([20000, 3, 0, 700], 16, 1, BF16, 128),
    ([9000, 9000], 4, 1, F16, 256),
    ([1] * 700, 2, 2, BF16, 64),       # more items than CTAs, less than a tile each
    ([600 + i for i in range(40)], 16, 16, F16, 128)])
def test_decode_split_over_ctas(lens, H, Hkv, dtype, D):
    """Long contexts, ragged batches and many small items; twice with one
    workspace, equal bit for bit."""
    c, out = run(lens=lens, H=H, Hkv=Hkv, dtype=dtype, D=D, seed=len(lens))
    again = c.decode()
    assert torch.equal(out, again)


def test_decode_more_sequences_than_two_ctas_of_schedule_hold():
    """The schedule's shared memory leaves one CTA per SM."""
    run(lens=[(i * 7) % 40 for i in range(2500)], H=2, Hkv=1, seed=3)


@pytest.mark.parametrize("magnitude,dtype", [(1e-6, F16), (1e-30, BF16), (1e3, BF16), (1e4, F16), (1e20, F32), (1e-35, F32)])
def test_decode_query_magnitudes(magnitude, dtype):
    """Queries far from 1 (the head's power of two keeps them in fp16), scores
    brought back by the scale."""
    c = Cache(lens=[100, 17], dtype=dtype, q_magnitude=magnitude, seed=5).to_gpu()
    c.scale = 1.0 / (math.sqrt(128) * magnitude)
    if c.scale > 3e38:
        c.scale = 3e38
    held_to(c.decode(), c.reference())


def test_decode_factors_and_flat_scores():
    run(lens=LENS, k_scale=0.01, v_scale=300.0, seed=6)
    run(lens=[3000, 90], k_scale=2.0, v_scale=2.0 ** -20, flat_scores=True, H=8, Hkv=2, seed=7)


def test_decode_zero_scales_and_one_token_per_weight():
    c = Cache(lens=[64, 5], seed=8)
    c.scales[:, 0] = torch.where(c.scales[:, 0] == 0x7F, c.scales[:, 0], torch.zeros_like(c.scales[:, 0]))  # K = 0: a mean
    c.to_gpu()
    held_to(c.decode(), c.reference())
    c = Cache(lens=[64, 5], q_magnitude=100.0, dtype=F32, seed=9).to_gpu()      # one weight is all
    held_to(c.decode(), c.reference())


def test_decode_nan_scale_inside_reaches_only_its_outputs():
    c = Cache(lens=[40, 40, 700], H=4, Hkv=2, seed=10)
    blk, slot = int(c.table[1, 1]), 3
    c.scales[blk, 1, 1, slot, 2] = 0x7F        # V, kv head 1, elements 32..47
    c.to_gpu()
    out = c.decode().cpu()
    nan = torch.isnan(out)
    want = torch.zeros_like(nan)
    want[1, 2:, 32:48] = True
    assert torch.equal(nan, want)
    c.scales[blk, 0, 0, slot, 0] = 0xFF        # K, kv head 0: every element of its heads
    c.to_gpu()
    nan = torch.isnan(c.decode().cpu())
    want[1, :2] = True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("lens", [[40, 40, 40, 40], [30000, 40, 30000, 40]])
def test_decode_errors_reported_and_zeroed(lens):
    c = Cache(lens=lens, H=8, Hkv=2, seed=11).to_gpu()
    table = c.g["table"].clone()
    table[1, 1] = -1
    table[2, lens[2] // 32] = c.NB
    bad = torch.tensor([lens[0], 40, lens[2], c.MB * c.bs + 1], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = c.decode(err=err, lens=bad, table=table)
    torch.cuda.synchronize()
    assert int(err.item()) == pa.DEVERR_BAD_BLOCK | pa.DEVERR_BAD_LEN
    assert not out[1:].any()
    want, tol = c.reference()
    held_to(out[:1], (want[:1], tol[:1]))
    assert not c.counters().any()
    bad[3] = -5
    out = c.decode(lens=bad, table=table)      # no err_word
    assert not out[1:].any()


def test_decode_tables_may_share_blocks():
    c = Cache(lens=[100, 100], seed=12)
    c.table[1] = c.table[0]
    c.to_gpu()
    held_to(c.decode(), c.reference())


def test_decode_workspace_is_refused_when_small_or_misaligned():
    c = Cache(lens=[100, 3]).to_gpu()
    n = pa.paged_attention_fp4_workspace(pa.decode_shape(c.g["q"], c.g["table"], num_kv_heads=c.Hkv, **c.kw))
    for ws, status in ((c.ws[:n - 1], pa.PA_ERR_WORKSPACE), (torch.zeros(n + 16, dtype=torch.uint8, device="cuda")[4:],
                                                              pa.PA_ERR_MISALIGNED)):
        with pytest.raises(pa.PagedAttnError) as e:
            c.decode(ws=ws)
        assert e.value.status == status


def test_decode_on_a_side_stream_and_in_graphs():
    """Captured with one set of lengths, replayed with others; two graphs that
    take turns on one workspace; two that overlap, each with its own."""
    c = Cache(lens=[3000, 50, 900], H=8, Hkv=2, seed=13).to_gpu()
    side = torch.cuda.Stream()
    lens = c.g["lens"].clone()
    outs = [torch.full_like(c.g["q"], math.nan) for _ in range(3)]
    other_ws = torch.zeros_like(c.ws)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.decode(out=outs[0])
    side.synchronize()
    held_to(outs[0], c.reference())
    graphs = []
    for out, ws in zip(outs, (c.ws, c.ws, other_ws)):
        with torch.cuda.stream(side):
            _, call = c.decode(out=out, ws=ws, lens=lens, prepare=True)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            call()
    new = torch.tensor([17, 50, 899], dtype=torch.int32)
    lens.copy_(new)
    torch.cuda.synchronize()
    for _ in range(3):
        graphs[0].replay()
        graphs[1].replay()
        with torch.cuda.stream(side):
            graphs[2].replay()
    torch.cuda.synchronize()
    for out in outs:
        held_to(out, c.reference(lens=new))


def test_decode_scores_far_below_any_reference():
    """Every score the same, about -1e34: all tokens of a tile weigh the same (a
    rounding of such a score would outweigh any other), the output is the
    values' mean."""
    c = Cache(lens=[32, 7], H=2, Hkv=2, dtype=F32, seed=14)
    c.pool[:, 0], c.scales[:, 0] = 0x22, torch.where(c.scales[:, 0] == 0x7F, c.scales[:, 0], torch.full_like(c.scales[:, 0], 0x38))
    c.q = torch.full_like(c.q, -1e33)          # keys of ones: 128 products of -1e33
    c.to_gpu()
    out = c.decode()
    for b, n in enumerate((32, 7)):
        v = ref.cached_rows(c.pool, c.scales, c.table[b], c.bs, 0, n, (1.0, 1.0))[1]
        mean, size = v.mean(1), v.abs().mean(1)
        # equal weights of 1: n/16 + 32 fp32 sums at most, the quotient, the last rounding
        off = (out[b].double().cpu() - mean).abs()
        assert (off <= size * (n / 16 + 36) * 2.0 ** -23).all()


def test_decode_of_empty_sequences_only():
    c = Cache(lens=[0, 0, 0], H=8, Hkv=2).to_gpu()
    assert not c.decode().any()


def test_decode_one_workspace_serves_smaller_shapes_too():
    big = Cache(lens=[3000] * 9, H=32, Hkv=8, seed=15).to_gpu()
    held_to(big.decode(), big.reference())
    for kw in (dict(lens=[5000], H=8, Hkv=1), dict(lens=[40000], H=4, Hkv=2, dtype=F32, D=64), dict(lens=[9, 700], D=256, dtype=F16)):
        c = Cache(seed=16, **kw).to_gpu()
        held_to(c.decode(ws=big.ws), c.reference())
    held_to(big.decode(), big.reference())
    assert not big.counters().any()


def test_decode_pools_in_any_order_and_apart():
    """Values before keys in a block; keys and values in allocations of their own."""
    c = Cache(lens=[100, 33], H=4, Hkv=2, seed=17).to_gpu()
    want, pool = c.decode(), c.g["pool"]
    call = lambda out, k, v, stride: pa.paged_attention_decode_fp4(
        out, c.g["q"], k, v, c.g["scales"], c.g["table"], c.g["lens"], c.scale, c.ws, num_kv_heads=c.Hkv,
        block_size=c.bs, num_blocks=c.NB, block_stride=stride)
    flipped, out = pool.flip(1).contiguous().view(-1), torch.empty_like(want)
    call(out, flipped[pool.stride(1):], flipped, pool.stride(0))
    assert torch.equal(out, want)
    k, v = pool[:, 0].contiguous(), pool[:, 1].contiguous()
    call(out.zero_(), k.view(-1), v.view(-1), k.stride(0))
    assert torch.equal(out, want)


def test_two_decodes_at_once_on_two_streams():
    """Each with its own workspace, many times over."""
    cs = [Cache(lens=[20000, 33], H=8, Hkv=2, seed=18).to_gpu(), Cache(lens=[700] * 12, H=8, Hkv=8, seed=19).to_gpu()]
    want = [c.decode() for c in cs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = []
    for c, stream in zip(cs, streams):
        with torch.cuda.stream(stream):
            outs.append(c.decode(prepare=True))
    for _ in range(20):
        for out, call in outs:
            call()
    torch.cuda.synchronize()
    for (out, _), w in zip(outs, want):
        assert torch.equal(out, w)


# --- reading rows back -------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("D,Hkv,bs", [(64, 1, 16), (64, 2, 3), (64, 3, 16), (64, 7, 8), (128, 8, 16), (128, 1, 1), (256, 5, 24),
                                       (256, 1, 16)])
def test_gather_rows(D, Hkv, bs, dtype):
    lens = [40, 0, 100, 7]
    c = Cache(lens=lens, H=Hkv, Hkv=Hkv, D=D, bs=bs, dtype=dtype, k_scale=0.375, v_scale=3.0, seed=D).to_gpu()
    T = 60
    starts, counts = [0, 0, 41, 6], [40, 0, 59, 1]
    k, v = (torch.full((4, T, Hkv, D), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    i32 = dict(dtype=torch.int32, device="cuda")
    err = torch.zeros(1, **i32)
    pa.paged_kv_gather_fp4(k, v, c.flat, c.flat[c.g["pool"].stride(1):], c.g["scales"], c.g["table"],
                           torch.tensor(starts, **i32), torch.tensor(counts, **i32), k_scale=c.kg, v_scale=c.vg,
                           err_word=err, **c.kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for b in range(4):
        n = counts[b]
        want = ref.cached_rows(c.pool, c.scales, c.table[b], bs, starts[b], starts[b] + n, (c.kg, c.vg)) if n else None
        for half, got in ((0, k), (1, v)):
            assert (got[b, n:] == 7.0).all()
            if n:
                # code * scale is exact, times the factor in fp32, rounded once more to the dtype
                w = want[half].transpose(0, 1).float().to(dtype)
                assert torch.equal(got[b, :n].cpu(), w)


def test_gather_errors():
    c = Cache(lens=[40, 40, 40, 40, 40], H=2, Hkv=2, seed=1).to_gpu()
    i32 = dict(dtype=torch.int32, device="cuda")
    table = c.g["table"].clone()
    table[1, 1] = -1
    k, v = (torch.full((5, 40, 2, 128), 7.0, dtype=BF16, device="cuda") for _ in range(2))
    err = torch.zeros(1, **i32)
    starts = torch.tensor([0, 10, -1, 0, c.MB * c.bs - 39], **i32)
    pa.paged_kv_gather_fp4(k, v, c.flat, c.flat[c.g["pool"].stride(1):], c.g["scales"], table, starts,
                           torch.tensor([40, 20, 5, 41, 40], **i32), err_word=err, **c.kw)
    torch.cuda.synchronize()
    assert int(err.item()) == pa.DEVERR_BAD_LEN | pa.DEVERR_BAD_POS | pa.DEVERR_BAD_BLOCK
    for half, got in ((0, k), (1, v)):
        rows = lambda b, n0, n1: ref.cached_rows(c.pool, c.scales, c.table[b], c.bs, n0, n1, (1.0, 1.0))[half].transpose(0, 1)
        assert torch.equal(got[0].double().cpu(), rows(0, 0, 40))
        assert torch.equal(got[1, :6].double().cpu(), rows(1, 10, 16))
        assert not got[1, 6:20].any() and (got[1, 20:] == 7.0).all()      # block 1 (tokens 16..31) is missing
        assert not got[2, :5].any() and (got[2, 5:] == 7.0).all()
        assert (got[3] == 7.0).all()
        assert not got[4].any()


# --- the operators together --------------------------------------------------------

@pytest.mark.parametrize("dtype,H,Hkv,D,bs", [(BF16, 8, 2, 128, 16), (F16, 4, 4, 64, 3), (F32, 6, 2, 256, 32)])
def test_prompt_then_decode_steps(dtype, H, Hkv, D, bs):
    """A ragged prompt into an empty cache, then steps of append and attention,
    as a serving loop issues them: every step against the values the cache
    holds, read back by the gather."""
    B, T, steps = 3, 50, 4
    g = torch.Generator(device="cuda").manual_seed(D)
    counts = torch.tensor([50, 1, 33], dtype=torch.int32, device="cuda")
    MB = -(-(T + steps) // bs)
    NB = B * MB + 2
    table = torch.randperm(NB, generator=torch.Generator().manual_seed(1))[:B * MB].view(B, MB).to(torch.int32).cuda()
    pool = torch.full((NB, 2, Hkv, bs, D // 2), 0xFF, dtype=torch.uint8, device="cuda")
    scales = torch.full((NB, 2, Hkv, bs, D // 16), 0x7F, dtype=torch.uint8, device="cuda")
    flat = pool.view(-1)
    kw = dict(block_size=bs, num_blocks=NB, block_stride=pool.stride(0))
    gf = dict(k_scale=0.5, v_scale=0.25)
    cs = pa.rope_table(MB * bs, D, device="cuda")
    qn, kn = (torch.randn(D, generator=g, device="cuda").mul(0.1).add(1).to(dtype) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")

    def append(n, counts):
        qkv = torch.randn((B, n, H + 2 * Hkv, D), generator=g, device="cuda").to(dtype)
        q = torch.zeros((B, n, H, D), dtype=dtype, device="cuda")
        pa.paged_kv_append_rope_fp4(q, qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:], flat,
                                    flat[pool.stride(1):], scales, table, lens, cs, counts=counts, q_norm=qn,
                                    k_norm=kn, err_word=err, **gf, **kw)
        return q

    append(T, counts)
    lens += counts
    ws = None
    for _ in range(steps):
        q = append(1, None).view(B, H, D)
        lens += 1
        ws = pa.fp4_workspace_for(q, table, num_kv_heads=Hkv, **kw) if ws is None else ws
        out = torch.empty_like(q)
        pa.paged_attention_decode_fp4(out, q, flat, flat[pool.stride(1):], scales, table, lens, D ** -0.5, ws,
                                      num_kv_heads=Hkv, err_word=err, **gf, **kw)
        torch.cuda.synchronize()
        held_to(out, ref.decode64(q.cpu(), pool.cpu(), scales.cpu(), table.cpu(), lens.cpu(), bs, D ** -0.5, 0, 0.5, 0.25))
    k, v = (torch.zeros((B, T + steps, Hkv, D), dtype=F32, device="cuda") for _ in range(2))
    pa.paged_kv_gather_fp4(k, v, flat, flat[pool.stride(1):], scales, table, torch.zeros_like(lens), lens, **gf, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for b in range(B):
        n = int(lens[b])
        want = ref.cached_rows(pool.cpu(), scales.cpu(), table[b].cpu(), bs, 0, n, (0.5, 0.25))
        assert torch.equal(k[b, :n].cpu().double(), want[0].transpose(0, 1))
        assert torch.equal(v[b, :n].cpu().double(), want[1].transpose(0, 1))

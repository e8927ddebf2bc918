"""GPU checks of paged_attention_chunk and paged_attention_chunk_diff against the
64-bit restatement of tests/chunk_ref.py, each element within a bound counted
from the roundings of its own row; everything no token may see is NaN."""
import math

import pytest
import torch

import pagedattention_decode_paged_gb300 as pa
from tests.chunk_ref import BF16, F16, F32, Chunk, run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


KINDS = [(F32, 16, False)] + [(t, d, f) for t in (F32, F16, BF16) for d in (32, 64, 128, 256) for f in (False, True)
                              if not (t == F32 and d == 256)]


@pytest.mark.parametrize("dtype,D,diff", KINDS)
def test_types_and_head_sizes(dtype, D, diff):
    run(dtype=dtype, D=D, diff=diff, B=3, T=70, H=4, Hkv=2, pos=[0, 61, 200], counts=[70, 1, 33])


@pytest.mark.parametrize("diff", [False, True])
@pytest.mark.parametrize("bs", [1, 3, 8, 16, 24, 32, 64, 128, 256])
def test_block_sizes(bs, diff):
    run(bs=bs, diff=diff, dtype=F16, D=128, B=2, T=40, H=4, Hkv=2, pos=[250, 5])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 3), (6, 2), (5, 1), (14, 2), (32, 2), (64, 1), (100, 1), (300, 1)])
def test_groups(H, Hkv, dtype):
    run(H=H, Hkv=Hkv, dtype=dtype, D=64, B=2, T=7, pos=[130, 0], counts=[7, 5])
    run(H=H, Hkv=Hkv, dtype=dtype, D=64, B=2, T=7, pos=[130, 0], counts=[7, 5], diff=True)


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("diff", [False, True])
@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 127, 128, 129, 300, 2 ** 31 - 1])
def test_windows(window, diff, dtype):
    run(window=window, diff=diff, dtype=dtype, D=64, B=3, T=150, H=4, Hkv=2, pos=[0, 100, 333], counts=[150, 150, 3])


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F32, 64), (F16, 64), (BF16, 256)])
@pytest.mark.parametrize("counts", [[0, 0, 0], [1, 0, 1], [0, 257, 0], [129, 128, 127], [1, 1, 1], None])
def test_counts(counts, dtype, D):
    run(counts=counts, T=257 if counts is None or max(counts) > 1 else 1, B=3, dtype=dtype, D=D, H=2, Hkv=1,
        pos=[0, 127, 128])


@pytest.mark.parametrize("diff", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pos", [0, 1, 62, 63, 64, 126, 127, 128, 129, 255, 256])
def test_single_tokens_at_tile_borders(pos, dtype, diff):
    run(pos=[pos], B=1, T=1, H=8, Hkv=2, D=128, dtype=dtype, diff=diff)


@pytest.mark.parametrize("layout", [dict(gap=64), dict(separate=True), dict(packed=False), dict(gap=8, bs=3),
                                    dict(separate=True, gap=128, bs=8)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layouts(layout, dtype):
    for diff in (False, True):
        run(**{**dict(dtype=dtype, D=64, B=2, T=40, H=4, Hkv=2, pos=[77, 0], diff=diff), **layout})


@pytest.mark.parametrize("dtype,D,diff", [(BF16, 128, False), (F16, 64, True), (F32, 64, False), (BF16, 64, False),
                                          (BF16, 128, True)])
def test_long_contexts_are_cut_and_joined(dtype, D, diff):
    run(dtype=dtype, D=D, diff=diff, B=1, T=3, H=8, Hkv=1, pos=[20011], bs=32, ref_device="cuda")
    run(dtype=dtype, D=D, diff=diff, B=2, T=40, H=8, Hkv=2, pos=[9000, 31], counts=[40, 2], bs=16, ref_device="cuda")


@pytest.mark.parametrize("dtype,D,diff", [(BF16, 128, False), (F16, 128, True), (BF16, 64, False), (F32, 128, False)])
def test_prompts(dtype, D, diff):
    run(dtype=dtype, D=D, diff=diff, B=3, T=700, H=16, Hkv=2, pos=[0, 300, 1000], counts=[700, 411, 5], ref_device="cuda")


@pytest.mark.parametrize("B", [1, 31, 300, 1025, 2600])
def test_batches(B):
    g = torch.Generator().manual_seed(B)
    cnt = torch.randint(0, 3, (B,), generator=g).tolist()
    pos = torch.randint(0, 70, (B,), generator=g).tolist()
    run(B=B, T=2, counts=cnt, pos=pos, H=2, Hkv=1, D=64, bs=8, dtype=F16)


def test_mixed_batch():
    B = 40
    run(B=B, T=300, counts=[1] * (B - 1) + [300], pos=[(211 * b) % 1500 for b in range(B)], H=8, Hkv=2, D=128,
        ref_device="cuda")


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 64), (F32, 64), (BF16, 256)])
def test_no_norm_and_no_difference(dtype, D):
    """Without a norm, and with lambda 0 the first map's attention."""
    run(dtype=dtype, D=D, diff=True, norm=False, B=2, T=9, pos=[40, 0])
    s = Chunk(dtype=dtype, D=D, diff=True, norm=False, B=2, T=9, pos=[40, 0], out_scale=1.0)
    s.lam.zero_()
    s.check(s.call())


@pytest.mark.parametrize("diff", [False, True])
@pytest.mark.parametrize("bs", [3, 16])
@pytest.mark.parametrize("dtype,D", [(F32, 64), (BF16, 128), (F16, 64), (BF16, 32)])
@pytest.mark.parametrize("odd", [math.inf, -math.inf, math.nan])
def test_values_that_are_not_finite_reach_only_rows_that_see_them(odd, dtype, D, bs, diff):
    s = Chunk(dtype=dtype, D=D, B=2, T=150, H=4, Hkv=2, bs=bs, pos=[30, 0], diff=diff, norm=False)
    for b, t, h, d in ((0, 100, 0, 5), (0, 175, 1, D - 1), (1, 3, 1, 0), (1, 149, 0, 17)):
        s.block(int(s.table[b, t // bs]), 1)[h, t % bs, d] = odd
    out = s.call()
    if diff:   # (a1 - lambda a2) odd and a1 odd - lambda a2 odd differ in kind: the rows that see it are not compared
        for b in range(2):
            n, p = s.n[b], int(s.pos[b])
            first = {0: 100 - 30, 1: 3}[b]
            want, tol = s.want(b)
            off = (out[b, :first].cpu().double() - want[:first]).abs() / tol[:first]
            assert (off <= 1).all()
    else:
        s.check(out)


@pytest.mark.parametrize("dtype,D", [(F32, 64), (BF16, 128), (F16, 64)])
def test_keys_that_are_not_finite_reach_only_rows_that_see_them(dtype, D):
    s = Chunk(dtype=dtype, D=D, B=1, T=90, H=2, Hkv=1, pos=[50])
    t = 110
    s.block(int(s.table[0, t // s.bs]), 0)[0, t % s.bs, 3] = math.nan
    got, (want, tol) = s.call()[0].cpu(), s.want(0)
    assert ((got[:60].double() - want[:60]).abs() <= tol[:60]).all()
    assert got[60:].isnan().all()


@pytest.mark.parametrize("window", [0, 130])
@pytest.mark.parametrize("dtype,D,bs", [(F32, 64, 16), (BF16, 128, 16), (F16, 64, 3), (BF16, 64, 8), (BF16, 128, 256)])
@pytest.mark.parametrize("diff", [False, True])
def test_bad_blocks(diff, dtype, D, bs, window):
    """Tokens that attend to a block out of range are zeros, others are not."""
    s = Chunk(dtype=dtype, D=D, bs=bs, B=3, T=200, H=4, Hkv=2, pos=[100, 0, 300], counts=[200, 200, 200], window=window,
              diff=diff)
    table, rows = s.table.clone(), {}
    for b, t, entry in ((0, 251, -1), (1, 120, s.NB), (2, 20, 2 ** 31 - 1)):
        j = t // bs
        table[b, j] = entry
        lo, hi = j * bs, j * bs + bs - 1           # positions of the block
        p = int(s.pos[b])
        rows[b] = [i for i in range(s.n[b]) if p + i >= lo and (not window or p + i - window + 1 <= hi)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = s.call(table=table, err=err)
    assert int(err.item()) == (pa.DEVERR_BAD_BLOCK if any(rows.values()) else 0)
    s.check(out, zero_rows=rows)


def test_bad_block_in_a_context_cut_between_ctas():
    for dtype in (BF16, F32):
        s = Chunk(dtype=dtype, B=1, T=2, H=8, Hkv=1, D=128, pos=[9000])
        table = s.table.clone()
        table[0, 100] = -7
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = s.call(table=table, err=err)
        assert int(err.item()) == pa.DEVERR_BAD_BLOCK
        s.check(out, zero=(0,))


@pytest.mark.parametrize("dtype,D", [(F32, 64), (BF16, 128), (F16, 64)])
def test_bad_counts_and_positions(dtype, D):
    s = Chunk(dtype=dtype, D=D, B=5, T=20, H=4, Hkv=2, pos=[10, 10, 10, 10, 10], counts=[20, 20, 20, 20, 20])
    counts, pos = s.counts.clone(), s.pos.clone()
    counts[0], counts[1] = -1, 21
    pos[2], pos[3] = -1, s.MB * s.bs - 19
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = s.call(positions=pos, counts=counts, err=err)
    assert int(err.item()) == pa.DEVERR_BAD_LEN | pa.DEVERR_BAD_POS
    s.check(out, skip=(0, 1), zero=(2, 3))
    pos.fill_(2 ** 31 - 1)
    s.check(s.call(positions=pos, err=err), zero=range(5))


def test_without_an_error_word():
    s = Chunk(B=2, T=20, pos=[100, 0])
    table = s.table.clone()
    table[1, 0] = -1
    s.check(s.call(table=table), zero=(1,))


@pytest.mark.parametrize("dtype,D,diff", [(F32, 64, False), (BF16, 128, False), (F16, 128, True)])
def test_results_repeat_and_workspaces_are_scratch(dtype, D, diff):
    s = Chunk(dtype=dtype, D=D, diff=diff, B=2, T=60, H=8, Hkv=2, pos=[3000, 5])
    first = s.call()
    ws = s.keep[5]
    for fill in (0, 0x7F, 0xFF):
        ws.fill_(fill)
        assert torch.equal(s.call(ws=ws), first)
    s.check(first, device="cuda")
    # the same workspace for another shape
    t = Chunk(dtype=dtype, D=D, diff=diff, B=7, T=1, H=4, Hkv=4, pos=[900 + b for b in range(7)], bs=8)
    t.check(t.call(ws=ws))


@pytest.mark.parametrize("dtype,D,diff", [(F32, 64, False), (BF16, 128, False), (F16, 128, True), (BF16, 64, False)])
def test_captured_calls_replay_on_new_contents(dtype, D, diff):
    s = Chunk(dtype=dtype, D=D, diff=diff, B=3, T=50, H=8, Hkv=2, pos=[2500, 5, 130], counts=[50, 50, 50])
    out, call = s.call(prepare=True)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa_stream = torch.cuda.current_stream()
        s2 = Chunk(dtype=dtype, D=D, diff=diff, B=3, T=50, H=8, Hkv=2, pos=[2500, 5, 130], counts=[50, 50, 50])
        q, flat, table, pos, cnt, ws, out = s.keep[:7]
        kw = dict(num_kv_heads=s.Hkv, block_size=s.bs, num_blocks=s.NB, block_stride=s.stride, counts=cnt, stream=pa_stream)
        if diff:
            pa.paged_attention_chunk_diff(out, q, flat, flat[s.v_at:], table, pos, s.keep[7], s.scale, ws, norm=s.keep[8],
                                          eps=s.eps, out_scale=s.out_scale, **kw)
        else:
            pa.paged_attention_chunk(out, q, flat, flat[s.v_at:], table, pos, s.scale, ws, **kw)
    for counts, posn in (([50, 50, 50], [2500, 5, 130]), ([1, 0, 50], [2549, 0, 0]), ([17, 33, 2], [12, 21, 170])):
        s2.counts, s2.pos = torch.tensor(counts, dtype=torch.int32), torch.tensor(posn, dtype=torch.int32)
        s2.n = counts
        cnt.copy_(s2.counts)
        pos.copy_(s2.pos)
        out.copy_(s2.out)
        q.copy_(s2.q)
        for b in range(3):   # query rows past the counts may hold anything
            q[b, counts[b]:] = math.nan
        graph.replay()
        torch.cuda.synchronize()
        s2.check(out, device="cuda")


def test_two_streams_with_workspaces_of_their_own():
    a = Chunk(B=2, T=60, H=8, Hkv=2, D=128, pos=[3000, 5], seed=1)
    b = Chunk(B=2, T=60, H=8, Hkv=2, D=128, pos=[2000, 77], seed=2)
    outs = []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    calls = [s.call(prepare=True, stream=st) for s, st in zip((a, b), streams)]
    torch.cuda.synchronize()
    for _ in range(20):
        for _, c in calls:
            c()
    torch.cuda.synchronize()
    for s, (out, _) in zip((a, b), calls):
        s.check(out, device="cuda")


@pytest.mark.parametrize("dtype,D,H,Hkv", [(BF16, 128, 16, 2), (F32, 64, 4, 4), (F16, 64, 8, 8)])
@pytest.mark.parametrize("window", [0, 40])
def test_single_tokens_agree_with_the_decode(dtype, D, H, Hkv, window):
    """With one token per sequence both entry points state the same attention."""
    s = Chunk(dtype=dtype, D=D, H=H, Hkv=Hkv, B=5, T=1, pos=[0, 15, 16, 200, 1000], window=window)
    out = s.call()
    s.check(out)
    q, flat, table, pos = s.keep[:4]
    ref = torch.empty((5, H, D), dtype=dtype, device="cuda")
    kw = dict(num_kv_heads=Hkv, block_size=s.bs, num_blocks=s.NB, block_stride=s.stride)
    q1 = q[:, 0].contiguous()
    if window:
        pa.paged_attention_decode_window(ref, q1, flat, flat[s.v_at:], table, pos + 1, s.scale, window, **kw)
    else:
        pa.paged_attention_decode(ref, q1, flat, flat[s.v_at:], table, pos + 1, s.scale, **kw)
    s.check(ref.view(5, 1, H, D))


def test_scales_of_either_sign_and_zero():
    for scale in (-0.2, 0.0, 3.0):
        run(scale=scale, B=2, T=70, H=2, Hkv=1, pos=[30, 0], D=64, dtype=F32)
        run(scale=scale, B=2, T=70, H=2, Hkv=1, pos=[30, 0], D=64, dtype=BF16)
        run(scale=scale, B=2, T=70, H=2, Hkv=1, pos=[30, 0], D=128, dtype=F16)


def test_scores_that_grow_along_the_context():
    """The running maximum moves with every tile; weights of early tiles vanish."""
    for dtype, D in ((BF16, 128), (F16, 64), (F32, 64), (BF16, 256)):
        s = Chunk(dtype=dtype, D=D, B=1, T=40, H=4, Hkv=1, pos=[700], scale=0.5)
        for j in range(-(-740 // s.bs)):
            k = s.block(int(s.table[0, j]), 0)
            k[:] = torch.where(k.isnan(), k, k * (0.01 * (j + 1)))
        s.check(s.call())


def test_three_operators_as_a_layer_runs_them():
    """Prompts with axes are written, attended to, continued by single tokens."""
    B, T, H, Hkv, D, bs = 2, 37, 8, 2, 64, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    MB, NB = 5, 12
    pool = torch.full((NB, 2, Hkv, bs, D), math.nan, dtype=BF16, device="cuda")
    flat = pool.view(-1)
    v_pool = flat[pool.stride(1):]
    table = torch.randperm(NB, generator=torch.Generator().manual_seed(1))[:B * MB].view(B, MB).int().cuda()
    kw = dict(block_size=bs, num_blocks=NB, block_stride=pool.stride(0))
    cs = pa.rope_table(256, D, device="cuda")
    pair_axis = pa.rope_axes((8, 12, 12))
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = None
    history = [[], []]
    for step, (t, counts) in enumerate(((T, [37, 20]), (1, [1, 1]), (4, [4, 2]))):
        qkv = torch.randn((B, t, H + 2 * Hkv, D), generator=g, device="cuda").to(BF16)
        q, k, v = qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]
        cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
        axis_pos = torch.randint(0, 256, (3, B, t), generator=g, device="cuda", dtype=torch.int32)
        q_out = torch.zeros((B, t, H, D), dtype=BF16, device="cuda")
        pa.paged_kv_append_rope_axes(q_out, q, k, v, flat, v_pool, table, pos, axis_pos, cs, pair_axis, counts=cnt,
                                     err_word=err, **kw)
        ws = pa.chunk_workspace_for(q_out, table, num_kv_heads=Hkv, **kw) if ws is None else ws
        out = torch.zeros_like(q_out)
        pa.paged_attention_chunk(out, q_out, flat, v_pool, table, pos, D ** -0.5, ws, counts=cnt, num_kv_heads=Hkv,
                                 err_word=err, **kw)
        for b in range(B):
            n, p = counts[b], int(pos[b])
            rows = pool[table[b].long()].transpose(2, 3).transpose(1, 2).flatten(0, 1)[:p + n].double()   # [L, 2, Hkv, D]
            assert torch.equal(rows[p:, 1], v[b, :n].double())
            x = torch.einsum("thgd,lhd->hgtl", q_out[b, :n].double().unflatten(1, (Hkv, -1)), rows[:, 0]) * D ** -0.5
            hidden = torch.arange(p + n, device="cuda")[None] > torch.arange(p, p + n, device="cuda")[:, None]
            a = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
            want = torch.einsum("hgtl,lhd->thgd", a, rows[:, 1]).flatten(1, 2)
            av = torch.einsum("hgtl,lhd->thgd", a, rows[:, 1].abs()).flatten(1, 2)
            # weights and the result rounded to bf16, 2^-8 each at most; what fp32 adds is far below 2^-12
            assert ((out[b, :n].double() - want).abs() <= 2.0 ** -8 * (av + want.abs()) + 2.0 ** -12 * av).all()
        pos += cnt
    assert int(err.item()) == 0


@pytest.mark.parametrize("H,Hkv", [(4, 4), (6, 2), (14, 2), (16, 1), (64, 1), (128, 1), (200, 1), (256, 1)])
@pytest.mark.parametrize("window", [0, 100])
def test_prompts_of_any_group(H, Hkv, window):
    """Tiles of whole tokens and tiles that cut one, several items of a head."""
    run(H=H, Hkv=Hkv, D=128, T=150, B=2, pos=[70, 0], counts=[150, 131], window=window, ref_device="cuda")
    run(H=H, Hkv=Hkv, D=64, T=150, B=2, pos=[70, 0], counts=[150, 131], window=window, diff=True, dtype=F16,
        ref_device="cuda")


@pytest.mark.parametrize("bs,gap", [(8, 1024), (16, 8 * 128), (128, 2048), (256, 1024), (24, 5 * 1024)])
def test_gaps_between_blocks(bs, gap):
    """Block strides that whole groups of 8 rows divide: gaps of poison are not read as rows."""
    for diff in (False, True):
        run(bs=bs, gap=gap, D=128, T=90, B=2, H=4, Hkv=2, pos=[200, 0], diff=diff)
        run(bs=bs, gap=gap, D=64, T=90, B=2, H=4, Hkv=2, pos=[200, 0], diff=diff, dtype=F16)


@pytest.mark.parametrize("dtype,D,bs", [(BF16, 128, 16), (F16, 64, 3), (F32, 64, 16)])
@pytest.mark.parametrize("B", [32, 33, 127, 128, 129])
def test_batches_around_those_a_warp_sums(B, dtype, D, bs):
    g = torch.Generator().manual_seed(B)
    cnt = torch.randint(0, 3, (B,), generator=g).tolist()
    cnt[0] = cnt[-1] = 0
    pos = torch.randint(0, 300, (B,), generator=g).tolist()
    run(B=B, T=2, counts=cnt, pos=pos, H=4, Hkv=2, D=D, bs=bs, dtype=dtype)


@pytest.mark.parametrize("dtype,D,bs,T", [(BF16, 128, 16, 5), (BF16, 128, 3, 5), (BF16, 128, 3, 80), (F16, 64, 16, 5),
                                          (F32, 64, 16, 5)])
def test_blocks_past_32_bit_offsets(dtype, D, bs, T):
    """Blocks near the end of pools of more than 2^32 bytes, queries and outputs in small tensors."""
    Hkv, H = 2, 4
    per = 2 * Hkv * bs * D
    es = torch.empty(0, dtype=dtype).element_size()
    NB = (1 << 32) // (per * es) + 50
    if torch.cuda.mem_get_info()[0] < NB * per * es + (1 << 30):
        pytest.skip("not enough memory")
    pool = torch.empty(NB * per, dtype=dtype, device="cuda")
    s = Chunk(dtype=dtype, D=D, B=1, T=T, H=H, Hkv=Hkv, bs=bs, pos=[4 * bs + 1])
    table = torch.full_like(s.table, -1)
    for j in range(s.MB):
        if int(s.table[0, j]) < 0:
            continue
        far = NB - 1 - 7 * j
        table[0, j] = far
        pool[far * per:(far + 1) * per] = s.flat[int(s.table[0, j]) * per:(int(s.table[0, j]) + 1) * per].cuda()
    q, out = s.q.contiguous().cuda(), s.out.cuda()
    table, pos = table.cuda(), s.pos.cuda()
    kw = dict(num_kv_heads=Hkv, block_size=bs, num_blocks=NB, block_stride=per)
    ws = pa.chunk_workspace_for(q, table, **kw)
    pa.paged_attention_chunk(out, q, pool, pool[Hkv * bs * D:], table, pos, s.scale, ws, **kw)
    s.check(out)


def test_many_calls_in_a_row_repeat():
    """Calls back to back, short and long ones in turn, with one workspace: each waits for
    the one before where it has to."""
    cases = [Chunk(B=1, T=1, H=8, Hkv=2, D=128, pos=[300]), Chunk(B=3, T=200, H=8, Hkv=2, D=128, pos=[0, 500, 33]),
             Chunk(B=2, T=3, H=8, Hkv=2, D=64, dtype=F16, pos=[2000, 7]), Chunk(B=1, T=4, H=4, Hkv=1, D=32, pos=[900]),
             Chunk(B=2, T=30, H=4, Hkv=2, D=128, diff=True, pos=[100, 700])]
    first = [c.call() for c in cases]
    ws = max((c.keep[5] for c in cases), key=lambda w: w.numel())
    calls = [c.call(ws=ws, prepare=True) for c in cases]
    for _ in range(30):
        for _, call in calls:
            call()
    torch.cuda.synchronize()
    for c, (out, _), want in zip(cases, calls, first):
        assert torch.equal(out, want)
        c.check(out, device="cuda")


# blocks that boxes of 8 rows do not fit, on either side of 128 query rows per kv head
@pytest.mark.parametrize("dtype,D,diff", [(BF16, 128, False), (F16, 64, False), (F16, 128, True), (BF16, 64, True)])
@pytest.mark.parametrize("bs", [1, 3, 5, 12, 130])
def test_rows_copied_one_by_one(bs, dtype, D, diff):
    run(bs=bs, dtype=dtype, D=D, diff=diff, B=3, T=131, H=8, Hkv=2, pos=[0, 61, 700], counts=[131, 1, 77])
    run(bs=bs, dtype=dtype, D=D, diff=diff, B=2, T=131, H=6, Hkv=2, pos=[500, 5], window=130)


@pytest.mark.parametrize("T", [31, 32, 33, 64, 65])
@pytest.mark.parametrize("bs,D", [(3, 128), (1, 64)])
def test_rows_copied_one_by_one_from_few_rows_on(bs, D, T):
    run(bs=bs, D=D, dtype=BF16, B=2, T=T, H=8, Hkv=2, pos=[300, 0], counts=[T, T - 1])


def test_rows_copied_one_by_one_in_long_contexts_and_many_sequences():
    run(bs=3, dtype=BF16, D=128, B=1, T=20, H=8, Hkv=1, pos=[9001], ref_device="cuda")
    run(bs=1, dtype=F16, D=64, B=2, T=40, H=16, Hkv=2, pos=[4000, 31], counts=[40, 2], ref_device="cuda")
    g = torch.Generator().manual_seed(7)
    cnt = torch.randint(0, 11, (300,), generator=g).tolist()
    pos = torch.randint(0, 70, (300,), generator=g).tolist()
    run(bs=3, dtype=BF16, D=128, B=300, T=10, counts=cnt, pos=pos, H=32, Hkv=2)


@pytest.mark.parametrize("window", [0, 130])
@pytest.mark.parametrize("dtype,D,diff", [(BF16, 128, False), (F16, 64, False), (BF16, 128, True)])
def test_bad_blocks_of_rows_copied_one_by_one(dtype, D, diff, window):
    s = Chunk(dtype=dtype, D=D, bs=1, B=2, T=200, H=4, Hkv=2, pos=[100, 0], counts=[200, 200], window=window, diff=diff)
    table, rows = s.table.clone(), {}
    for b, places, entry in ((0, (251, 259), -1), (1, (120,), s.NB)):
        for t in places:
            table[b, t] = entry
        rows[b] = [i for i in range(200) if any(t <= int(s.pos[b]) + i and (not window or t > int(s.pos[b]) + i - window)
                                                for t in places)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = s.call(table=table, err=err)
    assert int(err.item()) == pa.DEVERR_BAD_BLOCK
    s.check(out, zero_rows=rows)

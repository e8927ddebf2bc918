"""CPU checks of attention of several new tokens and of the rotary append with
axes: the headers as plain C against the binding, host-side refusals through the
C ABI and through the wrappers, and the helpers."""
import ctypes
import math
import subprocess
from pathlib import Path

import pytest
import torch

import pagedattention_decode_paged_gb300 as pa
from tests.chunk_ref import BF16, F16, F32, Chunk

ROOT = Path(__file__).resolve().parent.parent


@pytest.fixture(scope="module")
def lib():
    if not pa.LIB_PATH.exists():
        pytest.skip("library not built")
    return pa.load()


def test_headers_compile_as_plain_c_and_match_the_binding(tmp_path):
    src = tmp_path / "h.c"
    src.write_text('#include "pagedattn_chunk.h"\n#include "pagedattn_axes.h"\n#include <stdio.h>\n'
                   'int main(void){ printf("%zu %zu\\n", sizeof(pa_diff), sizeof(pa_rope_axes)); return 0; }\n')
    exe = tmp_path / "h"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-pedantic", f"-I{ROOT / 'include'}", str(src), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in out] == [ctypes.sizeof(pa.Diff), ctypes.sizeof(pa.RopeAxes)]


def shape(**over):
    a = dict(batch=2, num_heads=8, num_kv_heads=2, head_dim=128, block_size=16, max_blocks_per_seq=8, num_blocks=64,
             block_stride=2 * 2 * 16 * 128, dtype=BF16)
    a.update(over)
    return pa.make_shape(**a)


P = 4096   # an aligned address that is never read: every call here is refused first


def chunk(lib, s, *, out=P, q=P, q_stride=0, T=4, k=P, v=P, table=P, pos=P, counts=None, scale=0.1, window=0, ws=P,
          ws_bytes=0, diff=None):
    args = (out, q, q_stride, T, k, v, table, pos, counts, scale, window, ws, ws_bytes, None, None)
    sp = ctypes.byref(s) if s is not None else None
    if diff is None:
        return lib.paged_attention_chunk(sp, *args)
    return lib.paged_attention_chunk_diff(sp, ctypes.byref(diff) if diff != "null" else None, *args)


BAD_SHAPES = [(dict(batch=-1), 1), (dict(num_heads=0), 1), (dict(num_heads=7), 1), (dict(num_kv_heads=0), 1),
              (dict(head_dim=0), 1), (dict(block_size=0), 1), (dict(max_blocks_per_seq=0), 1), (dict(num_blocks=0), 1),
              (dict(dtype=7), 1), (dict(block_stride=100), 1), (dict(max_blocks_per_seq=2 ** 28), 1),
              (dict(max_blocks_per_seq=(2 ** 31 - 1) // 16), 2), (dict(head_dim=96), 2), (dict(head_dim=16), 2),
              (dict(head_dim=512), 2), (dict(dtype=F32, head_dim=256, block_stride=1 << 20), 2),
              (dict(block_stride=2 * 2 * 16 * 128 + 4), 3)]


@pytest.mark.parametrize("over,status", BAD_SHAPES)
def test_shapes_that_are_refused(lib, over, status):
    assert chunk(lib, shape(**over)) == status
    assert chunk(lib, shape(**over), diff=pa.Diff(P, None, 0.0, 1.0)) == status
    assert pa.paged_attention_chunk_workspace(shape(**over)) == 0


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), 1), (dict(window=-1), 1), (dict(scale=math.inf), 1), (dict(scale=math.nan), 1), (dict(scale=3e38), 1),
    (dict(q_stride=8 * 128 - 8), 1), (dict(out=None), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1),
    (dict(table=None), 1), (dict(pos=None), 1), (dict(ws=None), 1), (dict(T=2 ** 30), 1), (dict(out=P + 8), 3),
    (dict(q=P + 2), 3), (dict(k=P + 4), 3), (dict(v=P + 8), 3), (dict(ws=P + 8), 3), (dict(q_stride=8 * 128 + 4), 3)])
def test_arguments_that_are_refused(lib, over, status):
    assert chunk(lib, shape(), **over) == status
    assert chunk(lib, shape(), diff=pa.Diff(P, P, 1e-5, 1.0), **over) == status


def test_query_rows_past_int32_are_refused(lib):
    assert chunk(lib, shape(batch=1, num_heads=256, num_kv_heads=1), T=2 ** 23) == 2


@pytest.mark.parametrize("diff,status", [("null", 1), (pa.Diff(None, None, 0.0, 1.0), 1), (pa.Diff(P, P, -1.0, 1.0), 1),
                                         (pa.Diff(P, P, math.nan, 1.0), 1), (pa.Diff(P, None, 0.0, math.inf), 1),
                                         (pa.Diff(P, P + 2, 0.0, 1.0), 3)])
def test_differential_arguments_that_are_refused(lib, diff, status):
    assert chunk(lib, shape(), diff=diff) == status


def test_nothing_to_do_is_accepted(lib):
    assert chunk(lib, shape(batch=0), q=None, out=None, ws=None) == 0
    assert chunk(lib, shape(), T=0, q=None, out=None, ws=None) == 0
    assert chunk(lib, None) == 1
    assert chunk(lib, shape(dtype=F32, head_dim=16), diff=pa.Diff(P, None, 0.0, 1.0)) == 2


def axes_call(lib, *, rope=None, axes=None, T=1, **over):
    s = shape(**over)
    rows = pa.NewRows(P, P, P, 0, 0, 0, T)
    return lib.paged_kv_append_rope_axes(ctypes.byref(s), ctypes.byref(rope) if rope else None,
                                         ctypes.byref(axes) if axes else None, ctypes.byref(rows), P, P, P, P, P, None, None,
                                         None)


def test_axes_that_are_refused(lib):
    rope = pa.Rope(P, 100, 64, 0, None, None, 0.0)

    def axes(pair, n=3, pos=P):
        buf = ctypes.create_string_buffer(bytes(pair), len(pair))
        a = pa.RopeAxes(pos, n, ctypes.addressof(buf))
        a.keep = buf
        return a

    good = [0] * 10 + [1] * 10 + [2] * 12
    assert axes_call(lib, rope=rope) == 1
    assert axes_call(lib, axes=axes(good)) == 1
    assert axes_call(lib, rope=rope, axes=axes(good, n=0)) == 1
    assert axes_call(lib, rope=rope, axes=axes(good, n=5)) == 1
    assert axes_call(lib, rope=rope, axes=axes(good, n=2)) == 1
    assert axes_call(lib, rope=rope, axes=axes(good, pos=None)) == 1
    assert axes_call(lib, rope=rope, axes=pa.RopeAxes(P, 3, None)) == 1
    assert axes_call(lib, rope=pa.Rope(None, 0, 0, 0, None, None, 0.0), axes=axes(good)) == 1
    assert axes_call(lib, rope=pa.Rope(P, 100, 24, 0, None, None, 0.0), axes=axes(good)) == 1
    assert axes_call(lib, rope=rope, axes=axes(good), head_dim=96) == 2
    assert axes_call(lib, rope=rope, axes=axes(good), T=0) == 0


def test_rope_axes_helper():
    assert pa.rope_axes((2, 3, 1)) == bytes([0, 0, 1, 1, 1, 2])
    assert pa.rope_axes((2, 3, 1), cyclic=True) == bytes([0, 1, 2, 0, 1, 1])
    assert pa.rope_axes((0, 2)) == bytes([1, 1])
    with pytest.raises(ValueError):
        pa.rope_axes((1, 1, 1, 1, 1))
    with pytest.raises(ValueError):
        pa.rope_axes((1, -1))


def wrapper(s, **over):
    kw = dict(num_kv_heads=s.Hkv, block_size=s.bs, num_blocks=s.NB, block_stride=s.stride)
    args = dict(out=s.out, q=s.q, k_pool=s.flat, v_pool=s.flat[s.v_at:], block_table=s.table, positions=s.pos,
                scale=s.scale, workspace=torch.zeros(64, dtype=torch.uint8), counts=s.counts, **kw)
    fn = pa.paged_attention_chunk
    if s.diff:
        fn = pa.paged_attention_chunk_diff
        args.update(lambdas=s.lam, norm=s.w)
    args.update(over)
    return fn(**args)


@pytest.mark.parametrize("diff", [False, True])
def test_wrappers_refuse(lib, diff):
    s = Chunk(diff=diff)
    bad = [dict(out=s.out[:1]), dict(out=s.out.float()), dict(out=s.out.transpose(0, 1)), dict(q=s.q.float()),
           dict(q=s.q.transpose(2, 3)), dict(q=s.q[0, 0]), dict(block_table=s.table.long()), dict(block_table=s.table[:1]),
           dict(positions=s.pos[:1]), dict(positions=s.pos.long()), dict(counts=s.counts[:1]), dict(counts=s.counts.long()),
           dict(workspace=torch.zeros(64)), dict(k_pool=s.flat.float()), dict(v_pool=s.flat[-8:]),
           dict(num_blocks=s.NB + 1), dict(block_stride=s.stride + 8)]
    if diff:
        bad += [dict(lambdas=s.lam[:1]), dict(lambdas=s.lam.double()), dict(norm=s.w[:8]), dict(norm=s.w.float())]
    for over in bad:
        with pytest.raises(ValueError):
            wrapper(s, **over)
    with pytest.raises(ValueError, match="current CUDA device"):   # tensors of the host
        wrapper(s)


def test_axes_wrapper_refuses(lib):
    B, T, H, D = 2, 3, 2, 32
    x = torch.zeros((B, T, H, D), dtype=F16)
    pool = torch.zeros((4, 2, H, 16, D), dtype=F16)
    flat = pool.view(-1)
    args = dict(q_out=x, q=x, k_new=x, v_new=x, k_pool=flat, v_pool=flat[pool.stride(1):],
                block_table=torch.zeros((B, 2), dtype=torch.int32), positions=torch.zeros(B, dtype=torch.int32),
                axis_positions=torch.zeros((3, B, T), dtype=torch.int32), cos_sin=torch.zeros((9, D)),
                pair_axis=pa.rope_axes((6, 5, 5)), block_size=16, num_blocks=4, block_stride=pool.stride(0))
    for over in (dict(cos_sin=None), dict(axis_positions=None), dict(pair_axis=bytes(15)),
                 dict(axis_positions=torch.zeros((3, B, T + 1), dtype=torch.int32)),
                 dict(axis_positions=torch.zeros((3, B, T), dtype=torch.int64))):
        with pytest.raises(ValueError):
            pa.paged_kv_append_rope_axes(**{**args, **over})
    with pytest.raises(ValueError, match="current CUDA device"):
        pa.paged_kv_append_rope_axes(**args)

"""CPU checks of arguments that the wrappers of attention of several new tokens and of
the append with axes must not take for another operator's."""
import pytest
import torch

import pagedattention_decode_paged_gb300 as pa
from tests.chunk_ref import Chunk


@pytest.fixture
def issued(monkeypatch):
    """What would be issued, with every tensor taken for one of the current device."""
    calls = []
    monkeypatch.setattr(pa, "_launch_stream", lambda stream, what, *tensors: 0)
    monkeypatch.setattr(pa, "_issue", lambda fn, args, what, prepare, keep=(): calls.append((fn, what)))
    if not pa.LIB_PATH.exists():
        pytest.skip("library not built")
    return calls


def chunk_args(s):
    return (s.out, s.q, s.flat, s.flat[s.v_at:], s.table, s.pos), dict(
        num_kv_heads=s.Hkv, block_size=s.bs, num_blocks=s.NB, block_stride=s.stride)


@pytest.mark.parametrize("prepare", [False, True])
def test_the_differential_form_without_lambdas_is_refused(issued, prepare):
    """None is not the plain operator: norm, eps and out_scale would be lost without a word."""
    s = Chunk(diff=True)
    args, kw = chunk_args(s)
    ws = torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="lambdas"):
        pa.paged_attention_chunk_diff(*args, None, s.scale, ws, norm=s.w, out_scale=0.5, prepare=prepare, **kw)
    assert not issued
    pa.paged_attention_chunk_diff(*args, s.lam, s.scale, ws, norm=s.w, prepare=prepare, **kw)
    pa.paged_attention_chunk(*args, s.scale, ws, prepare=prepare, **kw)
    assert [what for _, what in issued] == ["paged_attention_chunk_diff", "paged_attention_chunk"]
    assert [fn.__name__ for fn, _ in issued] == [what for _, what in issued]


@pytest.mark.parametrize("prepare", [False, True])
@pytest.mark.parametrize("over", [dict(pair_axis=None), dict(axis_positions=None), dict(cos_sin=None),
                                  dict(axis_positions=torch.tensor(3, dtype=torch.int32))])
def test_the_append_with_axes_without_its_axes_is_refused(issued, over, prepare):
    """pair_axis=None went on to the entry point with another operator's arguments."""
    B, T, H, D = 2, 3, 2, 32
    x = torch.zeros((B, T, H, D), dtype=torch.float16)
    pool = torch.zeros((4, 2, H, 16, D), dtype=torch.float16)
    flat = pool.view(-1)
    args = dict(q_out=x, q=x, k_new=x, v_new=x, k_pool=flat, v_pool=flat[pool.stride(1):],
                block_table=torch.zeros((B, 2), dtype=torch.int32), positions=torch.zeros(B, dtype=torch.int32),
                axis_positions=torch.zeros((3, B, T), dtype=torch.int32), cos_sin=torch.zeros((9, D)),
                pair_axis=pa.rope_axes((6, 5, 5)), block_size=16, num_blocks=4, block_stride=pool.stride(0))
    with pytest.raises(ValueError, match="pair_axis"):
        pa.paged_kv_append_rope_axes(**{**args, **over}, prepare=prepare)
    assert not issued
    pa.paged_kv_append_rope_axes(**args, prepare=prepare)
    assert [what for _, what in issued] == ["paged_kv_append_rope_axes"]

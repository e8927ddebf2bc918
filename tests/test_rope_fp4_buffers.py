"""CPU checks that the wrappers of the rotary append and the 4-bit cache refuse
buffers that end before the sizes of the call do."""
import pytest
import torch

import pagedattention_decode_paged_gb300 as pa

B, H, Hkv, D, BS, NB = 2, 4, 2, 64, 16, 4
BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32
ON_HOST = "must be on the current CUDA device"      # the last check: what is right but for that gets there


def calls(k_pool, v_pool, scales, stride, wide=None):
    """Every entry point over these buffers; `wide`: pools of the rows' own type."""
    q, k = torch.zeros(B, H, D, dtype=BF), torch.zeros(B, Hkv, D, dtype=BF)
    table, at = torch.zeros(B, 2, dtype=I32), torch.zeros(B, dtype=I32)
    rows = torch.zeros(B, 3, Hkv, D, dtype=BF)
    kw = dict(block_size=BS, num_blocks=NB, block_stride=stride, stream=0)
    if wide is not None:
        return [lambda: pa.paged_kv_append_rope(q.clone(), q, k, k, *wide, table, at, None, **kw)]
    return [lambda: pa.paged_kv_append_rope_fp4(q.clone(), q, k, k, k_pool, v_pool, scales, table, at, None, **kw),
            lambda: pa.paged_kv_append_fp4(k, k, k_pool, v_pool, scales, table, at, **kw),
            lambda: pa.paged_kv_gather_fp4(rows, rows.clone(), k_pool, v_pool, scales, table, at, **kw),
            lambda: pa.paged_attention_decode_fp4(q.clone(), q, k_pool, v_pool, scales, table, at, 0.1,
                                                  torch.zeros(1 << 16, dtype=U8), num_kv_heads=Hkv, **kw)]


def refused(fn):
    with pytest.raises(ValueError) as e:
        fn()
    assert ON_HOST not in str(e.value)


def accepted(fn):
    with pytest.raises(ValueError, match=ON_HOST):
        fn()


HALF = Hkv * BS * D // 2                             # bytes of a block's keys in the 4-bit cache
SCALES = (NB, 2, Hkv, BS, D // 16)


@pytest.mark.parametrize("entry", range(4))
def test_scales_for_fewer_blocks_are_refused(entry):
    pool = torch.zeros(NB * 2 * HALF, dtype=U8)
    full = torch.zeros(SCALES, dtype=U8)
    for sc, ok in ((full, True), (full[:-1], False), (full.view(-1)[:-1], False), (torch.zeros(0, dtype=U8), False),
                   (torch.zeros((NB + 1, *SCALES[1:]), dtype=U8), True), (full.view(-1), True)):
        (accepted if ok else refused)(calls(pool, pool[HALF:], sc, 2 * HALF)[entry])


@pytest.mark.parametrize("entry", range(4))
def test_pools_that_end_early_are_refused(entry):
    sc = torch.zeros(SCALES, dtype=U8)
    pool = torch.zeros(NB * 2 * HALF, dtype=U8)
    apart = torch.zeros(NB * HALF, dtype=U8)
    cases = [(pool, pool[HALF:], 2 * HALF, True), (pool[HALF:], pool, 2 * HALF, True),      # values before keys
             (apart, apart.clone(), HALF, True), (apart, apart[16:], HALF, False), (pool, pool[HALF + 16:], 2 * HALF, False),
             (pool[2 * HALF:], pool, 2 * HALF, False), (apart, pool, 2 * HALF, False),
             (pool[:16], pool[HALF:HALF + 16], 2 * HALF, True),          # views that begin where the pools do
             (pool.view(NB, 2, Hkv, BS, D // 2)[:, 0], pool.view(NB, 2, Hkv, BS, D // 2)[:, 1], 2 * HALF, True)]
    for k, v, stride, ok in cases:
        (accepted if ok else refused)(calls(k, v, sc, stride)[entry])


def test_pools_of_the_rows_own_type():
    half = Hkv * BS * D
    pool = torch.zeros(NB * 2 * half, dtype=BF)
    accepted(calls(0, 0, 0, 2 * half, (pool, pool[half:]))[0])
    refused(calls(0, 0, 0, 2 * half, (pool, pool[half + 8:]))[0])
    refused(calls(0, 0, 0, 2 * half, (pool[:7 * half - 1].clone(), pool[half:]))[0])
    refused(calls(0, 0, 0, 2 * half + 8, (pool, pool[half:]))[0])

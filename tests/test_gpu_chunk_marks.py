"""GPU checks that no cached position is lost, counted twice or weighed wrongly where
contexts are cut between CTAs and joined: values zero but for marked positions, so that
an output element shows a few positions' weights and nothing else (the bounds are tried
against lost tiles in tests/test_chunk_marks.py)."""
import pytest
import torch

from tests.chunk_marks import APART, BF16, CASES, F16, F32, Marks, long_context, stairs, two_parts
from tests.chunk_ref import Chunk

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


def check(s, m):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = s.call(err=err).cpu()
    assert int(err.item()) == 0
    G, two = s.H // s.Hkv, two_parts(s)
    for b in (b for b in range(s.B) if s.n[b] > 0):
        for h, r in enumerate(m.offsets):
            want = m.want(b, r)
            for g in range(G):
                off = m.off(out[b, :s.n[b], h * G + g], want, two)
                assert off <= 1, f"sequence {b}, kv head {h} (marks at {r} of {APART}), head {g}: {off:.2f} of the bound"


@pytest.mark.parametrize("flat", [True, False])
@pytest.mark.parametrize("dtype,D,diff,bs", CASES)
def test_long_contexts_of_one_kv_head(dtype, D, diff, bs, flat):
    """About one tile a CTA."""
    for group in (1, 8):
        check(*long_context(dtype, D, diff, bs, 1, 20011, 3, group, None if flat else stairs(20014)))


@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("flat", [True, False])
@pytest.mark.parametrize("dtype,D,diff,bs", CASES)
def test_every_position_of_long_contexts_of_many_heads(dtype, D, diff, bs, flat, shift):
    """64 kv heads mark every second position between them, with many cuts at other places."""
    check(*long_context(dtype, D, diff, bs, 64, 4097, 2, 1, None if flat else stairs(4099), shift=shift))


@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("dtype,D,diff,bs", CASES)
def test_pieces_of_prompts_behind_long_contexts(dtype, D, diff, bs, window):
    check(*long_context(dtype, D, diff, bs, 4, 5003, 150, 2, stairs(5153), window))


@pytest.mark.parametrize("dtype,D,bs", [(F32, 64, 16), (BF16, 128, 16), (F16, 64, 16), (BF16, 32, 16), (BF16, 128, 1)])
def test_mixed_batches(dtype, D, bs):
    """Sequences of other lengths and counts: items begin and end inside slices everywhere."""
    pos = [0, 1, 127, 128, 1500, 63, 2999, 640, 5, 64]
    cnt = [257, 1, 1, 130, 1, 65, 2, 300, 0, 1]
    s = Chunk(dtype=dtype, D=D, bs=bs, B=10, T=300, H=8, Hkv=4, pos=pos, counts=cnt, scale=1.0)
    check(s, Marks(s, (0, 127, 17, 64), stairs(3100)))

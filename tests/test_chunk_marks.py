"""CPU check that the bounds of tests/chunk_marks.py tell a lost, doubled or misplaced
tile, and a lost position, from rounding."""
import pytest
import torch

from tests.chunk_marks import CASES, long_context, stairs, two_parts


@pytest.mark.parametrize("dtype,D,diff,bs", CASES)
@pytest.mark.parametrize("flat", [True, False])
def test_the_bound_rejects_a_lost_or_doubled_tile_and_a_lost_mark(dtype, D, diff, bs, flat):
    n = 20014
    s, m = long_context(dtype, D, diff, bs, 1, n - 3, 3, scores=None if flat else stairs(n))
    two = two_parts(s)
    want = m.want(0, 0)
    assert m.off(want, want, two) == 0
    assert m.off(want.to(dtype), want, two) <= 1
    for tile in [*range(0, n // 128 * 128, 5 * 128), n // 128 * 128 - 128]:
        for change in (dict(drop=range(tile, tile + 128)), dict(twice=range(tile, tile + 128)),
                       dict(drop=range(tile, tile + 64)), dict(drop=range(tile, tile + 1))):
            assert m.off(m.want(0, 0, **change).to(dtype), want, two) > 2, f"tile {tile}: {change}"
    if flat:       # lost from the sums that divide alone
        assert m.off((want * (n / (n - 128))).to(dtype), want, two) > 1


@pytest.mark.parametrize("window", [1, 64, 500])
def test_the_restatement_is_the_softmax_s(window):
    s, m = long_context(torch.float32, 64, False, 32, 1, 700, 4, scores=stairs(704), window=window)
    for t in range(4):
        p = 700 + t
        lo = max(0, p - window + 1)
        a = torch.softmax(m.x[lo:p + 1], 0)
        want = torch.zeros(64, dtype=torch.float64)
        for j in range(lo, p + 1):
            if j % 128 == 0:
                want[j // 128 % 64] += 64 * a[j - lo]
        assert torch.allclose(m.want(0, 0)[t], want, atol=1e-13, rtol=1e-12)

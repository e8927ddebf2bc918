"""GPU checks of the 4-bit decode where its fp16 parts could lose what the
header promises: query elements far below their head's largest, weights far
below the largest, scales whose product with a query leaves binary32.

Tolerances, with u = 2^-24, A = sum w |V| / sum w, S = the largest scale * sum
|q k|, E the error of a score:
- the last rounding: half a step of the dtype;
- a weight in the second product: 2^-11 of itself (16-bit queries) or 2^-22
  (fp32: two fp16 parts), and 2^-32 of the largest;
- scores: fp32 sums of D exact products, as counted in tests/fp4_ref.py:
  (D/8 + 8) 2 u S; 16-bit queries are exact but for elements below 2^-28 of the
  head's largest (none here), fp32 ones off by 2^-22 of themselves and 2^-39 of
  the largest, at each of which a key has its magnitude;
- sums of weights and weighted values: (n/16 + 32) 2 u A.
"""
import math

import pytest
import torch

from tests import fp4_ref as ref
from tests.test_gpu_fp4 import BF16, F16, F32, Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(cuda_ok):
    torch.cuda.synchronize()
    yield
    torch.cuda.synchronize()


def bounds(c):
    """(out, tolerance) in fp64 [B][H][D]."""
    B, H, D = c.q.shape
    u, wide = 2.0 ** -24, c.dtype == F32
    out, tol = torch.zeros(2, B, H, D, dtype=torch.float64)
    for b in range(B):
        n = int(c.lens[b])
        k, v = ref.cached_rows(c.pool, c.scales, c.table[b], c.bs, 0, n, (c.kg, c.vg))
        q = c.q[b].double().view(c.Hkv, H // c.Hkv, D)
        x = torch.einsum("hgd,hld->hgl", q, k) * c.scale
        w = torch.softmax(x, -1)
        o, A = torch.einsum("hgl,hld->hgd", w, v), torch.einsum("hgl,hld->hgd", w, v.abs())
        S = (torch.einsum("hgd,hld->hgl", q.abs(), k.abs()) * abs(c.scale)).amax(-1, keepdim=True)
        E = (D / 8 + 8) * 2 * u * S
        if wide:
            far = q.abs().amax(-1, keepdim=True) * k.abs().sum(-1).amax(-1)[:, None, None] * abs(c.scale)
            E = E + 2.0 ** -22 * S + 2.0 ** -39 * far
        t = A * ((2.0 ** -22 if wide else 2.0 ** -11) + 2 * E + (n / 16 + 32) * 2 * u)
        t = t + 2.0 ** -32 * w.amax(-1, keepdim=True) * v.abs().sum(1)[:, None]
        out[b], tol[b] = o.reshape(H, D), (t + ref.half_step(o.reshape(H, D), c.dtype).view_as(t)).reshape(H, D)
    return out, tol


def held(c):
    c.to_gpu()
    got = c.decode().double().cpu()
    want, tol = bounds(c)
    assert torch.isfinite(got).all()
    off = (got - want).abs()
    assert (off <= tol).all(), f"{float((off / tol.clamp(min=1e-300)).max()):.2f} of the bound"


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype,below", [(BF16, 20), (F16, 18), (F32, 12), (F32, 17)])
def test_query_elements_far_below_the_largest(dtype, below, D):
    """One element of each query is 2^below times the others, where every key is
    zero: the scores are those of the others."""
    c = Cache(lens=[100, 33, 1, 700], H=8, Hkv=2, D=D, dtype=dtype, seed=41)
    c.scales[:, 0, :, :, 0] = torch.where(c.scales[:, 0, :, :, 0] == 0x7F, 0x7F, 0).to(torch.uint8)
    c.q = (c.q.float() * 2.0 ** -(below - 8)).to(dtype)
    c.q[:, :, 5] = 256.0
    c.scale = 2.0 ** (below - 8) / math.sqrt(D)
    held(c)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("bits", [14.4, 20.6])
def test_weights_far_below_the_largest(bits, dtype, D):
    """The first token of every sequence takes nearly all the weight and has no
    value; what comes out is the others', each 2^-bits of it."""
    lens = [120 + 5 * i % 70 for i in range(130)]
    c = Cache(lens=lens, H=16, Hkv=8, D=D, dtype=dtype, seed=42)
    live = c.scales != 0x7F
    c.scales[:, 0] = torch.where(live[:, 0], 0, 0x7F).to(torch.uint8)            # keys of zero
    c.q[:] = 1.0
    for b in range(c.B):
        blk = int(c.table[b, 0])
        c.scales[blk, 0, :, 0, 1], c.pool[blk, 0, :, 0, 8:16] = 0x38, 0x22         # but the first: 16 ones
        c.scales[blk, 1, :, 0] = 0
    c.scale = bits * math.log(2.0) / 16
    held(c)


@pytest.mark.parametrize("dtype,D", [(F32, 64), (F32, 128), (BF16, 256)])
def test_a_scaled_query_past_binary32_where_keys_are_zero(dtype, D):
    """The query's largest element times the scale is no fp32 number; every key
    is zero there and the score finite."""
    c = Cache(lens=[100, 33, 1, 64], H=4, Hkv=2, D=D, dtype=dtype, seed=43)
    c.scales[:, 0, :, :, 0] = torch.where(c.scales[:, 0, :, :, 0] == 0x7F, 0x7F, 0).to(torch.uint8)
    c.q = torch.zeros_like(c.q)
    c.q[:, :, 5] = 1e38
    c.scale = 1e38
    held(c)

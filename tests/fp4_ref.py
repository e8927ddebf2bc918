"""Plain restatements of the rotary append and the 4-bit cache
(include/pagedattn_rope.h, include/pagedattn_fp4.h) for the tests: torch on the
CPU, one sequence at a time.  `turn64` and `decode64` are in 64 bits; `turn32`
is the stated order of binary32 operations, which decides codes exactly."""
from __future__ import annotations

import math

import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                    dtype=torch.float64)


def e4m3_value(byte: int) -> float:
    """OCP E4M3, from the bit fields."""
    sign = -1.0 if byte & 0x80 else 1.0
    e, m = (byte >> 3) & 15, byte & 7
    if e == 15 and m == 7:
        return math.nan
    return sign * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))


E4M3 = torch.tensor([e4m3_value(i) for i in range(256)], dtype=torch.float64)


def nearest(v: torch.Tensor, table: torch.Tensor) -> torch.Tensor:
    """Index of the entry of an ascending table nearest to each fp64 v >= 0,
    ties to the even index, saturating."""
    v = v.clamp(max=float(table[-1]))
    i = torch.searchsorted(table, v).clamp(1, table.numel() - 1)
    lo, hi = table[i - 1], table[i]
    up = (v - lo > hi - v) | ((v - lo == hi - v) & (i % 2 == 0))
    return torch.where(up, i, i - 1)


def quantise(x: torch.Tensor, g: float):
    """(code bytes [..., D/2], scale bytes [..., D/16]) of fp32 rows: quotients
    in binary32, then the nearest codes decided in fp64 (every binary32 number
    is one).  numpy's float32 division is IEEE division."""
    x = x.float()
    G = torch.where(torch.isnan(x), torch.zeros_like(x), x).unflatten(-1, (-1, 16))
    six_g = torch.tensor(6.0, dtype=torch.float32) * torch.tensor(g, dtype=torch.float32)
    a = torch.from_numpy(G.abs().amax(-1).numpy() / six_g.numpy())
    s = nearest(a.double(), E4M3[:127])
    t = (E4M3[s].float() * torch.tensor(g, dtype=torch.float32))[..., None]
    y = torch.where(t > 0, torch.from_numpy(G.numpy() / torch.where(t > 0, t, torch.ones_like(t)).numpy()),
                    torch.zeros_like(G))
    c = nearest(y.abs().double(), E2M1[:8]) | (torch.signbit(y).long() << 3)
    c = torch.where(t > 0, c, torch.zeros_like(c)).flatten(-2).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), s.to(torch.uint8)


def dequantise(codes: torch.Tensor, scales: torch.Tensor, g: float) -> torch.Tensor:
    """fp64 values of code bytes [..., D/2] and scale bytes [..., D/16]."""
    v = torch.stack((E2M1[(codes & 15).long()], E2M1[(codes >> 4).long()]), -1).flatten(-2)
    return v * E4M3[scales.long()].repeat_interleave(16, -1) * g


def _split(x, R, pairs):
    return (x[..., 0:R:2], x[..., 1:R:2]) if pairs else (x[..., :R // 2], x[..., R // 2:R])


def _join(x, a, b, R, pairs):
    y = x.clone()
    if pairs:
        y[..., 0:R:2], y[..., 1:R:2] = a, b
    else:
        y[..., :R // 2], y[..., R // 2:R] = a, b
    return y


def turn(x, w, cos_sin, pos, R, pairs, eps, dtype):
    """Norm (w) and rotation of rows x [n, heads, D] at positions pos, every
    operation rounded to `dtype` (float32: the stated order; float64: exact
    for the tests' purposes).  The mean square is taken in 64 bits either way."""
    x = x.to(dtype)
    if w is not None:
        v = (x.double().square().mean(-1, keepdim=True) + eps).to(dtype)
        x = (x * (1.0 / v.double().sqrt()).to(dtype)) * w.to(dtype)
    if R:
        cs = cos_sin[pos.long()][:, None].to(dtype)
        cos, sin = cs[..., :R // 2], cs[..., R // 2:]
        a, b = _split(x, R, pairs)
        x = _join(x, a * cos - b * sin, b * cos + a * sin, R, pairs)
    return x


def turn_bound(x, w, cos_sin, pos, R, pairs, eps):
    """Bound on the binary32 error of a turned row, per element, before its
    last rounding.  With u = 2^-24: the mean square's sum has at most 8 + 5
    roundings, half of which reach its root, which adds two (v, the root);
    two products with r and w: at most 11 u of the normed value.  A rotated
    element adds one product's and one sum's rounding to each of its two
    terms.  14 u covers both."""
    y = turn(x, w, cos_sin, pos, 0, pairs, eps, torch.float64).abs()
    if R:
        a, b = _split(y, R, pairs)
        y = _join(y, a + b, a + b, R, pairs)
    return 14 * 2.0 ** -24 * y


def half_step(ref, dtype):
    """Half a step of `dtype` at fp64 values (its smallest subnormal's half at least)."""
    f = torch.finfo(dtype)
    return (ref.abs() * (f.eps / 2)).clamp(min=f.smallest_normal * f.eps / 2)


def cached_rows(pool, scales, table_row, bs, n0, n1, g):
    """fp64 K and V values [2][Hkv][n1 - n0, D] of tokens n0..n1 of one sequence;
    pool uint8 [NB][2][Hkv][bs][D/2], scales uint8 [NB][2][Hkv][bs][D/16]."""
    pos = torch.arange(n0, n1)
    blk, slot = table_row[pos // bs].long(), pos % bs
    c, s = pool[blk, :, :, slot], scales[blk, :, :, slot]       # [n][2][Hkv][...]
    return dequantise(c, s, 1.0).permute(1, 2, 0, 3) * torch.tensor(g, dtype=torch.float64).view(2, 1, 1, 1)


def decode64(q, pool, scales, table, lens, bs, scale, window=0, k_scale=1.0, v_scale=1.0):
    """(out, tolerance) in fp64 [B][H][D]: textbook attention over the cached
    values, and how far a right kernel may be from it.

    With u = 2^-24, A = sum w |V| / sum w, S = the largest scale * sum |q k|:
    - the last rounding: half a step of the dtype;
    - the weights in the second product: 2^-11 of each for 16-bit queries
      (fp16), 2^-22 for fp32 (two fp16 parts);
    - scores: fp32 sums of D exact products, each of D/16 steps and the 16
      terms inside one rounding by at most 2 u of S (the tensor cores may
      truncate), plus the scaling: (D/8 + 8) 2 u S; fp32 queries in two parts:
      2^-21 S more; 16-bit ones lose at most 2^-24 of the head's largest
      element per element;  a score error e moves w by e, its normaliser too;
    - sums of weights and weighted values: a step of 16 tokens loses at most
      2 u, a merge a few: (n/16 + 32) 2 u A;
    - weights far below the largest: they are taken against a reference that no
      score passes by more than 2^8 and the largest reaches, so the largest is
      at least 1 there, and fp16 (one part or two, whose lower part is a
      multiple of 2^-24 as well) holds a weight below its normal range to
      2^-25; normalised by at least the largest weight's share:
      2^-25 max w sum |V|.
    """
    B, H, D = q.shape
    Hkv = pool.shape[2]
    grp = H // Hkv
    u = 2.0 ** -24
    out = torch.zeros((B, H, D), dtype=torch.float64)
    tol = torch.zeros((B, H, D), dtype=torch.float64)
    wide = q.dtype == torch.float32
    for b in range(B):
        n1 = int(lens[b])
        n0 = max(0, n1 - window) if window else 0
        if n1 == n0:
            continue
        k, v = cached_rows(pool, scales, table[b], bs, n0, n1, (k_scale, v_scale))
        qq = q[b].double().view(Hkv, grp, D)
        x = torch.einsum("hgd,hld->hgl", qq, k) * scale
        w = torch.softmax(x, -1)
        o = torch.einsum("hgl,hld->hgd", w, v)
        A = torch.einsum("hgl,hld->hgd", w, v.abs())
        S = (torch.einsum("hgd,hld->hgl", qq.abs(), k.abs()) * abs(scale)).amax(-1, keepdim=True)
        low = (qq.abs().amax(-1, keepdim=True) * k.abs().sum(-1).amax(-1)[:, None, None] * abs(scale)) * 2.0 ** -24
        E = (D / 8 + 8) * 2 * u * S + (2.0 ** -21 * S if wide else low)
        part = 2.0 ** -22 if wide else 2.0 ** -11
        t = A * (2 * part + 2 * E + ((n1 - n0) / 16 + 32) * 2 * u)
        t = t + 2.0 ** -25 * w.amax(-1, keepdim=True) * v.abs().sum(1)[:, None]
        out[b], tol[b] = o.reshape(H, D), (t + half_step(o, q.dtype)).reshape(H, D)
    return out, tol

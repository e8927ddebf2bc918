"""Inputs that show every cached position by itself: values are zero but for marked
positions, one in 128, each in a channel that at most a few others share.  An output
element is then the weight of one to a few positions over the sum of all, and a
position or a tile that is lost, doubled or weighed with another record's maximum
changes it by a good part of itself."""
import torch

from tests.chunk_ref import BF16, F16, F32, Chunk, half_step

APART = 128
MARK = 64.0                # far enough above fp16's smallest normal element after division by the context's length


class Marks:
    """Keys give position t the score scores[t] (0: all weigh the same) for every query row,
    head r marks the positions t % 128 == offsets[r] in channel t // 128 % D."""

    def __init__(self, s, offsets, scores=None, lam=0.25):
        self.s, self.offsets, self.lam = s, offsets, lam
        n = max(int(p) + c for p, c in zip(s.pos, s.n))
        e = s.D // 2 if s.diff else s.D
        x = torch.zeros(n, dtype=torch.float64) if scores is None else scores[:n].double()
        # two elements whose sum is the score in full, and queries of (1, 1, 0, ...), scale 1
        hi = x.to(s.dtype)
        key = torch.zeros((n, s.D), dtype=s.dtype)
        query = torch.zeros(s.D, dtype=s.dtype)
        for at in range(0, s.D, e):
            key[:, at], key[:, at + 1] = hi, (x - hi.double()).to(s.dtype)
            query[at:at + 2] = 1
        self.x = key[:, 0].double() + key[:, 1].double()
        s.q.copy_(torch.where(s.q.isnan(), s.q, query))
        s.lam.fill_(lam)
        t = torch.arange(n)
        value = torch.zeros((s.Hkv, n, s.D), dtype=s.dtype)
        for h, r in enumerate(offsets):
            marked = t[t % APART == r]
            value[h, marked, marked // APART % s.D] = MARK
        for b in range(s.B):
            held = int(s.pos[b]) + s.n[b]
            for j in range(-(-held // s.bs)):
                m = min(s.bs, held - j * s.bs)
                blk = int(s.table[b, j])
                s.block(blk, 0)[:, :m] = key[j * s.bs:j * s.bs + m]
                s.block(blk, 1)[:, :m] = value[:, j * s.bs:j * s.bs + m]

    def want(self, b, r, drop=(), twice=()):
        """[n, D] of sequence b in a head that marks t % 128 == r, in 64 bits; without the
        positions of range `drop`, those of `twice` counted once more."""
        s = self.s
        p, n = int(s.pos[b]), s.n[b]
        x = self.x[:p + n]
        w = (x - x.max()).exp()
        if len(drop):
            w[drop.start:drop.stop] = 0
        if len(twice):
            w[twice.start:twice.stop] *= 2
        marked = torch.arange(r, max(r, p + n), APART)
        y = torch.zeros((n, s.D), dtype=torch.float64)
        for t in range(n):
            lo, hi = max(0, p + t - s.window + 1) if s.window else 0, p + t + 1
            seen = marked[(marked >= lo) & (marked < hi)]
            y[t].index_add_(0, seen // APART % s.D, w[seen])
            y[t] *= MARK / w[lo:hi].sum()
        return y * (1 - self.lam) * s.out_scale if s.diff else y

    def room(self, two_parts):
        """How far an element may be off, relative to itself: its sums hold positive terms
        only.  Exponents by 4 roundings of fp32 of the largest score, the exponential to
        2^-22, weights rounded to the type or as two parts (equal ones are 1 and exact);
        sums along 128 positions of a tile, tile by tile and record by record, at most as
        many roundings as that (the tensor cores cut, twice a rounding); quotient, factors
        and the join of records 16 more; all that for numerator and denominator."""
        s, u = self.s, 2.0 ** -24
        n = len(self.x)
        big = float(self.x.abs().max())
        rel = 0.0
        if big > 0:
            rel += 4 * u * big + 2.0 ** -22
            if s.dtype != F32:
                # fp16 holds weights to 2^-25 of the largest
                small = float((self.x.min() - self.x.max()).exp())
                rel += half_step(s.dtype) ** (2 if two_parts else 1) + (2.0 ** -25 / small if s.dtype == F16 else 0.0)
            rel += (128 + n / 128 + 160) * 2 * u
        rel = 2 * rel + 16 * u
        return rel * (1 + self.lam) / (1 - self.lam) if s.diff else rel

    def off(self, got, want, two_parts):
        """The largest error over its bound; an element that should be zero is."""
        rel = self.room(two_parts)
        # below the normal elements half a step is that of the smallest of them
        small = torch.finfo(self.s.dtype).tiny * torch.finfo(self.s.dtype).eps / 2
        bound = want.abs() * (rel + half_step(self.s.dtype) * (1 + rel)) + small
        return float(((got.double() - want).abs() / bound).max())


def two_parts(s):
    return s.diff or (s.dtype != F32 and s.T * (s.H // s.Hkv) <= 128)


def stairs(n):
    """Scores that go up and down by up to 1, tiles by half of that: marks that share a
    channel weigh within a factor of 8 of one another."""
    t = torch.arange(n)
    return ((t * 37) % 29 - 14).double() / 32 + ((t // 128 * 11) % 17 - 8).double() / 16


CASES = [(F32, 64, False, 32), (BF16, 128, False, 32), (F16, 64, False, 32), (BF16, 64, False, 16), (BF16, 128, True, 32),
         (F16, 64, True, 32), (F16, 128, False, 3), (BF16, 32, False, 16), (F32, 32, True, 8)]


def long_context(dtype, D, diff, bs, heads, pos, T, group=1, scores=None, window=0, shift=0):
    s = Chunk(dtype=dtype, D=D, diff=diff, bs=bs, B=1, T=T, H=heads * group, Hkv=heads, pos=[pos], norm=False, scale=1.0,
              window=window, out_scale=1.0)
    offsets = [r * APART // heads + shift if heads > 4 else (0, 127, 64, 63)[r] for r in range(heads)]
    return s, Marks(s, offsets, scores)

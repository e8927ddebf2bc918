"""Plain 64-bit restatement of attention of several new tokens over a paged
cache (include/pagedattn_chunk.h), a bound on what its roundings may do to each
output, and inputs whose unused memory is poison."""
import math

import torch

import pagedattention_decode_paged_gb300 as pa

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


class Chunk:
    """One call: queries (a slice of a packed projection output), a table over
    shuffled blocks, positions and counts.  Whatever no token may see is NaN:
    slots past the last token, blocks of no sequence, query rows past the
    counts; out holds a pattern that shows a stray write."""

    def __init__(self, *, B=2, T=5, H=4, Hkv=2, D=64, bs=16, dtype=BF16, pos=None, counts="full", window=0, diff=False,
                 norm=True, lam=0.3, out_scale=0.75, eps=1e-5, seed=0, gap=0, packed=True, separate=False, scale=None,
                 device="cpu"):
        g = torch.Generator().manual_seed(seed)
        self.B, self.T, self.H, self.Hkv, self.D, self.bs, self.dtype, self.window = B, T, H, Hkv, D, bs, dtype, window
        self.diff, self.eps, self.out_scale = diff, eps, out_scale
        self.scale = scale if scale is not None else 1.0 / math.sqrt(D // 2 if diff else D)
        self.pos = torch.tensor(pos if pos is not None else [17 * b for b in range(B)], dtype=torch.int32)
        self.counts = None if counts is None else torch.full((B,), T, dtype=torch.int32) if isinstance(counts, str) \
            else torch.tensor(counts, dtype=torch.int32)
        self.n = [T if self.counts is None else int(self.counts[b]) for b in range(B)]
        held = [int(p) + n for p, n in zip(self.pos, self.n)]
        nblk = [max(0, -(-h // bs)) for h in held]
        self.MB, self.NB = max(max(nblk), 1) + 1, sum(nblk) + 3
        perm = torch.randperm(self.NB, generator=g).to(torch.int32)
        self.table = torch.full((B, self.MB), -1, dtype=torch.int32)
        at = 0
        for b, k in enumerate(nblk):
            self.table[b, :k] = perm[at:at + k]
            at += k
        # [NB][2][Hkv][bs][D] with a gap between blocks, or all of K then all of V
        row = Hkv * bs * D
        self.stride = (row if separate else 2 * row) + gap
        self.v_at = self.NB * self.stride if separate else row
        flat = torch.full((2 * self.NB * (row + gap),), math.nan, dtype=dtype)
        self.flat = flat
        for b, h in enumerate(held):
            for j in range(nblk[b]):
                m = min(bs, h - j * bs)
                if m > 0:
                    for half in (0, 1):
                        self.block(int(self.table[b, j]), half)[:, :m] = torch.randn((Hkv, m, D), generator=g).to(dtype)
        qkv = torch.randn((B, T, H + 2 * Hkv, D), generator=g).to(dtype)
        for b in range(B):
            qkv[b, max(self.n[b], 0):] = math.nan
        self.q = qkv[:, :, :H] if packed else qkv[:, :, :H].contiguous()
        self.out = torch.randint(0, 100, (B, T, H, D), generator=g).to(dtype)
        self.lam = lam + 0.1 * torch.randn(H, generator=g)
        self.w = (1 + 0.2 * torch.randn(D, generator=g)).to(dtype) if norm else None

    def block(self, blk, half):
        """Keys (half 0) or values of a block: [Hkv, bs, D], a view."""
        at = blk * self.stride + half * self.v_at
        return self.flat[at:at + self.Hkv * self.bs * self.D].view(self.Hkv, self.bs, self.D)

    def rows(self, b, half, n):
        """[n, Hkv, D] of the first n cached tokens of sequence b, as they are in the cache."""
        return torch.cat([self.block(int(self.table[b, j]), half) for j in range(-(-n // self.bs))], 1)[:, :n].transpose(0, 1)

    def call(self, *, table=None, positions="own", counts="own", err=None, ws=None, stream=None, prepare=False, out=None,
             device="cuda", window=None):
        """Issue the call on `device`; the tensors are kept, out is returned."""
        d = device
        if not self.q.is_contiguous():
            full = torch.full((self.B, self.T, self.H + 2 * self.Hkv, self.D), math.nan, dtype=self.dtype)
            full[:, :, :self.H] = self.q
            q = full.to(d)[:, :, :self.H]
        else:
            q = self.q.to(d)
        flat = self.flat.to(d)
        out = self.out.to(d) if out is None else out
        table = (self.table if table is None else table).to(d)
        pos = (self.pos if isinstance(positions, str) else positions).to(d)
        cnt = self.counts if isinstance(counts, str) else counts
        cnt = cnt.to(d) if cnt is not None else None
        kw = dict(num_kv_heads=self.Hkv, block_size=self.bs, num_blocks=self.NB, block_stride=self.stride)
        ws = pa.chunk_workspace_for(q, table, **kw).fill_(0xFF) if ws is None else ws
        kw.update(counts=cnt, window=self.window if window is None else window, err_word=err, stream=stream, prepare=prepare)
        self.keep = (q, flat, table, pos, cnt, ws, out)
        if self.diff:
            lam, w = self.lam.to(d), self.w.to(d) if self.w is not None else None
            self.keep += (lam, w)
            call = pa.paged_attention_chunk_diff(out, q, flat, flat[self.v_at:], table, pos, lam, self.scale, ws, norm=w,
                                                 eps=self.eps, out_scale=self.out_scale, **kw)
        else:
            call = pa.paged_attention_chunk(out, q, flat, flat[self.v_at:], table, pos, self.scale, ws, **kw)
        return (out, call) if prepare else out

    def want(self, b, device="cpu"):
        """(output [n, H, D] of sequence b in 64 bits, bound on each element's error)."""
        n, p, maps = self.n[b], int(self.pos[b]), 2 if self.diff else 1
        G, e = self.H // self.Hkv, self.D // maps
        k, v = (self.rows(b, half, p + n).to(device).double() for half in (0, 1))
        q = self.q[b, :n].to(device).double()
        own, at = torch.arange(p, p + n, device=device)[:, None], torch.arange(p + n, device=device)[None]
        seen = at <= own
        if self.window:
            seen &= at > own - self.window
        ys, tols = [], []
        u = 2.0 ** -24
        for h in range(self.H):
            kh, vh = k[:, h // G], v[:, h // G]
            o, t = [], []
            for m in range(maps):
                qm, km = q[:, h, m * e:(m + 1) * e], kh[:, m * e:(m + 1) * e]
                x = torch.where(seen, (qm @ torch.where(km.isfinite(), km, 0.0).T) * self.scale, -math.inf)
                w = (x - x.amax(-1, keepdim=True)).exp()
                total = w.sum(-1, keepdim=True)
                a = w / total
                # what a row does not see weighs nothing, whatever it holds
                plain = torch.where(vh.isfinite(), vh, 0.0)
                om = a @ plain
                for j in (~vh.isfinite()).any(-1).nonzero().flatten().tolist():
                    odd = torch.where(vh[j].isfinite(), 0.0, vh[j])
                    om += torch.where(seen[:, j:j + 1], a[:, j:j + 1] * odd, 0.0)
                o.append(om)
                # scores: e products and sums in fp32 (the tensor cores cut, 2^-23 each),
                # scale and exponent in base 2 with 2 more roundings of the score itself,
                # and the exponential to 2^-22: an error of the score is one of its weight,
                # once in the product and once in the sum
                big = ((qm.abs() @ torch.where(km.isfinite(), km, 0.0).abs().T) * abs(self.scale)).masked_fill(~seen, 0.0)
                xmax = torch.where(seen, x.abs(), 0.0).amax(-1, keepdim=True)
                score = (e + 2) * 2 * u * big.amax(-1, keepdim=True) + 4 * u * xmax + 2.0 ** -22
                # the weight's rounding to the type (as two parts in the differential form: the
                # rest's rounding), and fp16's smallest step
                weight = 0.0 if self.dtype == F32 else half_step(self.dtype) ** maps
                av = a @ plain.abs()
                tm = av * (2 * score + weight) * (1 + 2.0 ** -6)
                if self.dtype == F16:
                    tm = tm + 2.0 ** -25 * (seen.double() @ plain.abs()) / total
                # sums over the positions in fp32, of numerator and denominator, in some
                # order of tiles: as many roundings as positions at most, cut again
                tm = tm + av * 2 * (p + n + 8) * 2 * u
                t.append(tm)
            y, tol = o[0], t[0]
            if self.diff:
                lam = float(self.lam[h])
                y = o[0] - lam * o[1]
                tol = t[0] + abs(lam) * t[1] + 2 * u * (o[0].abs() + abs(lam) * o[1].abs())
                if self.w is not None:
                    r = 1.0 / (y.square().mean(-1, keepdim=True) + self.eps).sqrt()
                    wd = self.w.to(device).double()
                    # y r w: r moves by at most r times the root mean square of the errors of y, relatively
                    rel = r * tol.square().mean(-1, keepdim=True).sqrt()
                    tol = wd.abs() * r * (tol + y.abs() * rel) / (1 - rel).clamp(min=0.5)
                    y = y * r * wd
                    tol = tol + y.abs() * (self.D + 8) * u
                y, tol = y * self.out_scale, tol * abs(self.out_scale) + 2 * u * y.abs()
            ys.append(y)
            tols.append(tol + half_step(self.dtype) * (y.abs() + tol) + torch.finfo(self.dtype).tiny)
        return torch.stack(ys, 1), torch.stack(tols, 1)

    def check(self, out, *, zero=(), skip=(), zero_rows=None, device="cpu"):
        """Every element of out.  zero: sequences of zeros; skip: sequences left
        as they were; zero_rows: {sequence: tokens of zeros}."""
        got = out.cpu()
        worst = 0.0
        for b in range(self.B):
            n = max(0, self.n[b])
            assert torch.equal(got[b, n:], self.out[b, n:]), f"rows past the count of sequence {b} were written"
            if b in skip:
                assert torch.equal(got[b], self.out[b])
                continue
            if b in zero:
                assert not got[b, :n].any()
                continue
            if n == 0:
                continue
            want, tol = (t.cpu() for t in self.want(b, device))
            g = got[b, :n].double()
            zr = set(() if zero_rows is None else zero_rows.get(b, ()))
            for t in zr:
                assert not got[b, t].any(), f"token {t} of sequence {b} is not zeros"
            keep = torch.tensor([t not in zr for t in range(n)])
            g, want, tol = g[keep], want[keep], tol[keep]
            odd = ~want.isfinite()
            assert torch.equal(odd, ~g.isfinite()), f"sequence {b}: other elements are not finite"
            assert torch.equal(g[odd].isnan(), want[odd].isnan()) and torch.equal(g[odd].nan_to_num(), want[odd].nan_to_num())
            off = ((g - want).abs() / tol).nan_to_num(0.0)
            assert (off <= 1).all(), f"sequence {b}: {float(off.max()):.2f} of the bound"
            worst = max(worst, float(off.max()) if off.numel() else 0.0)
        return worst


def run(**over):
    dev = over.pop("ref_device", "cpu")
    s = Chunk(**over)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = s.call(err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    s.check(out, device=dev)
    return s, out

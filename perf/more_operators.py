"""Measured cases of attention of several new tokens per sequence over a paged
cache (prompts, chunks of them, speculative tokens, mixed batches), the same
with the difference of two softmax maps, and the rotary append with positions
of several axes.

`run` computes an operator in its plain form (elementary torch operations in
32 bits, rounded once at the end) or, with `own`, makes the call a user of
pagedattention_decode_paged_gb300 makes.  `exact` restates the definitions in
64 bits, one sequence and kv head at a time.

Token t of sequence b has cache position p = positions[b] + t; its keys and
values are in the cache already, and it attends to the positions
max(0, p - window + 1) .. p (window 0: from 0).

The two maps of a differential head: a key row of E elements holds the key of
the first map, then that of the second, E / 2 each; so does a query row; values
and outputs have E elements.
"""
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5
THETA = 10000.0
DEV = "cuda"


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _case(name, op, **kw):
    c = dict(name=name, op=op, B=1, T=1, cnt=1, lo=0, hi=0, H=8, Hkv=8, D=128, bs=16, dtype="bf16", window=0,
             norm=False, mixed=False, s0=0, s1=0, s2=0, cyclic=False, pairs=False)
    c.update(kw)
    return c


def listed():
    return [
        # the 4-request fp32 example with a few new tokens each: the smallest call, latency only
        _case("chunk 4 short f32", "chunk", B=4, T=4, cnt=1, H=4, Hkv=4, D=64, dtype="f32", lo=32, hi=128),
        # four speculative tokens of each request of the grouped-query layer at batch 32
        _case("chunk 32 x 4 tokens behind 2048", "chunk", B=32, T=4, cnt=4, H=64, Hkv=8, lo=2040, hi=2048),
        # a serving step that carries a 512-token piece of one prompt beside 63 requests with one token each
        _case("chunk mixed batch", "chunk", B=64, T=512, cnt=1, H=64, Hkv=8, lo=100, hi=4000, mixed=True),
        # whole prompts of a ragged batch, behind cached prefixes of other lengths
        _case("chunk prompts gqa", "chunk", B=8, T=2047, cnt=900, H=64, Hkv=8, lo=0, hi=700),
        # the Llama-7B-like layer's prompts, fp16, with a sliding window
        _case("chunk prompts mha window", "chunk", B=16, T=1000, cnt=450, H=32, Hkv=32, dtype="f16", bs=24, lo=0, hi=520,
              window=512),
        # fp32 prompts of an odd length over blocks of 8
        _case("chunk prompts f32", "chunk", B=3, T=517, cnt=33, H=12, Hkv=4, D=64, bs=8, dtype="f32", lo=0, hi=90),
        # one piece of a very long prompt: compute
        _case("chunk 4096 behind 28672", "chunk", B=1, T=4096, cnt=4096, H=64, Hkv=8, lo=28672, hi=28672, bs=32),
        # the next token of a differential grouped-query layer at batch 32
        _case("diff 32 x 1 token behind 2047", "diff", B=32, H=32, Hkv=8, lo=2047, hi=2047, norm=True),
        # ragged prompts of that layer
        _case("diff prompts", "diff", B=8, T=1023, cnt=300, H=32, Hkv=8, dtype="f16", lo=0, hi=200, norm=True),
        # one request's next token with axes: launch and dependent-load latency
        _case("axes append 1 token", "axes", H=64, Hkv=8, lo=2047, hi=2047, norm=True, s0=16, s1=24, s2=24),
        # prompts of text and images of a ragged batch, axes in turn
        _case("axes append prompts", "axes", B=8, T=2047, cnt=900, H=64, Hkv=8, lo=0, hi=700, norm=True, s0=24, s1=20,
              s2=20, cyclic=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng: random.Random):
    op = rng.choice(["chunk", "chunk", "chunk", "diff", "diff", "axes"])
    dtype = rng.choice(["f32", "f16", "f16", "bf16", "bf16", "bf16"])
    D = rng.choice([32, 64, 128, 128] + ([] if dtype == "f32" else [128, 256]))
    Hkv = rng.choice([1, 2, 3, 4, 5, 8, 8, 16, 32])
    grp = rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 8, 16])
    H = Hkv * grp if Hkv * grp <= 64 else Hkv
    c = dict(op=op, H=H, Hkv=Hkv, D=D, bs=rng.choice([1, 3, 8, 16, 16, 16, 24, 32, 64, 128]), dtype=dtype,
             norm=rng.random() < 0.6)
    if op == "axes":
        c["B"] = B = _log(rng, 1, 256)
        most = max(1, min(4096, (1 << 24) // (B * (H + 2 * Hkv) * D)))
        T = 1 if rng.random() < 0.4 else _log(rng, 1, most)
        half = rng.choice([r for r in (16, 32, 64, 128, 256) if r <= D] + [D, D]) // 2
        s0 = rng.randint(0, half)
        s1 = rng.randint(0, half - s0)
        c.update(T=T, cnt=rng.randint(1, T), hi=rng.randint(0, 2000), s0=s0, s1=s1, s2=half - s0 - s1,
                 cyclic=rng.random() < 0.4, pairs=rng.random() < 0.3)
    else:
        # up to 2^27 query elements, 2^28 cached ones of K and no more arithmetic than the largest listed case
        c["B"] = B = _log(rng, 1, 128)
        T = 1 if rng.random() < 0.3 else _log(rng, 1, max(1, min(4096, (1 << 27) // (B * H * D))))
        hi = _log(rng, 1, 65536) - 1
        hi = max(0, min(hi, (1 << 28) // (B * Hkv * D) - T))
        flops = 2e12 if dtype != "f32" else 1e11
        while T > 1 and 6.0 * D * H * B * T * (hi + T) > flops:
            T, hi = T // 2, hi // 2
        c.update(T=T, cnt=rng.randint(1, T), lo=rng.randint(0, hi), hi=hi, mixed=T > 1 and rng.random() < 0.25)
        c["window"] = _log(rng, 1, 4096) if rng.random() < 0.25 else 0
    full = _case("", op)
    full.update(c)
    del full["name"]
    return full


# --------------------------------------------------------------------------
# what a case's program has in hand
# --------------------------------------------------------------------------

def _lengths(case):
    """Cached tokens before, and new tokens of each sequence: part of the case, not of the seed."""
    c = case
    r = random.Random(f"{c['B']} {c['T']} {c['cnt']} {c['lo']} {c['hi']} {c['mixed']}")
    pos = [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    cnt = [1 if c["mixed"] else r.randint(c["cnt"], c["T"]) for _ in range(c["B"])]
    pos[-1], cnt[-1] = c["hi"], c["T"]
    return pos, cnt


def _pair_axis(case):
    """The axis of each pair: s0 pairs of axis 0, then s1, then s2; or (cyclic) in turn while an axis has some left."""
    left = [case["s0"], case["s1"], case["s2"]]
    if not case["cyclic"]:
        return bytes(a for a, n in enumerate(left) for _ in range(n))
    out = []
    while any(left):
        for a in range(3):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return bytes(out)


def _grid_positions(pos, cnt, T):
    """[3][B][T]: runs of text (all axes alike) and images (time, row, column) one after another, as image prompts have."""
    r = random.Random(f"{pos} {cnt}")
    out = torch.zeros((3, len(pos), T), dtype=torch.int32)
    for b, (p, n) in enumerate(zip(pos, cnt)):
        t, at = 0, p // 2
        while t < n:
            text = min(n - t, r.randint(1, 40))
            out[:, b, t:t + text] = torch.arange(at, at + text, dtype=torch.int32)
            t, at = t + text, at + text
            h, w = r.randint(1, 24), r.randint(1, 24)
            i = torch.arange(min(n - t, h * w), dtype=torch.int32)
            out[:, b, t:t + len(i)] = torch.stack((torch.full_like(i, at), at + i // w, at + i % w))
            t, at = t + len(i), at + max(h, w)
    return out


def _randn(gen, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32) * scale).to(dtype)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = DT[c["dtype"]]
    B, T, H, Hkv, D, bs = c["B"], c["T"], c["H"], c["Hkv"], c["D"], c["bs"]
    pos, cnt = _lengths(c)
    nblk = [-(-(p + n) // bs) for p, n in zip(pos, cnt)]
    MB, NB = max(nblk), sum(nblk) + 2
    perm = torch.randperm(NB, generator=gen, device=DEV).to(torch.int32).cpu()
    table = torch.full((B, MB), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(nblk):
        table[b, :n] = perm[at:at + n]
        at += n
    s = dict(case=c, table=table.to(DEV), NB=NB, dt=dt, pos=torch.tensor(pos, dtype=torch.int32, device=DEV),
             cnt=torch.tensor(cnt, dtype=torch.int32, device=DEV), host=(pos, cnt), ws={})
    s["pool"] = torch.empty((NB, 2, Hkv, bs, D), dtype=dt, device=DEV)
    step = max(1, (1 << 26) // (2 * Hkv * bs * D))
    for i in range(0, NB, step):
        s["pool"][i:i + step] = _randn(gen, (min(step, NB - i), 2, Hkv, bs, D), dt)
    # the packed output of the layer's projection, rows of all heads of q, k and v beside one another
    qkv = _randn(gen, (B, T, H + 2 * Hkv, D), dt)
    s["q"], s["k"], s["v"] = qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]
    s["out"] = torch.zeros((B, T, H, D), dtype=dt, device=DEV)

    def weight():
        return _randn(gen, (D,), torch.float32, 0.1).add_(1.0).to(dt) if c["norm"] else None

    if c["op"] == "axes":
        s["qw"], s["kw"] = weight(), weight()
        s["axis"], R = _pair_axis(c), 2 * (c["s0"] + c["s1"] + c["s2"])
        s["axis_pos"] = _grid_positions(pos, cnt, T).to(DEV)
        n = int(s["axis_pos"].max()) + 1
        freq = THETA ** (-torch.arange(0, R, 2, device=DEV, dtype=torch.float64) / R)
        ang = torch.arange(n, device=DEV, dtype=torch.float64)[:, None] * freq
        s["cos_sin"] = torch.cat((ang.cos(), ang.sin()), 1).float()
    if c["op"] == "diff":
        s["w"] = weight()
        # exp(a.b) - exp(c.d) + init with learned vectors of about 0.1
        l4 = _randn(gen, (4, H, D // 2), torch.float32, 0.1)
        s["lam"] = (l4[0] * l4[1]).sum(-1).exp() - (l4[2] * l4[3]).sum(-1).exp() + 0.5
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def _softmax_rows(x, seen):
    x = x.masked_fill_(~seen, -math.inf)
    w = (x - x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
    return w / w.sum(-1, keepdim=True).clamp(min=1e-30)


def _attend(s, b0, b1, h0, h1):
    """Rows of sequences [b0, b1) and kv heads [h0, h1): [b, h, g, t, D] in fp32."""
    c = s["case"]
    pos, cnt = s["host"]
    D, bs, G = c["D"], c["bs"], c["H"] // c["Hkv"]
    T = max(cnt[b0:b1])
    L = max(p + n for p, n in zip(pos[b0:b1], cnt[b0:b1]))
    first = min(max(0, p - c["window"] + 1) if c["window"] else 0 for p in pos[b0:b1]) // bs
    blk = s["table"][b0:b1, first:-(-L // bs)].clamp(min=0).long()
    at = first * bs + torch.arange(blk.shape[1] * bs, device=DEV)
    own_pos = s["pos"][b0:b1, None] + torch.arange(T, device=DEV)
    seen = (at <= own_pos[..., None]) & (torch.arange(T, device=DEV) < s["cnt"][b0:b1, None])[..., None]
    if c["window"]:
        seen &= at > own_pos[..., None] - c["window"]
    seen = seen[:, None, None]

    def rows(half):
        return s["pool"][:, half, h0:h1][blk].transpose(1, 2).flatten(2, 3).float()[:, :, None]

    q = s["q"][b0:b1, :T, h0 * G:h1 * G].float().unflatten(2, (h1 - h0, G)).permute(0, 2, 3, 1, 4)
    k, v = rows(0), rows(1)
    # rows that nothing of this batch holds may be anything: they weigh nothing, but not as 0 * NaN
    v = v.masked_fill(~(at < (s["pos"] + s["cnt"])[b0:b1, None])[:, None, None, :, None], 0.0)
    if c["op"] == "chunk":
        return _softmax_rows((q / math.sqrt(D)) @ k.transpose(-1, -2), seen) @ v
    e = D // 2
    q = q / math.sqrt(e)
    a = _softmax_rows(q[..., :e] @ k[..., :e].transpose(-1, -2), seen)
    a2 = _softmax_rows(q[..., e:] @ k[..., e:].transpose(-1, -2), seen)
    a -= s["lam"][h0 * G:h1 * G].view(1, h1 - h0, G, 1, 1) * a2
    o = a @ v
    if s["w"] is not None:
        o = o * (o.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["w"].float()
    return o * 0.5


def _plain_attention(s):
    c = s["case"]
    pos, cnt = s["host"]
    G, longest = c["H"] // c["Hkv"], max(p + n for p, n in zip(pos, cnt))
    whole = c["B"] * c["H"] * max(cnt) * longest <= 1 << 28 and c["B"] * c["Hkv"] * longest * c["D"] <= 1 << 28
    for b0, b1 in ([(0, c["B"])] if whole else [(b, b + 1) for b in range(c["B"])]):
        n, L = max(cnt[b0:b1]), max(p + k for p, k in zip(pos[b0:b1], cnt[b0:b1]))
        step = c["Hkv"] if whole else max(1, (1 << 30) // (G * n * L))
        for h0 in range(0, c["Hkv"], step):
            h1 = min(c["Hkv"], h0 + step)
            o = _attend(s, b0, b1, h0, h1).permute(0, 3, 1, 2, 4).flatten(2, 3).to(s["dt"])
            out = s["out"][b0:b1, :n, h0 * G:h1 * G]
            kept = torch.arange(n, device=DEV) < s["cnt"][b0:b1, None]
            out.copy_(torch.where(kept[..., None, None], o, out))


def _rotate(s, x, w, b, t):
    """Norm (when w is given) and rotation of rows x [n, heads, D] of tokens (b, t), in fp32."""
    c = s["case"]
    x = x.float()
    if w is not None:
        r = (x.double().square().mean(-1, keepdim=True) + EPS).float().double().rsqrt().float()
        x = (x * r) * w.float()
    half = len(s["axis"])
    i = torch.arange(half, device=DEV)
    p = s["axis_pos"][:, b, t].long()[torch.tensor(list(s["axis"]), device=DEV, dtype=torch.long)].T   # [n, half]
    cos, sin = s["cos_sin"][p, i][:, None], s["cos_sin"][p, half + i][:, None]
    y = x.clone()
    f, g = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if c["pairs"] else (slice(0, half), slice(half, 2 * half))
    y[..., f] = x[..., f] * cos - x[..., g] * sin
    y[..., g] = x[..., g] * cos + x[..., f] * sin
    return y


def _plain_axes(s):
    c = s["case"]
    b, t = torch.nonzero(torch.arange(c["T"], device=DEV) < s["cnt"][:, None], as_tuple=True)
    p = s["pos"][b].long() + t
    blk, slot = s["table"][b, p // c["bs"]].long(), p % c["bs"]
    s["out"][b, t] = _rotate(s, s["q"][b, t], s["qw"], b, t).to(s["dt"])
    s["pool"][blk, 0, :, slot] = _rotate(s, s["k"][b, t], s["kw"], b, t).to(s["dt"])
    s["pool"][blk, 1, :, slot] = s["v"][b, t]


def run(state):
    s = state
    c = s["case"]
    if own:
        import pagedattention_decode_paged_gb300 as pa
        flat = s["pool"].view(-1)
        k_pool, v_pool = flat, flat[s["pool"].stride(1):]
        kw = dict(block_size=c["bs"], num_blocks=s["NB"], block_stride=s["pool"].stride(0))
        if c["op"] == "axes":
            pa.paged_kv_append_rope_axes(s["out"], s["q"], s["k"], s["v"], k_pool, v_pool, s["table"], s["pos"],
                                         s["axis_pos"], s["cos_sin"], s["axis"], counts=s["cnt"],
                                         interleaved=c["pairs"], q_norm=s["qw"], k_norm=s["kw"], eps=EPS, **kw)
            return {"q": s["out"], "pool": s["pool"]}
        kw["num_kv_heads"] = c["Hkv"]
        if "ws" not in s["ws"]:   # kept for the life of the cache
            s["ws"]["ws"] = pa.chunk_workspace_for(s["q"], s["table"], **kw)
        if c["op"] == "chunk":
            pa.paged_attention_chunk(s["out"], s["q"], k_pool, v_pool, s["table"], s["pos"], 1.0 / math.sqrt(c["D"]),
                                     s["ws"]["ws"], counts=s["cnt"], window=c["window"], **kw)
        else:
            pa.paged_attention_chunk_diff(s["out"], s["q"], k_pool, v_pool, s["table"], s["pos"], s["lam"],
                                          1.0 / math.sqrt(c["D"] // 2), s["ws"]["ws"], counts=s["cnt"], norm=s["w"],
                                          eps=EPS, out_scale=0.5, window=c["window"], **kw)
        return s["out"]
    if c["op"] == "axes":
        _plain_axes(s)
        return {"q": s["out"], "pool": s["pool"]}
    _plain_attention(s)
    return s["out"]


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def _attended(case):
    """(pairs of a new token and a position it attends to, cached rows read) of all sequences."""
    w, pairs, rows = case["window"], 0, 0
    for p, n in zip(*_lengths(case)):
        rows += p + n - (max(0, p - w + 1) if w else 0)
        full = p * n + n * (n + 1) // 2
        if w:   # token t sees min(p + t + 1, w)
            cut = max(0, min(n, w - p))   # tokens whose window is not full yet
            full = p * cut + cut * (cut + 1) // 2 + (n - cut) * w
        pairs += full
    return pairs, rows


def work(case):
    c = case
    es = 4 if c["dtype"] == "f32" else 2
    H, Hkv, D = c["H"], c["Hkv"], c["D"]
    pos, cnt = _lengths(c)
    n = sum(cnt)
    if c["op"] == "axes":
        R = 2 * (c["s0"] + c["s1"] + c["s2"])
        b = n * (2 * H + 4 * Hkv) * D * es + n * 3 * 4
        return {"bytes": b, "flops": n * (H + Hkv) * (3 * R + (4 * D if c["norm"] else 0))}
    pairs, rows = _attended(c)
    return {"bytes": rows * 2 * Hkv * D * es + 2 * n * H * D * es,
            "flops": (4 if c["op"] == "chunk" else 6) * D * H * pairs}


# --------------------------------------------------------------------------
# the definitions in 64 bits, one sequence and kv head at a time
# --------------------------------------------------------------------------

def _exact_axes(s, x, w, b, n):
    """Rows x [n, heads, D] of sequence b normed and rotated as complex numbers."""
    c = s["case"]
    x = x.double()
    if w is not None:
        x = x / (x.pow(2).sum(-1, keepdim=True) / c["D"] + EPS).sqrt() * w.double()
    half = len(s["axis"])
    cs = s["cos_sin"].double()
    z = torch.empty((n, half), dtype=torch.complex128, device=DEV)
    for i, a in enumerate(s["axis"]):
        p = s["axis_pos"][a, b, :n].long()
        z[:, i] = torch.complex(cs[p, i], cs[p, half + i])
    head, rest = x[..., :2 * half], x[..., 2 * half:]
    pair = head.unflatten(-1, (half, 2)) if c["pairs"] else head.unflatten(-1, (2, half)).transpose(-1, -2)
    turned = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z[:, None])
    turned = turned if c["pairs"] else turned.transpose(-1, -2)
    return torch.cat((turned.flatten(-2), rest), -1)


def exact(case, seed):
    c = case
    if work(c)["flops"] > 6e12:
        return None
    s = prepare(c, seed)
    pos, cnt = s["host"]
    out = s["out"].double()
    D, bs, G = c["D"], c["bs"], c["H"] // c["Hkv"]
    if c["op"] == "axes":
        pool = s["pool"].double()
        for b, (p, n) in enumerate(zip(pos, cnt)):
            at = torch.arange(p, p + n, device=DEV)
            blk = s["table"][b].long()[at // bs]
            out[b, :n] = _exact_axes(s, s["q"][b, :n], s["qw"], b, n)
            pool[blk, 0, :, at % bs] = _exact_axes(s, s["k"][b, :n], s["kw"], b, n)
            pool[blk, 1, :, at % bs] = s["v"][b, :n].double()
        return {"q": out, "pool": pool}
    maps = 1 if c["op"] == "chunk" else 2
    e = D // maps
    for b, (p, n) in enumerate(zip(pos, cnt)):
        at = torch.arange(max(0, p - c["window"] + 1) if c["window"] else 0, p + n, device=DEV)
        kv = s["pool"][s["table"][b].long()[at // bs], :, :, at % bs]            # [L, 2, Hkv, D]
        ahead = at[None] - torch.arange(p, p + n, device=DEV)[:, None]           # 0: the token itself
        hidden = ahead > 0
        if c["window"]:
            hidden |= ahead <= -c["window"]
        for h in range(c["Hkv"]):
            k, v = kv[:, 0, h].double(), kv[:, 1, h].double()
            q = s["q"][b, :n, h * G:(h + 1) * G].double().transpose(0, 1).unflatten(-1, (maps, e))   # [G, n, maps, e]
            o = []
            for m in range(maps):
                x = q[:, :, m] @ k[:, m * e:(m + 1) * e].T
                x.div_(math.sqrt(e)).masked_fill_(hidden, -math.inf)
                o.append(torch.softmax(x, -1) @ v)
                del x
            y = o[0]
            if maps == 2:
                y = o[0] - s["lam"][h * G:(h + 1) * G].double()[:, None, None] * o[1]
                if s["w"] is not None:
                    y = y / (y.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * s["w"].double()
                y = y * 0.5
            out[b, :n, h * G:(h + 1) * G] = y.transpose(0, 1)
    return out

"""CPU checks of the rotary append and the 4-bit cache: the headers and the
library agree, bad arguments are refused before anything is enqueued, the
Python wrappers check their tensors, and the tests' own restatements hold on
hand-worked values."""
import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import pagedattention_decode_paged_gb300 as pa
from pagedattention_decode_paged_gb300 import _build
from tests import fp4_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADERS = ("pagedattn_rope.h", "pagedattn_fp4.h")
FAKE = 1 << 20          # a 16-byte aligned address that is never dereferenced on the host
OK, INVALID, UNSUPPORTED, MISALIGNED = pa.PA_OK, pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED, pa.PA_ERR_MISALIGNED


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return pa.load()


def declarations(name):
    """{function: the comment nearest above its declaration}."""
    text = open(os.path.join(ROOT, "include", name)).read()
    out, last = {}, ""
    for m in re.finditer(r"^/\*.*?\*/|^[A-Za-z_][\w\s\*]*?\b([a-z_][a-z0-9_]*)\s*\(", text, flags=re.S | re.M):
        if m.group(0).startswith("/*"):
            last = " ".join(re.sub(r"\n\s*\*(?!/)", " ", m.group(0)).split())
        elif m.group(1):
            out[m.group(1)] = last
    return out


def test_declared_symbols_are_exported_and_bound(lib):
    names = set()
    for h in HEADERS:
        for name, comment in declarations(h).items():
            names.add(name)
            assert hasattr(lib, name), name
            assert name in pa.EXPORTED and getattr(lib, name).argtypes, name
            assert any(t in comment for t in ("[BM]", "[KB]", "[BUG]", "[PG]")) or "no counterpart" in comment or \
                "paged_kv_append_rope" in comment, name
    assert names == {"paged_kv_append_rope", "paged_kv_append_fp4", "paged_kv_append_rope_fp4", "paged_kv_gather_fp4",
                     "paged_attention_fp4_workspace", "paged_attention_decode_fp4"}


@pytest.mark.parametrize("header", HEADERS)
def test_header_compiles_as_plain_c_and_matches_the_binding(tmp_path, header):
    src = tmp_path / "t.c"
    src.write_text(f'#include "{header}"\n#include <stdio.h>\nint main(void){{ printf("%zu %zu %zu\\n", '
                   'sizeof(pa_shape), sizeof(pa_rope), sizeof(pa_new_rows)); return 0; }\n')
    exe = tmp_path / "t"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", f"-I{ROOT}/include", str(src), "-o", str(exe)], check=True)
    sizes = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(s) for s in sizes] == [ctypes.sizeof(t) for t in (pa.Shape, pa.Rope, pa.NewRows)]


def shape(**over):
    d = dict(batch=2, num_heads=8, num_kv_heads=2, head_dim=128, block_size=16, max_blocks_per_seq=8, num_blocks=64,
             block_stride=2 * 2 * 16 * 128, dtype=pa.PA_BF16)
    d.update(over)
    return pa.make_shape(**d)


def shape4(**over):
    d = dict(block_stride=2 * 2 * 16 * 64)
    d.update(over)
    return shape(**d)


def rope(**over):
    d = dict(cos_sin=FAKE, max_position=64, rotary_dim=128, interleaved=0, q_weight=None, k_weight=None, eps=1e-6)
    d.update(over)
    return pa.Rope(**d)


def rows(**over):
    d = dict(q=FAKE, k=FAKE, v=FAKE, q_stride=0, k_stride=0, v_stride=0, max_tokens=1)
    d.update(over)
    return pa.NewRows(**d)


def ref_or_none(x):
    return None if x is None else ctypes.byref(x)


def call_rope(lib, s=None, r=None, n=None, q_out=FAKE, kp=FAKE, vp=FAKE, bt=FAKE, pos=FAKE, cnt=None, err=None):
    return lib.paged_kv_append_rope(ref_or_none(s), ref_or_none(r), ref_or_none(n), q_out, kp, vp, bt, pos, cnt, err,
                                    None)


def call_rope4(lib, s=None, r=None, n=None, q_out=FAKE, kp=FAKE, vp=FAKE, sc=FAKE, kg=1.0, vg=1.0, bt=FAKE, pos=FAKE):
    return lib.paged_kv_append_rope_fp4(ref_or_none(s), ref_or_none(r), ref_or_none(n), q_out, kp, vp, sc, kg, vg, bt,
                                        pos, None, None, None)


BAD_ROWS = [(dict(max_tokens=-1), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
            (dict(k=FAKE + 8), MISALIGNED), (dict(v=FAKE + 2), MISALIGNED), (dict(q=FAKE + 4), MISALIGNED),
            (dict(q_stride=8 * 128 - 8), INVALID), (dict(k_stride=128), INVALID), (dict(v_stride=-1024), INVALID),
            (dict(q_stride=8 * 128 + 4), MISALIGNED), (dict(k_stride=2 * 128 + 1), MISALIGNED)]
BAD_ROPE = [(dict(rotary_dim=-16), INVALID), (dict(rotary_dim=144), INVALID), (dict(rotary_dim=24), INVALID),
            (dict(cos_sin=None), INVALID), (dict(max_position=0), INVALID), (dict(cos_sin=FAKE + 4), MISALIGNED),
            (dict(q_weight=FAKE, eps=float("nan")), INVALID), (dict(k_weight=FAKE, eps=-1.0), INVALID),
            (dict(q_weight=FAKE + 2), MISALIGNED)]


@pytest.mark.parametrize("fp4", [False, True])
def test_append_refuses_bad_arguments(lib, fp4):
    call, s = (call_rope4, shape4()) if fp4 else (call_rope, shape())
    for over, status in BAD_ROWS:
        assert call(lib, s, rope(), rows(**over)) == status, over
    for over, status in BAD_ROPE:
        assert call(lib, s, rope(**over), rows()) == status, over
    assert call(lib, None, rope(), rows()) == INVALID
    assert call(lib, s, None, rows()) == INVALID
    assert call(lib, s, rope(), None) == INVALID
    for arg in ("q_out", "kp", "vp", "bt", "pos"):
        assert call(lib, s, rope(), rows(), **{arg: None}) == INVALID, arg
    for arg in ("q_out", "kp", "vp"):
        assert call(lib, s, rope(), rows(), **{arg: FAKE + 8}) == MISALIGNED, arg
    make = shape4 if fp4 else shape
    for over in (dict(batch=-1), dict(num_heads=0), dict(num_kv_heads=0), dict(head_dim=0), dict(block_size=0),
                 dict(max_blocks_per_seq=0), dict(num_blocks=0), dict(dtype=3), dict(block_stride=16),
                 dict(max_blocks_per_seq=1 << 28)):
        assert call(lib, make(**over), rope(), rows()) == INVALID, over
    assert call(lib, make(block_stride=2 * 2 * 16 * 128 + 4), rope(), rows()) == MISALIGNED
    for over in (dict(num_heads=65537), dict(num_kv_heads=65537, block_stride=1 << 40)):
        assert call(lib, make(**over), rope(), rows(q_stride=1 << 30, k_stride=1 << 30, v_stride=1 << 30)) == INVALID, over
    assert call(lib, make(batch=1 << 16), rope(), rows(max_tokens=1 << 15)) == INVALID
    # nothing to do: refused or accepted before any pointer is looked at
    assert call(lib, make(batch=0), rope(), rows()) == OK
    assert call(lib, s, rope(), rows(max_tokens=0, k=None), kp=None) == OK
    # unsupported head sizes
    for D in ((32, 96, 512) if fp4 else (16, 96, 512)):
        assert call(lib, make(head_dim=D, block_stride=1 << 20), rope(rotary_dim=0), rows()) == UNSUPPORTED, D
    if not fp4:
        assert call(lib, make(head_dim=256, dtype=pa.PA_F32, block_stride=1 << 20), rope(), rows()) == UNSUPPORTED


def test_fp4_refuses_bad_factors_and_scales(lib):
    for g in (0.0, -1.0, float("inf"), float("nan"), 2.0 ** -65, 2.0 ** 65):
        assert call_rope4(lib, shape4(), rope(), rows(), kg=g) == INVALID
        assert call_rope4(lib, shape4(), rope(), rows(), vg=g) == INVALID
    assert call_rope4(lib, shape4(), rope(), rows(), sc=None) == INVALID
    assert call_rope4(lib, shape4(), rope(), rows(), sc=FAKE + 8) == MISALIGNED
    app = lib.paged_kv_append_fp4
    s = shape4()
    tail = (FAKE, FAKE, None, None, None)
    assert app(ctypes.byref(s), ctypes.byref(rows(k=None)), FAKE, FAKE, FAKE, 1.0, 1.0, *tail) == INVALID
    assert app(ctypes.byref(s), ctypes.byref(rows()), FAKE, FAKE, None, 1.0, 1.0, *tail) == INVALID
    assert app(ctypes.byref(s), ctypes.byref(rows()), FAKE, FAKE + 4, FAKE, 1.0, 1.0, *tail) == MISALIGNED


def test_gather_refuses_bad_arguments(lib):
    f = lib.paged_kv_gather_fp4

    def call(s=shape4(), ko=FAKE, vo=FAKE, T=4, kp=FAKE, vp=FAKE, sc=FAKE, kg=1.0, vg=1.0, bt=FAKE, st=FAKE):
        return f(ref_or_none(s), ko, vo, T, kp, vp, sc, kg, vg, bt, st, None, None, None)

    assert call(s=None) == INVALID and call(T=-1) == INVALID and call(kg=0.0) == INVALID and call(vg=-2.0) == INVALID
    for arg in ("ko", "vo", "kp", "vp", "sc", "bt", "st"):
        assert call(**{arg: None}) == INVALID, arg
    for arg in ("ko", "vo", "kp", "vp", "sc"):
        assert call(**{arg: FAKE + 8}) == MISALIGNED, arg
    assert call(s=shape4(head_dim=32)) == UNSUPPORTED
    assert call(s=shape4(batch=0)) == OK and call(T=0) == OK


def test_decode_refuses_bad_arguments(lib):
    f = lib.paged_attention_decode_fp4

    def call(s=shape4(), out=FAKE, q=FAKE, kp=FAKE, vp=FAKE, sc=FAKE, kg=1.0, vg=1.0, bt=FAKE, sl=FAKE, scale=0.1,
             window=0, ws=FAKE):
        return f(ref_or_none(s), out, q, kp, vp, sc, kg, vg, bt, sl, scale, window, ws, 1 << 40, None, None)

    assert call(s=None) == INVALID and call(s=shape4(num_heads=7)) == INVALID
    assert call(window=-1) == INVALID and call(scale=float("inf")) == INVALID and call(kg=0.0) == INVALID
    for arg in ("out", "q", "kp", "vp", "sc", "bt", "sl", "ws"):
        assert call(**{arg: None}) == INVALID, arg
    for arg in ("out", "q", "kp", "vp", "sc", "ws"):
        assert call(**{arg: FAKE + 8}) == MISALIGNED, arg
    assert call(s=shape4(head_dim=96, block_stride=1 << 20)) == UNSUPPORTED
    assert call(s=shape4(block_stride=2 * 2 * 16 * 64 + 8)) == MISALIGNED
    assert call(s=shape4(block_stride=2 * 16 * 64 - 16)) == INVALID
    assert call(s=shape4(batch=0)) == OK
    # more tiles than the schedule's int32 indices hold
    assert call(s=shape4(batch=1 << 14, num_heads=64, num_kv_heads=64, max_blocks_per_seq=1 << 16,
                         block_stride=1 << 20)) == UNSUPPORTED
    assert call(s=shape4(block_size=1, max_blocks_per_seq=(1 << 31) - 1000, block_stride=1 << 20)) == UNSUPPORTED
    assert call(scale=3e38, kg=2.0) == INVALID
    assert pa.paged_attention_fp4_workspace(shape4(batch=0)) == 0
    assert pa.paged_attention_fp4_workspace(shape4(head_dim=32)) == 0


def test_wrappers_check_their_tensors(lib):
    B, H, Hkv, D, bs, NB = 2, 4, 2, 64, 16, 4
    bf, u8, i32 = torch.bfloat16, torch.uint8, torch.int32
    q, k = torch.zeros(B, H, D, dtype=bf), torch.zeros(B, Hkv, D, dtype=bf)
    pool, sc = torch.zeros(NB * 2 * Hkv * bs * D // 2, dtype=u8), torch.zeros(NB, 2, Hkv, bs, D // 16, dtype=u8)
    table, pos = torch.zeros(B, 2, dtype=i32), torch.zeros(B, dtype=i32)
    cs = pa.rope_table(8, D)
    kw = dict(block_size=bs, num_blocks=NB, block_stride=2 * Hkv * bs * D // 2, stream=0)

    def append(**over):
        a = dict(q_out=q.clone(), q=q, k=k, v=k, kp=pool, vp=pool, sc=sc, table=table, pos=pos, cs=cs)
        a.update({n: v for n, v in over.items() if n in a})
        more = {n: v for n, v in over.items() if n not in a}
        pa.paged_kv_append_rope_fp4(a["q_out"], a["q"], a["k"], a["v"], a["kp"], a["vp"], a["sc"], a["table"],
                                    a["pos"], a["cs"], **more, **kw)

    bad = [dict(v=k[:, :1]), dict(q=q.float()), dict(q=q[:1]), dict(q_out=None), dict(q_out=q[:, :2].clone()),
           dict(k=k.transpose(1, 2)), dict(v=torch.zeros(B, Hkv, 2 * D, dtype=bf)[..., ::2]), dict(kp=pool.view(torch.int8)),
           dict(sc=sc.float()), dict(table=table.long()), dict(table=table[:1]), dict(pos=pos[:1]), dict(cs=cs.double()),
           dict(rotary_dim=32), dict(q_norm=torch.ones(D)), dict(k_norm=torch.ones(D // 2, dtype=bf)),
           dict(counts=pos[:1]), dict(counts=pos.long())]
    on_host = "must be on the current CUDA device"      # the last check: what is right but for that gets there
    with pytest.raises(ValueError, match=on_host):
        append()

    def refused(fn):
        with pytest.raises((ValueError, TypeError)) as e:
            fn()
        assert on_host not in str(e.value)

    for over in bad:
        refused(lambda: append(**over))
    f64 = torch.float64
    refused(lambda: append(q=q.to(f64), k=k.to(f64), v=k.to(f64), q_out=q.to(f64)))
    out = torch.empty_like(q)
    ws = torch.zeros(1 << 16, dtype=u8)
    for over in (dict(out=out[:1]), dict(out=out.float()), dict(q=q.transpose(0, 1)), dict(ws=ws.float()),
                 dict(table=table[:1]), dict(lens=pos[:1]), dict(kp=pool.float())):
        a = dict(out=out, q=q, kp=pool, ws=ws, table=table, lens=pos)
        a.update(over)
        refused(lambda: pa.paged_attention_decode_fp4(a["out"], a["q"], a["kp"], pool, sc, a["table"], a["lens"], 0.1,
                                                      a["ws"], num_kv_heads=Hkv, **kw))
    rows_ = torch.zeros(B, 3, Hkv, D, dtype=bf)
    refused(lambda: pa.paged_kv_gather_fp4(rows_, rows_[:, :2], pool, pool, sc, table, pos, **kw))
    refused(lambda: pa.paged_kv_gather_fp4(rows_, rows_.float(), pool, pool, sc, table, pos, **kw))


def test_new_rows_accepts_slices_of_a_packed_projection():
    packed = torch.zeros(3, 5, 12, 64)
    assert pa._new_rows("q", packed[:, :, :8]) == (3, 5, 8, 64, 12 * 64)
    assert pa._new_rows("k", packed[:, :, 8:10]) == (3, 5, 2, 64, 12 * 64)
    assert pa._new_rows("k", packed[:, 0, 8:10]) == (3, 1, 2, 64, 5 * 12 * 64)
    assert pa._new_rows("k", packed[:, 1:2, 8:9]) == (3, 1, 1, 64, 5 * 12 * 64)
    with pytest.raises(ValueError):                     # sequences further apart than their tokens
        pa._new_rows("k", packed[:, :4, 8:10])
    assert pa._new_rows("k", packed[:, :0, 8:10]) == (3, 0, 2, 64, 128)      # no tokens: nothing to stride over
    one = torch.zeros(1, 1, 2, 64)
    assert pa._new_rows("k", one.expand(1, 1, 2, 64)) == (1, 1, 2, 64, 128)
    for x in (one.expand(3, 1, 2, 64), one.expand(1, 5, 2, 64), one[0].expand(3, 2, 64)):
        with pytest.raises(ValueError):                 # tokens that share their rows
            pa._new_rows("k", x)


# --- the restatements themselves -------------------------------------------------

def test_e4m3_values_are_torchs():
    lib_values = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double()
    assert torch.equal(torch.nan_to_num(lib_values, nan=-1e9), torch.nan_to_num(ref.E4M3, nan=-1e9))


def test_quantise_by_hand():
    x = torch.zeros(1, 32)
    # scale 1 exactly (largest 6): every tie of E2M1, to the even code
    x[0, :16] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -5.0, 0.26, 4.9, 5.1, -0.0, math.nan])
    x[0, 16:] = 0.0
    codes, s = ref.quantise(x, 1.0)
    lo, hi = codes[0] & 15, codes[0] >> 4
    nib = torch.stack((lo, hi), -1).flatten().tolist()
    assert nib[:16] == [7, 0, 2, 2, 4, 4, 6, 6, 8, 10, 14, 1, 6, 7, 8, 0]
    assert s[0].tolist() == [0x38, 0] and nib[16:] == [0] * 16
    assert ref.dequantise(codes, s, 1.0)[0, :8].tolist() == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]
    # the factor moves the scale, not the codes; a scale saturates at 448
    c2, s2 = ref.quantise(x * 0.5, 0.5)
    assert torch.equal(c2, codes) and torch.equal(s2, s)
    c3, s3 = ref.quantise(torch.full((1, 16), 1e9), 1.0)
    assert s3.tolist() == [[0x7E]] and (c3 == 0x77).all()
    c4, s4 = ref.quantise(torch.full((1, 16), math.inf), 1.0)
    assert s4.tolist() == [[0x7E]] and (c4 == 0x77).all()


def test_turn_by_hand():
    cs = pa.rope_table(4, 16, theta=100.0)
    assert torch.equal(cs[0], torch.cat((torch.ones(8), torch.zeros(8))))
    x = torch.randn(1, 2, 32, dtype=torch.float64)
    pos = torch.tensor([3])
    for pairs in (False, True):
        y = ref.turn(x, None, cs, pos, 16, pairs, 0.0, torch.float64)
        a = (0, 1) if pairs else (0, 8)
        z = complex(x[0, 1, a[0]], x[0, 1, a[1]]) * complex(math.cos(3.0), math.sin(3.0))
        assert abs(float(y[0, 1, a[0]]) - z.real) < 1e-6 and abs(float(y[0, 1, a[1]]) - z.imag) < 1e-6
        assert torch.equal(y[..., 16:], x[..., 16:])
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1), rtol=1e-6)
    w = torch.full((32,), 2.0, dtype=torch.float64)
    n = ref.turn(x, w, cs, pos, 0, False, 0.0, torch.float64)
    assert np.allclose(n.square().mean(-1).numpy(), 4.0)

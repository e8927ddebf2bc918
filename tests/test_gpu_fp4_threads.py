"""GPU check of the 4-bit decode called from two host threads at once, in a
process of its own so that its first calls are the library's: batches whose
schedules differ in size, each thread with its own stream and workspace."""
import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu

PROGRAM = r"""
import threading

import torch

import pagedattention_decode_paged_gb300 as pa
from tests.test_gpu_fp4 import BF16, F16, Cache, held_to

SIZES = [(3, 128, BF16), (900, 128, BF16), (40, 64, F16), (1500, 64, F16), (7, 256, BF16), (1200, 256, BF16)]
# made before the threads start: nothing but the calls themselves runs side by side
jobs = [[], []]
for i, (B, D, dtype) in enumerate(SIZES):
    for j in (0, 1):
        c = Cache(lens=[(k * 5) % 37 for k in range(B + j * 11)], H=2, Hkv=1, D=D, dtype=dtype, seed=i)
        c.g = {n: getattr(c, n).cuda() for n in ("pool", "scales", "table", "q", "lens")}
        c.kw = dict(block_size=c.bs, num_blocks=c.NB, block_stride=c.g["pool"].stride(0))
        c.flat = c.g["pool"].view(-1)
        c.ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
        jobs[j].append(c)
jobs[1].reverse()
streams, outs, errors = [torch.cuda.Stream() for _ in jobs], [[], []], []
torch.cuda.synchronize()
start = threading.Barrier(2)


def work(j):
    try:
        start.wait(30)
        with torch.cuda.stream(streams[j]):
            for c in jobs[j]:
                shape = pa.decode_shape(c.g["q"], c.g["table"], num_kv_heads=1, **c.kw)
                assert 0 < pa.paged_attention_fp4_workspace(shape) <= c.ws.numel()
                outs[j].append([c.decode() for _ in range(20)])
    except BaseException as e:
        errors.append(e)


threads = [threading.Thread(target=work, args=(j,)) for j in (0, 1)]
[t.start() for t in threads]
[t.join() for t in threads]
torch.cuda.synchronize()
assert not errors, errors
for j in (0, 1):
    for c, got in zip(jobs[j], outs[j]):
        want = c.reference()
        held_to(got[0], want)
        assert all(torch.equal(x, got[0]) for x in got)
print("both right")
"""


def test_first_calls_from_two_host_threads(cuda_ok):
    root = Path(__file__).resolve().parent.parent
    run = subprocess.run([sys.executable, "-c", PROGRAM], cwd=root, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0 and "both right" in run.stdout, run.stdout + run.stderr

"""CPU checks, by reading, of what no run of chunk_umma.cu can be made to show:
orders that the hardware need not break, and waits that run out."""
import re
from pathlib import Path

import pytest

SOURCE = Path(__file__).resolve().parent.parent / "pagedattention_decode_paged_gb300" / "csrc" / "chunk_umma.cu"


@pytest.fixture(scope="module")
def kernel():
    """The kernel's body, without comments."""
    text = re.sub(r"//[^\n]*", "", SOURCE.read_text())
    return text[text.index("chunk_umma_kernel("):text.index("plan_one(")]


def first(text, pattern, at):
    m = re.compile(pattern).search(text, at)
    return m.start() if m else len(text)


def test_waits_for_tensor_memory_are_followed_by_its_fence(kernel):
    """Barriers that order tensor memory between threads, or after the tensor core, order
    a thread's later tensor-memory instructions only with the fence after the wait."""
    waits = [m for m in re.finditer(r"wait(?:_loop)?\(bars? ?[(+][^;{]*?L::(S_FULL|S_FREE|P_EMPTY|P_HALF|P_FULL|O_DONE|O_FREE)\b", kernel)]
    assert {m.group(1) for m in waits} >= {"S_FULL", "P_HALF", "P_FULL", "O_DONE", "O_FREE"}
    for m in waits:
        use = first(kernel, r"\btmem_(ld|st)\w*\(|\bumma_\w+\(|\bput_record<|\bstore_row<", m.end())
        fence = first(kernel, r"tc05_fence_after_sync\(\)", m.end())
        leaves = first(kernel, r"\bcontinue;", m.end())            # rows that are not there touch none of it
        assert min(fence, leaves) < use, f"{m.group(1)}: {kernel[m.start():m.start() + 60]!r}"

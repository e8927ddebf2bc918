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


def test_a_warp_votes_before_it_acts_on_a_wait_that_gave_up(kernel):
    """Lanes may run out of polls apart: whatever leaves a loop, returns or goes on to
    what the whole warp does together is decided by a vote."""
    sets = [m.end() for m in re.finditer(r"\babort = true;", kernel)]
    assert len(sets) > 8
    warm = kernel.index("L::WARM), 0)) abort = true;")             # the first item's vote comes next
    for at in sets:
        vote = first(kernel, r"abort = __any_sync\(0xffffffffu, abort\);", at)
        if kernel[warm:at].count("\n") == 0 and at > warm:
            vote = first(kernel, r"= item\(i\)", at)
        acts = first(kernel, r"if \(abort\)|return abort|return !abort|&& !abort; |while \(has && !abort\)|__shfl_sync\(0xffffffffu, v, 0\)", at)
        if "auto wait = [&](uint32_t b, uint32_t bit)" in kernel[max(0, at - 160):at]:
            # the product warps' helper: its callers' step ends with the vote
            assert kernel.count("abort = __any_sync(0xffffffffu, abort);\n                    if (abort) break;\n                }\n                if (abort) break;") == 1
            continue
        assert vote < acts, kernel[at - 120:at + 200]


def test_no_wait_is_begun_by_a_product_warp_that_gave_up(kernel):
    products = kernel[kernel.index("auto wait = [&](uint32_t b, uint32_t bit)"):kernel.index("warp == kQWarp")]
    loops = [m.start() for m in re.finditer(r"mbar_wait_loop\(", products)]
    for at in loops:
        line = products[products.rindex("\n", 0, at):at]
        assert "!abort &&" in line or "L::END" in products[at:at + 60], line

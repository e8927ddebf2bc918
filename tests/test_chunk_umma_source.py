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


ACTS = r"if \(abort\)|return abort|return !abort|&& !abort; |while \(has && !abort\)|__shfl_sync\(|__syncwarp\(|__any_sync\(0xffffffffu, (?!abort)"
VOTE = r"abort = __any_sync\(0xffffffffu, abort\);"


def products(kernel):
    at = kernel.index("auto wait = [&](uint32_t b, uint32_t bit)")
    return at, kernel.index("umma_commit(bars + (L::END + s) * 8)", at)


def test_a_warp_votes_before_it_acts_on_a_wait_that_gave_up(kernel):
    """Lanes may run out of polls apart: what the whole warp leaves, returns from or does
    together is decided by a vote."""
    p0, p1 = products(kernel)
    warm = kernel.index("L::WARM), 0)) abort = true;")
    sets = [m.end() for m in re.finditer(r"\babort = true;", kernel)]
    outside = [at for at in sets if not warm < at < p1]
    assert len(outside) > 6
    for at in outside:
        assert first(kernel, VOTE, at) < first(kernel, ACTS, at), kernel[at - 120:at + 200]
    # every item is fetched with a vote, or through a role's own wait, which has one
    for m in re.finditer(r"L::ITEM_FULL \+", kernel):
        line = kernel[kernel.rindex("\n", 0, m.start()):m.start()]
        if "!wait(" not in line and "mbar_arrive" not in line and "i >= " not in line:
            assert first(kernel, VOTE, m.end()) < first(kernel, r"return abort", m.end())


def test_lanes_of_a_product_warp_that_part_meet_again_at_a_vote(kernel):
    """A lane that gave up leaves the steps of an item by itself: nothing in them, nor on
    the way to the next item's vote, is done by the whole warp."""
    p0, p1 = products(kernel)
    text = kernel[p0:p1]
    loop = text.index("for (int k = k0 - stride; k < k1; ++k)")
    assert "(x = item(i)) != nullptr" in text[:loop]
    steps = text[text.index("bool q_here"):]
    assert not re.search(r"_sync\(|__syncwarp|elect_one|return", steps.replace("tc05_fence_after_sync(", "").replace("tc05_fence_before_sync(", ""))
    assert re.findall(r"if \(abort\) \w+", steps) == ["if (abort) break"]

"""CPU check, by reading, of how the second launch of attention of several new tokens
reads what the first one left."""
import re
from pathlib import Path

SOURCE = Path(__file__).resolve().parent.parent / "pagedattention_decode_paged_gb300" / "csrc" / "chunk_merge.cu"


def test_records_and_cuts_are_not_read_through_the_read_only_path():
    """The launch before writes them while this one may be resident (programmatic launch);
    the read-only path is for what nothing writes while a kernel lives.  The caller's
    own arrays are that."""
    text = re.sub(r"//[^\n]*", "", SOURCE.read_text())
    read_only = re.findall(r"__ldg\(([^;]*?)\)", text)
    assert read_only and all(re.match(r"p\.(lambdas|counts)\b", r) for r in read_only), read_only
    assert "__restrict__" not in text and "ld.global.nc" not in text
    # and nothing is read before the wait for that launch
    kernel = text[text.index("chunk_merge_kernel("):]
    assert kernel.index("grid_dependency_wait()") < kernel.index("p.cuts[") < kernel.index("__ldcg(")

"""What only the source shows of the paged-cache kernels."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_compression_fkv_b200", "csrc")


def test_decode_warps_leave_a_wait_together():
    """A wait that ends early (time, or another warp's abort) may end for some lanes
    and not for others, and a warp that goes on in two parts never meets its next
    whole-warp instruction: warps wait through warp_wait, whose lanes agree."""
    with open(os.path.join(CSRC, "paged_decode.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    assert "warp_wait(" in text
    assert not re.search(r"\bmbar_wait\s*\(", text)

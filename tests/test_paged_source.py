"""What the paged cache's kernels must have that no run shows reliably, checked in their source."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mtp_speculative_decoding_spec_gb300", "csrc")


def source(name):
    """Without comments."""
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_the_commit_joins_its_warps_before_the_aligned_barrier():
    """A loop by lanes stands before it, and an aligned barrier needs all lanes of a warp together."""
    assert re.search(r"__syncwarp\(\);\s+asm volatile\(\"barrier\.cluster\.arrive\.aligned;", source("paged/commit.cu"))

"""Kernels that read shared memory which bulk copies fill: an arrival that hands a
buffer back to the copying warp follows a fence between the reads and the copy
(without it the arrival may overtake reads whose values nothing has used yet).
Looked up in the sources: no GPU is needed."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_tiled_attention_17_gb300", "csrc")


@pytest.mark.parametrize("name,hand_backs", [("paged_decode.cu", 3), ("paged4_decode.cu", 2), ("decode.cu", 1)])
def test_reads_are_fenced_before_a_buffer_is_handed_back(name, hand_backs):
    with open(os.path.join(CSRC, name)) as f:
        lines = [re.sub(r"//.*", "", x).strip() for x in f]
    lines = [x for x in lines if x]
    at = [i for i, x in enumerate(lines) if re.search(r"mbar_arrive\(.*(EMPTY|empty0)", x)]
    assert len(at) == hand_backs
    for i in at:
        assert lines[i - 2:i] == ["fence_proxy_async_smem();", "__syncwarp();"], lines[i - 3:i + 1]

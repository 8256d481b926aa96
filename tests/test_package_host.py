"""The Python package on the host: a torch without a 4-bit type (no GPU is needed)."""
import os
import subprocess
import sys

from test_abi_host import lib  # noqa: F401  (the fixture builds the library)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_other_types_without_a_4_bit_type(lib):  # noqa: F811
    code = """
import torch
if hasattr(torch, "float4_e2m1fn_x2"):
    del torch.float4_e2m1fn_x2
import exact_tiled_attention_17_gb300 as eta
for dtype, code in ((torch.bfloat16, eta.ATTN_BF16), (torch.float32, eta.ATTN_F32)):
    assert eta.attn_paged_workspace_size(8, 2, 1, 64, dtype) == eta.attn_paged_workspace_size(8, 2, 1, 64, code) > 0
    try:
        eta.PagedCache.empty(1, 4, 2, 16, 64, 2, 4, dtype=dtype, device="cpu")
    except ValueError as e:
        assert "CUDA" in str(e)      # the pools were made; they have to be on a GPU
    else:
        raise AssertionError("a cache on the CPU")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

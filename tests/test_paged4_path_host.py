"""Which kernel an attention call over 4-bit values takes, as its workspace shows (no
GPU is needed)."""
import pytest

from test_abi_host import lib  # noqa: F401  (the fixture builds and loads the library)
from test_paged4_host import E2M1
from test_paged_host import ci, sz


def size(lib, g, max_q, d=128):  # noqa: F811
    f = lib.attn_paged_workspace_size
    f.restype, f.argtypes = sz, [ci] * 5
    return f(2 * g, 2, max_q, d, E2M1)


@pytest.mark.parametrize("d", [32, 64, 96, 128])
def test_at_most_two_units_to_the_stream_kernel(lib, d):  # noqa: F811
    chunks = size(lib, 4, 1000, d)
    stream = size(lib, 16, 1, d)
    assert 0 < size(lib, 4, 2, d) < stream < chunks
    for g, new in ((1, 32), (4, 8), (4, 5), (5, 6), (7, 4), (8, 4), (13, 2), (16, 2), (9, 2)):
        assert size(lib, g, new, d) == stream, (g, new)
    # (a unit holds whole tokens: 6 x 5 rows would be three)
    for g, new in ((6, 5), (9, 3), (10, 3), (11, 3), (3, 11), (16, 3), (17, 1), (64, 1), (1, 33)):
        assert size(lib, g, new, d) == chunks, (g, new)

"""The largest sizes of the paged cache's calls, as far as the host refuses them (no GPU needed)."""
import ctypes

import pytest

from test_kv_abi_cpu import LIB, append, layer, pytestmark, rb, refused  # noqa: F401


@pytest.mark.parametrize("rows", [(1 << 25) - 1, 1 << 25, (1 << 31) - 1])
def test_rows_that_a_launch_cannot_hold(rows):
    """Two rows a workgroup of 256 lanes: a launch of 2^32 lanes is no launch."""
    b = rb()
    refused(b.lib().replay_kv_append(ctypes.byref(layer()), append(rows=rows), None), b.ERR_SHAPE)

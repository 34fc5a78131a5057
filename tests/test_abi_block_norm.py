"""Host-side sizes of the block-norm junction (CPU only)."""
import pytest

import selective_state_space_42_b200 as ss
from selective_state_space_42_b200 import build as ssbuild


@pytest.fixture(scope="module")
def lib():
    ssbuild.build()
    return ss.load_library()


def test_gradient_workspace_grows_with_the_blocks_that_run(lib):
    """Two float32 rows a block, and no more blocks than rows of this width are worked
    on at a time: two an SM of 512 threads, up to eight of 128."""
    f, sms = lib.selscan_block_norm_bwd_workspace_bytes, 148
    for dim, per_sm in ((64, 8), (1024, 8), (2048, 4), (2560, 3), (4096, 2), (16384, 2)):
        assert f(1 << 20, dim) == sms * per_sm * 2 * dim * 4, dim
        assert f(7, dim) == 7 * 2 * dim * 4

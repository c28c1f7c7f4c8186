"""Limits of the paged calls' arguments, on the host before any launch (CPU only)."""
import pytest

from tests.test_paged_args import INVALID, WORKSPACE, attn, good_batch, good_params, good_pool, lib  # noqa: F401


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_longest_table(lib, page):  # noqa: F811
    """A table may end 4096 positions before 2^31, which is what the kernels'
    32-bit positions look ahead at most; the check that follows (of the
    workspace) is reached at that length and not behind it."""
    most = (2 ** 31 - 4096) // page
    p = good_params(page_size=page)
    assert attn(lib, p, good_batch(max_blocks=most), good_pool(), None) == WORKSPACE
    assert attn(lib, p, good_batch(max_blocks=most + 1), good_pool(), None) == INVALID

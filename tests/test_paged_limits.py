"""Limits of the paged calls' arguments, on the host before any launch (CPU only)."""
import ctypes

import pytest
import torch

from long_context_sparse_compress_b200 import lib as L
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


def test_plan_refuses_outputs_in_the_place_of_other_arrays(lib):  # noqa: F811
    """Lengths written over their inputs, say, or over an array's last number."""
    out = ctypes.c_size_t(0)
    assert lib.lcsc_page_plan_workspace_size(3, ctypes.byref(out)) == 0
    names = ("cached", "n_new", "table", "free", "n_free", "left", "ctx", "q_start", "slots", "pos")
    sizes = dict(cached=3, n_new=3, table=12, free=10, n_free=1, left=1, ctx=3, q_start=4, slots=5, pos=5)
    at, apart = 1 << 16, {}
    for name in names:
        apart[name], at = at, at + 4 * sizes[name]  # one right behind the other

    def call(**kw):
        a = {**apart, **kw}
        return lib.lcsc_page_plan(64, 3, 5, 4, 10, *(a[n] for n in names), 256, out.value, None, None)

    for i, a in enumerate(names):
        for b in names[:i]:
            if (a, b) in (("n_new", "cached"), ("n_free", "cached"), ("n_free", "n_new"), ("left", "n_free")):
                continue
            for shift in {0, 4 * (sizes[b] - 1)}:  # the same place, and the other's last number
                assert call(**{a: apart[b] + shift}) == INVALID, (a, b, shift)


def test_status_words_of_no_alignment(lib):  # noqa: F811
    """A device atomic on such an address would be a fault."""
    p, c, b = good_params(), good_pool(), good_batch()
    out = ctypes.c_size_t(0)
    assert lib.lcsc_page_plan_workspace_size(3, ctypes.byref(out)) == 0
    for status in (1, 2, 4098):
        assert lib.lcsc_paged_attn(ctypes.byref(p), ctypes.byref(b), ctypes.byref(c), 4096, 1 << 40, status, None) == INVALID
        assert lib.lcsc_paged_store(ctypes.byref(p), ctypes.byref(c), 16, 256, 32, 256, 16, 1, status, None) == INVALID
        assert lib.lcsc_page_plan(64, 3, 5, 4, 10, *(1 << k for k in range(10, 20)), 256, out.value, status, None) == INVALID


def test_document_ends(lib):  # noqa: F811
    """Their alignment, and in the Python layer their type and size."""
    assert attn(lib, good_params(), good_batch(doc_end=5), good_pool()) == INVALID
    assert attn(lib, good_params(), good_batch(doc_end=4), good_pool(), None) == WORKSPACE
    p, cache = L.paged_params(4, 2, 64, 16), L.PagedCache(3, 2, 16, 64, device="cpu")
    q, i = torch.zeros((5, 4, 64), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    for ends in (torch.zeros(5), torch.zeros(4, dtype=torch.int32), torch.zeros(5, dtype=torch.int64)):
        with pytest.raises(L.LcscError, match="doc_end"):
            L.paged_attn(p, q, cache, torch.zeros((2, 3), dtype=torch.int32), i, torch.zeros(3, dtype=torch.int32), 1,
                         torch.zeros_like(q), doc_end=ends)

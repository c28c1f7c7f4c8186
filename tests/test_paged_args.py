"""Refusals of the paged calls, on the host before any launch (CPU only)."""
import ctypes

import pytest
import torch

from long_context_sparse_compress_b200 import build
from long_context_sparse_compress_b200 import lib as L

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(L.LIB_PATH):
        build.build()
    return L.load()


def good_params(**kw):
    p = L.paged_params(8, 2, 128, 64)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


def good_pool(**kw):
    return L.PagedPool(**{**dict(k=256, v=512, k_scale=1024, v_scale=2048, n_pages=10), **kw})


def good_batch(**kw):
    d = dict(B=2, n_tokens=5, max_new=4, max_blocks=3, q_start=16, ctx_len=32, block_table=48, q=64, q_stride=1024,
             out=128)
    return L.PagedBatch(**{**d, **kw})


BAD_PARAMS = [
    (INVALID, dict(n_heads=0)), (INVALID, dict(n_kv_heads=0)), (INVALID, dict(n_kv_heads=3)),
    (INVALID, dict(n_kv_heads=-2)), (INVALID, dict(q_dtype=2)), (INVALID, dict(x_dtype=-1)),
    (INVALID, dict(sm_scale=0.0)), (INVALID, dict(sm_scale=float("nan"))), (INVALID, dict(sm_scale=float("inf"))),
    (INVALID, dict(window=-1)), (INVALID, dict(softcap=-1.0)), (INVALID, dict(softcap=float("nan"))),
    (INVALID, dict(softcap=float("inf"))), (INVALID, dict(softcap=1e-7)), (INVALID, dict(softcap=1.1e4)),
    (UNSUPPORTED, dict(page_size=8)), (UNSUPPORTED, dict(page_size=48)),
    (UNSUPPORTED, dict(page_size=256)), (UNSUPPORTED, dict(page_size=0)), (UNSUPPORTED, dict(head_dim=96)),
    (UNSUPPORTED, dict(head_dim=512))]

BAD_POOLS = [
    dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(k=8), dict(v=520), dict(k_scale=1026),
    dict(n_pages=0), dict(n_pages=-1), dict(n_pages=1 << 26)]

BAD_BATCHES = [
    dict(B=0), dict(B=(1 << 20) + 1), dict(n_tokens=-1), dict(n_tokens=1 << 28), dict(max_new=0), dict(max_blocks=0),
    dict(max_blocks=1 << 26), dict(q_start=None), dict(ctx_len=None), dict(block_table=None), dict(q_start=18),
    dict(lse=6), dict(slopes=1), dict(sink=2), dict(prefix_len=3), dict(doc_start=5), dict(q=None), dict(q=72),
    dict(q_stride=1000), dict(q_stride=1020), dict(q_stride=1028), dict(q_stride=-1024), dict(out=None), dict(out=132)]


def attn(lib, p, b, c, ws=4096, n=1 << 40):
    return lib.lcsc_paged_attn(p and ctypes.byref(p), b and ctypes.byref(b), c and ctypes.byref(c), ws, n, None, None)


@pytest.mark.parametrize("code,kw", BAD_PARAMS)
def test_parameters(lib, code, kw):
    p, out = good_params(**kw), ctypes.c_size_t(0)
    assert lib.lcsc_paged_attn_workspace_size(ctypes.byref(p), 2, 5, 4, ctypes.byref(out)) == code
    assert attn(lib, p, good_batch(), good_pool()) == code
    assert lib.lcsc_paged_store(ctypes.byref(p), ctypes.byref(good_pool()), 16, 256, 32, 256, 16, 1, None, None) == code


@pytest.mark.parametrize("kw", BAD_POOLS)
def test_pools(lib, kw):
    p, c = good_params(), good_pool(**kw)
    assert attn(lib, p, good_batch(), c) == INVALID
    assert lib.lcsc_paged_store(ctypes.byref(p), ctypes.byref(c), 16, 256, 32, 256, 16, 1, None, None) == INVALID


def test_pool_whose_rows_of_all_heads_pass_32_bits(lib):
    assert attn(lib, good_params(), good_batch(), good_pool(n_pages=(1 << 24) + 1)) == UNSUPPORTED


@pytest.mark.parametrize("kw", BAD_BATCHES)
def test_batches(lib, kw):
    assert attn(lib, good_params(), good_batch(**kw), good_pool()) == INVALID


def test_null_structs_and_small_workspaces(lib):
    p, out = good_params(), ctypes.c_size_t(0)
    assert attn(lib, None, good_batch(), good_pool()) == INVALID
    assert attn(lib, p, None, good_pool()) == INVALID
    assert attn(lib, p, good_batch(), None) == INVALID
    assert lib.lcsc_paged_attn_workspace_size(ctypes.byref(p), 2, 5, 4, None) == INVALID
    assert lib.lcsc_paged_attn_workspace_size(ctypes.byref(p), 2, 5, 4, ctypes.byref(out)) == 0
    for ws, n in ((None, 1 << 40), (4096 + 8, 1 << 40), (4096, out.value - 1)):
        assert attn(lib, p, good_batch(), good_pool(), ws, n) == WORKSPACE
    # nothing to do: no launch, whatever the row pointers
    assert attn(lib, p, good_batch(n_tokens=0, q=None, out=None), good_pool()) == 0
    assert lib.lcsc_paged_store(ctypes.byref(p), ctypes.byref(good_pool()), None, 0, None, 0, None, 0, None, None) == 0


def test_workspace_does_not_grow_with_lengths(lib):
    p, sizes = good_params(), []
    for B, n in ((1, 1), (64, 64), (4096, 100000)):
        sizes.append(L.paged_attn_workspace(p, B, n, 1))
    assert len(set(sizes)) == 1


@pytest.mark.parametrize("args", [
    (None, 256, 32, 256, 16, 3), (16, 256, None, 256, 16, 3), (24, 256, 32, 256, 16, 3), (16, 255, 32, 256, 16, 3),
    (16, 256, 32, 128, 16, 3), (16, 260, 32, 256, 16, 3), (16, 256, 32, 256, None, 3), (16, 256, 32, 256, 18, 3),
    (16, 256, 32, 256, 16, -1), (16, 256, 32, 256, 16, 1 << 31)])
def test_store_rows(lib, args):
    k, ks, v, vs, slots, n = args
    p = good_params()
    assert lib.lcsc_paged_store(ctypes.byref(p), ctypes.byref(good_pool()), k, ks, v, vs, slots, n, None, None) == INVALID


def test_plan_arguments(lib):
    out = ctypes.c_size_t(0)
    assert lib.lcsc_page_plan_workspace_size(0, ctypes.byref(out)) == INVALID
    assert lib.lcsc_page_plan_workspace_size((1 << 20) + 1, ctypes.byref(out)) == INVALID
    assert lib.lcsc_page_plan_workspace_size(3, None) == INVALID
    assert lib.lcsc_page_plan_workspace_size(3, ctypes.byref(out)) == 0
    good = dict(page=64, B=3, n_tokens=5, max_blocks=4, n_pages=10, cached=16, n_new=16, table=16, free=16, n_free=16,
                left=16, ctx=16, q_start=16, slots=16, pos=None, ws=256, size=out.value)

    def call(**kw):
        return lib.lcsc_page_plan(*{**good, **kw}.values(), None, None)

    for kw in (dict(page=24), dict(page=256)):
        assert call(**kw) == UNSUPPORTED
    for kw in (dict(B=0), dict(n_tokens=-1), dict(max_blocks=0), dict(n_pages=0), dict(max_blocks=1 << 26),
               dict(n_pages=1 << 26), dict(slots=None), dict(slots=18), dict(pos=2)):
        assert call(**kw) == INVALID, kw
    for name in ("cached", "n_new", "table", "free", "n_free", "left", "ctx", "q_start"):
        assert call(**{name: None}) == INVALID and call(**{name: 19}) == INVALID
    for kw in (dict(ws=None), dict(ws=264), dict(size=out.value - 1)):
        assert call(**kw) == WORKSPACE


def test_python_layer_refuses_what_it_cannot_pass_on(lib):
    p = L.paged_params(4, 2, 64, 16)
    cache = L.PagedCache(3, 2, 16, 64, device="cpu")
    x = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    slots = torch.zeros(5, dtype=torch.int32)
    for k, v, s in ((x.float(), x, slots), (x[:, :1], x, slots), (x[:4], x, slots), (x, x[:4], slots),
                    (x, x.transpose(1, 2).contiguous().transpose(1, 2), slots), (x, x, slots.long()),
                    (x, x, torch.zeros(10, dtype=torch.int32)[::2])):
        with pytest.raises(L.LcscError):
            L.paged_store(p, cache, k, v, s)
    with pytest.raises(L.LcscError, match="current CUDA device"):
        L.paged_store(p, cache, x, x, slots)
    with pytest.raises(L.LcscError, match="pages"):
        L.paged_store(L.paged_params(4, 2, 64, 32), cache, x, x, slots)
    with pytest.raises(L.LcscError):
        L.PagedCache.of(cache.k, cache.v[:2], cache.k_scale, cache.v_scale)
    with pytest.raises(L.LcscError):
        L.PagedCache.of(cache.k, cache.v, cache.k_scale.double(), cache.v_scale)
    q, i = torch.zeros((5, 4, 64), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    table, start = torch.zeros((2, 3), dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    good = dict(q=q, cache=cache, block_table=table, ctx_len=i, q_start=start, max_new=1, out=torch.zeros_like(q))
    bad = [dict(q=q.float()), dict(out=q.float()), dict(out=q[:4]), dict(block_table=table[0]),
           dict(block_table=table[:1]), dict(q_start=i), dict(ctx_len=i.long()), dict(lse=torch.zeros(5)),
           dict(lse=torch.zeros((5, 4), dtype=torch.float64)), dict(slopes=torch.zeros(3)), dict(sink=torch.zeros(2)),
           dict(prefix_len=start), dict(doc_start=i), {}]
    for kw in bad:
        with pytest.raises(L.LcscError):
            L.paged_attn(p, **{**good, **kw})
    with pytest.raises(L.LcscError):
        L.page_plan(16, i, i, table[:1], i, i[:1], i[:1], i, start, slots)


def test_tables_that_end_at_the_last_position(lib):
    """Positions are 32-bit numbers, and the kernels look some tiles ahead of the last one."""
    b = good_batch(max_blocks=(1 << 25) - 1)
    assert attn(lib, good_params(), b, good_pool()) == INVALID

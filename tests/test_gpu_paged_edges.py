"""Edges of the paged attention's calls that the tests beside it do not reach."""
import numpy as np
import pytest
import torch

from long_context_sparse_compress_b200 import lib as L
from oracle import formats, paged
from tests.test_gpu_paged import BF16, F32, Case, check_plan, i32, run_plan, status0

pytestmark = pytest.mark.gpu

FEW, MANY = 1, 17  # hints that choose the form of few and of many rows


def set_page(codes, scale, page, values):
    """Values [heads][tokens][D] into a page, stored by the scale rule."""
    s = np.vectorize(paged.scale_of)(np.abs(values).max((1, 2)))
    scale[page] = s
    codes[page] = formats.e4m3_encode(values / s[:, None, None])


# -------------------------------------------------------------------- plan

@pytest.mark.parametrize("width", [3, 70, 1200])
def test_ended_requests_whose_early_pages_were_released(cuda_lib, width):
    """Entries below 0 do not come back to the stack; the others do, in their order."""
    rng = np.random.default_rng(width)
    B, P = 70, 16
    cached = rng.integers(1, width * P + 1, B)
    n_new = np.where(np.arange(B) % 3 == 0, 2, -1)
    cached = np.where(n_new < 0, cached, np.minimum(cached, width * P - 2))
    have = -(-cached // P)
    table = np.full((B, width), -1)
    pages = iter(rng.permutation(int(have.sum()) + 100))
    for b in range(B):
        for col in range(have[b]):
            gone = n_new[b] < 0 and (col < have[b] // 2 if b % 2 else rng.random() < 0.3)
            table[b, col] = -1 if gone else next(pages)
    rest = list(pages)
    free = np.array(rest + [-3] * (int(have.sum()) + 100 - len(rest)))
    args = (P, cached, n_new, table, free, len(rest), int(np.maximum(n_new, 0).sum()))
    want = paged.Plan(*args)
    assert not want.no_pages and -1 not in want.free[:len(rest)]
    got = run_plan(*args)
    top = len(rest) + int(((table >= 0) & (n_new < 0)[:, None]).sum())
    got["free"][top:] = i32(want.free[top:])  # above the stack
    check_plan(got, want)


# ------------------------------------------------------------------- store

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("P,holes", [(16, 1), (128, 1), (128, 100)])
def test_store_skips_what_comes_behind_a_hole_in_a_page(cuda_lib, dtype, P, holes):
    """Rows of a page behind skipped ones would be a second visit beside the
    first, with a scale of its own: they are skipped and reported; other pages
    behind skipped rows are stored."""
    rng = np.random.default_rng(P + holes)
    slots = np.concatenate([[3 * P + 1, 3 * P + 2], [-1] * holes, 3 * P + 3 + holes + np.arange(4) % (P - 3 - holes),
                            [-1], np.arange(5 * P, 6 * P), [-1] * 130, [2 * P + 5]]).astype(np.int32)
    x = torch.from_numpy(rng.standard_normal((len(slots), 2, 64)).astype(np.float32)).to(dtype)
    x[2 + holes:6 + holes] *= 64
    codes, scale = (rng.integers(0, 0x7E, (7, 2, P, 64)).astype(np.uint8), np.exp2(rng.integers(-9, 3, (7, 2))).astype(np.float32))
    cache = L.PagedCache.of(*(torch.from_numpy(codes).cuda() for _ in "kv"), *(torch.from_numpy(scale).cuda() for _ in "kv"))
    st = status0()
    L.paged_store(L.paged_params(2, 2, 64, P, x_dtype="f32" if dtype == F32 else "bf16"), cache, x.cuda(), x.cuda(),
                  i32(slots), status=st)
    assert st.item() == L.DEV_BAD_INDEX
    slots[2 + holes:6 + holes] = -1
    paged.store(codes, scale, x.float().numpy(), slots, P)
    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        assert np.array_equal(s.cpu().numpy(), scale) and np.array_equal(c.cpu().numpy(), codes)


# ------------------------------------------------------- V scales far apart

@pytest.mark.parametrize("dtype,form,ratio", [(F32, FEW, 2.0 ** -30)] + [
    (BF16, f, 2.0 ** -r) for f, rs in ((FEW, (3, 8, 12, 20, 60)), (MANY, (8, 12, 20))) for r in rs])
@pytest.mark.parametrize("hidden", [False, True])
def test_pages_of_small_values_beside_large_ones(cuda_lib, dtype, form, ratio, hidden):
    """Two pages of one tile, V of one `ratio` times the other's.  The large
    one's keys weigh nothing (scores 2 x 22 below), or are hidden from most rows
    by the documents while the first row sees them: the small one's values
    come out with their own precision, not that of the neighbour's."""
    P, D, H, n = 32, 128, 2, 5
    c = Case([64, 64], [n, n], 2 * H, H, D, P, dtype, seed=31)
    rng = np.random.default_rng(6)
    small = np.array([[0, 1], [1, 0]])  # request b's small page: its second, its first
    vsmall = 0.0
    for b in range(2):
        for col in range(2):
            page, is_small = c.table[b, col], col == small[b, 1]
            K = rng.standard_normal((H, P, D)) * 0.5
            if not hidden:
                K[..., 0] = 16.0 if is_small else -16.0
            V = rng.standard_normal((H, P, D)) * (ratio if is_small else 1.0)
            set_page(c.k, c.ks, page, K)
            set_page(c.v, c.vs, page, V)
            if is_small:
                vsmall = max(vsmall, np.abs(V).max() * 1.1)
    q = c.q.float()
    if not hidden:
        q[..., 0] = 16.0
    c.q = q.to(dtype)
    kw = {}
    if hidden:  # request 0's rows but the first see its second page only; request 1's see everything
        docs = np.zeros(c.N, np.int32)
        docs[1:n] = P
        kw["docs"] = docs
    c.run(max_new=form, **kw)
    torch.cuda.synchronize()
    assert c.status.item() == 0
    want, lse, dot, _ = paged.attention(q.to(dtype).float().numpy(), c.k, c.v, c.ks, c.vs, c.table, c.ctx, c.q_start,
                                        np.float32(D ** -0.5), **kw)
    rows = slice(1, n) if hidden else slice(0, 2 * n)
    got = c.out.double().cpu().numpy()[rows]
    want, dot = want[rows], dot[rows]
    # score errors as in Case.check; a weight's: half a step of its 11 bits
    # (2^-11) and of its third E4M3 term (2^-12), and what lies below the terms'
    # last step (2^-17 of the row's largest, for each of 32 keys: 2^-12)
    ds = (D + 8) * 2.0 ** -24 * dot / D ** 0.5 + 2.0 ** -21 * (1 + dot / D ** 0.5)
    dp = 0.0
    if dtype == BF16:
        ds = ds + 2.0 ** -17 * dot / D ** 0.5
        dp = 2.0 ** -11 + 2.0 ** -12 + 2.0 ** -12
    tol = (2 * ds + dp + 64 * 2.0 ** -24)[..., None] * vsmall + np.abs(want) * torch.finfo(dtype).eps / 2
    err = np.abs(got - want)
    assert np.abs(want).max() < 2 * vsmall  # the neighbour's share is nothing
    assert (err <= tol).all(), float((err / tol).max())


def test_pages_of_zeros_beside_others(cuda_lib):
    """A page of zeros has the least scale there is."""
    for form in (FEW, MANY):
        c = Case([190, 64], [1, 3], 4, 2, 64, 16, BF16, seed=32)
        for page in (c.table[0, 3], c.table[0, 4], c.table[1, 0]):
            set_page(c.v, c.vs, page, np.zeros((2, 16, 64)))
        c.run(max_new=form).check()


# --------------------------------------------------- one key above very many

@pytest.mark.parametrize("gap", [16, 18])
@pytest.mark.parametrize("form,rows", [(FEW, 1), (MANY, 1), (MANY, 130)])
def test_a_key_that_outweighs_very_many(cuda_lib, form, rows, gap):
    """2^17 equal keys `gap` below two others of no value, walked by one CTA as
    one piece (a request for each CTA, all over the same pages): what the many
    add up to is kept."""
    n, P, D = 1 << 17, 128, 64
    B = torch.cuda.get_device_properties(0).multi_processor_count * (2 if form == FEW else 1)
    k, v = (torch.zeros((n // P, 1, P, D), dtype=torch.uint8) for _ in range(2))
    v.fill_(int(formats.e4m3_encode(np.float32(1.0))))
    top = int(formats.e4m3_encode(np.float32(gap)))
    assert formats.e4m3_decode(np.uint8(top)) == gap
    for page in (0, 1):  # key 0 of the first and of the second tile
        k[page, 0, 0, 0], v[page, 0, 0] = top, 0
    one = torch.ones((n // P, 1))
    cache = L.PagedCache.of(*(x.cuda() for x in (k, v, one, one)))
    p = L.paged_params(1, 1, D, P)
    q = torch.zeros((B * rows, 1, D), dtype=BF16)
    q[..., 0] = 8.0  # 8 * gap / sqrt(D) = gap
    out, lse, st = torch.zeros_like(q).cuda(), torch.zeros((B * rows, 1)).cuda(), status0()
    table = torch.arange(n // P, dtype=torch.int32).repeat(B, 1).cuda()
    L.paged_attn(p, q.cuda(), cache, table, i32([n] * B), i32(np.arange(B + 1) * rows), form if rows == 1 else rows, out,
                 lse, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    others = n - rows + np.arange(rows) + 1 - 2.0  # keys that row i sees beside the two
    den = 2 + others * np.exp(-float(gap))
    want = others * np.exp(-float(gap)) / den
    got = out.double().cpu().numpy().reshape(B, rows, D)
    # a weight's half step: 2^-11 of it, or 2^-25 over 2^7 (or more) of the row's largest,
    # for each of n keys over a sum of 2; the products' float32 sums, which add 16
    # keys at a time (n / 16 steps of 2^-23: 2^-10) and the weights' own (a step a
    # tile: 2^-13); the output's rounding.  Three E4M3 terms lose 2^-12 more.
    tol = want * (2.0 ** -11 + 2.0 ** -10 + 2.0 ** -13 + 2.0 ** -9 + (2.0 ** -12 if form == FEW else 0)) + n * 2.0 ** -32 / 2
    err = np.abs(got - want[None, :, None])
    assert (err <= tol[None, :, None]).all(), (float(got.mean()), float(want.mean()))
    d = np.abs(lse.double().cpu().numpy().reshape(B, rows) - float(gap) - np.log(den))
    assert d.max() <= 2.0 ** -13


# --------------------------------------------- queries near the least magnitude

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new,form", [([1, 3], FEW), ([1, 3], MANY), ([60, 30], 60)])
def test_queries_near_the_least_magnitude(cuda_lib, dtype, new, form):
    """Queries down to subnormal numbers against keys near the largest."""
    c = Case([150, 40], new, 8, 2, 64, 16, dtype, seed=33)
    small = 2.0 ** -np.array([119, 121, 123, 124, 125, 126, 128, 130.0])
    c.q = (c.q.float() * torch.from_numpy(small).float()[None, :, None]).to(dtype)
    c.ks *= np.float32(2.0 ** 120)
    c.run(max_new=form).check()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new,form", [([1, 3], FEW), ([1, 3], MANY), ([160, 200], 200)])
@pytest.mark.parametrize("exponent", [16, 24, 27, 34, 60])
def test_scores_of_any_size(cuda_lib, dtype, new, form, exponent):
    """Scores of 2^18 to 2^62: the softmax is all on the largest, and what is
    left of float32's bits decides which, but it is a number."""
    c = Case([1500, 240], new, 8, 2, 64, 16, dtype, seed=39)
    c.ks *= np.float32(2.0 ** exponent)
    c.run(max_new=form).check()
    live = int(c.q_start[-1])
    assert torch.isfinite(c.out[:live]).all() and torch.isfinite(c.lse[:live]).all()
    assert (c.out[:live].float().abs().amax(2) > 0).all()


# ------------------------------------------------- what no query of a step sees

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("new", [[1, 4], [40, 30]])
def test_documents_pass_over_released_pages(cuda_lib, dtype, new):
    """Pages before every row's document may be gone from the table."""
    c = Case([300, 500], new, 8, 2, 128, 16, dtype, seed=34)
    docs = np.repeat([150, 333], new).astype(np.int32)
    docs = np.concatenate([docs, np.zeros(c.N - len(docs), np.int32)])
    table = c.table.copy()
    table[0, :150 // 16], table[1, :333 // 16] = -1, c.n_pages + 5
    c.run(table=table, docs=docs).check(docs=docs)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("new", [[1, 4], [40, 30]])
@pytest.mark.parametrize("mask", ["window", "docs"])
def test_rows_of_a_page_before_the_first_visible_may_hold_anything(cuda_lib, dtype, new, mask):
    c = Case([300, 500], new, 8, 2, 128, 64, dtype, seed=35)
    if mask == "window":
        kw, first = dict(window=40), [max(0, t - n + 1 - 40) for t, n in zip(c.ctx, new)]
    else:
        first = [150, 333]
        docs = np.repeat(first, new).astype(np.int32)
        kw = dict(docs=np.concatenate([docs, np.zeros(c.N - len(docs), np.int32)]))
    for b, lo in enumerate(first):
        assert lo % 64
        for codes in (c.k, c.v):
            codes[c.table[b, lo // 64], :, :lo % 64] = 0x7F
    c.run(**kw).check(**kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("new", [[1, 4, 2], [40, 30, 2]])
@pytest.mark.parametrize("behind", [0, 5, 1 << 30])
def test_requests_whose_documents_begin_behind_the_last_token(cuda_lib, dtype, new, behind):
    """They see nothing, also where what lies behind the last token is in its tile and page."""
    c = Case([300, 500, 100], new, 8, 2, 128, 128, dtype, seed=38)
    docs = np.zeros(c.N, np.int32)
    docs[:new[0]] = 300 + behind
    docs[new[0] + new[1]:] = 100 + behind
    kw = dict(docs=docs, sink=np.linspace(-3, 3, 8).astype(np.float32))
    c.run(**kw).check(**kw)
    c.run(docs=docs).check(docs=docs)


# ------------------------------------------------------- documents with an end

def run_with_ends(c, ends, max_new=None, table=None, **kw):
    c.run(max_new=max_new, table=table, **kw)
    c.out.fill_(77), c.lse.fill_(77), c.status.zero_()
    L.paged_attn(*c.pos, **{**c.args, "doc_end": i32(ends)})
    return c.check(ends=ends, **kw)


@pytest.mark.parametrize("dtype,cap", [(F32, 5.0), (BF16, 0.0), (BF16, 5.0)])
@pytest.mark.parametrize("Hq,Hkv,D,P", [(12, 4, 64, 16), (8, 1, 128, 128)])
def test_packed_documents_with_ends_under_a_prefix(cuda_lib, dtype, cap, Hq, Hkv, D, P):
    """No query sees another document, however far the prefix goes; blocks of
    rows whose documents end tiles before the prefix does, chunks that begin
    inside a document, single tokens and requests without new ones."""
    new = [700, 1, 0, 257, 300] if dtype == BF16 else [150, 1, 0, 57, 60]
    ctx = np.array([700, 900, 40, 300, 700] if dtype == BF16 else [150, 400, 40, 90, 260])
    c = Case(ctx, new, Hq, Hkv, D, P, dtype, seed=41)
    pos = np.concatenate([t - n + np.arange(n) for t, n in zip(ctx, new)] + [np.zeros(c.N - sum(new), int)])
    every = np.repeat([40, 333, 7, 90, 257], new)
    every = np.concatenate([every, np.full(c.N - len(every), 9)])
    starts = (pos // every * every).astype(np.int32)
    ends = (starts + every).astype(np.int32)
    for prefix in (ctx, ctx // 2):
        kw = dict(docs=starts, prefix=prefix.astype(np.int32), cap=cap)
        run_with_ends(c, ends, **kw)
        run_with_ends(c, ends, window=33, sink=np.linspace(-2, 2, Hq).astype(np.float32), **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("new", [[5, 5, 3, 1], [130, 60, 3, 1]])
@pytest.mark.parametrize("docs", [False, True])
def test_ends_anywhere(cuda_lib, dtype, new, docs):
    """Ends before the query, before the first token, behind the last one and at
    the type's least and largest numbers, with starts and without."""
    c = Case([140, 300, 60, 7], new, 10, 2, 64, 16, dtype, seed=42)
    rng = np.random.default_rng(9)
    ends = rng.integers(-20, 330, c.N).astype(np.int64)
    ends[rng.random(c.N) < 0.1] = 2 ** 31 - 1
    ends[rng.random(c.N) < 0.1] = -2 ** 31
    ends[c.q_start[2]:c.q_start[3]] = -2 ** 31  # a request that sees nothing
    kw = dict(prefix=rng.integers(0, 330, 4).astype(np.int32), sink=rng.standard_normal(10).astype(np.float32),
              slopes=np.exp2(-np.arange(10.0)).astype(np.float32))
    if docs:
        kw["docs"] = rng.integers(-5, 200, c.N).astype(np.int32)
    run_with_ends(c, ends.astype(np.int32), **kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("new", [[4, 5], [60, 70]])
def test_ends_pass_over_pages_behind_them(cuda_lib, dtype, new):
    """Pages behind every row's document may be missing, under a prefix that goes on."""
    c = Case([300, 500], new, 8, 2, 128, 16, dtype, seed=43)
    ends = np.concatenate([np.repeat([100, 333], new), np.zeros(c.N - sum(new), int)]).astype(np.int32)
    table = c.table.copy()
    table[0, -(-100 // 16):19], table[1, -(-333 // 16):32] = -1, c.n_pages + 5
    run_with_ends(c, ends, table=table, prefix=np.array([300, 480], np.int32))


# -------------------------------------------------------- parts of a batch

@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_call_for_each_kind_of_request(cuda_lib, dtype):
    """Decodes and prompts of one batch in calls of their own, over slices of its
    arrays: each writes its requests' rows and no other."""
    c = Case([300, 170, 65, 200, 90], [1, 1, 1, 130, 77], 8, 2, 128, 32, dtype, seed=44)
    prefix = np.array([0, 100, 0, 150, 90], np.int32)
    c.run(prefix=prefix).check(prefix=prefix)
    p, q, cache, table, ctx, q_start, _, out = c.pos
    for first, last, hint in ((3, 5, 130), (0, 3, 1)):
        out.fill_(77), c.lse.fill_(77), c.status.zero_()
        L.paged_attn(p, q, cache, table[first:last], ctx[first:last], q_start[first:last + 1], hint, out, c.lse,
                     prefix_len=c.args["prefix_len"][first:last], status=c.status)
        rows = slice(int(c.q_start[first]), int(c.q_start[last]))
        kept, kept_lse = out[rows].clone(), c.lse[rows].clone()
        out[rows], c.lse[rows] = 77, 77
        assert (out == 77).all() and (c.lse == 77).all()
        c.run(prefix=prefix, max_new=hint)  # the whole batch in the same form
        torch.cuda.synchronize()
        c.out[rows], c.lse[rows] = kept, kept_lse
        c.check(prefix=prefix)
        p, q, cache, table, ctx, q_start, _, out = c.pos


# ------------------------------------------------------------------- sinks

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("new", [[1, 1, 1], [40, 3, 30]])
def test_sinks_of_any_size(cuda_lib, dtype, new):
    """The largest and least values of the type, and none (minus infinity), of
    rows that see something and of rows that see nothing."""
    big = float(np.finfo(np.float32).max)
    c = Case([3000, 40, 64], new, 8, 2, 64, 16, dtype, seed=36)
    docs = np.zeros(c.N, np.int32)
    docs[c.q_start[1]:c.q_start[2]] = 1 << 30
    kw = dict(sink=np.array([big, -big, -np.inf, 2.5e38, 3e38, -3e38, 80.0, 0.0], np.float32), docs=docs)
    c.run(**kw).check(**kw)


# -------------------------------------------------------------- workspaces

def test_a_workspace_of_the_call_belongs_to_its_stream(cuda_lib):
    """Memory that a call takes for itself is not given to another stream while
    the call may still run."""
    c = Case([400, 300], [3, 1], 8, 2, 64, 16, BF16, seed=37).run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ints = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    plan = (16, i32([5, 0]), i32([1, 3]), i32([[0, -1], [-1, -1]]), i32([1, 2, 3]), i32([3]), ints(1), ints(2), ints(3),
            ints(4))
    torch.cuda.synchronize()
    for call in (lambda: L.paged_attn(*c.pos, **{**c.args, "ws": None, "stream": s}),
                 lambda: L.page_plan(*plan, stream=s)):
        ws = call()
        at, n = ws.data_ptr(), ws.numel()
        del ws
        again = [L.workspace(n) for _ in range(4)]
        assert at not in [x.data_ptr() for x in again]
        s.synchronize()
    c.check()


# ------------------------------------------------------------ failure path

@pytest.mark.parametrize("stall", [True, False])
@pytest.mark.parametrize("new", [[1, 1, 1], [1, 30, 3], [90, 60, 5]])
def test_waits_that_give_up_at_once(cuda_lib, new, stall):
    """A limit of a nanosecond ends roles while copies and products of their CTA
    are in flight; each CTA waits for those, and the next call is right."""
    c = Case([3000, 400, 7000], new, 8, 2, 128, 64, BF16, seed=30)
    c.run().check()
    for _ in range(20):
        L.set_wait_test(1, stall)
        try:
            c.run()
            torch.cuda.synchronize()
        finally:
            L.set_wait_test(0, False)
        assert c.status.item() in ((L.DEV_TIMEOUT,) if stall else (0, L.DEV_TIMEOUT))
    c.run().check()

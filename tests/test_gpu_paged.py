"""The paged 8-bit cache on the GPU against the oracle: plan, store, attention
(every form, mask and layout) and a run of them together."""
import numpy as np
import pytest
import torch

from long_context_sparse_compress_b200 import lib as L
from oracle import formats, paged

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


def i32(v):
    return torch.as_tensor(np.asarray(v, np.int32)).cuda()


def status0():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# -------------------------------------------------------------------- plan

def run_plan(page, cached, n_new, table, free, n_free, n_tokens, in_place=False):
    d = dict(table=i32(table), free=i32(free), ctx=i32([-7] * len(cached)), q_start=i32([-7] * (len(cached) + 1)),
             slots=i32([-7] * n_tokens), pos=i32([-7] * n_tokens), n_free=i32([n_free]), status=status0())
    d["left"] = d["n_free"] if in_place else i32([-7])
    L.page_plan(page, i32(cached), i32(n_new), d["table"], d["free"], d["n_free"], d["left"], d["ctx"], d["q_start"],
                d["slots"], d["pos"], status=d["status"])
    return d


def check_plan(d, want):
    for name, w in (("ctx", want.ctx), ("q_start", want.q_start), ("table", want.table), ("free", want.free),
                    ("slots", want.slots), ("pos", want.pos), ("left", [want.n_free])):
        assert np.array_equal(d[name].cpu().numpy(), w), name
    assert d["status"].item() == (2 if want.bad_length else 0) + (16 if want.no_pages else 0)


@pytest.mark.parametrize("B,page,top,spare", [(1, 16, 40, 0), (7, 16, 100, 5), (37, 64, 700, -40), (1025, 32, 90, 100),
                                              (2100, 128, 9, -200), (3, 128, 6000, 9)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_matches_oracle(cuda_lib, B, page, top, spare, in_place):
    rng = np.random.default_rng(B + page)
    cached = rng.integers(0, top, B)
    n_new = np.where(rng.random(B) < 0.2, -1, rng.integers(0, top, B))
    width = -(-2 * top // page)
    have = -(-cached // page)
    need = np.where(n_new < 0, 0, -(-(cached + np.maximum(n_new, 0)) // page) - have).sum()
    back = have[n_new < 0].sum()
    n_free = max(0, int(need + spare - back))  # spare < 0: the pages do not reach every request
    pool = n_free + int(have.sum())
    order = rng.permutation(max(pool, 1))
    table = np.full((B, width), -1)
    at = n_free
    for b in range(B):
        table[b, :have[b]] = order[at:at + have[b]]
        at += have[b]
    free = np.full(max(pool, 1), -3)
    free[:n_free] = order[:n_free]
    n_tokens = int(np.maximum(n_new, 0).sum()) + 17
    want = paged.Plan(page, cached, n_new, table, free, n_free, n_tokens)
    d = run_plan(page, cached, n_new, table, free, n_free, n_tokens, in_place)
    check_plan(d, want)
    if not in_place:  # the same call again gives the same plan
        L.page_plan(page, i32(cached), i32(n_new), d["table"], d["free"], d["n_free"], d["left"], d["ctx"],
                    d["q_start"], d["slots"], d["pos"], status=d["status"])
        check_plan(d, want)


def test_plan_refusals_on_the_device(cuda_lib):
    """Lengths past the table, rows past the arrays, negative counts, a stack
    that would grow past the pool."""
    table = np.full((5, 2), -1)
    table[4, 0] = 3
    args = (16, [0, -5, 0, 0, 4], [33, 2, 3, 9, 1], table, [0, 1, 2, 3, 4], 3, 47)
    want = paged.Plan(*args)
    assert want.bad_length and want.ctx.tolist() == [0, 0, 3, 9, 0]
    check_plan(run_plan(*args), want)
    table = np.array([[5, 6, 7]])  # three pages back onto a stack of two in a pool of four
    d = run_plan(16, [40], [-1], table, [0, 1, 2, 3], 2, 0)
    assert d["left"].item() == 4 and d["status"].item() == 1 and d["free"].tolist() == [0, 1, 5, 6]
    d = run_plan(16, [0], [5], np.full((1, 1), -1), [77, 1], 1, 5)  # a page outside the pool on the stack
    assert d["status"].item() == 1 and (d["slots"] == -1).all()


# ------------------------------------------------------------------- store

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("D,P,H,runs", [
    (128, 64, 2, [(0, 64), (64 + 63, 1), (128, 3), (131, 61 + 64)]),
    (64, 16, 3, [(5, 11), (16, 16), (33, 1), (50, 2)]),
    (128, 128, 1, [(1, 127), (128, 128), (256 + 9, 100)]),
    (64, 32, 1, [(i * 32 + (7 * i) % 32, 1) for i in range(40)]),
    (128, 16, 2, [(i * 48 + i % 16, 30) for i in range(60)])])
def test_store_matches_oracle(cuda_lib, dtype, D, P, H, runs):
    rng = np.random.default_rng(D + P + len(runs))
    n_pages = max(a + n for a, n in runs) // P + 2
    slots = np.concatenate([np.arange(a, a + n) for a, n in runs] + [[-1, -1]]).astype(np.int32)
    if len(runs) == 40:  # padded rows between the runs too
        slots = np.insert(slots, [3, 17], [-1, -1]).astype(np.int32)
    N = len(slots)
    x = {}
    for name in "kv":
        r = rng.standard_normal((N, H, D)) * np.exp2(rng.integers(-9, 9, (N, H, 1)))
        r[rng.random((N, H)) < 0.1] = 0
        x[name] = torch.from_numpy(r.astype(np.float32)).to(dtype)
    codes = {n: rng.integers(0, 0x7E, (n_pages, H, P, D)).astype(np.uint8) for n in "kv"}
    scale = {n: np.exp2(rng.integers(-12, 3, (n_pages, H))).astype(np.float32) for n in "kv"}
    cache = L.PagedCache.of(*(torch.from_numpy(codes[n]).cuda() for n in "kv"),
                            *(torch.from_numpy(scale[n]).cuda() for n in "kv"))
    # K and V rows are slices of one wider array
    pad = torch.zeros((N, 1, D), dtype=dtype)
    both = torch.cat([pad, x["k"], pad, x["v"]], 1).cuda()
    st = status0()
    p = L.paged_params(H, H, D, P, x_dtype="f32" if dtype == F32 else "bf16")
    L.paged_store(p, cache, both[:, 1:1 + H], both[:, 2 + H:], i32(slots), status=st)
    assert st.item() == 0
    for n, got, gs in (("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale)):
        paged.store(codes[n], scale[n], x[n].float().numpy(), slots, P)
        assert np.array_equal(gs.cpu().numpy(), scale[n])
        assert np.array_equal(got.cpu().numpy(), codes[n])


def test_store_extremes(cuda_lib):
    """Zeros, subnormal and largest values, values that are not finite, slots out
    of order or outside the pool."""
    D, P = 64, 16
    rows = np.zeros((8, 1, D), np.float32)
    rows[1, 0, 0], rows[1, 0, 1] = 3e38, -1.0
    rows[2, 0, 0] = 1e-42
    rows[3, 0, :3] = [np.nan, np.inf, 2.0]
    rows[4:] = 1.5
    cache = L.PagedCache(6, 1, P, D)
    p = L.paged_params(1, 1, D, P, x_dtype="f32")
    st, x = status0(), torch.from_numpy(rows).cuda()
    L.paged_store(p, cache, x, x, i32([0, 16, 32, 48, 64, 64, 65, 6 * 16]), status=st)
    assert st.item() == L.DEV_RANGE | L.DEV_BAD_INDEX
    assert cache.k_scale[:, 0].tolist() == [2.0 ** -100, paged.scale_of(np.float32(3e38)), 2.0 ** -100, 2.0 ** -7,
                                            paged.scale_of(1.5), 1.0]
    assert formats.e4m3_decode(cache.k[3, 0, 0, :4].cpu().numpy()).tolist() == [0, 0, 256, 0]
    assert (cache.k[4, 0, 0].cpu() == int(formats.e4m3_encode(np.float32(384)))).all()
    assert (cache.k[4, 0, 1:] == 0).all() and (cache.k[5] == 0).all()  # the second 64, and 65 after it, are skipped
    assert torch.equal(cache.k, cache.v)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("P,n", [(128, 100), (64, 64), (16, 16), (32, 5)])
def test_store_of_values_that_are_not_finite(cuda_lib, dtype, P, n):
    """They are stored as zeros, left out of the scale and reported, in runs of every length."""
    rng = np.random.default_rng(P)
    x = torch.from_numpy(rng.standard_normal((n, 2, 128)).astype(np.float32)).to(dtype)
    for i, v in enumerate((float("nan"), float("inf"), -float("inf"), -float("nan"))):
        x[i, 0, 5 + 31 * i] = v
    cache = L.PagedCache(2, 2, P, 128)
    p, st = L.paged_params(2, 2, 128, P, x_dtype="f32" if dtype == F32 else "bf16"), status0()
    clean = torch.nan_to_num(x.float(), 0, 0, 0).to(dtype)
    L.paged_store(p, cache, x.cuda(), clean.cuda(), i32(np.arange(n)), status=st)
    assert st.item() == L.DEV_RANGE
    assert torch.equal(cache.k, cache.v) and torch.equal(cache.k_scale, cache.v_scale)
    codes, scale = np.zeros((2, 2, P, 128), np.uint8), np.ones((2, 2), np.float32)
    paged.store(codes, scale, x.float().numpy(), np.arange(n), P)
    assert np.array_equal(cache.k.cpu().numpy(), codes) and np.array_equal(cache.k_scale.cpu().numpy(), scale)


# --------------------------------------------------------------- attention

class Case:
    """Requests with random caches, lengths and masks; the pool's other bytes
    and the pages' tails hold garbage, NaN codes among it."""

    def __init__(self, ctx, new, Hq, Hkv, D, P, dtype, seed=0, spread=3, q_mul=2.0, pad=3):
        rng = np.random.default_rng(seed)
        self.ctx, self.new = np.asarray(ctx), np.asarray(new)
        B = len(ctx)
        self.Hq, self.Hkv, self.D, self.P, self.dtype = Hq, Hkv, D, P, dtype
        self.q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.N = int(self.q_start[-1]) + pad  # rows behind the last request
        used = [max(0, -(-int(c) // P)) for c in ctx]
        self.n_pages = sum(used) + 2
        order = rng.permutation(self.n_pages)
        self.table = np.full((B, max(used + [1]) + 1), -1, np.int32)
        at = 0
        self.k, self.v = (rng.integers(0, 256, (self.n_pages, Hkv, P, D)).astype(np.uint8) for _ in range(2))
        self.ks, self.vs = (np.full((self.n_pages, Hkv), np.nan, np.float32) for _ in range(2))
        for b, u in enumerate(used):
            pages = order[at:at + u]
            at += u
            self.table[b, :u] = pages
            for c, s in ((self.k, self.ks), (self.v, self.vs)):
                live = u * P if u == 0 else int(ctx[b])
                val = rng.standard_normal((u, Hkv, P, D)) * np.exp2(rng.integers(-spread, spread + 1, (u, Hkv, 1, 1)))
                sc = np.vectorize(paged.scale_of)(np.abs(val).max((2, 3))) if u else np.zeros((0, Hkv))
                s[pages] = sc
                code = formats.e4m3_encode(val / sc[:, :, None, None]) if u else np.zeros((0, Hkv, P, D), np.uint8)
                keep = (np.arange(u * P) < live).reshape(u, 1, P, 1)
                c[pages] = np.where(keep, code, c[pages])
        q = rng.standard_normal((self.N, Hq, D)) * q_mul
        self.q = torch.from_numpy(q.astype(np.float32)).to(dtype)
        self.rng = rng

    def run(self, cache=None, max_new=None, wide=False, stream=None, ws=None, p=None, table=None, **kw):
        name = "f32" if self.dtype == F32 else "bf16"
        self.p = L.paged_params(self.Hq, self.Hkv, self.D, self.P, q_dtype=name,
                                window=kw.get("window", 0), softcap=kw.get("cap", 0.0))
        self.cache = cache or L.PagedCache.of(*(torch.from_numpy(x).cuda() for x in (self.k, self.v, self.ks, self.vs)))
        q = self.q.cuda()
        if wide:  # the queries are a slice of a wider projection
            q = torch.cat([q, q + 1, q[:, :1]], 1)[:, :self.Hq]
        self.out = torch.full((self.N, self.Hq, self.D), 77.0, dtype=self.dtype, device="cuda")
        self.lse = torch.full((self.N, self.Hq), 77.0, device="cuda")
        self.status = status0()
        f = lambda n: None if kw.get(n) is None else torch.as_tensor(np.asarray(kw[n], np.float32)).cuda()
        g = lambda n: None if kw.get(n) is None else i32(kw[n])
        self.args = dict(lse=self.lse, slopes=f("slopes"), sink=f("sink"), prefix_len=g("prefix"), doc_start=g("docs"),
                         status=self.status, ws=ws, stream=stream)
        self.pos = (self.p, q, self.cache, i32(self.table if table is None else table), i32(self.ctx),
                    i32(self.q_start), max_new or max(1, int(self.new.max())), self.out)
        L.paged_attn(*self.pos, **self.args)
        return self

    def check(self, status=0, table=None, **kw):
        torch.cuda.synchronize()
        assert self.status.item() == status
        scale = self.D ** -0.5
        want, lse, dot, vmax = paged.attention(
            self.q.float().numpy(), self.k, self.v, self.ks, self.vs, self.table if table is None else table, self.ctx,
            self.q_start, np.float32(scale), **kw)
        live = int(self.q_start[-1])
        assert (self.out[live:] == 77).all() and (self.lse[live:] == 77).all()
        got, got_lse = self.out[:live].double().cpu().numpy(), self.lse[:live].double().cpu().numpy()
        want, lse, dot, vmax = want[:live], lse[:live], dot[:live], vmax[:live]
        # bound of a score's error: D products and their sums in float32 (half a
        # step 2^-24 each, on sums of at most `dot`), its scale, cap, bias and
        # exponential (2^-21 in all, times the score's and the bias' size); the
        # bf16 query's E4M3 terms add 2^-17 of its largest value per key value
        n = max(self.ctx.max(), 1)
        size = scale * dot + (np.max(kw["slopes"]) * n if kw.get("slopes") is not None else 0)
        ds = (self.D + 8) * 2.0 ** -24 * scale * dot + 2.0 ** -21 * (1 + size)
        dp = 0.0
        if self.dtype == BF16:
            ds = ds + 2.0 ** -17 * scale * dot
            dp = 2.0 ** -11 + 2.0 ** -16  # the weights, and V's terms against the largest |V|
        # |out' - out| <= (2 ds + dp + sums of up to n terms) max |V|, then one rounding
        tol = (2 * ds + dp + n * 2.0 ** -24)[..., None] * vmax[..., None]
        tol = tol + np.abs(want) * torch.finfo(self.dtype).eps / 2 + 1e-30
        err = np.abs(got - want)
        assert (err <= tol).all(), (np.unravel_index(np.argmax(err / tol), err.shape), float((err / tol).max()))
        empty = np.isneginf(lse)
        assert np.array_equal(np.isneginf(got_lse), empty)
        assert (got[empty] == 0).all()
        d = np.abs(got_lse - lse)[~empty]
        lim = (ds + (n + 8) * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(np.where(empty, 0, lse))))[~empty]
        assert (d <= lim).all(), float((d / lim).max())
        return self


LAYOUTS = [  # Hq, Hkv, D, page
    (1, 1, 128, 64), (8, 8, 64, 16), (8, 1, 128, 16), (6, 2, 128, 32), (64, 8, 128, 64), (20, 4, 64, 128),
    (16, 1, 64, 32), (32, 1, 128, 128), (64, 1, 128, 64), (40, 2, 64, 16)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Hq,Hkv,D,P", LAYOUTS)
def test_decode_lengths(cuda_lib, dtype, Hq, Hkv, D, P):
    """One new token per request, at lengths around every tile and page border."""
    ctx = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200, 257, 391]
    Case(ctx, [1] * len(ctx), Hq, Hkv, D, P, dtype, seed=Hq + D).run().check()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Hq,Hkv,D,P", [(8, 1, 128, 16), (6, 2, 64, 32), (16, 2, 128, 64)])
def test_decode_long(cuda_lib, dtype, Hq, Hkv, D, P):
    """Requests long enough to be split over many CTAs, beside short ones."""
    Case([9000, 1, 3333], [1, 1, 1], Hq, Hkv, D, P, dtype, seed=5).run().check()


MASKS = {
    "plain": {}, "window1": dict(window=1), "window100": dict(window=100), "cap": dict(cap=4.0),
    "slopes": dict(slopes=True), "sink": dict(sink=True), "prefix": dict(prefix=True), "docs": dict(docs=True),
    "all": dict(window=90, cap=30.0, slopes=True, sink=True, prefix=True, docs=True),
}


def mask_args(c, kw):
    kw = dict(kw)
    rng = np.random.default_rng(8)
    if kw.get("slopes"):
        kw["slopes"] = np.exp2(-8.0 * np.arange(1, c.Hq + 1) / c.Hq).astype(np.float32)
    if kw.get("sink"):
        kw["sink"] = rng.standard_normal(c.Hq).astype(np.float32) * 3
    if kw.get("prefix"):
        kw["prefix"] = rng.integers(0, c.ctx.max() + 20, len(c.ctx)).astype(np.int32)
    if kw.get("docs"):  # some documents start after their query: those rows see nothing
        kw["docs"] = rng.integers(-5, c.ctx.max() + 40, c.N).astype(np.int32)
    return kw


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("mask", sorted(MASKS))
@pytest.mark.parametrize("Hq,Hkv,D,P", [(8, 2, 128, 64), (10, 2, 64, 16)])
def test_draft_tokens_with_masks(cuda_lib, dtype, mask, Hq, Hkv, D, P):
    c = Case([5, 140, 300, 7], [5, 5, 3, 1], Hq, Hkv, D, P, dtype, seed=11)
    kw = mask_args(c, MASKS[mask])
    c.run(wide=True, **kw).check(**kw)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("mask", sorted(MASKS))
@pytest.mark.parametrize("Hq,Hkv,D,P", [(4, 2, 128, 32), (6, 1, 64, 128), (8, 1, 128, 16)])
def test_prompts_with_masks(cuda_lib, dtype, mask, Hq, Hkv, D, P):
    """Chunks of prompts beside single tokens and a request without new ones."""
    c = Case([150, 70, 90, 33], [97, 1, 0, 33], Hq, Hkv, D, P, dtype, seed=12)
    kw = mask_args(c, MASKS[mask])
    c.run(wide=True, **kw).check(**kw)


@pytest.mark.parametrize("cap", [0.0, 5.0])
@pytest.mark.parametrize("Hq,Hkv,D,P", [(12, 4, 64, 16), (64, 1, 128, 128), (16, 2, 128, 32)])
def test_packed_documents(cuda_lib, Hq, Hkv, D, P, cap):
    """Whole prompts of packed documents, whose blocks of rows begin at later and
    later tiles of keys; a document at a block's first and last token, one that
    starts behind every key, and requests without documents of their own."""
    new = [700, 1, 0, 257, 64, 1000]
    c = Case([700, 900, 40, 300, 64, 1000], new, Hq, Hkv, D, P, BF16, seed=21)
    rng = np.random.default_rng(3)
    docs, every = [], (40, 1, 1, 257, 5000, 333)
    for b, n in enumerate(new):
        pos = int(c.ctx[b]) - n + np.arange(n)
        docs.append(pos // every[b] * every[b])
    docs = np.concatenate(docs + [np.zeros(c.N - sum(new), int)]).astype(np.int32)
    docs[int(c.q_start[5]) + 256:int(c.q_start[5]) + 512] = 1 << 30
    prefix = rng.integers(0, 400, len(new)).astype(np.int32)
    c.run(docs=docs).check(docs=docs)
    kw = dict(docs=docs, prefix=prefix, cap=cap, window=150)
    c.run(**kw).check(**kw)


@pytest.mark.parametrize("cap", [0.0, 5.0])
@pytest.mark.parametrize("G,D,P", [(8, 128, 64), (5, 64, 16), (20, 128, 32)])
def test_many_short_prompts(cuda_lib, G, D, P, cap):
    """Several short items a CTA, of one and two tiles of rows in turn, each a
    single tile of keys; again and again with the same result."""
    n = np.random.default_rng(G).integers(1, 41, 70)
    c = Case(n, n, 8 * G, 8, D, P, BF16, seed=22)
    c.run(cap=cap).check(cap=cap)
    first, lse = c.out.clone(), c.lse.clone()
    for _ in range(20):
        c.run(cap=cap)
        torch.cuda.synchronize()
        assert torch.equal(c.out, first) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_what_ran_before_changes_no_bit(cuda_lib, dtype, new):
    """Capped scores of lengths that end inside a tile, after calls that leave
    small and large keys behind the last one in the shared memory."""
    ctx = np.random.default_rng(new).integers(40, 700, 60)
    c = Case(ctx, [new] * 60, 10, 2, 64, 16, dtype, seed=23)
    prefix = np.random.default_rng(4).integers(0, 900, 60).astype(np.int32)
    kw = dict(cap=5.0, prefix=prefix)
    c.run(**kw).check(**kw)
    first, lse = c.out.clone(), c.lse.clone()
    other = [Case([900] * 4, [new] * 4, 10, 2, 64, 16, dtype, seed=i, spread=1 + 5 * i) for i in range(2)]
    for i in range(20):
        other[i % 2].run()
        c.run(**kw)
        torch.cuda.synchronize()
        assert torch.equal(c.out, first) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("new", [[1, 1, 1, 1], [70, 5, 60, 1]])
def test_bad_pages_lengths_and_absent_requests(cuda_lib, dtype, new):
    """A page number outside the pool hides its tokens; ctx_len 0 takes no part;
    lengths that do not fit give zeros; each sets its bit."""
    c = Case([200, 65, 60, 130], new, 4, 2, 128, 16, dtype, seed=13)
    table = c.table.copy()
    table[0, 3], table[0, 11], table[3, 0] = -1, c.n_pages, 1 << 30
    c.run(table=table).check(status=L.DEV_BAD_INDEX, table=table)
    whole = c.ctx.copy()
    c.ctx = np.array([200, 0, 60, 130])
    c.run().check()
    for bad in (-3, 16 * c.table.shape[1] + 1) + ((4,) if max(new) > 1 else ()):
        c.ctx = np.array([200, bad, 60, 130])
        c.run()
        c.ctx = np.array([200, 0, 60, 130])
        c.check(status=L.DEV_BAD_LENGTH)
    c.ctx = whole
    # rows of a q_start that falls or passes the array are left as they were
    q_start = c.q_start.copy()
    c.q_start = q_start.copy()
    c.q_start[-1] = c.N + 1
    c.run()
    torch.cuda.synchronize()
    assert c.status.item() == L.DEV_BAD_LENGTH and (c.out[q_start[-2]:] == 77).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_window_passes_over_released_pages(cuda_lib, dtype):
    """Pages left of every window may be gone from the table."""
    c = Case([300, 500], [1, 4], 8, 2, 128, 16, dtype, seed=14)
    table = c.table.copy()
    table[0, :(300 - 40) // 16], table[1, :(500 - 4 - 40) // 16] = -1, c.n_pages + 5
    c.run(table=table, window=40).check(window=40)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("new", [[1, 1], [40, 30]])
def test_caps_far_above_and_below_the_scores(cuda_lib, dtype, new):
    """A cap of ten thousand nearly changes nothing, and is not to cost precision; one
    far below the scores leaves little more than their signs."""
    c = Case([190, 64], new, 8, 2, 128, 16, dtype, seed=22)
    c.run(cap=1e4).check(cap=1e4)
    c.run(cap=0.25).check(cap=0.25)


def test_page_scales_far_apart(cuda_lib):
    """Neighbouring pages whose scales differ by 2^40, the small ones weighing most."""
    for dtype in (F32, BF16):
        c = Case([190, 64], [1, 40], 4, 1, 128, 16, dtype, seed=15, spread=20, q_mul=0.001)
        c.run().check()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_hint_does_not_change_what_is_computed(cuda_lib, dtype):
    """max_new chooses the form only: a wrong one still gives every row its result."""
    c = Case([150, 40, 90], [60, 2, 17], 8, 2, 128, 64, dtype, seed=16)
    for hint in (1, 5, 60, 4000):
        c.run(max_new=hint).check()


def test_many_short_requests(cuda_lib):
    rng = np.random.default_rng(2)
    ctx = rng.integers(0, 50, 700)
    c = Case(ctx, np.minimum(ctx, 1), 2, 1, 64, 16, BF16, seed=17)
    c.run().check()


def test_repeats_streams_graphs_and_two_calls_at_once(cuda_lib):
    a = Case([3000, 77, 900], [1, 1, 1], 16, 2, 128, 64, BF16, seed=18).run()
    b = Case([400, 300], [130, 60], 8, 2, 64, 16, BF16, seed=19).run()
    torch.cuda.synchronize()
    first = [(c.out.clone(), c.lse.clone()) for c in (a, b)]
    sizes = [L.paged_attn_workspace(c.p, len(c.ctx), c.N, int(c.new.max())) for c in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [L.workspace(n) for n in sizes]

    def both():
        for c, s, ws in zip((a, b), streams, spaces):
            L.paged_attn(*c.pos, **{**c.args, "ws": ws, "stream": s})

    for _ in range(20):  # two calls at once, each with its workspace
        both()
    torch.cuda.synchronize()
    graphs = []
    for c, s, ws in zip((a, b), streams, spaces):
        c.out.fill_(77)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            L.paged_attn(*c.pos, **{**c.args, "ws": ws})
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for c, (out, lse) in zip((a, b), first):
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
        c.check()


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_serving_steps(cuda_lib, dtype):
    """Requests come, decode, end and make room for others: every step planned,
    stored and attended on the device, against the oracle's own state."""
    rng = np.random.default_rng(21)
    B, P, Hq, Hkv, D, pool, width = 5, 16, 6, 2, 64, 40, 12
    td = F32 if dtype == "f32" else BF16
    p = L.paged_params(Hq, Hkv, D, P, q_dtype=dtype, x_dtype=dtype, softcap=20.0)
    cache = L.PagedCache(pool, Hkv, P, D)
    ok, ov = (np.zeros((pool, Hkv, P, D), np.uint8) for _ in range(2))
    oks, ovs = (np.ones((pool, Hkv), np.float32) for _ in range(2))
    table, free, n_free = i32(np.full((B, width), -1)), i32(rng.permutation(pool)), i32([pool])
    cached = np.zeros(B, np.int64)
    steps = [[50, 3, 0, 1, 17], [1, 1, 1, 1, 1], [1, -1, 40, 5, 1], [1, 120, 1, -1, 1], [1, 1, 1, 90, 1], [3, 1, -1, 1, 1]]
    for n_new in steps:
        n_new = np.array(n_new)
        n_tokens = int(np.maximum(n_new, 0).sum()) + 2
        want = paged.Plan(P, cached, n_new, table.cpu().numpy(), free.cpu().numpy(), n_free.item(), n_tokens)
        ctx, q_start, slots = i32(np.zeros(B)), i32(np.zeros(B + 1)), i32(np.zeros(n_tokens))
        st = status0()
        L.page_plan(P, i32(cached), i32(n_new), table, free, n_free, n_free, ctx, q_start, slots, status=st)
        k, v, q = (torch.from_numpy(rng.standard_normal((n_tokens, h, D)).astype(np.float32)).to(td)
                   for h in (Hkv, Hkv, Hq))
        L.paged_store(p, cache, k.cuda(), v.cuda(), slots, status=st)
        out = torch.zeros((n_tokens, Hq, D), dtype=td, device="cuda")
        L.paged_attn(p, q.cuda(), cache, table, ctx, q_start, int(n_new.max()), out, status=st)
        torch.cuda.synchronize()
        assert st.item() == 0
        assert np.array_equal(ctx.cpu().numpy(), want.ctx) and np.array_equal(slots.cpu().numpy(), want.slots)
        assert n_free.item() == want.n_free and np.array_equal(table.cpu().numpy(), want.table)
        for x, codes, scale in ((k, ok, oks), (v, ov, ovs)):
            paged.store(codes, scale, x.float().numpy(), want.slots, P)
        assert np.array_equal(cache.k.cpu().numpy(), ok) and np.array_equal(cache.v_scale.cpu().numpy(), ovs)
        ref, _, _, vmax = paged.attention(q.float().numpy(), ok, ov, oks, ovs, want.table, want.ctx, want.q_start,
                                          np.float32(D ** -0.5), cap=20.0)
        live = want.q_start[-1]
        eps = torch.finfo(td).eps / 2
        err = np.abs(out.double().cpu().numpy()[:live] - ref[:live])
        # one rounding of the output, and the weights' and scores' errors of the attention tests' bound
        assert (err <= np.abs(ref[:live]) * eps + (2.0 ** -10 if td == BF16 else 2.0 ** -16) * vmax[:live, :, None]).all()
        cached = np.where(n_new < 0, 0, cached + np.maximum(n_new, 0))


# ------------------------------------------------------------ failure path

@pytest.mark.parametrize("new", [[1, 1], [1, 30], [90, 60]])
def test_wait_runs_out_then_recovers(cuda_lib, new):
    """A bounded wait of the tensor-core forms that runs out (only that: every
    CTA ends by itself) is reported, and the next call is right."""
    c = Case([3000, 400], new, 8, 2, 128, 64, BF16, seed=20)
    L.set_wait_test(20_000_000, True)
    try:
        c.run()
        torch.cuda.synchronize()
        assert c.status.item() == L.DEV_TIMEOUT
    finally:
        L.set_wait_test(0, False)
    c.run().check()

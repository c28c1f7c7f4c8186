"""Cases of the paged 8-bit cache operators: the plan of a serving step
(block tables and slot maps from request lengths), the store of new K and V
rows and the attention over the cached tokens.

``run`` computes a case in plain torch operations, or, where ``own`` is true,
makes the library's calls.  Lengths, document starts and the like follow from
the case alone; values and the order of the pages follow from the seed.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
SCALE_FLOOR = -100  # least exponent of a page scale


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a small server: every request adds a token
        dict(name="plan_decode_16", op="plan", B=16, page=64, lo=1, hi=8192, new="one", pool=2048),
        # a busy server's step: prompts beside decodes, some requests have ended, short pages
        dict(name="plan_mixed_512", op="plan", B=512, page=16, lo=0, hi=32768, new="mixed", pool=1048576),
        # the tokens of a decode step join partly filled pages
        dict(name="store_decode_16", op="store", B=16, page=64, Hkv=8, D=128, lo=1, hi=8192, new="one", x="bf16"),
        # four prompt chunks of 4096 tokens
        dict(name="store_chunk_4x4096", op="store", B=4, page=64, Hkv=8, D=128, lo=0, hi=8192, new="chunk4096", x="bf16"),
        # short prompts and decodes in float32, short pages, an odd count of heads
        dict(name="store_mixed_f32", op="store", B=37, page=16, Hkv=3, D=64, lo=0, hi=900, new="mixed", x="f32"),
        # one request in float32 at 4096 tokens, a KV head for each of 8 heads
        dict(name="attn_decode_4k_f32", op="attn", B=1, page=64, Hq=8, Hkv=8, D=128, q="f32", lo=4096, hi=4096,
             new="one", window=0, cap=0.0, bias=False, sink=False, prefix=False, docs=False),
        # a sliding-window layer's decode step: 128 tokens, a sink logit for each head
        dict(name="attn_window_16", op="attn", B=16, page=64, Hq=64, Hkv=8, D=128, q="bf16", lo=3, hi=8192,
             new="one", window=128, cap=0.0, bias=False, sink=True, prefix=False, docs=False),
        # plain decode of a batch of long requests
        dict(name="attn_decode_16_64k", op="attn", B=16, page=64, Hq=64, Hkv=8, D=128, q="bf16", lo=16384, hi=65536,
             new="one", window=0, cap=0.0, bias=False, sink=False, prefix=False, docs=False),
        # one request at a million tokens, all heads on one KV head, scores capped
        dict(name="attn_decode_1m_mqa", op="attn", B=1, page=128, Hq=64, Hkv=1, D=128, q="bf16", lo=1048576,
             hi=1048576, new="one", window=0, cap=30.0, bias=False, sink=False, prefix=False, docs=False),
        # five draft tokens to verify, a bias by distance
        dict(name="attn_draft5_8_32k", op="attn", B=8, page=32, Hq=64, Hkv=8, D=128, q="bf16", lo=9000, hi=32768,
             new="five", window=0, cap=0.0, bias=True, sink=False, prefix=False, docs=False),
        # a prompt chunk of 4096 tokens on a context of 4096
        dict(name="attn_chunk_4096", op="attn", B=1, page=64, Hq=64, Hkv=8, D=128, q="bf16", lo=8192, hi=8192,
             new="chunk4096", window=0, cap=0.0, bias=False, sink=False, prefix=False, docs=False),
        # packed documents with a bidirectional prefix, half-size heads, short pages, odd lengths
        dict(name="attn_docs_prefix", op="attn", B=5, page=16, Hq=12, Hkv=4, D=64, q="bf16", lo=11, hi=3001,
             new="whole", window=0, cap=50.0, bias=False, sink=True, prefix=True, docs=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "store", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        B = _log(rng, 1, 512)
        hi = _log(rng, 2, 32768)
        new = rng.choice(["one", "five", "mixed", "whole"])
        return dict(op=op, B=B, page=page, lo=0, hi=hi, new=new, pool=B * ((hi + 5) // page + 2) + rng.randint(0, 99))
    Hkv = rng.choice([1, 2, 3, 4, 8])
    D = rng.choice([64, 128])
    if op == "store":
        hi = _log(rng, 5, 8192)
        B = _log(rng, 1, max(2, min(64, 32768 // hi)))
        return dict(op=op, B=B, page=page, Hkv=Hkv, D=D, lo=rng.randint(0, hi // 2), hi=hi,
                    new=rng.choice(["one", "five", "mixed", "whole"]), x=rng.choice(["bf16", "bf16", "f32"]))
    G = rng.choice([1, 2, 4, 5, 8, 16])
    new = rng.choice(["one", "one", "five", "whole", "mixed"])
    hi = _log(rng, 5, 65536) if new in ("one", "five") else _log(rng, 5, 4096)
    B = _log(rng, 1, max(2, min(32, 262144 // hi if new in ("one", "five") else 8192 // hi)))
    q = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if q == "f32" and new in ("whole", "mixed"):
        hi, B = min(hi, 1024), min(B, 4)
    return dict(op=op, B=B, page=page, Hq=Hkv * G, Hkv=Hkv, D=D, q=q, lo=rng.randint(min(hi, 5), hi), hi=hi, new=new,
                window=rng.choice([0, 0, 128, 2048, rng.randint(1, 300)]), cap=rng.choice([0.0, 0.0, 30.0, 50.0]),
                bias=rng.random() < 0.3, sink=rng.random() < 0.4, prefix=rng.random() < 0.3,
                docs=rng.random() < 0.3)


def lengths(case):
    """(tokens cached before the step, new tokens) of each request; -1 new
    tokens: the request has ended."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k in ("op", "B", "page", "lo", "hi", "new"))))
    cached, fresh = [], []
    for _ in range(case["B"]):
        total = r.randint(case["lo"], case["hi"])
        if case["new"] == "one":
            n = 1
        elif case["new"] == "five":
            n = 5
        elif case["new"] == "whole":
            n = total
        elif case["new"].startswith("chunk"):
            n = int(case["new"][5:])
            total = max(total, n)
        else:  # mixed: mostly single tokens, prompts of up to 512, a few requests that ended
            kind = r.random()
            n = 1 if kind < 0.7 else r.randint(1, 512) if kind < 0.9 or case["op"] != "plan" else -1
        n = min(n, max(total, 1))
        cached.append(max(total - max(n, 0), 0))
        fresh.append(n)
    return cached, fresh


# ----------------------------------------------------------------- inputs

def _pow2_scale(amax):
    """The least power of two s with amax <= 448 s (not below 2^-100)."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, SCALE_FLOOR)).clamp(min=SCALE_FLOOR)
    return torch.ldexp(torch.ones_like(amax), e)


def _tables(case, g, cached, total, n_pages):
    """Block table over a random order of the pages; places not in use hold -1."""
    P = case["page"]
    width = max(1, max(-(-t // P) for t in total))
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    used = torch.tensor([-(-c // P) for c in cached], device="cuda")
    start = torch.cumsum(used, 0) - used
    col = torch.arange(width, device="cuda")
    at = (start[:, None] + col).clamp(max=n_pages - 1)
    table = torch.where(col < used[:, None], order[at], torch.full_like(order[at], -1))
    return table.contiguous(), order, int(used.sum())


def _rows(g, n, heads, D, dtype, spread):
    """Rows whose heads differ in size, as projections' heads do."""
    x = torch.randn((n, heads, D), generator=g, device="cuda")
    s = torch.exp2(torch.rand((heads, 1), generator=g, device="cuda") * spread - spread / 2)
    return (x * s).to(dtype)


def _filled(g, pages, Hkv, P, D, live):
    """Codes and scales of `pages` pages, of which the first live[i] tokens of page i hold values."""
    codes = torch.zeros((pages, Hkv, P, D), dtype=torch.uint8, device="cuda")
    scale = torch.full((pages, Hkv), 2.0 ** SCALE_FLOOR, device="cuda")
    step = max(1, (1 << 26) // (Hkv * P * D))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        x = torch.randn((n, Hkv, P, D), generator=g, device="cuda")
        x *= torch.exp2(torch.rand((n, Hkv, 1, 1), generator=g, device="cuda") * 2 - 1)
        x *= (torch.arange(P, device="cuda") < live[a:a + n, None])[:, None, :, None]
        s = _pow2_scale(x.abs().amax((2, 3)))
        codes[a:a + n] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scale[a:a + n] = s
    return codes, scale


def _live(table, counts, P, n_pages):
    """Tokens held by each page, from the block table and the tokens of each request."""
    col = torch.arange(table.shape[1], device="cuda")
    held = (counts[:, None] - col * P).clamp(0, P)
    live = torch.zeros(n_pages, dtype=torch.int64, device="cuda")
    ok = (table >= 0) & (held > 0)
    live[table[ok].long()] = held[ok]
    return live


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    cached, fresh = lengths(case)
    P, B = case["page"], case["B"]
    total = [c + max(n, 0) for c, n in zip(cached, fresh)]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    st = dict(case=case, cached=i32(cached), fresh=i32(fresh))
    N = sum(max(n, 0) for n in fresh)
    st["N"] = N
    if case["op"] == "plan":
        table, order, used = _tables(case, g, cached, total, case["pool"])
        width = table.shape[1]
        st["table"] = table
        st["free"] = torch.cat([order[used:], order[:used] * 0 - 1]).contiguous()
        st["n_free"] = i32([case["pool"] - used])
        if own:
            from long_context_sparse_compress_b200 import lib as L
            st["ws"] = L.workspace(L.page_plan_workspace(B))
            new = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")
            st.update(L=L, ctx=new(B), q_start=new(B + 1), slots=new(N), pos=new(N), left=new(1))
        assert width * P >= max(total)
        return st
    # every request's pages, those of the new tokens among them, in a random order of the pool
    n_pages = sum(-(-t // P) for t in total) + 3
    table, _, _ = _tables(case, g, total, total, n_pages)
    st["table"] = table
    st["ctx"] = i32(total)
    st["q_start"] = i32([0] + [sum(fresh[:i + 1]) for i in range(B)])
    Hkv, D = case["Hkv"], case["D"]
    held = torch.tensor(cached if case["op"] == "store" else total, device="cuda")
    live = _live(table, held, P, n_pages)
    st["k"], st["k_scale"] = _filled(g, n_pages, Hkv, P, D, live)
    st["v"], st["v_scale"] = _filled(g, n_pages, Hkv, P, D, live)
    if case["op"] == "store":
        dt = torch.float32 if case["x"] == "f32" else torch.bfloat16
        # K and V rows are slices of one projection's output
        both = torch.cat([_rows(g, N, Hkv, D, dt, 4.0), _rows(g, N, Hkv, D, dt, 4.0)], 1)
        st["x_k"], st["x_v"] = both[:, :Hkv], both[:, Hkv:]
        req = torch.repeat_interleave(torch.arange(B, device="cuda"), st["fresh"].long())
        pos = torch.arange(N, device="cuda") - st["q_start"][:-1].long()[req] + st["cached"].long()[req]
        st["slots"] = (table[req, pos // P].long() * P + pos % P).to(torch.int32)
    else:
        Hq = case["Hq"]
        dt = torch.float32 if case["q"] == "f32" else torch.bfloat16
        st["q"] = _rows(g, N, Hq, D, dt, 3.0)
        st["max_new"] = max(fresh)
        st["slopes"] = (torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq).float().contiguous()
                        if case["bias"] else None)
        st["sink"] = torch.randn(Hq, generator=g, device="cuda") if case["sink"] else None
        r = random.Random(B * 131 + case["hi"])
        st["prefix"] = i32([r.randint(0, t) for t in total]) if case["prefix"] else None
        st["docs"] = None
        if case["docs"]:  # a document starts every so many tokens of each request
            per = [max(1, t // r.randint(1, 4)) for t in total]
            req = torch.repeat_interleave(torch.arange(B, device="cuda"), st["fresh"].long())
            pos = torch.arange(N, device="cuda") - st["q_start"][:-1].long()[req] + st["cached"].long()[req]
            every = torch.tensor(per, device="cuda")[req]
            st["docs"] = (pos // every * every).to(torch.int32)
    if own:
        from long_context_sparse_compress_b200 import lib as L
        st["L"] = L
        st["cache"] = L.PagedCache.of(st["k"], st["v"], st["k_scale"], st["v_scale"])
        if case["op"] == "store":
            st["p"] = L.paged_params(Hkv, Hkv, D, P, x_dtype=case["x"])
        else:
            st["p"] = L.paged_params(case["Hq"], Hkv, D, P, q_dtype=case["q"], window=case["window"],
                                     softcap=case["cap"])
            st["ws"] = L.workspace(L.paged_attn_workspace(st["p"], B, N, st["max_new"]))
            st["out"] = torch.empty_like(st["q"])
            st["lse"] = torch.empty((N, case["Hq"]), device="cuda")
    return st


# -------------------------------------------------------------------- run

def run(state):
    op = state["case"]["op"]
    if own:
        return {"plan": _own_plan, "store": _own_store, "attn": _own_attn}[op](state)
    return {"plan": _plan, "store": _store, "attn": _attn}[op](state)


def _own_plan(st):
    st["L"].page_plan(st["case"]["page"], st["cached"], st["fresh"], st["table"], st["free"], st["n_free"], st["left"],
                      st["ctx"], st["q_start"], st["slots"], st["pos"], ws=st["ws"])
    return {k: st[k] for k in ("ctx", "q_start", "slots", "pos", "table", "free", "left")}


def _own_store(st):
    st["L"].paged_store(st["p"], st["cache"], st["x_k"], st["x_v"], st["slots"])
    return _stored(st)


def _own_attn(st):
    st["L"].paged_attn(st["p"], st["q"], st["cache"], st["table"], st["ctx"], st["q_start"], st["max_new"], st["out"],
                       st["lse"], slopes=st["slopes"], sink=st["sink"], prefix_len=st["prefix"], doc_start=st["docs"],
                       ws=st["ws"])
    return {"out": st["out"], "lse": st["lse"]}


def _stored(st):
    e4m3 = torch.float8_e4m3fn
    return {"k": st["k"].view(e4m3), "v": st["v"].view(e4m3), "k_scale": st["k_scale"], "v_scale": st["v_scale"]}


def _plan(st):
    P, N = st["case"]["page"], st["N"]
    table, free = st["table"], st["free"]
    cached, fresh = st["cached"].long(), st["fresh"].long()
    B, width = table.shape
    ended = fresh < 0
    new = fresh.clamp(min=0)
    col = torch.arange(width, device="cuda")
    have = (cached + P - 1) // P
    # the pages of ended requests go on top of the free ones
    back = ended[:, None] & (col < have[:, None])
    given = torch.where(ended, have, 0)
    n_free = st["n_free"].long()
    place = n_free + (torch.cumsum(given, 0) - given)[:, None] + col
    free[place[back]] = table[back]
    top = n_free + given.sum()
    # pages from the top, in request order; a request that they do not reach takes no part
    q_end = torch.cumsum(new, 0)
    fits = ~ended & (cached + new <= width * P) & (q_end <= N)
    need = torch.where(fits, (cached + new + P - 1) // P - have, 0)
    upto = torch.cumsum(need, 0)
    part = fits & ((need == 0) | (upto <= top))
    take = part[:, None] & (col >= have[:, None]) & (col < (have + need)[:, None])
    order = (upto - need)[:, None] + col - have[:, None]
    table[take] = free[(top - 1 - order)[take]]
    left = top - torch.where(part, need, 0).sum()
    ctx = torch.where(part, cached + new, 0)
    q_start = torch.cat([torch.zeros_like(q_end[:1]), q_end])
    row = torch.arange(N, device="cuda")
    req = torch.searchsorted(q_end, row, right=True).clamp(max=B - 1)
    pos = row - q_start[req] + cached[req]
    live = part[req] & (row < q_end[-1])
    page = table[req, (pos // P).clamp(max=width - 1)].long()
    slots = torch.where(live, page * P + pos % P, -1)
    pos = torch.where(live, pos, -1)
    i32 = lambda x: x.to(torch.int32)
    return {"ctx": i32(ctx), "q_start": i32(q_start), "slots": i32(slots), "pos": i32(pos), "table": table, "free": free,
            "left": i32(left)}


def _store_one(x, codes, scale, page, off):
    x = x.float()
    fresh = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda")
    fresh[page[off == 0]] = True
    new = torch.where(fresh[:, None], 0.0, scale)
    new = new.index_reduce(0, page, _pow2_scale(x.abs().amax(2)), "amax")
    touched = torch.unique(page)
    ratio = torch.where(fresh[:, None], 1.0, scale / new)[touched]
    old = codes[touched].view(torch.float8_e4m3fn).float() * ratio[:, :, None, None]
    codes[touched] = old.to(torch.float8_e4m3fn).view(torch.uint8)
    codes[page, :, off] = (x / new[page][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    scale[touched] = new[touched]


def _store(st):
    P = st["case"]["page"]
    slots = st["slots"].long()
    _store_one(st["x_k"], st["k"], st["k_scale"], slots // P, slots % P)
    _store_one(st["x_v"], st["v"], st["v_scale"], slots // P, slots % P)
    return _stored(st)


def _gathered(codes, scale, table):
    """The cached values of every request, [B][Hkv][tokens][D]."""
    x = codes[table].view(torch.float8_e4m3fn).float() * scale[table][..., None, None]
    B, n, H, P, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, H, n * P, D)


def _attn(st):
    c = st["case"]
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    G, T, dt = Hq // Hkv, st["max_new"], st["q"].dtype
    table = st["table"].long().clamp(min=0)
    L, q0 = st["ctx"].long(), st["q_start"].long()
    n = q0[1:] - q0[:-1]
    B = L.shape[0]
    i = torch.arange(T, device="cuda")
    row = q0[:-1, None] + i  # [B][T]
    live = i < n[:, None]
    row = torch.where(live, row, 0)
    q = st["q"][row].float().reshape(B, T, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, D)
    s = torch.matmul(q, _gathered(st["k"], st["k_scale"], table).transpose(2, 3)).view(B, Hkv, G, T, -1)
    s *= 1.0 / math.sqrt(D)
    if c["cap"]:
        s = c["cap"] * torch.tanh(s / c["cap"])
    pos = (L - n)[:, None] + i  # [B][T]
    j = torch.arange(s.shape[-1], device="cuda")
    if c["bias"]:
        away = (pos[..., None] - j).abs().float()
        s = s - st["slopes"].view(1, Hkv, G, 1, 1) * away[:, None, None]
    hi = pos + 1
    if c["prefix"]:
        hi = torch.maximum(hi, st["prefix"].long()[:, None])
    hi = torch.minimum(hi, L[:, None])
    lo = torch.zeros_like(pos)
    if c["window"]:
        lo = (pos - c["window"] + 1).clamp(min=0)
    if c["docs"]:
        lo = torch.maximum(lo, st["docs"].long()[row])
    seen = (j >= lo[..., None]) & (j < hi[..., None])
    s.masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(-1)
    if c["sink"]:
        top = torch.maximum(top, st["sink"].view(1, Hkv, G, 1))
    top = torch.where(top == -math.inf, 0.0, top)
    s = torch.exp(s - top[..., None])
    den = s.sum(-1)
    if c["sink"]:
        den = den + torch.exp(st["sink"].view(1, Hkv, G, 1) - top)
    o = torch.matmul(s.view(B, Hkv, G * T, -1), _gathered(st["v"], st["v_scale"], table)).view(B, Hkv, G, T, D)
    o = torch.where(den[..., None] > 0, o / den[..., None], 0.0)
    lse = top + torch.log(den)
    out = o.permute(0, 3, 1, 2, 4).reshape(B * T, Hq, D)[live.view(-1)].to(dt)
    return {"out": out, "lse": lse.permute(0, 3, 1, 2).reshape(B * T, Hq)[live.view(-1)]}


# ------------------------------------------------------------------- work

def _spans(case):
    """For each request the (first, past the last) visible position of each new token."""
    cached, fresh = lengths(case)
    r = random.Random(case["B"] * 131 + case["hi"])
    total = [c + n for c, n in zip(cached, fresh)]
    prefix = [r.randint(0, t) for t in total] if case["prefix"] else [0] * len(total)
    every = [max(1, t // r.randint(1, 4)) for t in total] if case["docs"] else None
    for b, (c, n) in enumerate(zip(cached, fresh)):
        p = torch.arange(c, c + n)
        hi = torch.clamp(torch.clamp(p + 1, min=prefix[b]), max=total[b])
        lo = torch.clamp(p - case["window"] + 1, min=0) if case["window"] else torch.zeros_like(p)
        if every:
            lo = torch.maximum(lo, p // every[b] * every[b])
        yield lo, torch.maximum(hi, lo)


def work(case):
    cached, fresh = lengths(case)
    P, N = case["page"], sum(max(n, 0) for n in fresh)
    if case["op"] == "plan":
        pages = sum(-(-(c + n) // P) - -(-c // P) if n >= 0 else -(-c // P) for c, n in zip(cached, fresh))
        return {"bytes": 16 * case["B"] + 8 * N + 8 * pages, "flops": 0}
    H, D = case["Hkv"], case["D"]
    if case["op"] == "store":
        size = 4 if case["x"] == "f32" else 2
        return {"bytes": 2 * N * H * D * (size + 1) + 4 * N, "flops": 0}
    size = 4 if case["q"] == "f32" else 2
    keys, pairs = 0, 0
    for lo, hi in _spans(case):
        keys += int(hi.max() - lo.min())
        pairs += int((hi - lo).sum())
    Hq = case["Hq"]
    return {"bytes": 2 * keys * H * (D + 4 / P) + 2 * N * Hq * D * size + 4 * N * Hq + 4 * keys // P,
            "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------ exact

def exact(case, seed):
    st = prepare(case, seed)
    return {"plan": _exact_plan, "store": _exact_store, "attn": _exact_attn}[case["op"]](st)


def _exact_plan(st):
    return None  # whole numbers: the two sides are compared with each other


def _e4m3_values():
    """The non-negative values of E4M3, code by code (the last code holds no number)."""
    v = [(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64, device="cuda")


def _nearest(x):
    """x (|x| <= 448) rounded to the nearest E4M3 value, ties to the even code."""
    grid = _e4m3_values()
    a = x.abs()
    up = torch.searchsorted(grid, a).clamp(max=126)
    dn = (up - 1).clamp(min=0)
    du, dd = grid[up] - a, a - grid[dn]
    code = torch.where((du < dd) | ((du == dd) & (up % 2 == 0)) | (du == 0), up, dn)
    return torch.copysign(grid[code], x)


def _exact_store(st):
    P = st["case"]["page"]
    slots = st["slots"].tolist()
    by_page = {}
    for t, s in enumerate(slots):
        by_page.setdefault(s // P, []).append((t, s % P))
    if len(by_page) > 20000:
        return None
    out = {}
    for name in ("k", "v"):
        x = st["x_" + name].double()
        val = st[name].view(torch.float8_e4m3fn).double()
        scale = st[name + "_scale"].double()
        for page, rows in by_page.items():
            t = torch.tensor([r[0] for r in rows], device="cuda")
            off = torch.tensor([r[1] for r in rows], device="cuda")
            a = x[t].abs().amax((0, 2)) / E4M3_MAX  # [Hkv]
            e = torch.ceil(torch.log2(a.clamp(min=2.0 ** -120)))
            e = torch.where(torch.exp2(e - 1) >= a, e - 1, torch.where(torch.exp2(e) < a, e + 1, e))
            s = torch.exp2(e.clamp(min=SCALE_FLOOR))
            first = min(r[1] for r in rows)
            if first > 0:
                s = torch.maximum(s, scale[page])
                val[page, :, :first] = _nearest(val[page, :, :first] * (scale[page] / s)[:, None, None])
            val[page][:, off] = _nearest(x[t] / s[None, :, None]).transpose(0, 1)
            scale[page] = s
        out[name], out[name + "_scale"] = val, scale
    return out


def _exact_attn(st):
    c = st["case"]
    Hq, Hkv, D, P = c["Hq"], c["Hkv"], c["D"], c["page"]
    G, N = Hq // Hkv, st["N"]
    out = torch.zeros((N, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((N, Hq), dtype=torch.float64, device="cuda")
    starts, ctx = st["q_start"].tolist(), st["ctx"].tolist()
    for b, L in enumerate(ctx):
        r0, r1 = starts[b], starts[b + 1]
        pages = st["table"][b, :-(-L // P)].long()
        p = torch.arange(L - (r1 - r0), L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")[None]
        seen = j <= p
        if c["prefix"]:
            seen = seen | (j < st["prefix"][b])
        if c["window"]:
            seen = seen & (j > p - c["window"])
        if c["docs"]:
            seen = seen & (j >= st["docs"][r0:r1, None])
        for h in range(Hkv):
            val = lambda n: (st[n][pages, h].view(torch.float8_e4m3fn).double()
                             * st[n + "_scale"][pages, h].double()[:, None, None]).reshape(-1, D)[:L]
            K, V = val("k"), val("v")
            for a in range(h * G, (h + 1) * G):
                x = st["q"][r0:r1, a].double() @ K.T / math.sqrt(D)
                if c["cap"]:
                    x = c["cap"] * torch.tanh(x / c["cap"])
                if c["bias"]:
                    x = x - st["slopes"][a].double() * (p - j).abs()
                x = torch.where(seen, x, -math.inf)
                if c["sink"]:
                    x = torch.cat([x, st["sink"][a].double().expand(r1 - r0, 1)], 1)
                z = torch.logsumexp(x, 1)
                lse[r0:r1, a] = z
                w = torch.exp(x[:, :L] - torch.where(z == -math.inf, 0.0, z)[:, None])
                out[r0:r1, a] = w @ V
    return {"out": out, "lse": lse}

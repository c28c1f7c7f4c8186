"""Raw tokens in a paged 8-bit cache: plan, store and attention (oracle side).

Test infrastructure only (see ``oracle/__init__.py``).  Plain numpy: the plan in
Python integers, stored codes decided in float32, everything else float64.
"""
import numpy as np

from . import formats

SCALE_FLOOR = -100


def scale_of(amax):
    """The least power of two s with amax <= 448 s, not below 2^-100."""
    e = SCALE_FLOOR
    while float(amax) > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


class Plan:
    """What one plan call leaves: the arrays lcsc_page_plan writes."""

    def __init__(self, page, cached, n_new, table, free, n_free, n_tokens):
        B, width = table.shape
        self.table, self.free = table.copy(), free.copy()
        self.ctx = np.zeros(B, np.int32)
        self.q_start = np.zeros(B + 1, np.int32)
        self.slots = np.full(n_tokens, -1, np.int32)
        self.pos = np.full(n_tokens, -1, np.int32)
        stack = list(free[:n_free])
        self.no_pages = self.bad_length = False
        for b in range(B):
            if n_new[b] < 0:
                stack += [x for x in table[b, :-(-int(cached[b]) // page)] if x >= 0]
        self.free[:len(stack)] = stack
        row, starved = 0, False
        for b in range(B):
            c, n = int(cached[b]), max(int(n_new[b]), 0)
            self.q_start[b] = min(row, n_tokens)
            first, row = row, row + n
            if n_new[b] < 0:
                continue
            if c < 0 or c + n > width * page or row > n_tokens:
                self.bad_length = True
                continue
            have, want = -(-c // page), -(-(c + n) // page)
            if want > have and (starved or want - have > len(stack)):
                starved = self.no_pages = True
                continue
            for col in range(have, want):
                self.table[b, col] = stack.pop()
            self.ctx[b] = c + n
            for i in range(n):
                self.pos[first + i] = c + i
                self.slots[first + i] = self.table[b, (c + i) // page] * page + (c + i) % page
        self.q_start[B] = min(row, n_tokens)
        self.n_free = len(stack)


def store(codes, scale, x, slots, page):
    """Rows x [tokens][heads][D] into codes [pages][heads][page][D] and scale
    [pages][heads], in place; slots < 0 are skipped."""
    heads = codes.shape[1]
    t = 0
    while t < len(slots):
        if slots[t] < 0:
            t += 1
            continue
        n = 1
        while t + n < len(slots) and slots[t + n] == slots[t + n - 1] + 1 and slots[t + n] % page:
            n += 1
        pg, first = int(slots[t]) // page, int(slots[t]) % page
        for h in range(heads):
            rows = np.asarray(x[t:t + n, h], np.float32)
            rows = np.where(np.isfinite(rows), rows, np.float32(0))
            s = scale_of(np.abs(rows).max())
            if first > 0 and s <= scale[pg, h]:
                s = float(scale[pg, h])
            elif first > 0:
                old = formats.e4m3_decode(codes[pg, h, :first]) * (float(scale[pg, h]) / s)
                codes[pg, h, :first] = formats.e4m3_encode(old)
            codes[pg, h, first:first + n] = formats.e4m3_encode(rows.astype(np.float64) / s)
            scale[pg, h] = s
        t += n


def attention(q, k, v, k_scale, v_scale, table, ctx, q_start, sm_scale, window=0, cap=0.0, slopes=None, sink=None,
              prefix=None, docs=None, ends=None):
    """(out, lse, bound) of every row of every request; rows of no request stay
    NaN.  bound[row, head] is the largest sum_d |q_d K_d| over the visible keys, and
    vmax[row, head] their largest |V|, for error bounds."""
    N, Hq, D = q.shape
    Hkv, P = k.shape[1], k.shape[2]
    G = Hq // Hkv
    out = np.full((N, Hq, D), np.nan)
    lse = np.full((N, Hq), np.nan)
    dot = np.zeros((N, Hq))
    vmax = np.zeros((N, Hq))
    for b in range(len(ctx)):
        L, r0, r1 = int(ctx[b]), int(q_start[b]), int(q_start[b + 1])
        n = r1 - r0
        pages = table[b, :-(-L // P)]
        ok = (pages >= 0) & (pages < k.shape[0])
        pages = np.where(ok, pages, 0)
        there = np.repeat(ok, P)[:L]
        for g in range(Hkv):
            K = (formats.e4m3_decode(k[pages, g]) * k_scale[pages, g, None, None]).reshape(-1, D)[:L]
            V = (formats.e4m3_decode(v[pages, g]) * v_scale[pages, g, None, None]).reshape(-1, D)[:L]
            for i in range(n):
                p = L - n + i
                j = np.arange(L)
                seen = (j <= p) | (j < (prefix[b] if prefix is not None else 0))
                seen &= there
                if window:
                    seen &= j > p - window
                if docs is not None:
                    seen &= j >= docs[r0 + i]
                if ends is not None:
                    seen &= j < ends[r0 + i]
                for h in range(g * G, (g + 1) * G):
                    row = q[r0 + i, h].astype(np.float64)
                    x = K[seen] @ row * sm_scale
                    if cap:
                        x = cap * np.tanh(x / cap)
                    if slopes is not None:
                        x = x - float(slopes[h]) * np.abs(p - j[seen])
                    terms = list(x)
                    if sink is not None and L > 0:
                        terms.append(float(sink[h]))
                    top = max(terms, default=-np.inf)
                    if top == -np.inf:
                        out[r0 + i, h], lse[r0 + i, h] = 0.0, -np.inf
                        continue
                    e = np.exp(x - top)
                    den = np.exp(np.array(terms) - top).sum()
                    out[r0 + i, h] = (e[:, None] * V[seen]).sum(0) / den
                    lse[r0 + i, h] = top + np.log(den)
                    if seen.any():
                        dot[r0 + i, h] = (np.abs(K[seen]) @ np.abs(row)).max()
                        vmax[r0 + i, h] = np.abs(V[seen]).max()
    return out, lse, dot, vmax

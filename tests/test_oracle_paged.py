"""Pins of the paged oracle: scales against a closed form, codes against torch's
E4M3 cast, attention against torch's library attention and its own limits."""
import numpy as np
import pytest
import torch

from oracle import formats, paged


def test_scale_is_the_least_power_of_two():
    for amax in (448.0, 448.00003, 447.9, 1.0, 3.5, 3.5000002, 1e-20, 1e30, 7.0, 7.0000005):
        amax = float(np.float32(amax))
        s = paged.scale_of(amax)
        assert np.log2(s) == round(np.log2(s)) and amax <= 448 * s and amax > 448 * s / 2
    assert paged.scale_of(0.0) == 2.0 ** -100 == paged.scale_of(1e-38)


def test_store_codes_are_torchs_cast_and_order_matters_only_below_normal_codes():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((40, 2, 64)).astype(np.float32)
    x[20:] *= 64  # the page's scale grows by 2^6 half way
    slots = np.arange(40)
    one, two = np.zeros((2, 2, 32, 64), np.uint8), np.zeros((2, 2, 32, 64), np.uint8)
    s1, s2 = np.ones((2, 2)), np.ones((2, 2))
    paged.store(one, s1, x, slots, 32)
    for t in range(40):
        paged.store(two, s2, x[t:t + 1], slots[t:t + 1], 32)
    assert np.array_equal(s1, s2)
    a, b = formats.e4m3_decode(one), formats.e4m3_decode(two)
    full = np.zeros_like(a)
    for t in range(40):
        full[t // 32, :, t % 32] = x[t] / s1[t // 32, :, None]
    normal = np.abs(full) >= 2.0 ** -6
    assert np.array_equal(a[normal], b[normal])
    assert np.abs(a - b).max() <= 2.0 ** -9
    want = torch.from_numpy(x[:32, 0] / np.float32(s1[0, 0])).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(one[0, 0], want)


def test_plan_reuses_and_refuses():
    table = np.full((4, 3), -1, np.int32)
    table[0, :2], table[2, 0] = [7, 3], 5
    p = paged.Plan(16, [17, 0, 9, 0], [15, 40, -1, 1], table, np.array([1, 2, 4, 6, 0, 0, 0, 0], np.int32), 4, 60)
    # request 0 fits in its pages, request 2 gives page 5 back, request 1 takes 5, 6, 4, request 3 takes 2
    assert p.table.tolist() == [[7, 3, -1], [5, 6, 4], [5, -1, -1], [2, -1, -1]]
    assert p.ctx.tolist() == [32, 40, 0, 1] and p.q_start.tolist() == [0, 15, 55, 55, 56]
    assert p.n_free == 1 and p.slots[15] == 80 and p.slots[55] == 32 and (p.slots[56:] == -1).all()
    p = paged.Plan(16, [0, 0, 3], [40, 1, 1], np.array([[-1] * 3, [-1] * 3, [0, -1, -1]]), np.array([1, 2]), 2, 42)
    assert p.no_pages and p.ctx.tolist() == [0, 0, 4] and p.n_free == 2  # the first is not reached, nor the next


@pytest.mark.parametrize("window", [0, 5])
def test_attention_is_library_attention(window):
    rng = np.random.default_rng(3)
    Hq, Hkv, D, P = 4, 2, 64, 16
    ctx, new = [37, 16], [37, 2]
    q_start = np.array([0, 37, 39])
    k = rng.integers(0, 120, (5, Hkv, P, D)).astype(np.uint8)
    v = rng.integers(128, 250, (5, Hkv, P, D)).astype(np.uint8)
    ks, vs = np.exp2(rng.integers(-9, -6, (5, Hkv))), np.exp2(rng.integers(-3, 3, (5, Hkv)))
    table = np.array([[3, 0, 4], [1, -1, -1]])
    q = rng.standard_normal((39, Hq, D)).astype(np.float32)
    out, lse, _, _ = paged.attention(q, k, v, ks, vs, table, ctx, q_start, D ** -0.5, window=window)
    for b in range(2):
        pages = table[b, :-(-ctx[b] // P)]
        val = lambda c, s: (formats.e4m3_decode(c[pages]) * s[pages][:, :, None, None]).transpose(1, 0, 2, 3).reshape(
            Hkv, -1, D)[:, :ctx[b]]
        K, V = (torch.from_numpy(np.repeat(val(c, s), Hq // Hkv, 0)) for c, s in ((k, ks), (v, vs)))
        Q = torch.from_numpy(q[q_start[b]:q_start[b + 1]].astype(np.float64)).transpose(0, 1)
        p = torch.arange(ctx[b] - new[b], ctx[b])[:, None]
        j = torch.arange(ctx[b])
        mask = (j <= p) & ((j > p - window) if window else True)
        want = torch.nn.functional.scaled_dot_product_attention(Q, K, V, attn_mask=mask)
        assert np.allclose(out[q_start[b]:q_start[b + 1]], want.transpose(0, 1).numpy(), rtol=1e-12, atol=1e-12)


def test_attention_limits():
    """A document that starts after the query leaves nothing; a prefix over
    everything makes every row see every key; a large cap changes nothing."""
    rng = np.random.default_rng(4)
    D, P = 64, 16
    k, v = (rng.integers(0, 120, (1, 1, P, D)).astype(np.uint8) for _ in range(2))
    ones, table = np.full((1, 1), 0.02), np.zeros((1, 1), int)
    q = rng.standard_normal((6, 1, D))
    run = lambda **kw: paged.attention(q, k, v, ones, ones, table, [6], [0, 6], 0.125, **kw)
    out, lse, _, _ = run(docs=np.full(6, 99))
    assert (out == 0).all() and (lse == -np.inf).all()
    out, lse, _, _ = run(docs=np.full(6, 99), sink=np.array([0.25]))
    assert (out == 0).all() and np.allclose(lse, 0.25)
    full = run(prefix=[6])[0]
    K, V = formats.e4m3_decode(k[0, 0, :6]) * 0.02, formats.e4m3_decode(v[0, 0, :6]) * 0.02
    w = np.exp(q[:, 0] @ K.T * 0.125)
    assert np.allclose(full[:, 0], w @ V / w.sum(1, keepdims=True))
    assert np.allclose(run(cap=1e6)[0], run()[0], rtol=1e-9)

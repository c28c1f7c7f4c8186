"""Pins of the paged oracle's document masks: an explicit mask of who is in whose
document, given to torch's library attention."""
import numpy as np
import pytest
import torch

from oracle import formats, paged


def document_mask(sizes, prefix, shared):
    """[L][L]: query p sees j of its own document (or, with `shared`, of the
    first `prefix` tokens too) that is not behind it or that is in the prefix."""
    doc = np.repeat(np.arange(len(sizes)), sizes)
    L = len(doc)
    p, j = np.arange(L)[:, None], np.arange(L)[None]
    same = doc[:, None] == doc[None]
    return (same | (shared & (j < prefix))) & ((j <= p) | (j < prefix))


@pytest.mark.parametrize("new", [37, 20, 1])
@pytest.mark.parametrize("prefix", [0, 5, 12, 30, 37])
def test_documents_under_a_prefix(prefix, new):
    """doc_start and doc_end keep documents apart whatever the prefix; without
    starts every query sees the prefix whole, which a document's end does not
    shorten where it is given as the length."""
    rng = np.random.default_rng(prefix)
    sizes = [10, 1, 14, 12]
    L, D, P, Hq, Hkv = 37, 64, 16, 4, 2
    starts = np.repeat(np.cumsum([0] + sizes[:-1]), sizes)
    ends = np.repeat(np.cumsum(sizes), sizes)
    k, v = (rng.integers(0, 120, (3, Hkv, P, D)).astype(np.uint8) for _ in range(2))
    s = np.exp2(rng.integers(-9, -6, (3, Hkv)).astype(float))
    table = np.array([[2, 0, 1]])
    q = rng.standard_normal((new, Hq, D)).astype(np.float32)
    full = lambda c: torch.from_numpy(np.repeat(
        (formats.e4m3_decode(c[table[0]]) * s[table[0]][:, :, None, None]).transpose(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :L],
        Hq // Hkv, 0))
    Q = torch.from_numpy(q.astype(np.float64)).transpose(0, 1)
    run = lambda **kw: paged.attention(q, k, v, s, s, table, [L], [0, new], D ** -0.5, prefix=[prefix], **kw)[0]
    for kw, mask in ((dict(docs=starts[-new:], ends=ends[-new:]), document_mask(sizes, prefix, False)),
                     (dict(ends=np.full(new, L)), document_mask([L], prefix, True))):
        want = torch.nn.functional.scaled_dot_product_attention(Q, full(k), full(v),
                                                                attn_mask=torch.from_numpy(mask[-new:]))
        assert np.allclose(run(**kw), want.transpose(0, 1).numpy(), rtol=1e-12, atol=1e-12)


def test_a_start_alone_leaves_a_document_open_under_a_prefix():
    """The rule as documented: what follows a document is seen as far as the prefix goes."""
    rng = np.random.default_rng(1)
    k, v = (rng.integers(0, 120, (1, 1, 16, 64)).astype(np.uint8) for _ in range(2))
    one, q = np.full((1, 1), 0.02), rng.standard_normal((6, 1, 64)).astype(np.float32)
    run = lambda **kw: paged.attention(q, k, v, one, one, np.zeros((1, 1), int), [6], [0, 6], 0.125, prefix=[5], **kw)[0]
    docs = np.array([0, 0, 2, 2, 4, 4])
    open_, wide = run(docs=docs), run(docs=docs, ends=np.full(6, 5))
    assert np.array_equal(open_[:4], wide[:4])
    assert not np.allclose(open_[0], run(docs=docs, ends=docs + 2)[0])

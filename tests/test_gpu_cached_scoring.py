"""The new operators together, as a service runs them: documents pooled, projected and stored in an 8-bit cache,
then scored for queries by a stack with norms around its blocks, against a 64-bit chain.

The chain rounds to bf16 where the path stores bf16 (normed inputs, projections, attention outputs, the residual stream)
and reads the cached K/V from the cache itself (their quantisation is tested bit for bit elsewhere and here).  Scores of
plain stacks are held to the scoring path's stated 1e-3; the stacks here are at most three layers deep.

Stacks with norms: a block's output y is small beside the residual stream (weights of 0.02), and in the plain stack its
rounding errors are as small; its norm scales it, errors included, to unit size, so their share of the score grows.  With
r = 1.7e-3 the root mean square of a bf16 rounding's relative error (2^-7 / sqrt(12) of the binade): the probabilities'
rounding, which the chain lacks, moves o by r; o and y are rounded on both sides at values that differ by about a step, so
independently: sqrt(2) r each; h likewise: in all sqrt(1 + 2 + 2 + 2) r = sqrt(7) r of h, independent from element to element.
The margin h . (w_yes - w_no) then has the standard deviation sqrt(H) * 0.02 * sqrt(2) * sqrt(7) r * rms(h) with rms(h) =
sqrt(1 + 0.2^2), and the score a quarter of it at most: sigma = 3.3e-5 sqrt(H).  A further layer adds its own errors
and those that the changed h brings into its logits, no larger: variance 2 L - 1 times as large.  Six sigma."""
import dataclasses

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle
import synthetic
from tests.gpu_util import from_dev, rand_bf16, to_dev
from tests.test_gpu_cache import quantise

pytestmark = pytest.mark.gpu

SCORE_TOL = 1e-3


@pytest.fixture(scope="module")
def kalm():
    import __graft_entry__
    __graft_entry__.build()
    import encoder_decoder_document_b200 as k
    k.kalm_device_check()
    return k


def score_tol(q, with_norms):
    return 6 * 3.3e-5 * (q.hidden * (2 * q.layers - 1)) ** 0.5 if with_norms else SCORE_TOL


def bf(bits):
    return oracle.bf16_bits_to_f64(bits)


def norm_weights(q, seed, **kw):
    """(device weights, the same as float64) of a stack with norms."""
    from encoder_decoder_document_b200.scorer import DeviceWeights
    rng = np.random.default_rng(seed)
    n = dict(w_norm_pre=rand_bf16(rng, (q.layers, q.hidden), 0.2), w_norm_post=rand_bf16(rng, (q.layers, q.hidden), 0.2),
             gate=oracle.bf16_round(1 + 0.3 * rng.standard_normal((q.layers, q.hidden))),
             w_norm_final=rand_bf16(rng, (q.hidden,), 0.2))
    dev = {k: to_dev(oracle.f64_to_bf16_bits(v)) for k, v in n.items()}
    w = dataclasses.replace(DeviceWeights.from_bits(q.weights), **dev, norm_weight_offset=1.0, norm_eps=1e-5, **kw)
    return w, n


def norm(v, w, eps=1e-5):
    return v / np.sqrt((v * v).mean(-1, keepdims=True) + eps) * (w + 1.0)


def chain(q, x0, kv, n=None, residual_scale=1.0):
    """One document's (margin, score): the decoder stack over its cached K/V rows [Nc][L][2][n_kv][D]."""
    w, D, lq = q.weights, q.head_dim, x0.shape[0]
    r = oracle.bf16_round
    x = x0
    h = r(norm(x, n["w_norm_pre"][0])) if n else x
    for l in range(q.layers):
        qkv = oracle.linear(h, bf(w.w_qkv[l]))
        a, b = q.n_q * D, (q.n_q + q.n_kv) * D
        o, _ = oracle.merged_attention_doc(qkv[:, :a].reshape(lq, q.n_q, D), qkv[:, a:b].reshape(lq, q.n_kv, D),
                                           qkv[:, b:].reshape(lq, q.n_kv, D), kv[:, l, 0], kv[:, l, 1], D ** -0.5)
        if n is None:
            x = h = oracle.linear(o.reshape(lq, a), bf(w.w_o[l]), residual=x)
            continue
        y = oracle.linear(o.reshape(lq, a), bf(w.w_o[l]))
        t = residual_scale * x + n["gate"][l] * norm(y, n["w_norm_post"][l])
        x = r(t)
        h = r(norm(t, n["w_norm_pre"][l + 1] if l + 1 < q.layers else n["w_norm_final"]))
    _, _, m, s = oracle.yes_no_score(h[-1:], bf(w.w_yes), bf(w.w_no))
    return float(m[0]), float(s[0])


def cached_kv(q, cache, key):
    rows, _ = cache.get([key])
    return from_dev(rows).reshape(-1, q.layers, 2, q.n_kv, q.head_dim)


@pytest.mark.parametrize("name,kw", [("tiny", dict(layers=1)), ("tiny", dict(layers=3)),
                                     ("large", dict(n_docs=3, layers=2, lq=40)), ("tiny", dict(layers=2, lq=1))])
@pytest.mark.parametrize("prune", [True, False])
@pytest.mark.parametrize("with_norms", [False, True])
def test_cached_documents_score_as_the_chain(kalm, name, kw, prune, with_norms):
    from encoder_decoder_document_b200.scorer import DeviceWeights, FBNLScorer
    q = synthetic.make_query(name, **kw)
    weights, n = norm_weights(q, 7, residual_scale=0.8) if with_norms else (DeviceWeights.from_bits(q.weights), None)
    sc = FBNLScorer(weights, q.n_q, q.n_kv, prune=prune)
    cache = sc.new_cache(40, page_rows=16)
    keys = [f"doc {i}" for i in range(q.n_docs)]
    cut = q.n_docs // 2  # in two calls, the second one's pages after the first's
    for lo, hi in ((0, cut), (cut, q.n_docs)):
        sc.cache_put(cache, keys[lo:hi], q.enc[q.tok_off[lo]:q.tok_off[hi]], q.doc_len[lo:hi])
    ask = keys[::-1] + keys[:1]  # another order, one document twice
    got = sc.score_rows_cached(q.x0, cache, ask)
    want = np.array([chain(q, bf(q.x0), cached_kv(q, cache, k), n, 0.8 if with_norms else 1.0) for k in ask])
    assert np.abs(got[:, 3] - want[:, 1]).max() <= score_tol(q, with_norms)
    assert np.array_equal(got[0], sc.score_rows_cached(q.x0, cache, ask[:1])[0])  # alone as in the batch
    assert np.array_equal(got[-1], got[len(keys) - 1])                             # named twice, scored alike
    ranked = sc.rerank_cached(q.x0, cache, ask, top_n=2)
    assert [r["index"] for r in ranked] == sorted(range(len(ask)), key=lambda i: (-got[i, 2], i))[:2]


def test_cache_put_stores_the_projection_quantised(kalm):
    """What cache_put stores is, bit for bit, the quantised cross K/V that the uncached path computes."""
    from encoder_decoder_document_b200.scorer import DeviceWeights, FBNLScorer
    q = synthetic.make_query("tiny", layers=2)
    sc = FBNLScorer(DeviceWeights.from_bits(q.weights), q.n_q, q.n_kv)
    sc.rerank(q.x0, q.enc, q.doc_len)
    cache = sc.new_cache(8, page_rows=32)
    sc.cache_put(cache, range(q.n_docs), q.enc, q.doc_len)
    codes, scales = quantise(from_dev(sc.kv_cross[:sc.total_pooled]))
    v = cache.view(list(range(q.n_docs)))
    table, off = v.page_table.cpu().numpy(), v.row_off.cpu().numpy()
    for d in range(q.n_docs):
        i = np.arange(off[d + 1] - off[d])
        at = torch.from_numpy(table[d, i // 32].astype(np.int64) * 32 + i % 32).cuda()
        np.testing.assert_array_equal(cache.codes[at].cpu().numpy(), codes[off[d]:off[d + 1]])
        np.testing.assert_array_equal(cache.scales[at].cpu().numpy(), scales[off[d]:off[d + 1]])


def test_eight_bits_keep_the_ranking(kalm):
    """Scores over the 8-bit cache beside the bf16 path's: e4m3's rounding (2^-4 of a value at most, 32 columns a scale)
    changes them, but not the order of documents whose bf16 scores lie further apart than twice the largest change."""
    from encoder_decoder_document_b200.scorer import DeviceWeights, FBNLScorer
    q = synthetic.make_query("nano", n_docs=24, layers=2)
    sc = FBNLScorer(DeviceWeights.from_bits(q.weights), q.n_q, q.n_kv)
    plain = sc.score_rows(q.x0, q.enc, q.doc_len)
    cache = sc.new_cache(24 * 4)
    sc.cache_put(cache, range(24), q.enc, q.doc_len)
    got = sc.score_rows_cached(q.x0, cache, list(range(24)))
    off = np.abs(got[:, 3] - plain[:, 3]).max()
    assert 0 < off < 0.05
    i, j = np.nonzero(plain[:, 3][:, None] - plain[:, 3][None] > 2 * off)
    assert (got[i, 3] > got[j, 3]).all()


def test_the_plain_path_after_the_cached_one(kalm):
    """A scorer goes back and forth between its own documents and cached ones without a trace."""
    from encoder_decoder_document_b200.scorer import DeviceWeights, FBNLScorer
    q = synthetic.make_query("tiny", layers=2)
    sc = FBNLScorer(DeviceWeights.from_bits(q.weights), q.n_q, q.n_kv)
    before = sc.score_rows(q.x0, q.enc, q.doc_len)
    cache = sc.new_cache(8, page_rows=32)
    sc.cache_put(cache, range(4), q.enc, q.doc_len)
    cached = sc.score_rows_cached(q.x0, cache, [2, 0])
    assert np.array_equal(sc.score_rows(q.x0, q.enc, q.doc_len), before)
    assert np.array_equal(sc.score_rows_cached(q.x0, cache, [2, 0]), cached)
    cache.drop([0])
    with pytest.raises(KeyError):
        sc.rerank_cached(q.x0, cache, [0])
    assert np.array_equal(sc.score_rows_cached(q.x0, cache, [2]), cached[:1])
    assert sc.score_rows_cached(q.x0, cache, []).shape == (0, 4)


def test_empty_documents(kalm):
    from encoder_decoder_document_b200.scorer import DeviceWeights, FBNLScorer
    q = synthetic.make_query("tiny", doc_len=np.array([0, 5, 0]))
    sc = FBNLScorer(DeviceWeights.from_bits(q.weights), q.n_q, q.n_kv)
    cache = sc.new_cache(2, page_rows=8)
    sc.cache_put(cache, "abc", q.enc, q.doc_len)
    for ask in ("abc", "ac", "a"):
        got = sc.score_rows_cached(q.x0, cache, ask)
        want = np.array([chain(q, bf(q.x0), cached_kv(q, cache, k))[1] for k in ask])
        assert np.abs(got[:, 3] - want).max() <= SCORE_TOL


@pytest.mark.parametrize("graph", [False, True])
def test_norms_without_a_cache(kalm, graph):
    """The stack with norms over a query's own documents, eagerly and as a captured graph."""
    from encoder_decoder_document_b200.scorer import FBNLScorer
    q = synthetic.make_query("tiny", layers=3)
    weights, n = norm_weights(q, 9)
    sc = FBNLScorer(weights, q.n_q, q.n_kv)
    res = sc.score_rows(q.x0, q.enc, q.doc_len)
    if graph:
        sc.capture()
        for g in (sc.graphs[0], sc.graphs_decode[0]):
            sc.result.zero_()
            g.replay()
            assert np.array_equal(sc.scores_to_host().numpy().T, res)
        kalm.kalm_check_device_errors()
    kv = oracle.linear(oracle.chunk_pool(bf(q.enc), q.tok_off, q.doc_len)[0],
                       bf(q.weights.w_kv_cross).reshape(-1, q.hidden)).reshape(-1, q.layers, 2, q.n_kv, q.head_dim)
    off = np.concatenate([[0], np.cumsum(oracle.pooled_counts(q.doc_len))])
    want = np.array([chain(q, bf(q.x0), kv[off[d]:off[d + 1]], n)[1] for d in range(q.n_docs)])
    assert np.abs(res[:, 3] - want).max() <= score_tol(q, True)


@pytest.mark.parametrize("name,kw", [("tiny", dict(layers=2)), ("large", dict(n_docs=2, layers=2, lq=24))])
def test_block_stages_with_norms(kalm, name, kw):
    """Each stage of a block from the tensors that the stage before it left: one bf16 step and fp32 effects."""
    from encoder_decoder_document_b200.scorer import FBNLScorer
    q = synthetic.make_query(name, **kw)
    weights, n = norm_weights(q, 3, residual_scale=0.7)
    sc = FBNLScorer(weights, q.n_q, q.n_kv, prune=False)
    sc.rerank(q.x0, q.enc, q.doc_len)
    sc.documents()
    kalm.kalm_broadcast_rows(sc.x0, sc.q_off, sc.x)
    for l in range(q.layers):
        x0 = from_dev(sc.x)
        if l == 0:
            h = from_dev(sc.first_norm(sc.x, sc.h))
            want = norm(x0, n["w_norm_pre"][0])
            assert (np.abs(h - want) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(want)).all()
        sc.layer_qkv(l)
        sc.layer_attention(l)
        sc.block_out(l)
        u = n["gate"][l] * norm(from_dev(sc.y), n["w_norm_post"][l])
        t = 0.7 * x0 + u
        loose = 2.0 ** -20 * (np.abs(x0) + np.abs(u))
        assert (np.abs(from_dev(sc.x) - t) <= 2.0 ** -8 * np.abs(t) + loose).all()
        w = n["w_norm_pre"][l + 1] if l + 1 < q.layers else n["w_norm_final"]
        want = norm(t, w)
        f = np.abs(w + 1.0) / np.sqrt((t * t).mean(-1, keepdims=True) + 1e-5)
        assert (np.abs(from_dev(sc.h) - want) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(want) + 2 * loose * f).all()
    kalm.kalm_check_device_errors()


def test_norm_options_that_do_not_go_together(kalm):
    from encoder_decoder_document_b200.scorer import FBNLScorer
    q = synthetic.make_query("tiny")
    w, _ = norm_weights(q, 1)
    with pytest.raises(ValueError):
        FBNLScorer(w, q.n_q, q.n_kv, fused_out=True)
    with pytest.raises(ValueError):
        FBNLScorer(dataclasses.replace(w, w_norm_pre=None), q.n_q, q.n_kv)
    sc = FBNLScorer(w, q.n_q, q.n_kv)
    with pytest.raises(ValueError):
        sc.cache_put(kalm_cache_of(64), ["a"], q.enc, q.doc_len[:1])


def kalm_cache_of(width):
    from encoder_decoder_document_b200.document_cache import DocumentCache
    return DocumentCache(1, width)


def test_pooled_vectors_in_a_cache(kalm):
    """The other use of a cache: pooled vectors kept in 8 bits, read back and projected for a query."""
    from encoder_decoder_document_b200.document_cache import DocumentCache
    q = synthetic.make_query("tiny", layers=2)
    pooled, off = oracle.chunk_pool(bf(q.enc), q.tok_off, q.doc_len)
    counts = np.diff(off)
    cache = DocumentCache(12, q.hidden, page_rows=8)
    dev = to_dev(oracle.f64_to_bf16_bits(pooled))
    cache.put(range(4), counts, dev)
    cache.append([2], [3], dev[:3])
    cache.drop([1])
    codes, scales = quantise(pooled)
    from tests.test_gpu_cache import dequantise
    val = dequantise(codes, scales)
    rows, row_off = cache.get([2, 0])
    want = np.concatenate([val[off[2]:off[3]], val[:3], val[off[0]:off[1]]])
    np.testing.assert_array_equal(from_dev(rows), want)
    assert row_off.tolist() == [0, counts[2] + 3, counts[2] + 3 + counts[0]]
    kv = torch.empty(rows.shape[0], q.layers * 2 * q.n_kv * q.head_dim, dtype=torch.bfloat16, device="cuda")
    kalm.kalm_cross_kv_proj(rows, to_dev(q.weights.w_kv_cross), kv, q.n_kv)
    ref = oracle.linear(want, bf(q.weights.w_kv_cross).reshape(-1, q.hidden))
    assert (np.abs(from_dev(kv) - ref) <= 2.0 ** -7 * np.abs(ref) + 1e-4).all()  # one bf16 step of the projection
    kalm.kalm_check_device_errors()

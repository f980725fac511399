"""Scoring from a document cache leaves what a scorer prepared, captured or cached for its own documents as it was."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import synthetic

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kalm():
    import __graft_entry__
    __graft_entry__.build()
    import encoder_decoder_document_b200 as k
    k.kalm_device_check()
    return k


def pinned(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).pin_memory()


def scorer(q, **kw):
    from encoder_decoder_document_b200.scorer import DeviceWeights, FBNLScorer
    return FBNLScorer(DeviceWeights.from_bits(q.weights), q.n_q, q.n_kv, **kw)


@pytest.mark.parametrize("instrument", [False, True])
def test_graphs_and_cached_documents_survive(kalm, instrument):
    """The prepared set, its captured graphs and the bf16 document cache, used before and after queries from a cache of
    another number of documents and another query length."""
    q = synthetic.make_query("tiny", layers=3)
    other = synthetic.make_query("tiny", layers=3, lq=17)
    sc = scorer(q)
    plain = sc.score_rows(q.x0, q.enc, q.doc_len)
    sc.capture(instrument=instrument)
    kept = (sc.graph, list(sc.graphs), list(sc.graphs_decode), sc.graph_inst, sc.pool_off, sc.kv_cross, sc.result, sc._shape)
    cache = sc.new_cache(16, page_rows=16)
    sc.cache_put(cache, range(q.n_docs), q.enc, q.doc_len)
    cached = [sc.score_rows_cached(other.x0, cache, [2, 0]), sc.score_rows_cached(q.x0, cache, [1]),
              sc.score_rows_cached(other.x0, cache, [2, 0])]
    np.testing.assert_array_equal(cached[0], cached[2])
    assert (sc.graph, list(sc.graphs), list(sc.graphs_decode), sc.graph_inst, sc._shape) == (*kept[:4], kept[7])
    assert sc.pool_off is kept[4] and sc.kv_cross is kept[5] and sc.result is kept[6]
    np.testing.assert_array_equal(sc.scores_to_host().numpy().T, plain)  # the last query's scores are still there
    # captured graphs
    sc.result.zero_()
    sc.run()
    np.testing.assert_array_equal(sc.scores_to_host().numpy().T, plain)
    outs = [torch.zeros(4, q.n_docs).pin_memory() for _ in range(3)]
    sc.score_cached_stream([pinned(q.x0)] * 3, outs)
    sc.check_errors()
    for out in outs:
        np.testing.assert_array_equal(out.numpy().T, plain)
    if instrument:
        n = len(sc.marks)
        sc.graph_inst.replay()
        torch.cuda.synchronize()
        times = sc.kernel_times()
        sc.score_rows_cached(q.x0, cache, [1])
        assert len(sc.marks) == n and sorted(sc.kernel_times()) == sorted(times)
        sc.marks = None
    # eagerly: the query side over the documents of the last full forward, and a new capture
    sc.result.zero_()
    sc.forward(cached=True)
    np.testing.assert_array_equal(sc.scores_to_host().numpy().T, plain)
    sc.score_rows_cached(other.x0, cache, [2, 0])
    sc.capture()
    sc.score_rows_cached(other.x0, cache, [0])
    sc.graphs_decode[0].replay()
    np.testing.assert_array_equal(sc.scores_to_host().numpy().T, plain)
    kalm.kalm_check_device_errors()


def test_a_scorer_that_has_only_cached_documents(kalm):
    """Nothing prepared before: cached queries work, and the scorer's own documents after them."""
    q = synthetic.make_query("tiny", layers=2)
    sc, ref = scorer(q), scorer(q)
    cache = sc.new_cache(8, page_rows=32)
    sc.cache_put(cache, range(q.n_docs), q.enc, q.doc_len)
    first = sc.score_rows_cached(q.x0, cache, [0, 3])
    assert sc._shape is None and sc.graph is None
    with pytest.raises(KeyError):
        sc.score_rows_cached(q.x0, cache, ["none"])
    np.testing.assert_array_equal(sc.score_rows(q.x0, q.enc, q.doc_len), ref.score_rows(q.x0, q.enc, q.doc_len))
    np.testing.assert_array_equal(sc.score_rows_cached(q.x0, cache, [0, 3]), first)


def test_a_refused_query_changes_nothing(kalm, monkeypatch):
    """An error in the middle of a cached query: the scorer's own set is in place again."""
    q = synthetic.make_query("tiny", layers=2)
    sc = scorer(q)
    plain = sc.score_rows(q.x0, q.enc, q.doc_len)
    cache = sc.new_cache(8, page_rows=32)
    sc.cache_put(cache, range(q.n_docs), q.enc, q.doc_len)
    good = sc.score_rows_cached(q.x0, cache, [1])

    def refuse():
        raise RuntimeError("refused")
    monkeypatch.setattr(sc, "readout", refuse)
    with pytest.raises(RuntimeError, match="refused"):
        sc.score_rows_cached(q.x0, cache, [1, 2])
    monkeypatch.undo()
    assert sc.view is None
    np.testing.assert_array_equal(sc.scores_to_host().numpy().T, plain)
    sc.forward(cached=True)
    np.testing.assert_array_equal(sc.scores_to_host().numpy().T, plain)
    np.testing.assert_array_equal(sc.score_rows_cached(q.x0, cache, [1]), good)
    kalm.kalm_check_device_errors()


def test_a_prepared_set_without_documents_yet(kalm):
    """Between prepare() and the first documents a step or a capture sees empty documents, not memory's leftovers."""
    q = synthetic.make_query("tiny", layers=2)
    for _ in range(3):  # leave bytes in the allocator's blocks that offsets and lengths must not be made of
        torch.full((1 << 20,), 0x7F, dtype=torch.uint8, device="cuda")
    want = scorer(q).score_rows(q.x0, q.enc[:0], np.zeros(q.n_docs, dtype=np.int32))
    sc = scorer(q)
    sc.prepare(q.n_docs, int(q.doc_len.sum()), 500, q.x0.shape[0])
    for t in (sc.slots[0]["doc_len"], sc.slots[1]["doc_len"], sc.pool_off, sc.tok_off):
        assert int(t.abs().max()) == 0
    assert sorted(sc.order.tolist()) == list(range(len(sc.order)))
    sc.x0.copy_(pinned(q.x0))
    sc.forward(cached=True)
    np.testing.assert_array_equal(sc.scores_to_host().numpy().T, want)
    kalm.kalm_check_device_errors()
    sc.capture()
    sc.run()
    np.testing.assert_array_equal(sc.scores_to_host().numpy().T, want)
    with pytest.raises(kalm.KalmError) as e:  # the pooling was promised 500 rows
        sc.check_errors()
    assert e.value.name == "KALM_ERR_DEVICE_ARG"


@pytest.mark.parametrize("cached", [False, True])
def test_an_allocation_that_fails_is_made_again(kalm, monkeypatch, cached):
    """Out of memory in the middle of prepare(): the same query, asked again, gets its buffers."""
    import encoder_decoder_document_b200.scorer as module
    q = synthetic.make_query("tiny", layers=2)
    sc = scorer(q)
    cache = sc.new_cache(8, page_rows=32)
    sc.cache_put(cache, range(q.n_docs), q.enc, q.doc_len)
    ask = (lambda: sc.score_rows_cached(q.x0, cache, [0, 2])) if cached else (lambda: sc.score_rows(q.x0, q.enc, q.doc_len))

    def refuse(*a, **k):
        raise torch.cuda.OutOfMemoryError("no memory")
    monkeypatch.setattr(module, "kalm_linear_chain_sync_len", refuse)
    with pytest.raises(torch.cuda.OutOfMemoryError):
        ask()
    monkeypatch.undo()
    ref = scorer(q)
    want = ref.score_rows_cached(q.x0, cache, [0, 2]) if cached else ref.score_rows(q.x0, q.enc, q.doc_len)
    np.testing.assert_array_equal(ask(), want)


def test_a_failed_allocation_leaves_nothing_to_run(kalm, monkeypatch):
    """After prepare() failed for another shape: no graph over the old buffers, no step over a mix of both."""
    import encoder_decoder_document_b200.scorer as module
    q = synthetic.make_query("tiny", layers=2)
    sc = scorer(q)
    plain = sc.score_rows(q.x0, q.enc, q.doc_len)
    sc.capture()

    def refuse(*a, **k):
        raise torch.cuda.OutOfMemoryError("no memory")
    monkeypatch.setattr(module, "kalm_attention_items", refuse)
    with pytest.raises(torch.cuda.OutOfMemoryError):
        sc.prepare(2 * q.n_docs, 1000, 250, q.x0.shape[0])
    monkeypatch.undo()
    for call in (sc.run, sc.forward, lambda: sc.forward(cached=True), sc.capture, lambda: sc.score_stream([], []),
                 lambda: sc.score_cached_stream([], [])):
        with pytest.raises(RuntimeError):
            call()
    np.testing.assert_array_equal(sc.score_rows(q.x0, q.enc, q.doc_len), plain)
    with pytest.raises(RuntimeError):
        scorer(q).forward()

"""cache_put in groups of documents: the same cache, bit for bit, as in one; all documents are stored, or none."""
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


@pytest.fixture
def scorer(kalm):
    from encoder_decoder_document_b200.scorer import DeviceWeights, FBNLScorer
    q = synthetic.make_query("tiny", layers=2, doc_len=np.array([90, 0, 300, 1, 64, 1024, 0, 33]))
    return q, FBNLScorer(DeviceWeights.from_bits(q.weights), q.n_q, q.n_kv)


def limit(monkeypatch, sc, rows):
    """At most so many pooled rows a group."""
    import encoder_decoder_document_b200.scorer as module
    monkeypatch.setattr(module, "CACHE_PUT_BYTES", rows * sc.L * 2 * sc.n_kv * sc.D * 2)
    return module


@pytest.mark.parametrize("rows", [1, 40, 100, 257])
def test_groups_store_what_one_call_stores(kalm, scorer, monkeypatch, rows):
    q, sc = scorer
    one, many = (sc.new_cache(64, page_rows=16) for _ in range(2))
    sc.cache_put(one, range(q.n_docs), q.enc, q.doc_len)
    limit(monkeypatch, sc, rows)
    sc.cache_put(many, range(q.n_docs), q.enc, q.doc_len)
    assert torch.equal(one.codes, many.codes) and torch.equal(one.scales, many.scales)
    assert one._docs == many._docs and one.free_pages == many.free_pages
    kalm.kalm_check_device_errors()


def test_all_or_none(kalm, scorer, monkeypatch):
    q, sc = scorer
    cache = sc.new_cache(64, page_rows=16)
    sc.cache_put(cache, ["held"], q.enc[:90], q.doc_len[:1])
    before = (cache.free_pages, dict(cache._docs))
    module = limit(monkeypatch, sc, 100)
    calls = []

    def refuse(*a, **k):
        calls.append(1)
        if len(calls) == 3:
            raise RuntimeError("refused")
        return project(*a, **k)
    project = module.kalm_cross_kv_proj
    monkeypatch.setattr(module, "kalm_cross_kv_proj", refuse)
    with pytest.raises(RuntimeError, match="refused"):  # in the third group
        sc.cache_put(cache, range(q.n_docs), q.enc, q.doc_len)
    assert len(calls) == 3 and (cache.free_pages, cache._docs) == before
    # refused before any work: a known key in the last group, too few pages
    for keys, kept in (([*range(q.n_docs - 1), "held"], KeyError), ([0, 1, 2, 3, 4, 5, 6, 0], ValueError)):
        with pytest.raises(kept):
            sc.cache_put(cache, keys, q.enc, q.doc_len)
    small = sc.new_cache(20, page_rows=16)
    with pytest.raises(MemoryError):
        sc.cache_put(small, range(q.n_docs), q.enc, q.doc_len)
    assert len(calls) == 3 and len(small) == 0 and (cache.free_pages, cache._docs) == before
    monkeypatch.undo()
    sc.cache_put(cache, range(q.n_docs), q.enc, q.doc_len)
    assert len(cache) == q.n_docs + 1
    kalm.kalm_check_device_errors()


def test_scratch_of_many_documents(kalm, scorer, monkeypatch):
    """The bf16 scratch is that of a group, not of the call."""
    q, sc = scorer
    n, rows = 300, 100  # 300 documents of 64 rows; groups of 100 rows: one document each
    width = sc.L * 2 * sc.n_kv * sc.D
    limit(monkeypatch, sc, rows)
    cache = sc.new_cache(n * 4, page_rows=16)
    enc = np.zeros((n * 256, q.hidden), dtype=np.uint16)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    sc.cache_put(cache, range(n), enc, np.full(n, 256))
    peak = torch.cuda.max_memory_allocated() - before
    one = 64 * width * 2 + 256 * q.hidden * 2 + 64 * q.hidden * 2
    assert peak <= 3 * one + (8 << 20) < n * 64 * width * 2
    kalm.kalm_check_device_errors()

"""The document cache's calls on offsets and lengths that the host cannot check: flagged, with a defined result and an
end, in the order of the calls' own bounds and not of the numbers found there.  Tolerances as in test_gpu_cache.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.gpu_util import f64_to_dev, from_dev, i32, i64, rand_bf16
from tests.test_gpu_cache import attention, check, dequantise, plain_attention, quantise, run_attention

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kalm():
    import __graft_entry__
    __graft_entry__.build()
    import encoder_decoder_document_b200 as k
    k.kalm_device_check()
    return k


def flagged(kalm):
    with pytest.raises(kalm.KalmError) as e:
        kalm.kalm_check_device_errors()
    return e.value.name == "KALM_ERR_DEVICE_ARG"


def with_zero_rows(want, lse, vmax, extra):
    """The softmax with `extra` more keys of score 0 and value 0, from the one without: log-sum-exp and output."""
    more = np.logaddexp(lse, np.log(extra))
    return want * np.exp(lse - more)[..., None], more, vmax


@pytest.mark.parametrize("lq,n_q,n_kv", [([1, 1], 4, 1), ([1, 1, 1], 4, 4), ([2, 1], 2, 1), ([4, 2], 1, 1)])
@pytest.mark.parametrize("extra", [1, 7, 100_000])
def test_few_rows_that_claim_more_than_the_table(kalm, lq, n_q, n_kv, extra):
    """Rows past the table's places count as zeros, as many as are claimed, without a step for each."""
    rng = np.random.default_rng(70 + extra % 13)
    page_rows, nc = 16, [32] * len(lq)  # the table's places, all used
    a = attention(rng, lq, nc, n_q, n_kv, page_rows)
    want = plain_attention(a)
    claim = dict(a, p_off=np.arange(len(lq) + 1) * (32 + extra))
    got, lse = run_attention(kalm, claim)
    assert flagged(kalm)
    check(got, lse, *with_zero_rows(*want, extra))


def test_few_rows_of_a_wild_length(kalm):
    """A claim of 2^40 rows (stale offsets): the walk ends at the table, the sum holds the rest."""
    a = attention(np.random.default_rng(71), [1, 1], [32, 32], 4, 1, 16)
    out, lse, vmax = plain_attention(a)
    got, got_lse = run_attention(kalm, dict(a, p_off=np.array([0, 1 << 40, (1 << 40) + 32])))
    assert flagged(kalm)
    first = with_zero_rows(out[:1], lse[:1], vmax[:1], 2.0 ** 40 - 32)
    check(got[:1], got_lse[:1], *first)
    check(got[1:], got_lse[1:], out[1:], lse[1:], vmax[1:])


def test_few_rows_of_a_negative_length(kalm):
    """Offsets that go back: no cached rows for that document, flagged; the others have theirs."""
    a = attention(np.random.default_rng(72), [1, 1, 1], [20, 0, 20], 4, 1, 16)
    want = plain_attention(a)
    got, lse = run_attention(kalm, dict(a, p_off=np.array([0, 20, 10, 30])))
    assert flagged(kalm)
    check(got, lse, *want)


@pytest.mark.parametrize("ws_rows,past", [(198, []), (197, [1]), (133, [1]), (127, [0, 1])])
def test_documents_past_the_workspace(kalm, ws_rows, past):
    """General form: a document whose widened rows do not fit the workspace is flagged and has no cached rows; the others
    and the decoder rows' own attention are what they were."""
    lq, nc = [40, 3], [70, 20]  # workspace rows 0 .. 127 (two tiles) and 134 .. 197
    a = attention(np.random.default_rng(73), lq, nc, 4, 1, 16)
    got, lse = run_attention(kalm, a, ws_rows=ws_rows)
    if past:
        assert flagged(kalm)
    seen = dict(a, nc=[0 if d in past else n for d, n in enumerate(nc)])
    check(got, lse, *plain_attention(seen))
    assert kalm.kalm_check_device_errors() == 0


def test_lengths_that_no_workspace_holds(kalm):
    """General form: a negative length, and ones past 32 bits and past the workspace, are flagged and count as none."""
    lq, nc = [33, 5, 40], [20, 30, 9]
    a = attention(np.random.default_rng(74), lq, nc, 4, 1, 16)
    for off, left in (([0, 20, 10, 19], [20, 0, 9]),             # document 1 ends before it starts
                      ([0, 20, (1 << 32) + 50, 59], [20, 0, 0]),  # 2^32 + 30 rows, then a start past the workspace
                      ([0, 20, 1 << 50, 1 << 50], [20, 0, 0])):
        got, lse = run_attention(kalm, dict(a, p_off=np.array(off)), ws_rows=59 + 3 * 64)
        assert flagged(kalm)
        check(got, lse, *plain_attention(dict(a, nc=left)))


@pytest.mark.parametrize("lq", [[40, 3, 130], [1, 1, 1], [2, 1, 2]])
@pytest.mark.parametrize("start", [5, 1000, -7, 1 << 40])
def test_offsets_that_start_elsewhere(kalm, lq, start):
    """Only the differences of the cached rows' offsets count, in every form and with the workspace sized by them."""
    nc = [70, 0, 20]
    a = attention(np.random.default_rng(75), lq, nc, 4, 1, 16)
    want = run_attention(kalm, a)
    moved = dict(a, p_off=a["p_off"] + start)
    for ws_rows in (None, kalm.kalm_merged_attention_cache_rows(90, 3)):
        got = run_attention(kalm, moved, ws_rows=ws_rows)
        np.testing.assert_array_equal(got[0], want[0])
        np.testing.assert_array_equal(got[1], want[1])
    assert kalm.kalm_check_device_errors() == 0


@pytest.mark.parametrize("lq,n_q,n_kv", [(1, 4, 1), (2, 4, 1), (8, 1, 1), (3, 2, 1), (1, 8, 1), (2, 16, 4), (3, 4, 1), (40, 4, 1)])
def test_a_document_in_any_company(kalm, lq, n_q, n_kv):
    """A document's result, bit for bit: alone, beside one whose pages widen the table, and among many."""
    rng = np.random.default_rng(76 + lq + n_q)
    n = 300
    a = attention(rng, [lq] * n, [40, 700] + [int(k) for k in rng.integers(0, 100, n - 2)], n_q, n_kv, 16)

    def some(docs):
        rows = np.concatenate([np.arange(a["q_off"][d], a["q_off"][d + 1]) for d in docs])
        nc = [a["nc"][d] for d in docs]
        width = max(1, max(-(-c // 16) for c in nc))
        part = dict(a, lq=[lq] * len(docs), nc=nc, q_off=np.arange(len(docs) + 1) * lq, p_off=np.concatenate([[0], np.cumsum(nc)]),
                    table=a["table"][list(docs), :width].copy(), q=a["q"][rows], ks=a["ks"][rows], vs=a["vs"][rows])
        out, lse = run_attention(kalm, part)
        return out.reshape(len(docs), lq, n_q, 256), lse.reshape(len(docs), lq, n_q)

    alone = [some([d]) for d in (0, 1, 5)]
    for docs in ([0, 1, 5], range(n)):
        out, lse = some(list(docs))
        for d, (o, l) in zip((0, 1, 5), alone):
            np.testing.assert_array_equal(out[list(docs).index(d)], o[0])
            np.testing.assert_array_equal(lse[list(docs).index(d)], l[0])
    assert kalm.kalm_check_device_errors() == 0


def test_a_cached_document_scores_alone_as_beside_a_long_one(kalm):
    """Two decoder rows of four heads a KV head through the scorer: a short document's score, bit for bit."""
    import synthetic
    from encoder_decoder_document_b200.scorer import DeviceWeights, FBNLScorer
    q = synthetic.make_query("tiny", layers=2, lq=2, doc_len=np.array([90, 1024, 7, 600]))
    sc = FBNLScorer(DeviceWeights.from_bits(q.weights), q.n_q, q.n_kv)
    cache = sc.new_cache(40, page_rows=16)
    sc.cache_put(cache, range(4), q.enc, q.doc_len)
    together = sc.score_rows_cached(q.x0, cache, [0, 1, 2, 3])
    for d in range(4):
        np.testing.assert_array_equal(sc.score_rows_cached(q.x0, cache, [d])[0], together[d])


@pytest.mark.parametrize("lq,n_q,n_kv", [([2, 1], 4, 1), ([8, 5], 1, 1), ([1, 1], 8, 1)])
def test_few_rows_take_no_workspace(kalm, lq, n_q, n_kv):
    """Up to eight packed rows over documents of any length: nothing is rounded before the output, no workspace is needed."""
    a = attention(np.random.default_rng(77), lq, [900, 33], n_q, n_kv, 64)
    want, want_lse, vmax = plain_attention(a)
    got, lse = run_attention(kalm, a, ws_rows=0)
    check(got, lse, want, want_lse, vmax)
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -15 * vmax[..., None]).all()
    assert kalm.kalm_check_device_errors() == 0


def test_the_default_workspace_of_uneven_documents(kalm):
    """Told how many cached rows there are, the call allocates for those and not for every place of a wide page table."""
    rng = np.random.default_rng(78)
    n, lq = 200, 12
    nc = [4000] + [int(k) for k in rng.integers(0, 30, n - 1)]
    a = attention(rng, [lq] * n, nc, 4, 1, 64)
    qkv = torch.cat([f64_to_dev(a[k].reshape(n * lq, -1)) for k in ("q", "ks", "vs")], 1)
    codes, scales = torch.from_numpy(a["codes"]).cuda(), torch.from_numpy(a["scales"]).cuda()
    out, ref = (torch.empty(n * lq, 1024, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    args = (qkv[:, :1024], qkv[:, 1024:1280], qkv[:, 1280:], codes[:, :256], scales[:, :8], codes[:, 256:], scales[:, 8:],
            i32(a["table"]), 64, i64(a["q_off"]), i64(a["p_off"]), lq, 4, 1)

    def peak(call):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        call()
        return torch.cuda.max_memory_allocated() - before

    wide = peak(lambda: kalm.kalm_merged_attention_cache(*args, ref))
    rows = kalm.kalm_merged_attention_cache_rows(sum(nc), n)
    assert peak(lambda: kalm.kalm_merged_attention_cache(*args, out, total_pool=sum(nc))) <= rows * 1024 + (1 << 20) < wide // 20
    assert torch.equal(out, ref)
    with pytest.raises(kalm.KalmError):
        kalm.kalm_merged_attention_cache(*args, out, total_pool=-1)
    # calls of few rows allocate nothing
    few = torch.empty(n, 2048, dtype=torch.bfloat16, device="cuda")
    a8 = (torch.randn(n, 2048, device="cuda").bfloat16(), args[1][:n], args[2][:n], *args[3:9], i64(np.arange(n + 1)), args[10],
          1, 8, 1)
    assert peak(lambda: kalm.kalm_merged_attention_cache(*a8, few)) == 0
    assert kalm.kalm_check_device_errors() == 0


@pytest.mark.parametrize("q_off,total_q,in_off,skipped", [
    ([0, 40, 43, 83], 50, None, [2]),                    # the last document's rows reach past the output's
    ([0, 40, 1 << 40, 43], 83, None, [1, 2]),            # 2^40 rows, and a start past the output
    ([0, 40, 43, 42], 83, None, [2]),                    # a document that ends before it starts
    ([-5, 35, 38, 83], 83, None, [0]),                   # rows before the output; 45 rows of at most 40
    ([0, 40, 43, 83], 43, [0, 40, 43], [2]),             # inputs that exist, an output that does not
])
def test_decoder_rows_outside_the_call(kalm, q_off, total_q, in_off, skipped):
    """General form: flagged; nothing outside the output and nothing of another document is written."""
    rng = np.random.default_rng(79)
    a = attention(rng, [40, 3, 40], [70, 20, 5], 4, 1, 16)
    qkv = torch.cat([f64_to_dev(a[k].reshape(83, -1)) for k in ("q", "ks", "vs")], 1)
    codes, scales = torch.from_numpy(a["codes"]).cuda(), torch.from_numpy(a["scales"]).cuda()
    whole = torch.full((300, 1024), 7.0, dtype=torch.bfloat16, device="cuda")  # the output, with rows on either side
    out = whole[100:200]

    kalm.kalm_merged_attention_cache(qkv[:, :1024], qkv[:, 1024:1280], qkv[:, 1280:], codes[:, :256], scales[:, :8],
                                     codes[:, 256:], scales[:, 8:], i32(a["table"]), 16, i64(q_off), i64(a["p_off"]), 40, 4, 1,
                                     out, total_q=total_q, in_off=None if in_off is None else i64(in_off))
    assert flagged(kalm)
    want, _, vmax = plain_attention(a)
    got = from_dev(out).reshape(100, 4, 256)
    written = np.zeros(100, bool)
    for d in range(3):
        if d not in skipped:
            lo, hi = q_off[d], q_off[d + 1]
            written[lo:hi] = True
            src = slice(a["q_off"][d], a["q_off"][d + 1])
            if (lo, hi) == (src.start, src.stop):
                bound = 2.0 ** -8 * np.abs(want[src]) + (2.0 ** -8 + 2.0 ** -15) * vmax[src][..., None]
                assert (np.abs(got[lo:hi] - want[src]) <= bound).all()
    assert (got[~written] == 7.0).all()
    assert bool((whole[:100] == 7.0).all()) and bool((whole[200:] == 7.0).all())


# ------------------------------------------------------------------ offsets past the rows in memory
@pytest.mark.parametrize("rows,off", [(20, [0, 12, 25]), (20, [0, 20, 20, 21]), (20, [-3, 5, 20]), (0, [0, 4])])
def test_write_and_read_of_rows_that_do_not_exist(kalm, rows, off):
    """Documents whose offsets leave the tensor: the rows that exist are stored and read, the call is flagged."""
    rng = np.random.default_rng(80)
    v = rand_bf16(rng, (rows, 64))
    src = f64_to_dev(v) if rows else torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    n = len(off) - 1
    codes = torch.full((n * 32, 64), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((n * 32, 2), 0x7F, dtype=torch.uint8, device="cuda")
    table = i32(np.arange(n * 4).reshape(n, 4))
    kalm.kalm_cache_write(src, i64(off), table, 8, codes, scales)
    assert flagged(kalm)
    want_c = np.full((n * 32, 64), 0x55, np.uint8)
    c, _ = quantise(v) if rows else (None, None)
    for d in range(n):
        for r in range(max(off[d], 0), min(off[d + 1], rows)):
            want_c[32 * d + r - off[d]] = c[r]
    np.testing.assert_array_equal(codes.cpu().numpy(), want_c)
    dst = torch.full((rows + 9, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    kalm.kalm_cache_read(codes, scales, i64(off), table, 8, dst[:rows])
    assert flagged(kalm)
    assert bool((dst[rows:] == 3.0).all())
    in_doc = [r for r in range(rows) if any(a <= r < b for a, b in zip(off, off[1:]))]
    stored = dequantise(want_c, scales.cpu().numpy())
    for r in in_doc:
        d = next(i for i in range(n) if off[i] <= r < off[i + 1])
        np.testing.assert_array_equal(from_dev(dst[r:r + 1])[0], stored[32 * d + r - off[d]])
    # offsets that end where the tensor does, or before, are as before
    kalm.kalm_cache_write(src, i64([0] * n + [rows]), table, 8, codes, scales)
    kalm.kalm_cache_write(src, i64([0] * n + [rows // 2]), table, 8, codes, scales)
    assert kalm.kalm_check_device_errors() == 0


# ------------------------------------------------------------------ a single row
def test_one_row_of_any_stride(kalm):
    """A single decoder row: the self K and V may be slices of one row or tensors of their own."""
    a = attention(np.random.default_rng(81), [1], [20], 4, 1, 8)
    want, want_lse = run_attention(kalm, a)
    q, ks, vs = (f64_to_dev(a[k].reshape(1, -1)) for k in ("q", "ks", "vs"))
    row = torch.cat([q, ks, vs, vs], 1)
    codes, scales = torch.from_numpy(a["codes"]).cuda(), torch.from_numpy(a["scales"]).cuda()
    out = torch.empty(1, 1024, dtype=torch.bfloat16, device="cuda")
    for k, v in ((ks, vs), (row[:, 1024:1280], vs), (ks, row[:, 1536:]), (ks.expand(3, 256)[1:2], torch.stack([vs, vs], 1)[:, 1])):
        kalm.kalm_merged_attention_cache(q, k, v, codes[:, :256], scales[:, :8], codes[:, 256:], scales[:, 8:], i32(a["table"]), 8,
                                         i64([0, 1]), i64([0, 20]), 1, 4, 1, out.zero_())
        np.testing.assert_array_equal(from_dev(out).reshape(want.shape), want)
    with pytest.raises(kalm.KalmError):  # not a row of consecutive values
        kalm.kalm_merged_attention_cache(q, ks, torch.cat([vs, vs], 1)[:, ::2], codes[:, :256], scales[:, :8], codes[:, 256:],
                                         scales[:, 8:], i32(a["table"]), 8, i64([0, 1]), i64([0, 20]), 1, 4, 1, out)


@pytest.mark.parametrize("lq", [[1, 1], [40, 3]])
@pytest.mark.parametrize("far", [(1 << 63) - 1, (1 << 63) - 40, -(1 << 63), 1 << 32])
def test_input_rows_at_the_ends_of_64_bits(kalm, lq, far):
    """First input rows so far out that adding a length to them would wrap: flagged, the other document as it was."""
    a = attention(np.random.default_rng(82), lq, [9, 30], 4, 1, 16)
    want, want_lse, vmax = plain_attention(a)
    got, lse = run_attention(kalm, a, in_off=[0, far])
    assert flagged(kalm)
    n = lq[0]
    check(got[:n], lse[:n], want[:n], want_lse[:n], vmax[:n])

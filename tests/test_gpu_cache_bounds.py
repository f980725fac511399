"""The document cache's calls on offsets and lengths that the host cannot check: flagged, with a defined result and an
end, in the order of the calls' own bounds and not of the numbers found there.  Tolerances as in test_gpu_cache.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_cache import attention, check, plain_attention, run_attention

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

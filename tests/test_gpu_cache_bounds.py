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

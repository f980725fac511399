"""The norms on offsets that the host cannot check, and on no rows at all.  Tolerances as in test_gpu_norm.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.gpu_util import f64_to_dev, from_dev, i64, rand_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kalm():
    import __graft_entry__
    __graft_entry__.build()
    import encoder_decoder_document_b200 as k
    k.kalm_device_check()
    return k


@pytest.mark.parametrize("width", [64, 640, 2560, 8192])
@pytest.mark.parametrize("rows,off", [(6, [0, 2, 9]), (6, [0, 6, 6, 7]), (6, [-2, 3, 6]), (0, [0, 5])])
def test_documents_whose_rows_are_not_there(kalm, width, rows, off):
    """Offsets that leave the tensors: the rows that exist are computed with their own gates, the call is flagged."""
    rng = np.random.default_rng(width + rows)
    n = len(off) - 1
    y, x, gate = rand_bf16(rng, (rows, width)), rand_bf16(rng, (rows, width)), rand_bf16(rng, (n, width))
    w = rand_bf16(rng, (width,), 0.3)
    dev = lambda a: f64_to_dev(a) if a.size else torch.empty(a.shape, dtype=torch.bfloat16, device="cuda")
    whole = torch.full((rows + 8, width), 5.0, dtype=torch.bfloat16, device="cuda")
    kalm.kalm_norm_residual(dev(y), dev(x), whole[:rows], w_post=f64_to_dev(w), gate=f64_to_dev(gate), q_off=i64(off))
    with pytest.raises(kalm.KalmError) as e:
        kalm.kalm_check_device_errors()
    assert e.value.name == "KALM_ERR_DEVICE_ARG" and "0x902" in str(e.value)
    doc = np.array([next(d for d in range(n) if off[d] <= r < off[d + 1]) for r in range(rows)], dtype=int)
    u = y / np.sqrt((y * y).mean(-1, keepdims=True) + 1e-6) * w * gate[doc]
    got = from_dev(whole)
    assert (np.abs(got[:rows] - (x + u)) <= 2.0 ** -8 * np.abs(x + u) + 2.0 ** -20 * (np.abs(x) + np.abs(u))).all()
    assert (got[rows:] == 5.0).all()
    # offsets that end with the tensor, or before it, are as before
    kalm.kalm_norm_residual(dev(y), dev(x), whole[:rows], gate=f64_to_dev(gate), q_off=i64([0] * n + [rows]))
    kalm.kalm_norm_residual(dev(y), dev(x), whole[:rows], gate=f64_to_dev(gate), q_off=i64([0] * n + [rows // 2]))
    assert kalm.kalm_check_device_errors() == 0

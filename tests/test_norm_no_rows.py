"""The norm between two blocks on tensors without rows, whose addresses are NULL: nothing to compute, nothing to refuse."""
import pytest

from tests.test_cache_norm_refusals import RESIDUAL, lib  # noqa: F401


def test_no_rows_are_not_refused(lib):  # noqa: F811
    import torch
    none = RESIDUAL | dict(rows=0, y=None, x=None, x_out=None, h=None)
    for more in (dict(), dict(gate=None, ld_gate=0, q_off=None), dict(gate=None, ld_gate=0, q_off=None, w_post=None)):
        if torch.cuda.is_available() and (none | more)["q_off"]:
            continue  # its offsets would be read
        assert lib.kalm_norm_residual(*(none | more).values()) == (0 if torch.cuda.is_available() else 3)


@pytest.mark.gpu
def test_no_rows_through_the_binding():
    import torch
    import encoder_decoder_document_b200 as kalm
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    w = bf(640)
    for q_off, gate in ((None, None), (None, w), (torch.zeros(3, dtype=torch.int64, device="cuda"), bf(2, 640)),
                        (torch.zeros(1, dtype=torch.int64, device="cuda"), bf(0, 640))):
        kalm.kalm_norm_residual(bf(0, 640), bf(0, 640), bf(0, 640), h=bf(0, 640), w_post=w, w_pre=w, gate=gate, q_off=q_off)
        kalm.kalm_norm_residual(bf(0, 640), bf(0, 640), bf(0, 640), gate=gate, q_off=q_off)
    kalm.kalm_rms_norm(bf(0, 640), w, bf(0, 640))
    assert kalm.kalm_check_device_errors() == 0

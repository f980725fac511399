"""Refusals of the document cache's and the norms' entry points.  Sizes, strides and pointers are checked before
anything touches a device, so these run on any machine: the addresses below are never read."""
import pytest

A = 1 << 20  # an aligned address that no call may reach


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    import encoder_decoder_document_b200 as k
    return k.load()


WRITE = dict(src=A, ld_src=64, row_off=A, n_docs=2, total_rows=9, width=64, first_row=None, page_table=A, ld_table=3,
             page_rows=16, n_pages=7, codes=A, ld_codes=64, scales=A, ld_scales=2, stream=None)
READ_ORDER = ("codes", "ld_codes", "scales", "ld_scales", "row_off", "n_docs", "total_rows", "width", "first_row",
              "page_table", "ld_table", "page_rows", "n_pages", "src", "ld_src", "stream")
ATTENTION = dict(q=A, ldq=1024, k_self=A, v_self=A, ld_self=256, k_codes=A, v_codes=A, ld_codes=512, k_scales=A, v_scales=A,
                 ld_scales=16, page_table=A, ld_table=3, page_rows=16, n_pages=7, q_off=A, in_off=None, total_in=40,
                 pool_off=A, n_docs=2, max_q=20, total_q=40, n_q=4, n_kv=1, head_dim=256, scale=0.0625, last=0,
                 order=None, workspace=A, workspace_rows=200, out=A, ldo=1024, lse=None, stream=None)
NORM = dict(x=A, ldx=64, w=A, h=A, ldh=64, rows=3, width=64, eps=1e-6, off=0.0, stream=None)
RESIDUAL = dict(y=A, ldy=64, x=A, ldx=64, w_post=A, gate=A, ld_gate=64, q_off=A, n_docs=2, scale=1.0, x_out=A, ldxo=64,
                w_pre=A, h=2 * A, ldh=64, rows=3, width=64, eps=1e-6, off=0.0, stream=None)

BAD_CACHE = [dict(n_docs=-1), dict(total_rows=-1), dict(width=0), dict(width=48), dict(width=-32), dict(page_rows=4),
             dict(page_rows=24), dict(page_rows=2048), dict(page_rows=0), dict(n_pages=-1), dict(n_pages=1 << 31),
             dict(ld_table=-1), dict(ld_src=60), dict(ld_src=32), dict(ld_codes=72), dict(ld_codes=32), dict(ld_scales=1),
             dict(src=None), dict(row_off=None), dict(page_table=None), dict(codes=None), dict(scales=None),
             dict(src=A + 2), dict(codes=A + 8), dict(total_rows=1 << 55)]


@pytest.mark.parametrize("bad", BAD_CACHE, ids=lambda b: "-".join(map(str, *b.items())))
def test_cache_calls_refuse(lib, bad):
    a = WRITE | bad
    assert lib.kalm_cache_write(*a.values()) == 1, lib.kalm_last_error()
    assert lib.kalm_last_error().startswith(b"kalm_cache_write")
    assert lib.kalm_cache_read(*(a[k] for k in READ_ORDER)) == 1
    assert lib.kalm_last_error().startswith(b"kalm_cache_read")


@pytest.mark.parametrize("bad,status", [
    (dict(head_dim=128), 2), (dict(n_q=3, n_kv=2), 1), (dict(n_q=3), 2), (dict(max_q=513), 1), (dict(n_docs=-1), 1),
    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(q=None), 1), (dict(out=None), 1),
    (dict(q_off=None), 1), (dict(pool_off=None), 1), (dict(ldq=1020), 1), (dict(ldo=512), 1), (dict(ld_self=128), 1),
    (dict(k_codes=None), 1), (dict(v_scales=None), 1), (dict(page_table=None), 1), (dict(k_codes=A + 4), 1),
    (dict(ld_codes=520), 1), (dict(ld_codes=240), 1), (dict(ld_scales=7), 1), (dict(workspace=None), 1), (dict(workspace_rows=0), 1),
    (dict(workspace_rows=-1), 1), (dict(workspace=A + 8), 1), (dict(workspace=A + 16), 1), (dict(n_docs=70000), 1), (dict(page_rows=12), 1), (dict(page_rows=2048), 1),
    (dict(n_pages=-1), 1), (dict(ld_table=-2), 1), (dict(in_off=A, total_in=0), 1), (dict(total_q=-1), 1),
], ids=str)
def test_attention_refuses(lib, bad, status):
    assert lib.kalm_merged_attention_cache(*(ATTENTION | bad).values()) == status


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(rows=1 << 31), dict(width=0), dict(width=60), dict(width=16392, ldx=1 << 15, ldh=1 << 15), dict(eps=0.0),
    dict(eps=-1.0), dict(eps=float("nan")), dict(off=float("inf")), dict(x=None), dict(w=None), dict(h=None), dict(ldx=56),
    dict(ldh=68), dict(x=A + 8), dict(w=A + 2)], ids=str)
def test_rms_norm_refuses(lib, bad):
    assert lib.kalm_rms_norm(*(NORM | bad).values()) == 1
    assert lib.kalm_last_error().startswith(b"kalm_rms_norm")


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(width=12), dict(eps=0.0), dict(scale=float("nan")), dict(n_docs=-1), dict(ld_gate=-8), dict(q_off=None),
    dict(h=None), dict(w_pre=None), dict(y=None), dict(x=None), dict(x_out=None), dict(h=A), dict(ldy=8), dict(ldxo=60),
    dict(ld_gate=32), dict(ld_gate=68), dict(gate=A + 4), dict(w_post=A + 4), dict(ldh=8)], ids=str)
def test_norm_residual_refuses(lib, bad):
    assert lib.kalm_norm_residual(*(RESIDUAL | bad).values()) == 1
    assert lib.kalm_last_error().startswith(b"kalm_norm_residual")


def test_good_arguments_reach_the_device_check(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("checks the no-device path")
    assert lib.kalm_cache_write(*WRITE.values()) == 3
    assert lib.kalm_cache_read(*(WRITE[k] for k in READ_ORDER)) == 3
    assert lib.kalm_merged_attention_cache(*ATTENTION.values()) == 3
    assert lib.kalm_rms_norm(*NORM.values()) == 3
    assert lib.kalm_norm_residual(*RESIDUAL.values()) == 3
    # nothing to do still needs a device (no silent success without one)
    assert lib.kalm_cache_write(*(WRITE | dict(n_docs=0)).values()) == 3


def test_binding_refuses_host_tensors():
    import torch
    import encoder_decoder_document_b200 as k
    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    off = torch.zeros(2, dtype=torch.int64)
    u8, table = torch.zeros(16, 64, dtype=torch.uint8), torch.zeros(1, 2, dtype=torch.int32)
    for call in (lambda: k.kalm_cache_write(t, off, table, 8, u8, u8[:, :2]),
                 lambda: k.kalm_cache_read(u8, u8[:, :2], off, table, 8, t),
                 lambda: k.kalm_rms_norm(t, t[0], t), lambda: k.kalm_norm_residual(t, t, t),
                 lambda: k.kalm_merged_attention_cache(t, t, t, u8, u8, u8, u8, table, 8, off, off, 4, 1, 1, t)):
        with pytest.raises(k.KalmError) as e:
            call()
        assert e.value.name == "KALM_ERR_INVALID_ARG"

"""The cache attention's log-sum-exp where only its output was looked at: in a captured graph replayed on new contents, and
over a cache past 4 GB.  Tolerances as in test_gpu_cache.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.gpu_util import f64_to_dev, from_dev, i32, i64, rand_bf16
from tests.test_gpu_cache import attention, check, offsets, plain_attention, quantise

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kalm():
    import __graft_entry__
    __graft_entry__.build()
    import encoder_decoder_document_b200 as k
    k.kalm_device_check()
    return k


@pytest.mark.parametrize("lq", [[33, 40], [1, 1], [2, 1]])
def test_replayed_with_new_contents(kalm, lq):
    rng = np.random.default_rng(90 + sum(lq))
    nc, n_q, r = [40, 70], 4, sum(lq)
    a = attention(rng, lq, nc, n_q, 1, 16)
    qkv = torch.empty(r, 1536, dtype=torch.bfloat16, device="cuda")
    codes, scales = (torch.zeros(a[k].shape, dtype=torch.uint8, device="cuda") for k in ("codes", "scales"))
    out, lse = torch.empty(r, 1024, dtype=torch.bfloat16, device="cuda"), torch.empty(r, n_q, device="cuda")
    table, q_off, p_off = i32(a["table"]), i64(a["q_off"]), i64(a["p_off"])

    def step():
        kalm.kalm_merged_attention_cache(qkv[:, :1024], qkv[:, 1024:1280], qkv[:, 1280:], codes[:, :256], scales[:, :8],
                                         codes[:, 256:], scales[:, 8:], table, 16, q_off, p_off, max(lq), n_q, 1, out, lse=lse)
    qkv.zero_()
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        a = dict(attention(rng, lq, nc, n_q, 1, 16), table=a["table"])
        qkv.copy_(torch.cat([f64_to_dev(a[k].reshape(r, -1)) for k in ("q", "ks", "vs")], 1))
        codes.copy_(torch.from_numpy(a["codes"])), scales.copy_(torch.from_numpy(a["scales"]))
        out.fill_(float("nan")), lse.fill_(float("nan"))
        g.replay()
        want = plain_attention(a)
        check(from_dev(out).reshape(want[0].shape), lse.cpu().numpy().astype(np.float64), *want)
    assert kalm.kalm_check_device_errors() == 0


@pytest.mark.parametrize("lq", [[40, 2], [1, 1], [2, 2]])
def test_past_four_gigabytes(kalm, lq):
    """The last columns of the last pages of a cache of more than 2^32 bytes."""
    width, page_rows = 9216, 64
    n_pages = (1 << 32) // (width * page_rows) + 40
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB of device memory")
    codes = torch.zeros(n_pages * page_rows, width, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(n_pages * page_rows, width // 32, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(91)
    nc, r = [100, 3], sum(lq)
    c, s = quantise(rand_bf16(rng, (103, 512), 0.7))
    pages = [[n_pages - 1, n_pages - 3], [n_pages - 2, -1]]
    for row in range(103):
        d, i = (0, row) if row < 100 else (1, row - 100)
        at = pages[d][i // page_rows] * page_rows + i % page_rows
        codes[at, width - 512:], scales[at, width // 32 - 16:] = torch.from_numpy(c[row]).cuda(), torch.from_numpy(s[row]).cuda()
    a = dict(lq=lq, nc=nc, n_q=4, n_kv=1, page_rows=128, q_off=offsets(lq), p_off=offsets(nc), table=np.array([[0], [1]]),
             codes=np.zeros((256, 512), np.uint8), scales=np.zeros((256, 16), np.uint8), q=rand_bf16(rng, (r, 4, 256), 0.7),
             ks=rand_bf16(rng, (r, 1, 256), 0.7), vs=rand_bf16(rng, (r, 1, 256)))
    a["codes"][:100], a["codes"][128:131], a["scales"][:100], a["scales"][128:131] = c[:100], c[100:], s[:100], s[100:]
    qkv = torch.cat([f64_to_dev(a[n].reshape(r, -1)) for n in ("q", "ks", "vs")], 1)
    out, lse = torch.empty(r, 1024, dtype=torch.bfloat16, device="cuda"), torch.empty(r, 4, device="cuda")
    kalm.kalm_merged_attention_cache(qkv[:, :1024], qkv[:, 1024:1280], qkv[:, 1280:], codes[:, width - 512:width - 256],
                                     scales[:, -16:-8], codes[:, width - 256:], scales[:, -8:], i32(pages), page_rows,
                                     i64(a["q_off"]), i64(a["p_off"]), max(lq), 4, 1, out, lse=lse)
    want = plain_attention(a)
    check(from_dev(out).reshape(want[0].shape), lse.cpu().numpy().astype(np.float64), *want)
    assert kalm.kalm_check_device_errors() == 0

"""The norms around a decoder block on the GPU against plain 64-bit implementations.

Tolerance.  One rounding to bf16 per output is at most 2^-8 of the value (half a step).  Before it everything is fp32:
n-term sums of squares of positive terms in any order, relative error below (n / 32 + 16) * 2^-24 for the partial
sums used (at most 64 serial terms a lane, then trees), rsqrt within 2^-22, and a handful of products; the residual
sum can cancel, so its absolute error is 2^-21 of |residual_scale x| + |gate u|.  Bounds: 2^-8 |x_out| + 2^-20 (|residual
part| + |block part|); for h the same sums again, divided by the row's root mean square and times the weight.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.gpu_util import f64_to_dev, from_dev, i64, rand_bf16

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(scope="module")
def kalm():
    import __graft_entry__
    __graft_entry__.build()
    import encoder_decoder_document_b200 as k
    k.kalm_device_check()
    return k


def norm(v, w, off, eps=EPS):
    return v / np.sqrt((v * v).mean(-1, keepdims=True) + eps) * (w + off)


def strided(a, extra=8):
    """A device copy of a 2-D array whose rows lie further apart than their width."""
    t = torch.full((a.shape[0], a.shape[1] + extra), float("nan"), dtype=torch.bfloat16, device="cuda")
    t[:, :a.shape[1]] = f64_to_dev(a)
    return t[:, :a.shape[1]]


@pytest.mark.parametrize("rows,width", [(1, 8), (1, 640), (3, 256), (7, 264), (33, 640), (9, 1024), (5, 1032), (130, 1152),
                                        (64, 2560), (2, 16384), (5, 16376), (0, 640)])
@pytest.mark.parametrize("off", [0.0, 1.0])
def test_rms_norm(kalm, rows, width, off):
    rng = np.random.default_rng(rows + width)
    x, w = rand_bf16(rng, (rows, width), 3.0), rand_bf16(rng, (width,), 0.3)
    if rows > 1:
        x[1] = 0.0
    h = strided(np.zeros((rows, width)))
    kalm.kalm_rms_norm(strided(x), f64_to_dev(w), h, eps=EPS, weight_offset=off)
    want = norm(x, w, off)
    assert (np.abs(from_dev(h) - want) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(want)).all()
    if rows:  # in place
        y = strided(x)
        kalm.kalm_rms_norm(y, f64_to_dev(w), y, eps=EPS, weight_offset=off)
        assert torch.equal(y, h)
    assert kalm.kalm_check_device_errors() == 0


@pytest.mark.parametrize("lens,width,post,gate,pre,scale", [
    ([1], 640, True, "none", True, 1.0),
    ([3, 0, 5, 1], 640, True, "doc", True, 0.5),
    ([3, 0, 5, 1], 2560, True, "doc", True, 0.5),
    ([128, 7], 1152, True, "row", False, 1.0),
    ([17], 8, False, "row", True, -1.0),
    ([6, 6], 1032, False, "none", False, 0.0),
    ([100, 1, 0, 0, 50] * 9, 136, True, "doc", True, 1.0),
    ([2, 2], 16384, True, "doc", True, 2.0),
])
def test_norm_residual(kalm, lens, width, post, gate, pre, scale):
    rng = np.random.default_rng(sum(lens) + width)
    rows, n = sum(lens), len(lens)
    extra = 3  # rows behind the last document
    y, x = rand_bf16(rng, (rows + extra, width)), rand_bf16(rng, (rows + extra, width), 2.0)
    wp, wq = rand_bf16(rng, (width,), 0.3), rand_bf16(rng, (width,), 0.3)
    g = {"none": None, "row": rand_bf16(rng, (width,)), "doc": rand_bf16(rng, (n, width))}[gate]
    x_out, h = (torch.full((rows + extra, width + 16), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kalm.kalm_norm_residual(strided(y), strided(x), x_out[:, :width], h=h[:, :width] if pre else None,
                            w_post=f64_to_dev(wp) if post else None, w_pre=f64_to_dev(wq) if pre else None,
                            gate=None if g is None else (strided(g) if gate == "doc" else f64_to_dev(g)),
                            q_off=i64(np.concatenate([[0], np.cumsum(lens)])), residual_scale=scale, eps=EPS,
                            weight_offset=1.0)
    assert kalm.kalm_check_device_errors() == 0
    u = norm(y[:rows], wp, 1.0) if post else y[:rows]
    if gate != "none":
        u = u * (np.repeat(g, lens, 0) if gate == "doc" else g)
    t = scale * x[:rows] + u
    loose = 2.0 ** -20 * (np.abs(scale * x[:rows]) + np.abs(u))
    got = from_dev(x_out)
    assert (np.abs(got[:rows, :width] - t) <= 2.0 ** -8 * np.abs(t) + loose).all()
    assert (got[rows:] == 5.0).all() and (got[:, width:] == 5.0).all()
    if pre:
        want = norm(t, wq, 1.0)
        f = np.abs(wq + 1.0) / np.sqrt((t * t).mean(-1, keepdims=True) + EPS)
        got = from_dev(h)
        assert (np.abs(got[:rows, :width] - want) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(want) + 2 * loose * f).all()
        assert (got[rows:] == 5.0).all() and (got[:, width:] == 5.0).all()


@pytest.mark.parametrize("width", [640, 2560])
def test_in_place_and_without_offsets(kalm, width):
    """x_out may be x or y, h may be y; without q_off every row is computed; results do not depend on it."""
    rng = np.random.default_rng(width)
    y, x = rand_bf16(rng, (37, width)), rand_bf16(rng, (37, width))
    wp, wq = f64_to_dev(rand_bf16(rng, (width,))), f64_to_dev(rand_bf16(rng, (width,)))
    ref_x, ref_h = torch.empty(37, width, dtype=torch.bfloat16, device="cuda"), torch.empty(37, width, dtype=torch.bfloat16, device="cuda")
    kalm.kalm_norm_residual(f64_to_dev(y), f64_to_dev(x), ref_x, h=ref_h, w_post=wp, w_pre=wq)
    a, b = f64_to_dev(y), f64_to_dev(x)
    kalm.kalm_norm_residual(a, b, b, h=a, w_post=wp, w_pre=wq)
    assert torch.equal(b, ref_x) and torch.equal(a, ref_h)
    a, b = f64_to_dev(y), f64_to_dev(x)
    h = torch.empty_like(a)
    kalm.kalm_norm_residual(a, b, a, h=h, w_post=wp, w_pre=wq, q_off=i64([0, 37]))
    assert torch.equal(a, ref_x) and torch.equal(h, ref_h)


def test_documents_that_start_late(kalm):
    """Rows before the first document and after the last are not touched, empty documents take none."""
    rng = np.random.default_rng(5)
    y, x = f64_to_dev(rand_bf16(rng, (12, 64))), f64_to_dev(rand_bf16(rng, (12, 64)))
    out = torch.full((12, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    kalm.kalm_norm_residual(y, x, out, q_off=i64([2, 2, 6, 6, 9, 9]))
    got, want = from_dev(out), from_dev(x) + from_dev(y)
    assert (got[:2] == 5.0).all() and (got[9:] == 5.0).all()
    assert (np.abs(got[2:9] - want[2:9]) <= 2.0 ** -8 * np.abs(want[2:9]) + 2.0 ** -20).all()


def test_a_row_of_nan_stays_a_row(kalm):
    rng = np.random.default_rng(6)
    x = rand_bf16(rng, (4, 1152))
    clean = torch.empty(4, 1152, dtype=torch.bfloat16, device="cuda")
    w = f64_to_dev(rand_bf16(rng, (1152,)))
    kalm.kalm_rms_norm(f64_to_dev(x), w, clean)
    t = f64_to_dev(x)
    t[2, 7] = float("nan")
    h = torch.empty_like(clean)
    kalm.kalm_rms_norm(t, w, h)
    assert torch.isnan(h[2]).all() and torch.equal(h[[0, 1, 3]], clean[[0, 1, 3]])


def test_captured_and_on_another_stream(kalm):
    rng = np.random.default_rng(8)
    y, x = f64_to_dev(rand_bf16(rng, (40, 640))), f64_to_dev(rand_bf16(rng, (40, 640)))
    w, g = f64_to_dev(rand_bf16(rng, (640,))), f64_to_dev(rand_bf16(rng, (3, 640)))
    off = i64([0, 10, 10, 40])
    out, h = torch.empty_like(x), torch.empty_like(x)
    call = lambda s=None: kalm.kalm_norm_residual(y, x, out, h=h, w_post=w, w_pre=w, gate=g, q_off=off, stream=s)
    call()
    want = out.clone(), h.clone()
    side = torch.cuda.Stream()
    out.zero_(), h.zero_()
    torch.cuda.synchronize()
    call(side)
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(h, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    x.mul_(2), y.mul_(0.5)
    graph.replay()
    got = out.clone(), h.clone()
    call()
    assert torch.equal(out, got[0]) and torch.equal(h, got[1]) and not torch.equal(out, want[0])


def test_binding_refuses(kalm):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    x, w = bf(4, 64), bf(64)
    for bad in (dict(x=x.half()), dict(x=x[0]), dict(w=bf(63)), dict(w=w.float()), dict(h=bf(3, 64)), dict(h=bf(4, 72)),
                dict(eps=0.0), dict(x=bf(64, 4).t()), dict(x=x.cpu()), dict(w=bf(128)[::2])):
        with pytest.raises(kalm.KalmError):
            kalm.kalm_rms_norm(**(dict(x=x, w=w, h=bf(4, 64)) | bad))
    off = i64([0, 2, 4])
    good = dict(y=bf(4, 64), x=x, x_out=bf(4, 64), h=bf(4, 64), w_post=w, w_pre=w, gate=bf(2, 64), q_off=off)
    kalm.kalm_norm_residual(**good)
    for bad in (dict(y=bf(5, 64)), dict(y=bf(4, 56)), dict(h=None), dict(w_pre=None), dict(q_off=None), dict(gate=bf(3, 64)),
                dict(gate=bf(2, 72)), dict(gate=bf(63)), dict(q_off=off.int()), dict(q_off=off[:0]), dict(x_out=bf(3, 64)),
                dict(h=good["x_out"]), dict(residual_scale=float("inf")), dict(w_post=bf(8)), dict(y=bf(4, 64).cpu())):
        with pytest.raises(kalm.KalmError):
            kalm.kalm_norm_residual(**(good | bad))
    assert kalm.kalm_check_device_errors() == 0


@pytest.mark.parametrize("width", [64, 72, 512, 520, 1280, 1288, 2048, 5120, 6400, 6408, 8192, 12296, 16376])
def test_widths_where_a_rows_threads_change(kalm, width):
    """Rows of 8 lanes, of a warp, of a block of five and of four units a thread, on either side of each change."""
    for case in [(([3, 0, 2], width, True, "doc", True, 0.5)), ([1, 9], width, True, "row", False, 1.0)]:
        test_norm_residual(kalm, *case)
    test_rms_norm(kalm, 6, width, 1.0)

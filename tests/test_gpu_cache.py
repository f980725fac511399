"""The 8-bit document cache on the GPU: quantising rows as they are written, reading them back, and the merged
attention over cached rows, against plain 64-bit implementations.

Tolerances.  Codes, scales and read-back values are exact.  The attention: the stored keys and values are the
operands, so what is off is (a) the output's rounding to bf16, at most 2^-8 of it (half a step), (b) each
probability's rounding to bf16, 2^-8 of it, so at most 2^-8 * sum_j p_j |v_j| <= 2^-8 max|v|, and (c) fp32
effects: logits up to 40 in magnitude with 2^-22 relative error and ex2 with 2^-22, below 2^-16 max|v|.
A bound of 2^-8 |o| + 2^-8 max|v| + 2^-15 max|v| per element holds for all.  The log-sum-exp: 256-term fp32 sums of
exact products, error below 2^-24 * 256 * sum|q k| / 16 < 1e-4 for the inputs here, plus ex2 / log2 effects of 2^-20.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle
from tests.gpu_util import f64_to_dev, from_dev, i32, i64, rand_bf16

pytestmark = pytest.mark.gpu

GROUP = 32


@pytest.fixture(scope="module")
def kalm():
    import __graft_entry__
    __graft_entry__.build()
    import encoder_decoder_document_b200 as k
    k.kalm_device_check()
    return k


# ------------------------------------------------------------------ plain forms, 64 bits
def e4m3_value(codes):
    c = codes.astype(np.int64)
    exp, frac = (c >> 3) & 15, c & 7
    mag = np.where(exp == 0, frac * 2.0 ** -9, (1 + frac / 8) * 2.0 ** (exp - 7.0))
    mag = np.where((c & 127) == 127, np.nan, mag)
    return np.where(c >= 128, -mag, mag)


ALL = e4m3_value(np.arange(127))  # the non-negative codes' values, ascending


def nearest_code(t):
    """Nearest e4m3 number of |t| <= 448, ties to the even code."""
    hi = np.clip(np.searchsorted(ALL, t), 1, 126)
    lo = hi - 1
    dl, dh = t - ALL[lo], ALL[hi] - t
    return np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))


def quantise(v):
    """Codes and scale bytes of [rows][width] bf16-valued float64 rows, from the definition."""
    g = v.reshape(v.shape[0], -1, GROUP)
    fine = np.isfinite(g)
    top = np.where(fine, np.abs(g), 0.0).max(-1)
    e = np.full(top.shape, -120)
    while (top > 448.0 * 2.0 ** e).any():
        e = e + (top > 448.0 * 2.0 ** e)
    t = np.abs(np.where(fine, g, 0.0)) / 2.0 ** e[..., None]
    t = np.where((e >= 120)[..., None], np.minimum(t, 240.0), t)
    code = nearest_code(t)
    code = np.where(fine, code, 127)
    # the sign bit of a NaN's code is not specified
    code = np.where(np.signbit(g) & fine, code + 128, code)
    return code.reshape(v.shape).astype(np.uint8), (e + 127).astype(np.uint8)


def dequantise(codes, scales):
    return e4m3_value(codes) * np.repeat(2.0 ** (scales.astype(np.float64) - 127), GROUP, -1)


def make_pages(rng, rows, page_rows, spare=2):
    need = [-(-int(r) // page_rows) for r in rows]
    n_pages = sum(need) + spare
    perm = rng.permutation(n_pages)
    table = np.full((len(rows), max(max(need, default=0), 1)), -1, np.int32)
    k = 0
    for d, n in enumerate(need):
        table[d, :n] = perm[k:k + n]
        k += n
    return table, n_pages


def row_index(table, page_rows, d, first, n):
    i = np.arange(first, first + n)
    return table[d, i // page_rows].astype(np.int64) * page_rows + i % page_rows


def offsets(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int64)


def same_codes(got, want):
    """Equal codes, any NaN for a NaN, and either zero for a zero that was rounded to."""
    nan = (want & 127) == 127
    assert (((got & 127) == 127) == nan).all()
    np.testing.assert_array_equal(got[~nan], want[~nan])


# ------------------------------------------------------------------ write
@pytest.mark.parametrize("rows,first,width,page_rows", [
    ([1], [0], 32, 8),                       # one row, one group
    ([1, 1, 1], [40, 7, 63], 640, 64),       # single rows appended, at a page's end too
    ([0, 5, 0, 0, 17, 1], None, 96, 8),      # empty documents, odd counts
    ([256, 33, 64, 129], None, 640, 64),
    ([70, 3], [5, 250], 9216, 16),           # every layer's cross K/V of a wide stack
    ([1] * 300, None, 32, 8),                # a warp's rows span many documents
    ([1000], [24], 64, 1024),
])
def test_write(kalm, rows, first, width, page_rows):
    rng = np.random.default_rng(sum(rows) + width)
    n0 = np.zeros(len(rows), int) if first is None else np.asarray(first)
    table, n_pages = make_pages(rng, np.asarray(rows) + n0, page_rows)
    off = offsets(rows)
    total = int(off[-1])
    v = rand_bf16(rng, (total, width)) * 2.0 ** rng.integers(-6, 7, (total, 1))
    v[:, ::7] *= 2.0 ** -9   # below the group's normal range
    src = torch.full((total + 3, width + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    src[:total, :width] = f64_to_dev(v)
    codes = torch.full((n_pages * page_rows, width + 16), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((n_pages * page_rows, width // 32 + 3), 0x11, dtype=torch.uint8, device="cuda")
    want_c, want_s = codes.cpu().numpy(), scales.cpu().numpy()
    c, s = quantise(v)
    for d in range(len(rows)):
        at = row_index(table, page_rows, d, n0[d], rows[d])
        want_c[at, :width], want_s[at, :width // 32] = c[off[d]:off[d + 1]], s[off[d]:off[d + 1]]
    # three rows behind the last document, and strides wider than the rows: left as they were
    kalm.kalm_cache_write(src[:, :width], i64(off), i32(table), page_rows, codes[:, :width], scales[:, :width // 32],
                          first_row=None if first is None else i32(first))
    assert kalm.kalm_check_device_errors() == 0
    np.testing.assert_array_equal(codes.cpu().numpy(), want_c)
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)


def test_write_special_values(kalm):
    """Zeros, subnormals, the borders of a scale, ties, the largest values, NaN and infinities."""
    big = float(torch.finfo(torch.bfloat16).max)
    rows = [[0.0] * 32, [-0.0] * 32, [2.0 ** -133] * 32, [448.0, 447.0] * 16, [450.0, 1.0] * 16, [1.75, 1.7578125] * 16,
            [big, -big] * 16, [big, 1.0] * 16, [2.0 ** 127, 3.0] * 16, [float("nan"), 1.0] * 16,
            [float("inf"), -2.0] * 16, [float("-inf")] * 32, [448.0] + [(k + 0.5) * 2.0 ** -9 for k in range(31)],
            [448.0] + [17.0, 19.0, 21.0, 23.0] * 7 + [0.0, -0.0, 2.0 ** -10]]
    v = oracle.bf16_round(np.array(rows)) if np.isfinite(np.array(rows)).all() else np.array(rows)
    t = torch.tensor(rows, dtype=torch.float64).to(torch.bfloat16)
    v = t.double().numpy()
    want_c, want_s = quantise(v)
    n = len(rows)
    codes = torch.zeros(16, 32, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(16, 1, dtype=torch.uint8, device="cuda")
    kalm.kalm_cache_write(t.cuda(), i64([0, n]), i32([[1, 0]]), 8, codes, scales)
    at = row_index(np.array([[1, 0]]), 8, 0, 0, n)
    got_c, got_s = codes.cpu().numpy()[at], scales.cpu().numpy()[at]
    same_codes(got_c, want_c)
    np.testing.assert_array_equal(got_s, want_s)
    assert want_s.min() >= 7 and want_s.max() <= 247
    # what is read back is the exact number, finite wherever the source was
    dst = torch.empty(n, 32, dtype=torch.bfloat16, device="cuda")
    kalm.kalm_cache_read(codes, scales, i64([0, n]), i32([[1, 0]]), 8, dst)
    back = dst.double().cpu().numpy()
    np.testing.assert_array_equal(np.isfinite(back), np.isfinite(v))
    np.testing.assert_array_equal(back[np.isfinite(v)], dequantise(want_c, want_s)[np.isfinite(v)])
    assert kalm.kalm_check_device_errors() == 0


def test_every_code_and_scale_reads_back_exactly(kalm):
    """All 256 codes under the scales that kalm_cache_write writes."""
    bytes_ = np.arange(7, 248)
    codes = np.tile(np.arange(256, dtype=np.uint8), (len(bytes_), 1))
    scales = np.repeat(bytes_.astype(np.uint8)[:, None], 8, 1)
    want = dequantise(codes, scales)
    n = len(bytes_)
    pad = -(-n // 8) * 8
    c = torch.zeros(pad, 256, dtype=torch.uint8, device="cuda")
    s = torch.zeros(pad, 8, dtype=torch.uint8, device="cuda")
    c[:n], s[:n] = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    dst = torch.empty(n, 256, dtype=torch.bfloat16, device="cuda")
    kalm.kalm_cache_read(c, s, i64([0, n]), i32(np.arange(pad // 8)[None]), 8, dst)
    got = dst.double().cpu().numpy()
    held = np.abs(want) < 2.0 ** 128  # kalm_cache_write never stores more than 240 under its largest scale
    np.testing.assert_array_equal(got[held & ~np.isnan(want)], want[held & ~np.isnan(want)])
    assert np.isnan(got[np.isnan(want)]).all()


# ------------------------------------------------------------------ read
@pytest.mark.parametrize("rows,first,width,page_rows", [
    ([1], [9], 32, 8),
    ([0, 5, 0, 17], None, 640, 16),
    ([100, 1, 64, 65], [3, 0, 64, 1], 2560, 64),
    ([1] * 200, None, 64, 8),
])
def test_read(kalm, rows, first, width, page_rows):
    rng = np.random.default_rng(sum(rows) + width + 1)
    n0 = np.zeros(len(rows), int) if first is None else np.asarray(first)
    table, n_pages = make_pages(rng, np.asarray(rows) + n0, page_rows)
    codes, scales = quantise(rand_bf16(rng, (n_pages * page_rows, width)))
    full_c = torch.zeros(n_pages * page_rows, width + 32, dtype=torch.uint8, device="cuda")
    full_s = torch.zeros(n_pages * page_rows, width // 32 + 1, dtype=torch.uint8, device="cuda")
    full_c[:, 32:], full_s[:, 1:] = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()  # a column window
    off = offsets(rows)
    total = int(off[-1])
    dst = torch.full((total + 2, width + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    kalm.kalm_cache_read(full_c[:, 32:], full_s[:, 1:], i64(off), i32(table), page_rows, dst[:, :width],
                         first_row=None if first is None else i32(first))
    assert kalm.kalm_check_device_errors() == 0
    want = np.full((total + 2, width + 8), 7.0)
    for d in range(len(rows)):
        at = row_index(table, page_rows, d, n0[d], rows[d])
        want[off[d]:off[d + 1], :width] = dequantise(codes[at], scales[at])
    np.testing.assert_array_equal(from_dev(dst), want)


def test_read_names_a_document_twice(kalm):
    rng = np.random.default_rng(3)
    codes, scales = quantise(rand_bf16(rng, (32, 64)))
    c, s = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    dst = torch.empty(40, 64, dtype=torch.bfloat16, device="cuda")
    kalm.kalm_cache_read(c, s, i64([0, 20, 40]), i32([[3, 0, 2], [3, 0, 2]]), 8, dst)
    got = from_dev(dst)
    np.testing.assert_array_equal(got[:20], got[20:])
    assert kalm.kalm_check_device_errors() == 0


def test_bad_pages_are_flagged_and_skipped(kalm):
    """Page numbers outside the cache and rows past the table: nothing is written or read there."""
    src = torch.ones(30, 32, dtype=torch.bfloat16, device="cuda")
    codes = torch.full((16, 32), 3, dtype=torch.uint8, device="cuda")
    scales = torch.full((16, 1), 5, dtype=torch.uint8, device="cuda")
    # document 0: page 1, then a page that does not exist, then -1; the last rows lie past the table
    table = i32([[1, 2, -1]])
    kalm.kalm_cache_write(src, i64([0, 30]), table, 8, codes, scales)
    with pytest.raises(kalm.KalmError) as e:
        kalm.kalm_check_device_errors()
    assert e.value.name == "KALM_ERR_DEVICE_ARG"
    got = codes.cpu().numpy()
    assert (got[:8] == 3).all() and (got[8:] == quantise(np.ones((8, 32)))[0]).all()
    dst = torch.full((30, 32), 9.0, dtype=torch.bfloat16, device="cuda")
    kalm.kalm_cache_read(codes, scales, i64([0, 30]), table, 8, dst)
    with pytest.raises(kalm.KalmError):
        kalm.kalm_check_device_errors()
    back = from_dev(dst)
    assert (back[:8] == 1.0).all() and (back[8:] == 9.0).all()
    # a first row before the document's start
    kalm.kalm_cache_write(src[:4], i64([0, 4]), table, 8, codes, scales, first_row=i32([-2]))
    with pytest.raises(kalm.KalmError):
        kalm.kalm_check_device_errors()


# ------------------------------------------------------------------ attention over the cache
def attention(rng, lq, nc, n_q, n_kv, page_rows, q_std=0.7, c_std=0.7, window=0, spare=2):
    """Inputs: decoder rows, and a cache whose columns hold `window` other columns before this layer's K and V."""
    d = 256
    q_off, p_off = offsets(lq), offsets(nc)
    table, n_pages = make_pages(rng, nc, page_rows, spare)
    n = n_pages * page_rows
    cache = rand_bf16(rng, (n, 2 * n_kv * d), c_std)
    codes, scales = quantise(cache)
    r = int(q_off[-1])
    a = dict(lq=lq, nc=nc, n_q=n_q, n_kv=n_kv, page_rows=page_rows, q_off=q_off, p_off=p_off, table=table,
             q=rand_bf16(rng, (r, n_q, d), q_std), ks=rand_bf16(rng, (r, n_kv, d), q_std), vs=rand_bf16(rng, (r, n_kv, d)),
             codes=codes, scales=scales, window=window)
    return a


def cached_rows(a, d):
    return row_index(a["table"], a["page_rows"], d, 0, a["nc"][d])


def plain_attention(a, scale=1 / 16, in_off=None):
    """64-bit: out [rows][n_q][256], lse [rows][n_q], and a bound's ingredients (max |v| of each row's document)."""
    n_q, n_kv, d = a["n_q"], a["n_kv"], 256
    r = int(a["q_off"][-1])
    out, lse, vmax = np.zeros((r, n_q, d)), np.zeros((r, n_q)), np.zeros((r, n_q))
    val = dequantise(a["codes"], a["scales"])
    for i in range(len(a["lq"])):
        r0, r1 = a["q_off"][i], a["q_off"][i + 1]
        s0 = r0 if in_off is None else in_off[i]
        n = r1 - r0
        c = val[cached_rows(a, i)].reshape(-1, 2, n_kv, d)
        for h in range(n_q):
            g = h // (n_q // n_kv)
            q, k, v = a["q"][s0:s0 + n, h], a["ks"][s0:s0 + n, g], a["vs"][s0:s0 + n, g]
            ls = np.where(np.tri(n, dtype=bool), q @ k.T * scale, -np.inf)
            logits = np.concatenate([ls, q @ c[:, 0, g].T * scale], 1)
            m = logits.max(1, keepdims=True)
            p = np.exp(logits - m)
            z = p.sum(1, keepdims=True)
            vv = np.concatenate([v, c[:, 1, g]])
            out[r0:r1, h] = p / z @ vv
            lse[r0:r1, h] = (m + np.log(z))[:, 0]
            vmax[r0:r1, h] = np.abs(vv).max() if vv.size else 0
    return out, lse, vmax


def run_attention(kalm, a, scale=1 / 16, order=None, in_off=None, last=False, poison=False, stream=None, page_table=None,
                  max_q=None, ws_rows=None):
    d, n_q, n_kv = 256, a["n_q"], a["n_kv"]
    rows = a["q"].shape[0]
    q_off, p_off = i64(a["q_off"]), i64(a["p_off"])
    r = int(a["q_off"][-1])
    qkv = torch.cat([f64_to_dev(a[k].reshape(rows, a[k].shape[1] * d)) for k in ("q", "ks", "vs")], 1)
    w, win = n_kv * d, a["window"]
    n = a["codes"].shape[0]
    codes = torch.full((n, win + 2 * w), 0x7F, dtype=torch.uint8, device="cuda")
    scales = torch.full((n, (win + 2 * w) // 32), 0x7F, dtype=torch.uint8, device="cuda")
    codes[:, win:] = torch.from_numpy(a["codes"]).cuda()
    scales[:, win // 32:] = torch.from_numpy(a["scales"]).cuda()
    if poison:  # every cached row that belongs to no document's attended rows holds NaN
        used = np.zeros(n, bool)
        for i in range(len(a["nc"])):
            used[cached_rows(a, i)] = True
        codes[torch.from_numpy(~used).cuda()] = 0x7F
    out = torch.full((r, n_q * d), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((r, n_q), float("nan"), dtype=torch.float32, device="cuda")
    kc, vc = codes[:, win:win + w], codes[:, win + w:]
    ksc, vsc = scales[:, win // 32:(win + w) // 32], scales[:, (win + w) // 32:]
    kalm.kalm_merged_attention_cache(
        qkv[:, :n_q * d], qkv[:, n_q * d:n_q * d + w], qkv[:, n_q * d + w:], kc, ksc, vc, vsc,
        i32(a["table"]) if page_table is None else page_table, a["page_rows"], q_off, p_off, max_q or max(a["lq"]),
        n_q, n_kv, out,
        scale, lse, in_off=None if in_off is None else i64(in_off), last_tile_only=last,
        order=order(q_off, p_off) if order else None, stream=stream,
        workspace=None if ws_rows is None else torch.full((ws_rows, 2 * w), float("nan"), dtype=torch.bfloat16, device="cuda"))
    if stream is not None:
        stream.synchronize()
    return from_dev(out).reshape(r, n_q, d), lse.cpu().numpy().astype(np.float64)


def check(got, lse, want, want_lse, vmax):
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -15) * vmax[..., None]
    over = np.abs(got - want) / bound
    assert np.isfinite(got).all()
    assert over.max() <= 1.0, over.max()
    assert np.abs(lse - want_lse).max() <= 1e-4 + 2.0 ** -20 * np.abs(want_lse).max()


SHAPES = [
    ([1], [1], 1, 1, 8),                                   # one position, one cached row, one head
    ([1, 1, 1], [0, 64, 200], 4, 1, 64),                   # single tokens
    ([32, 32, 32, 32], [3, 16, 9, 1], 4, 1, 16),           # Tiny shape
    ([128] * 6, [256, 16, 1, 0, 255, 64], 4, 1, 64),       # Nano shape, an empty document, ragged tails
    ([1, 2, 31, 33, 65, 130], [0, 5, 64, 65, 128, 129], 4, 1, 32),
    ([256, 100], [75, 256], 8, 4, 8),                      # Large heads, pages that end inside a tile
    ([512, 3], [1024, 2], 4, 1, 1024),                     # query budget, chunk 1
    ([17, 64, 200], [7, 0, 100], 2, 2, 16),                # one query head per KV head
    ([40, 130], [20, 70], 8, 1, 128),                      # 8 query heads per KV head
    ([5, 9], [0, 0], 4, 1, 8),                             # nothing cached in the whole batch
    ([3] * 200, list(range(0, 200)), 4, 1, 16),            # more items than CTAs
    # up to four packed rows a KV head: the few-row form, at each of its row counts, and the first beyond it
    ([1] * 5, [0, 1, 63, 64, 300], 2, 2, 8),               # 1 row
    ([1, 0, 1], [17, 5, 1024], 4, 2, 16),                  # 2 rows, a document without decoder rows
    ([2, 1, 2], [9, 130, 0], 1, 1, 64),                    # 2 rows of one head: causal self keys
    ([1] * 160, [7 * i % 131 for i in range(160)], 4, 1, 32),
    ([4, 3, 1, 2], [1000, 33, 64, 8], 1, 1, 128),          # 4 rows, 4 positions
    ([2, 1], [70, 257], 8, 4, 16),
    ([1, 1], [256, 65], 8, 1, 64),                         # 8 rows, one position of 8 heads
    ([8, 5, 0, 1], [40, 0, 3, 600], 2, 2, 8),              # 8 positions
    ([2, 2, 1], [5, 64, 513], 4, 1, 64),
]


@pytest.mark.parametrize("lq,nc,n_q,n_kv,page_rows", SHAPES)
def test_attention(kalm, lq, nc, n_q, n_kv, page_rows):
    a = attention(np.random.default_rng(sum(lq) + sum(nc) + n_q), lq, nc, n_q, n_kv, page_rows, window=0 if n_kv > 1 else 512)
    got, lse = run_attention(kalm, a, poison=True)
    assert kalm.kalm_check_device_errors() == 0
    check(got, lse, *plain_attention(a))


@pytest.mark.parametrize("lq,nc,n_q,n_kv", [([1] * 30, list(range(30)), 4, 1), ([2, 1], [300, 64], 4, 2)])
def test_few_rows_agree_with_many(kalm, lq, nc, n_q, n_kv):
    """The two forms of the attention on the same documents: a call sized for more positions takes the other one."""
    a = attention(np.random.default_rng(n_q), lq, nc, n_q, n_kv, 32)
    few, few_lse = run_attention(kalm, a)
    many, many_lse = run_attention(kalm, a, max_q=64)
    want, want_lse, vmax = plain_attention(a)
    check(few, few_lse, want, want_lse, vmax)
    check(many, many_lse, want, want_lse, vmax)
    # nothing is rounded before the few-row form's output: half a bf16 step and fp32 effects
    assert (np.abs(few - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -15 * vmax[..., None]).all()


def test_few_rows_of_nan_free_documents(kalm):
    """NaN in pages that no attended row names, and scores that jump by far more than fp32's exponent range allows."""
    rng = np.random.default_rng(77)
    a = attention(rng, [1, 1], [100, 40], 4, 1, 16)
    a["scales"][cached_rows(a, 0)[50], :8] += 12   # one key of document 0 dominates
    a["scales"][cached_rows(a, 1)[0], :8] += 14
    got, lse = run_attention(kalm, a, poison=True)
    want, want_lse, vmax = plain_attention(a)
    assert np.isfinite(got).all() and (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -12 * vmax[..., None]).all()
    # logits of up to 1e4 in fp32: relative 2^-20
    assert (np.abs(lse - want_lse) <= 2.0 ** -20 * np.abs(want_lse) + 1e-4).all()
    assert kalm.kalm_check_device_errors() == 0


# ------------------------------------------------------------------ the ways a program calls them
def test_attention_shared_inputs_order_and_last_tile(kalm):
    """Documents that share their decoder rows, a work order, and the last-tile-only mode."""
    n_q, n_kv, lq, nc = 4, 1, 70, [5, 130, 0, 64]
    rng = np.random.default_rng(34)
    a = attention(rng, [lq] * 4, nc, n_q, n_kv, 16)
    for k in ("q", "ks", "vs"):
        a[k] = a[k][:lq]
    in_off = [0] * 4
    want, want_lse, vmax = plain_attention(a, in_off=in_off)

    def order(q_off, p_off):
        o = torch.empty(kalm.kalm_attention_items(4, lq, n_q, n_kv), dtype=torch.int32, device="cuda")
        kalm.kalm_attention_schedule(q_off, p_off, lq, n_q, n_kv, o)
        return o

    got, lse = run_attention(kalm, a, in_off=in_off, poison=True)
    check(got, lse, want, want_lse, vmax)
    again, _ = run_attention(kalm, a, in_off=in_off, order=order)
    np.testing.assert_array_equal(again, got)
    last, _ = run_attention(kalm, a, in_off=in_off, last=True)
    first = (lq - 1) // 32 * 32  # 128 / 4 positions a tile
    for d in range(4):
        np.testing.assert_array_equal(last[d * lq + first:(d + 1) * lq], got[d * lq + first:(d + 1) * lq])
        assert np.isnan(last[d * lq:d * lq + first]).all()
    assert kalm.kalm_check_device_errors() == 0


def test_attention_equals_the_uncached_kernel_over_read_rows(kalm):
    """Bit for bit kalm_merged_attention over what kalm_cache_read returns (the tensor-core form)."""
    lq, nc, n_q, n_kv = [64, 7, 130], [100, 256, 33], 8, 4
    a = attention(np.random.default_rng(8), lq, nc, n_q, n_kv, 8)
    got, lse = run_attention(kalm, a)
    w, d = n_kv * 256, 256
    codes, scales = torch.from_numpy(a["codes"]).cuda(), torch.from_numpy(a["scales"]).cuda()
    kv = torch.empty(sum(nc), 2 * w, dtype=torch.bfloat16, device="cuda")
    kalm.kalm_cache_read(codes, scales, i64(a["p_off"]), i32(a["table"]), 8, kv)
    r = sum(lq)
    qkv = torch.cat([f64_to_dev(a[k].reshape(r, -1)) for k in ("q", "ks", "vs")], 1)
    out = torch.empty(r, n_q * d, dtype=torch.bfloat16, device="cuda")
    ref_lse = torch.empty(r, n_q, device="cuda")
    kalm.kalm_merged_attention(qkv[:, :n_q * d], qkv[:, n_q * d:n_q * d + w], qkv[:, n_q * d + w:], kv[:, :w], kv[:, w:],
                               i64(a["q_off"]), i64(a["p_off"]), max(lq), n_q, n_kv, out, 1 / 16, ref_lse)
    np.testing.assert_array_equal(from_dev(out).reshape(got.shape), got)
    np.testing.assert_array_equal(ref_lse.cpu().numpy().astype(np.float64), lse)


@pytest.mark.parametrize("n,top", [(3000, 100), (9000, 40)])
def test_attention_over_many_documents(kalm, n, top):
    """More documents than the widening has blocks for each part of: bit for bit the uncached kernel over the read rows."""
    rng = np.random.default_rng(n)
    nc, lq, page_rows = rng.integers(0, top, n), [5] * n, 8
    table, n_pages = make_pages(rng, nc, page_rows)
    codes = torch.from_numpy(rng.integers(0, 0x50, (n_pages * page_rows, 512), dtype=np.uint8)).cuda()
    scales = torch.from_numpy(rng.integers(115, 122, (n_pages * page_rows, 16), dtype=np.uint8)).cuda()
    q_off, p_off = i64(offsets(lq)), i64(offsets(nc))
    qkv = torch.randn(5 * n, 1536, device="cuda").bfloat16()
    q, k, v = qkv[:, :1024], qkv[:, 1024:1280], qkv[:, 1280:]
    kv = torch.zeros(int(nc.sum()) + 64, 512, dtype=torch.bfloat16, device="cuda")  # (rows past the last: zeros)
    kalm.kalm_cache_read(codes, scales, p_off, i32(table), page_rows, kv)
    out, ref = (torch.empty(5 * n, 1024, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.full((kalm.kalm_merged_attention_cache_rows(int(nc.sum()), n), 512), float("nan"), dtype=torch.bfloat16,
                    device="cuda")
    kalm.kalm_merged_attention_cache(q, k, v, codes[:, :256], scales[:, :8], codes[:, 256:], scales[:, 8:], i32(table), page_rows,
                                     q_off, p_off, 5, 4, 1, out, workspace=ws)
    kalm.kalm_merged_attention(q, k, v, kv[:, :256], kv[:, 256:], q_off, p_off, 5, 4, 1, ref)
    assert torch.equal(out, ref) and bool(torch.isfinite(out).all())
    assert kalm.kalm_check_device_errors() == 0


def test_attention_bad_pages_and_short_workspace(kalm):
    """Rows without a page count as zeros and are flagged, in both forms; a workspace that is too short is flagged."""
    for lq in ([40, 3], [1, 1]):
        a = attention(np.random.default_rng(9), lq, [70, 20], 4, 1, 16)
        table = a["table"].copy()
        table[0, 2], table[1, 0] = -1, 10_000_000
        got, _ = run_attention(kalm, a, page_table=i32(table))
        with pytest.raises(kalm.KalmError) as e:
            kalm.kalm_check_device_errors()
        assert e.value.name == "KALM_ERR_DEVICE_ARG"
        codes = a["codes"].copy()
        codes[row_index(a["table"], 16, 0, 32, 16)] = 0
        codes[row_index(a["table"], 16, 1, 0, 16)] = 0
        want, _, vmax = plain_attention(dict(a, codes=codes))
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -15) * vmax[..., None]).all()
    lq, nc = [40, 3], [70, 20]
    q = torch.zeros(43, 6 * 256, dtype=torch.bfloat16, device="cuda")
    c = torch.zeros(7 * 16, 512, dtype=torch.uint8, device="cuda")
    s = torch.zeros(7 * 16, 16, dtype=torch.uint8, device="cuda")
    out = torch.zeros(43, 1024, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(150, 512, dtype=torch.bfloat16, device="cuda")  # 90 + 2 * 64 rows are needed
    kalm.kalm_merged_attention_cache(q[:, :1024], q[:, 1024:1280], q[:, 1280:], c[:, :256], s[:, :8], c[:, 256:], s[:, 8:],
                                     i32([[0, 1, 2, 3, 4], [5, 6, 0, 0, 0]]), 16, i64([0, 40, 43]), i64([0, 70, 90]), 40, 4, 1,
                                     out, workspace=ws)
    with pytest.raises(kalm.KalmError) as e:
        kalm.kalm_check_device_errors()
    assert e.value.name == "KALM_ERR_DEVICE_ARG"


def test_rows_that_are_not_32_byte_aligned(kalm):
    """bf16 rows at 16-byte places (the other load and store width of write and read)."""
    rng = np.random.default_rng(10)
    v = rand_bf16(rng, (37, 96))
    base = torch.zeros(37, 96 + 8, dtype=torch.bfloat16, device="cuda")
    odd = base[:, 8:]   # 16 bytes past a 32-byte place, a stride of 208 bytes
    odd.copy_(f64_to_dev(v))
    codes, scales = torch.zeros(40, 96, dtype=torch.uint8, device="cuda"), torch.zeros(40, 3, dtype=torch.uint8, device="cuda")
    table = i32([[4, 3, 2, 1, 0]])
    kalm.kalm_cache_write(odd, i64([0, 37]), table, 8, codes, scales)
    c, s = quantise(v)
    at = row_index(np.array([[4, 3, 2, 1, 0]]), 8, 0, 0, 37)
    np.testing.assert_array_equal(codes.cpu().numpy()[at], c)
    np.testing.assert_array_equal(scales.cpu().numpy()[at], s)
    back = torch.full((37, 104), 3.0, dtype=torch.bfloat16, device="cuda")
    kalm.kalm_cache_read(codes, scales, i64([0, 37]), table, 8, back[:, 8:])
    np.testing.assert_array_equal(from_dev(back)[:, 8:], dequantise(c, s))
    assert (from_dev(back)[:, :8] == 3.0).all() and kalm.kalm_check_device_errors() == 0


def test_captured_and_replayed_with_new_contents(kalm):
    """Write, read and both forms of the attention in one graph, replayed after the inputs changed in place; two
    graphs, each with its own scratch, replayed in turn."""
    n_q, n_kv, d = 4, 1, 256
    rng = np.random.default_rng(11)
    lq, nc = [33, 33], [40, 70]
    graphs = []
    for k in range(2):
        a = attention(rng, lq, nc, n_q, n_kv, 16)
        r, n = sum(lq), a["codes"].shape[0]
        st = dict(a=a, qkv=torch.empty(r, (n_q + 2 * n_kv) * d, dtype=torch.bfloat16, device="cuda"),
                  src=torch.empty(sum(nc), 2 * d, dtype=torch.bfloat16, device="cuda"),
                  back=torch.empty(sum(nc), 2 * d, dtype=torch.bfloat16, device="cuda"),
                  codes=torch.zeros(n, 2 * d, dtype=torch.uint8, device="cuda"),
                  scales=torch.zeros(n, 16, dtype=torch.uint8, device="cuda"),
                  out=torch.empty(r, n_q * d, dtype=torch.bfloat16, device="cuda"),
                  one=torch.empty(2, n_q * d, dtype=torch.bfloat16, device="cuda"), table=i32(a["table"]),
                  q_off=i64(a["q_off"]), one_off=i64([0, 1, 2]), p_off=i64(a["p_off"]))

        def step(s=st):
            q, ks, vs = s["qkv"][:, :n_q * d], s["qkv"][:, n_q * d:n_q * d + d], s["qkv"][:, n_q * d + d:]
            kalm.kalm_cache_write(s["src"], s["p_off"], s["table"], 16, s["codes"], s["scales"])
            kalm.kalm_cache_read(s["codes"], s["scales"], s["p_off"], s["table"], 16, s["back"])
            kv = (s["codes"][:, :d], s["scales"][:, :8], s["codes"][:, d:], s["scales"][:, 8:], s["table"], 16)
            kalm.kalm_merged_attention_cache(q, ks, vs, *kv, s["q_off"], s["p_off"], 33, n_q, n_kv, s["out"])
            kalm.kalm_merged_attention_cache(q[:2], ks[:2], vs[:2], *kv, s["one_off"], s["p_off"], 1, n_q, n_kv, s["one"])

        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append((g, st))
    for round_ in range(3):
        for g, s in graphs:
            a = s["a"]
            new = attention(rng, lq, nc, n_q, n_kv, 16)
            a.update({k: new[k] for k in ("q", "ks", "vs")})
            src = rand_bf16(rng, (sum(nc), 2 * d))
            s["src"].copy_(f64_to_dev(src))
            s["qkv"].copy_(torch.cat([f64_to_dev(a[k].reshape(sum(lq), -1)) for k in ("q", "ks", "vs")], 1))
            s["out"].zero_(), s["one"].zero_(), s["back"].zero_()
            c, sc = quantise(src)
            for i in range(2):
                at = cached_rows(a, i)
                a["codes"][at], a["scales"][at] = c[a["p_off"][i]:a["p_off"][i + 1]], sc[a["p_off"][i]:a["p_off"][i + 1]]
            g.replay()
        torch.cuda.synchronize()
        for g, s in graphs:
            a = s["a"]
            val = dequantise(a["codes"], a["scales"])
            np.testing.assert_array_equal(from_dev(s["back"]), np.concatenate([val[cached_rows(a, i)] for i in range(2)]))
            want, want_lse, vmax = plain_attention(a)
            check(from_dev(s["out"]).reshape(want.shape), want_lse, want, want_lse, vmax)
            one = dict(a, lq=[1, 1], q_off=np.array([0, 1, 2]), q=a["q"][:2], ks=a["ks"][:2], vs=a["vs"][:2])
            want, want_lse, vmax = plain_attention(one)
            check(from_dev(s["one"]).reshape(want.shape), want_lse, want, want_lse, vmax)
    assert kalm.kalm_check_device_errors() == 0


def test_two_streams_at_once(kalm):
    """Calls on two side streams, each with its own scratch (the default one of either stream)."""
    a = [attention(np.random.default_rng(20 + k), [130, 64], [256, 90], 4, 1, 64) for k in range(2)]
    alone = [run_attention(kalm, x)[0] for x in a]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got, _ = run_attention(kalm, a[k], stream=streams[k])
            np.testing.assert_array_equal(got, alone[k])
    # both in flight, the arguments' streams given instead of entered
    outs = []
    n_q, d = 4, 256
    for k in range(2):
        x = a[k]
        qkv = torch.cat([f64_to_dev(x[n].reshape(194, -1)) for n in ("q", "ks", "vs")], 1)
        c, s = torch.from_numpy(x["codes"]).cuda(), torch.from_numpy(x["scales"]).cuda()
        outs.append((qkv, c, s, i32(x["table"]), i64(x["q_off"]), i64(x["p_off"]),
                     torch.empty(194, n_q * d, dtype=torch.bfloat16, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(10):
        for k in range(2):
            qkv, c, s, table, q_off, p_off, out = outs[k]
            kalm.kalm_merged_attention_cache(qkv[:, :1024], qkv[:, 1024:1280], qkv[:, 1280:], c[:, :256], s[:, :8], c[:, 256:],
                                             s[:, 8:], table, 64, q_off, p_off, 130, 4, 1, out, stream=streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        np.testing.assert_array_equal(from_dev(outs[k][-1]).reshape(alone[k].shape), alone[k])


def test_cache_offsets_past_32_bits(kalm):
    """A cache of more than 4 GB: pages near its end are written, read and attended to at their own places."""
    width, page_rows = 9216, 64
    n_pages = (1 << 32) // (width * page_rows) + 40
    free, _ = torch.cuda.mem_get_info()
    if free < 8 << 30:
        pytest.skip("needs 8 GB of device memory")
    codes = torch.zeros(n_pages * page_rows, width, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(n_pages * page_rows, width // 32, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(12)
    rows = [100, 3]
    v = rand_bf16(rng, (103, width), 0.7)
    table = np.array([[n_pages - 1, n_pages - 3], [n_pages - 2, -1]], np.int32)
    off = i64([0, 100, 103])
    kalm.kalm_cache_write(f64_to_dev(v), off, i32(table), page_rows, codes, scales)
    c, s = quantise(v)
    for d, (lo, hi) in enumerate(((0, 100), (100, 103))):
        at = torch.from_numpy(row_index(table, page_rows, d, 0, hi - lo)).cuda()
        np.testing.assert_array_equal(codes[at].cpu().numpy(), c[lo:hi])
        np.testing.assert_array_equal(scales[at].cpu().numpy(), s[lo:hi])
    assert int(codes[:(n_pages - 3) * page_rows].count_nonzero()) == 0
    back = torch.empty(103, width, dtype=torch.bfloat16, device="cuda")
    kalm.kalm_cache_read(codes, scales, off, i32(table), page_rows, back)
    np.testing.assert_array_equal(from_dev(back), dequantise(c, s))
    for lq in ([40, 2], [1, 1]):
        k = 17 * 512  # the last layer's columns of 18
        a = dict(lq=lq, nc=rows, n_q=4, n_kv=1, page_rows=128, q_off=offsets(lq), p_off=offsets(rows),
                 table=np.array([[0], [1]]), codes=np.zeros((256, 512), np.uint8), scales=np.zeros((256, 16), np.uint8),
                 q=rand_bf16(rng, (sum(lq), 4, 256), 0.7), ks=rand_bf16(rng, (sum(lq), 1, 256), 0.7),
                 vs=rand_bf16(rng, (sum(lq), 1, 256)))
        a["codes"][:100], a["codes"][128:131] = c[:100, k:], c[100:, k:]
        a["scales"][:100], a["scales"][128:131] = s[:100, k // 32:], s[100:, k // 32:]
        qkv = torch.cat([f64_to_dev(a[n].reshape(sum(lq), -1)) for n in ("q", "ks", "vs")], 1)
        out = torch.empty(sum(lq), 1024, dtype=torch.bfloat16, device="cuda")
        kalm.kalm_merged_attention_cache(qkv[:, :1024], qkv[:, 1024:1280], qkv[:, 1280:], codes[:, k:k + 256],
                                         scales[:, k // 32:k // 32 + 8], codes[:, k + 256:], scales[:, k // 32 + 8:],
                                         i32(table), page_rows, i64(a["q_off"]), off, max(lq), 4, 1, out)
        want, want_lse, vmax = plain_attention(a)
        check(from_dev(out).reshape(want.shape), want_lse, want, want_lse, vmax)
    assert kalm.kalm_check_device_errors() == 0


def test_repeated_calls_are_bit_identical(kalm):
    a = attention(np.random.default_rng(13), [128] * 5 + [1], [256, 3, 0, 77, 128, 64], 4, 1, 16)
    first = run_attention(kalm, a)
    few = attention(np.random.default_rng(14), [1] * 40, list(range(20, 60)), 4, 1, 16)
    few_first = run_attention(kalm, few)
    for _ in range(5):
        for x, y in ((a, first), (few, few_first)):
            again = run_attention(kalm, x)
            np.testing.assert_array_equal(again[0], y[0])
            np.testing.assert_array_equal(again[1], y[1])


def test_binding_refuses(kalm):
    """What the Python calls check before the library does: types, shapes, strides, lengths."""
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")
    src, off, table = bf(20, 64), i64([0, 12, 20]), i32([[0, 1], [2, -1]])
    codes, scales = u8(32, 64), u8(32, 2)
    good = dict(src=src, row_off=off, page_table=table, page_rows=8, codes=codes, scales=scales)
    kalm.kalm_cache_write(**good)
    for bad in (dict(src=src.float()), dict(src=src[0]), dict(src=bf(64, 20).t()), dict(row_off=off.int()), dict(row_off=off[:0]),
                dict(row_off=off[::2]), dict(page_table=table[:1]), dict(page_table=table.long()), dict(page_table=i32([0, 1])),
                dict(page_table=i32([[0, 0, 0, 1], [2, 0, 0, 0]])[:, ::2]), dict(page_rows=7), dict(page_rows=0), dict(page_rows=-8),
                dict(codes=codes[:, :32]), dict(codes=u8(32, 65)[:, :64]), dict(scales=scales[:16]), dict(scales=u8(32, 3)),
                dict(codes=codes.view(torch.int8)), dict(first_row=i32([0])), dict(first_row=i64([0, 0])), dict(src=src.cpu()),
                dict(codes=codes.cpu())):
        with pytest.raises(kalm.KalmError) as e:
            kalm.kalm_cache_write(**(good | bad))
        assert e.value.name == "KALM_ERR_INVALID_ARG", bad
    q, out = bf(6, 6 * 256), bf(6, 4 * 256)
    kc, ks = u8(32, 512), u8(32, 16)
    good = dict(q=q[:, :1024], k_self=q[:, 1024:1280], v_self=q[:, 1280:], k_codes=kc[:, :256], k_scales=ks[:, :8],
                v_codes=kc[:, 256:], v_scales=ks[:, 8:], page_table=table, page_rows=8, q_off=i64([0, 3, 6]), pool_off=off,
                max_q=3, n_q=4, n_kv=1, out=out)
    kalm.kalm_merged_attention_cache(**good)
    for bad in (dict(q=q), dict(v_self=q[:, 1280:].contiguous()), dict(v_codes=kc[:, 256:].contiguous()), dict(v_scales=ks[:, :16]),
                dict(out=out[:, :768]), dict(q_off=i64([0, 6])), dict(q_off=i32([0, 3, 6])), dict(in_off=i64([0])),
                dict(total_q=7), dict(lse=torch.zeros(6, 3, device="cuda")), dict(lse=torch.zeros(5, 4, device="cuda")),
                dict(lse=torch.zeros(6, 4, device="cuda").half()), dict(order=i32([0])), dict(order=i64([0, 0, 0, 0])),
                dict(workspace=bf(148, 256)), dict(workspace=bf(148, 1024)[:, :512]), dict(workspace=bf(148, 512).float()),
                dict(max_q=513), dict(n_q=3), dict(scale=float("nan")), dict(scale=0.0), dict(head_dim=128), dict(n_kv=2),
                dict(total_q=-1), dict(q=q[:, :1024].cpu())):
        with pytest.raises(kalm.KalmError):
            kalm.kalm_merged_attention_cache(**(good | bad))
    assert kalm.kalm_check_device_errors() == 0


@pytest.mark.parametrize("lq", [[5, 40, 64, 1, 130], [1, 1, 1, 1, 1], [70, 63, 65, 2, 17]])
def test_one_documents_nan_stays_its_own(kalm, lq):
    """NaN and infinities in every self row and cached row of some documents leave the others' results, bit for bit."""
    rng = np.random.default_rng(sum(lq))
    a = attention(rng, lq, [30, 7, 65, 0, 100], 4, 1, 16)
    clean, clean_lse = run_attention(kalm, a)
    b = dict(a, **{k: a[k].copy() for k in ("q", "ks", "vs", "codes")})
    for d, x in ((1, np.nan), (3, np.inf), (4, -np.inf)):
        rows = slice(a["q_off"][d], a["q_off"][d + 1])
        b["ks"][rows], b["vs"][rows] = x, x
        b["q"][rows] = np.nan
        b["codes"][cached_rows(a, d)] = 0x7F
    got, lse = run_attention(kalm, b, poison=True)
    for d in (0, 2):
        rows = slice(a["q_off"][d], a["q_off"][d + 1])
        np.testing.assert_array_equal(got[rows], clean[rows])
        np.testing.assert_array_equal(lse[rows], clean_lse[rows])
    assert np.isfinite(clean).all() and not np.isfinite(got[a["q_off"][1]]).any()
    assert kalm.kalm_check_device_errors() == 0


@pytest.mark.parametrize("lq,page_rows,places", [([40, 3], 16, 2), ([40, 3], 8, 1), ([40, 3], 8, 0), ([1, 1], 16, 2), ([1, 1], 8, 0)])
def test_attention_rows_past_the_table(kalm, lq, page_rows, places):
    """Documents that claim more rows than their table has places for: the rest count as zeros and are flagged."""
    nc = [200, 70]
    a = attention(np.random.default_rng(15), lq, nc, 4, 1, page_rows)
    codes = np.zeros_like(a["codes"])
    for d in range(2):
        at = cached_rows(a, d)[:places * page_rows]
        codes[at] = a["codes"][at]
    got, lse = run_attention(kalm, a, page_table=i32(a["table"][:, :places].copy()), ws_rows=270 + 2 * 64)
    with pytest.raises(kalm.KalmError) as e:
        kalm.kalm_check_device_errors()
    assert e.value.name == "KALM_ERR_DEVICE_ARG"
    check(got, lse, *plain_attention(dict(a, codes=codes)))


def test_numpy_numbers_as_sizes(kalm):
    a = attention(np.random.default_rng(16), [3, 20], [9, 30], 4, 1, 8)
    got, _ = run_attention(kalm, a, scale=np.float32(1 / 16), max_q=np.int64(20))
    want, _ = run_attention(kalm, a)
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("lq,nc,n_q,n_kv,page_rows", [
    ([3, 40], [5000, 1], 4, 1, 256),       # a document far longer than the passages' limit
    ([1, 1], [5000, 4097], 4, 1, 8),
    ([0, 0], [10, 20], 4, 1, 16),          # no decoder rows at all
    ([], [], 4, 1, 16),                    # no documents
    ([20, 0, 7], [30, 40, 0], 16, 1, 16),  # 16 query heads per KV head
])
def test_attention_outer_sizes(kalm, lq, nc, n_q, n_kv, page_rows):
    a = attention(np.random.default_rng(sum(nc)), lq, nc, n_q, n_kv, page_rows)
    got, lse = run_attention(kalm, a, poison=True, max_q=max(lq, default=0) or 1)
    want, want_lse, vmax = plain_attention(a)
    if got.size:
        check(got, lse, want, want_lse, vmax)
    assert got.shape == want.shape and kalm.kalm_check_device_errors() == 0


def test_few_rows_shared_inputs_and_last_tile(kalm):
    """The few-row form with shared decoder rows; its last-tile mode computes every row (they fit one tile)."""
    a = attention(np.random.default_rng(35), [2] * 5, [5, 130, 0, 64, 9], 2, 1, 16)
    for k in ("q", "ks", "vs"):
        a[k] = a[k][:2]
    want, want_lse, vmax = plain_attention(a, in_off=[0] * 5)
    got, lse = run_attention(kalm, a, in_off=[0] * 5)
    check(got, lse, want, want_lse, vmax)
    last, _ = run_attention(kalm, a, in_off=[0] * 5, last=True)
    np.testing.assert_array_equal(last, got)
    assert kalm.kalm_check_device_errors() == 0


def test_few_rows_flag_more_rows_than_sized_for(kalm):
    """A document with more decoder rows than max_q, or rows past the inputs: flagged, its output left alone."""
    a = attention(np.random.default_rng(36), [1, 3, 1], [9, 9, 9], 1, 1, 16)
    got, _ = run_attention(kalm, a, max_q=2)
    with pytest.raises(kalm.KalmError):
        kalm.kalm_check_device_errors()
    assert np.isnan(got[1:4]).all() and np.isfinite(got[[0, 4]]).all()


def test_twenty_thousand_documents(kalm):
    """Offsets of more documents than two rounds of the search: single rows written, read, and normed with a gate each."""
    n, width = 20000, 32
    rng = np.random.default_rng(37)
    rows = rng.integers(0, 3, n)
    off = offsets(rows)
    total = int(off[-1])
    v = rand_bf16(rng, (total, width))
    table = rng.permutation(n).astype(np.int32)[:, None]
    codes = torch.zeros(n * 8, width, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(n * 8, 1, dtype=torch.uint8, device="cuda")
    first = rng.integers(0, 6, n)
    kalm.kalm_cache_write(f64_to_dev(v), i64(off), i32(table), 8, codes, scales, first_row=i32(first))
    c, s = quantise(v)
    at = np.concatenate([table[d, 0] * 8 + first[d] + np.arange(rows[d]) for d in range(n)])
    np.testing.assert_array_equal(codes.cpu().numpy()[at], c)
    np.testing.assert_array_equal(scales.cpu().numpy()[at], s)
    back = torch.empty(total, width, dtype=torch.bfloat16, device="cuda")
    kalm.kalm_cache_read(codes, scales, i64(off), i32(table), 8, back, first_row=i32(first))
    np.testing.assert_array_equal(from_dev(back), dequantise(c, s))
    gate = rand_bf16(rng, (n, width))
    out = torch.empty(total, width, dtype=torch.bfloat16, device="cuda")
    kalm.kalm_norm_residual(f64_to_dev(v), torch.zeros_like(out), out, gate=f64_to_dev(gate), q_off=i64(off))
    want = oracle.bf16_round(v * np.repeat(gate, rows, 0))  # exact products of bf16 numbers, one rounding
    np.testing.assert_array_equal(from_dev(out), want)
    assert kalm.kalm_check_device_errors() == 0


@pytest.mark.parametrize("lq,n_q,n_kv", [([4, 3], 1, 1), ([2, 2], 4, 2)])
def test_few_rows_do_not_see_later_values(kalm, lq, n_q, n_kv):
    """A NaN in a self K / V row stays out of the decoder rows before it; those after it have it."""
    a = attention(np.random.default_rng(40), lq, [30, 70], n_q, n_kv, 16)
    want, want_lse, vmax = plain_attention(a)
    last = lq[0] - 1  # of the first document
    a["vs"][last] = np.nan
    a["ks"][last] = np.nan
    got, lse = run_attention(kalm, a)
    assert np.isnan(got[last]).all() and np.isnan(lse[last]).all()
    keep = np.arange(sum(lq)) != last
    check(got[keep], lse[keep], want[keep], want_lse[keep], vmax[keep])
    assert kalm.kalm_check_device_errors() == 0


def test_few_rows_stay_inside_the_output(kalm):
    """A document whose rows lie past total_q (its inputs do exist): flagged, the rows behind total_q left alone."""
    a = attention(np.random.default_rng(41), [1, 1, 1], [9, 9, 9], 1, 1, 16)
    d = 256
    q, ks, vs = (f64_to_dev(a[k].reshape(3, d)) for k in ("q", "ks", "vs"))
    codes, scales = torch.from_numpy(a["codes"]).cuda(), torch.from_numpy(a["scales"]).cuda()
    out = torch.full((3, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    kalm.kalm_merged_attention_cache(q, ks, vs, codes[:, :d], scales[:, :d // 32], codes[:, d:], scales[:, d // 32:],
                                     i32(a["table"]), 16, i64(a["q_off"]), i64(a["p_off"]), 1, 1, 1, out,
                                     in_off=i64([0, 1, 2]), total_q=2)
    with pytest.raises(kalm.KalmError):
        kalm.kalm_check_device_errors()
    got = from_dev(out)
    assert np.isfinite(got[:2]).all() and np.isnan(got[2]).all()


@pytest.mark.parametrize("lq,nc,n_q,n_kv,page_rows", [
    ([8, 7, 1, 0, 5, 8], [16, 0, 1, 15, 33, 64], 1, 1, 64),          # eight positions, self keys in two groups
    ([2, 1, 2], [64, 3, 0], 4, 1, 32),
    ([2, 2, 1, 0], [48, 17, 9, 5], 16, 4, 16),
    ([1, 1], [13, 64], 8, 1, 8),
    ([3], [40], 4, 2, 8),                                            # six rows of eight
    ([8] * 150, [int(n) for n in np.arange(150) * 7 % 129], 1, 1, 128),   # many documents of two pages' length
    ([2] * 160, [int(n) for n in np.arange(160) * 11 % 257], 16, 4, 256),
])
def test_short_documents(kalm, lq, nc, n_q, n_kv, page_rows):
    """Five to eight rows over short or many documents take the few-row launch: nothing is rounded before its output."""
    a = attention(np.random.default_rng(50 + n_q + len(lq)), lq, nc, n_q, n_kv, page_rows)
    got, lse = run_attention(kalm, a, poison=True)
    assert kalm.kalm_check_device_errors() == 0
    want, want_lse, vmax = plain_attention(a)
    check(got, lse, want, want_lse, vmax)
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -15 * vmax[..., None]).all()
    order = lambda q_off, p_off: _order(kalm, q_off, p_off, max(lq), n_q, n_kv)
    last, _ = run_attention(kalm, a, order=None, last=True)
    again, _ = run_attention(kalm, a, order=order)
    np.testing.assert_array_equal(last, got)
    np.testing.assert_array_equal(again, got)


def _order(kalm, q_off, p_off, lq, n_q, n_kv):
    out = torch.empty(kalm.kalm_attention_items(len(q_off) - 1, lq, n_q, n_kv), dtype=torch.int32, device="cuda")
    kalm.kalm_attention_schedule(q_off, p_off, lq, n_q, n_kv, out)
    return out


def test_short_documents_do_not_see_later_values(kalm):
    """Self keys in two groups: a NaN in row 5 of 8 stays out of rows 0 to 4 and reaches 5 to 7."""
    a = attention(np.random.default_rng(60), [8], [20], 1, 1, 32)
    want, want_lse, vmax = plain_attention(a)
    a["vs"][5] = np.nan
    got, lse = run_attention(kalm, a)
    assert np.isnan(got[5:]).all()
    check(got[:5], lse[:5], want[:5], want_lse[:5], vmax[:5])


def test_group_sizes_that_do_not_divide_a_tile(kalm):
    """Three query heads a KV head are refused in a call of few rows as in any other."""
    a = attention(np.random.default_rng(61), [2], [40], 6, 2, 8)
    with pytest.raises(kalm.KalmError, match="must divide 128"):
        run_attention(kalm, a)

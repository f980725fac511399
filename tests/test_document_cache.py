"""The document cache's host side (pages, tables, refusals), without a GPU: the two kernels are replaced by a
plain copy of rows into the pages that the calls name."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from encoder_decoder_document_b200 import document_cache as dc


class Rows:
    """What the calls did: the source row (as its first value) at each cache row."""

    def write(self, src, row_off, table, page_rows, codes, scales, first_row=None):
        off, first = row_off.tolist(), [0] * (len(row_off) - 1) if first_row is None else first_row.tolist()
        for d in range(len(off) - 1):
            for i in range(off[d + 1] - off[d]):
                r = first[d] + i
                page = int(table[d, r // page_rows])
                assert 0 <= page < codes.shape[0] // page_rows
                codes[page * page_rows + r % page_rows] = int(src[off[d] + i, 0])

    def read(self, codes, scales, row_off, table, page_rows, out, first_row=None):
        off = row_off.tolist()
        for d in range(len(off) - 1):
            for i in range(off[d + 1] - off[d]):
                out[off[d] + i] = float(codes[int(table[d, i // page_rows]) * page_rows + i % page_rows, 0])


@pytest.fixture
def cache(monkeypatch):
    rows = Rows()
    monkeypatch.setattr(dc, "kalm_cache_write", rows.write)
    monkeypatch.setattr(dc, "kalm_cache_read", rows.read)
    return dc.DocumentCache(6, 32, page_rows=8, device="cpu")


def numbered(*counts, start=1):
    n = sum(counts)
    return torch.arange(start, start + n, dtype=torch.float32)[:, None].expand(n, 32).to(torch.bfloat16)


def test_put_get_append_drop(cache):
    cache.put(["a", "b", "c"], [3, 0, 9], numbered(3, 0, 9))
    assert len(cache) == 3 and "b" in cache and cache.rows("c") == 9 and cache.free_pages == 3
    rows, off = cache.get(["c", "a", "c"])
    assert off.tolist() == [0, 9, 12, 21]
    assert rows[:, 0].tolist() == [*range(4, 13), 1, 2, 3, *range(4, 13)]
    # one row at a time, across a page's end
    for k in range(7):
        cache.append(["a"], [1], numbered(1, start=50 + k))
    assert cache.rows("a") == 10 and cache.free_pages == 2
    assert cache.get(["a"])[0][:, 0].tolist() == [1, 2, 3, *range(50, 57)]
    cache.append(["b", "a"], [2, 1], numbered(2, 1, start=70))
    assert cache.get(["b", "a"])[0][:, 0].tolist() == [70, 71, 1, 2, 3, *range(50, 57), 72]
    # freed pages are handed out again, other documents keep their rows
    cache.drop(["c"])
    assert "c" not in cache and cache.free_pages == 3
    cache.put(["d"], [24], numbered(24, start=100))
    assert cache.free_pages == 0
    assert cache.get(["d", "b"])[0][:, 0].tolist() == [*range(100, 124), 70, 71]
    assert cache.get([])[0].shape == (0, 32)
    pages = [p for k in ("a", "b", "d") for p in cache._docs[k][0]]
    assert sorted(pages) == list(range(6))  # no page twice


def test_refusals_change_nothing(cache):
    cache.put(["a"], [8], numbered(8))
    before = (cache.free_pages, len(cache))
    for err, call in [
        (KeyError, lambda: cache.put(["a"], [1], numbered(1))),
        (KeyError, lambda: cache.append(["x"], [1], numbered(1))),
        (KeyError, lambda: cache.drop(["x"])),
        (KeyError, lambda: cache.drop(["a", "x"])),
        (KeyError, lambda: cache.view(["x"])),
        (ValueError, lambda: cache.put(["p", "p"], [1, 1], numbered(2))),
        (ValueError, lambda: cache.append(["a", "a"], [1, 1], numbered(2))),
        (ValueError, lambda: cache.drop(["a", "a"])),
        (ValueError, lambda: cache.put(["p"], [-1], numbered(1))),
        (ValueError, lambda: cache.put(["p"], [2], numbered(1))),
        (ValueError, lambda: cache.put(["p", "q"], [1], numbered(1))),
        (MemoryError, lambda: cache.put(["p"], [41], numbered(41))),
        (MemoryError, lambda: cache.append(["a"], [41], numbered(41))),
        (ValueError, lambda: cache.get(["a"], out=torch.empty(7, 32))),
    ]:
        with pytest.raises(err):
            call()
        assert (cache.free_pages, len(cache)) == before and cache.rows("a") == 8
    for kw in (dict(n_pages=-1, width=32), dict(n_pages=1, width=40), dict(n_pages=1, width=0)):
        with pytest.raises(ValueError):
            dc.DocumentCache(**kw, device="cpu")
    with pytest.raises(ValueError):
        dc.DocumentCache(1, 32, page_rows=12, device="cpu")


def test_a_refused_write_takes_no_pages(cache, monkeypatch):
    def refuse(*a, **k):
        raise RuntimeError("refused")
    monkeypatch.setattr(dc, "kalm_cache_write", refuse)
    with pytest.raises(RuntimeError):
        cache.put(["a"], [9], numbered(9))
    assert "a" not in cache and cache.free_pages == 6


def test_tables(cache):
    cache.put([1, 2], [17, 1], numbered(17, 1))
    v = cache.view([2, 1])
    assert v.page_table.dtype == torch.int32 and v.row_off.tolist() == [0, 1, 18] and v.rows == [1, 17]
    assert v.page_table.shape == (2, 3) and v.page_table[0, 1:].tolist() == [-1, -1]
    assert (v.page_table[1] >= 0).all() and v.total_rows == 18
    assert np.array_equal(cache.view([]).row_off.numpy(), [0])

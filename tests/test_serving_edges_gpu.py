"""Serving over a paged KV cache in the states that follow a shortage or bad input."""

import numpy as np
import pytest

from _serving import Pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(cuda_ok):
    import torch

    return torch.device("cuda", 0)


@pytest.fixture(autouse=True)
def no_device_error(cuda_ok):
    import split_kv_decode_bsr_gb300 as sta

    sta.sta_device_error(reset=True)
    yield
    assert sta.sta_device_error(reset=True) == 0


def _i32(dev, a):
    import torch

    return torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)


def _indptr(dev, lens):
    return _i32(dev, np.concatenate([[0], np.cumsum(lens)]))


def _state(pool, dev):
    return _i32(dev, pool.ref), _i32(dev, pool.ptr), _i32(dev, pool.idx), _indptr(dev, pool.kv)


def _buffers(pool, dev, n, elems):
    import torch

    host = [np.random.default_rng(b).integers(0, 1 << 15, (pool.n_pages, elems)).astype(np.int16) for b in range(n)]
    return host, [torch.from_numpy(h.copy()).to(dev) for h in host]


def _same(pool, ref, idx, host=(), bufs=()):
    assert ref.tolist() == pool.ref and idx.tolist() == pool.idx
    for h, b in zip(host, bufs):
        assert np.array_equal(b.cpu().numpy(), h)


# ---- lists with entries that hold no page


def test_pages_compact_passes_over_entries_without_a_page(dev):
    """A pool that ran out of pages is compacted under its grown lengths: the entries that got no page
    stay -1, and nothing is reported."""
    import split_kv_decode_bsr_gb300 as sta

    pool = Pool(90, [20, 30, 0, 9], 8, 8, 10)
    ref, ptr, idx, kv = _state(pool, dev)
    host, bufs = _buffers(pool, dev, 2, 16)
    new = [40, 30, 0, 60]
    assert sta.sta_pages_grow(ref, ptr, idx, kv, _indptr(dev, new), 8).tolist() == pool.grow(new) == [1, 7]
    pool.kv = new
    sta.sta_pages_free(ref, ptr, idx, _indptr(dev, new), _i32(dev, [1]), 8)
    pool.free([1])
    pool.kv[1] = 0
    page_map, status = sta.sta_pages_compact(bufs, ref, ptr, idx, _indptr(dev, pool.kv), 8)
    goes, want = pool.compact(host)
    assert want[1] > 0 and pool.idx[3 * 8:4 * 8].count(-1) == 6
    assert status.tolist() == want and page_map.tolist() == goes
    _same(pool, ref, idx, host, bufs)
    assert sta.sta_device_error() == 0


def test_pages_compact_reports_entries_past_the_pool(dev):
    import split_kv_decode_bsr_gb300 as sta

    pool = Pool(91, [20, 0, 30], 8, 5, 12)
    pool.idx[2], pool.idx[12] = 12, -9
    ref, ptr, idx, kv = _state(pool, dev)
    sta.sta_pages_compact([], ref, ptr, idx, kv, 8)
    got = idx.tolist()
    assert got[2] == 12 and got[12] == -9  # left as they were
    assert sta.sta_device_error(reset=True) == 0x601

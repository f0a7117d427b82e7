"""Serving over a paged KV cache in the states that follow a shortage or bad input: lists with entries
that hold no page, and queries that are no numbers."""

import numpy as np
import pytest

from _serving import PagedCase, Pool, check_chunk

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


def _fork(pool, bufs, parent, child):
    """Pool.fork for parents with entries that hold no page: the child's is -1, and no page is taken for it."""
    free = iter([p for p in range(pool.n_pages) if pool.ref[p] == 0])
    got = missing = 0
    for a, c in zip(parent, child):
        for e in range(pool.need(pool.kv[a])):
            old = pool.idx[pool.ptr[a] + e]
            at = pool.ptr[c] + e
            if not 0 <= old < pool.n_pages:
                pool.idx[at] = -1
            elif (e + 1) * pool.P <= pool.kv[a]:
                pool.idx[at] = old
                pool.ref[old] += 1
            else:
                p = pool.idx[at] = next(free, -1)
                if p < 0:
                    missing += 1
                    continue
                pool.ref[p], got = 1, got + 1
                for b in bufs:
                    b[p] = b[old]
    return [got, missing]


@pytest.mark.parametrize("n_forks", [2, 1300])  # forks that are looked at once, and twice
@pytest.mark.parametrize("entry", [0, 2])       # a whole page; the last, partly filled one
@pytest.mark.parametrize("bad", [-1, -(1 << 31), 0, (1 << 31) - 1])
def test_pages_fork_of_a_parent_without_a_page(dev, bad, entry, n_forks):
    import split_kv_decode_bsr_gb300 as sta

    pool = Pool(92, [20, 30] + [0] * n_forks, 8, 5, 7 + n_forks)
    pool.idx[entry] = bad + pool.n_pages if bad == 0 else bad  # (0: the first number past the pool)
    pool.idx[10:] = [5] * (len(pool.idx) - 10)  # what a child's list held before
    ref, ptr, idx, kv = _state(pool, dev)
    host, bufs = _buffers(pool, dev, 2, 16)
    parent, child = [i % 2 for i in range(n_forks)], [2 + i for i in range(n_forks)]
    status = sta.sta_pages_fork(bufs, ref, ptr, idx, kv, _i32(dev, parent), _i32(dev, child), 8)
    want = _fork(pool, host, parent, child)
    assert want == [n_forks // 2 if entry == 2 else n_forks, 0]
    assert status.tolist() == want
    _same(pool, ref, idx, host, bufs)
    assert sta.sta_device_error(reset=True) == 0x601


def test_pages_fork_after_pages_ran_out(dev):
    """A parent that grew into a shortage is forked under its grown length: its child lacks the same pages."""
    import split_kv_decode_bsr_gb300 as sta

    pool = Pool(93, [20, 9, 0, 0], 8, 8, 7)
    ref, ptr, idx, kv = _state(pool, dev)
    host, bufs = _buffers(pool, dev, 1, 16)
    new = [20, 60, 0, 0]
    assert sta.sta_pages_grow(ref, ptr, idx, kv, _indptr(dev, new), 8).tolist() == pool.grow(new) == [2, 4]
    pool.kv = new
    sta.sta_pages_free(ref, ptr, idx, _indptr(dev, new), _i32(dev, [0]), 8)
    pool.free([0])
    pool.kv[0] = 0
    status = sta.sta_pages_fork(bufs, ref, ptr, idx, _indptr(dev, pool.kv), _i32(dev, [1]), _i32(dev, [2]), 8)
    assert status.tolist() == _fork(pool, host, [1], [2]) == [0, 0]
    _same(pool, ref, idx, host, bufs)
    assert sta.sta_device_error(reset=True) == 0x601


def test_pages_free_leaves_entries_that_it_reports(dev):
    """An entry past the pool, and one whose page is free already, are reported and stay as they were."""
    import split_kv_decode_bsr_gb300 as sta

    for what, code in (("past", 0x601), ("free", 0x603)):
        pool = Pool(94, [30, 20, 40], 8, 6, 20)
        page = pool.idx[1]
        if what == "past":
            pool.idx[1] = 20
        else:
            pool.ref[page] = 0
        ref, ptr, idx, kv = _state(pool, dev)
        sta.sta_pages_free(ref, ptr, idx, kv, _i32(dev, [0, 2, 0]), 8)  # (one named twice)
        stays = pool.idx[1]
        pool.idx[1] = -1
        pool.free([0, 2])
        pool.idx[1] = stays
        _same(pool, ref, idx)
        assert sta.sta_device_error(reset=True) == code


# ---- queries that are no numbers


@pytest.mark.parametrize("splits", [1, 2])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,kv,Hq,Hkv,win,sinks", [(128, 328, 2, 2, 64, 0), (32, 300, 8, 2, 32, 0), (128, 584, 1, 1, 64, 256)])
def test_chunk_nan_query_under_a_window(dev, new, kv, Hq, Hkv, win, sinks, d, splits):
    """A NaN query of a token whose window begins in a later key tile than that of its query tile's first
    token: the LSE is NaN, not that of a token without a key, and the other rows do not change."""
    import split_kv_decode_bsr_gb300 as sta

    c = PagedCase(95, [new, 1], [kv, 40], Hq, Hkv, d, 16)
    x = c.dev(dev)
    kw = dict(pattern=sta.MaskSource.pattern(causal=True, win_lo=1 - win, n_global_cols=sinks), num_splits=splits)
    clean, clean_lse = sta.sta_chunk_fwd_paged(**x, **kw)
    check_chunk(clean, clean_lse, c.ref(d ** -0.5, causal=True, win_lo=1 - win, n_global=sinks), new + 1)
    x["q"][new - 1, 0, 3] = float("nan")
    o, lse = sta.sta_chunk_fwd_paged(**x, **kw)
    assert o[new - 1, 0].isnan().all() and lse[new - 1, 0].isnan()
    o[new - 1, 0], lse[new - 1, 0] = clean[new - 1, 0], clean_lse[new - 1, 0]
    assert o.equal(clean) and lse.equal(clean_lse)

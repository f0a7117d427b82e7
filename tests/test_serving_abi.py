"""CPU checks of the serving calls: every refusal happens on the host, before anything is launched,
and the plain forms that the GPU tests compare with hold on closed cases."""

import ctypes as C
import math

import numpy as np
import pytest

import split_kv_decode_bsr_gb300 as sta
from _serving import Pool, chunk_ref, freqs, rope_ref
from split_kv_decode_bsr_gb300 import build as sta_build

P = 1 << 20  # an aligned pointer value that nothing dereferences
OK, INVALID, UNSUPPORTED, WORKSPACE = sta.STA_OK, sta.STA_ERR_INVALID_ARG, sta.STA_ERR_UNSUPPORTED, sta.STA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    sta_build.build()
    return sta.lib()


def _rope(lib, rope=None, x=P, y=P, pos=P, n=0, H=4, d=64, xs=256, ys=256, tr=0, dtype=sta.STA_BF16, **kw):
    r = sta.Rope(64, **kw) if rope is None else rope
    return lib.sta_rope(x, y, pos, C.byref(r.struct) if r else None, n, H, d, xs, ys, tr, dtype, None)


def test_rope_refusals(lib):
    assert _rope(lib) == OK  # no tokens: nothing launched
    assert _rope(lib, x=None, y=None, pos=None) == OK
    assert _rope(lib, rope=False) == INVALID
    assert _rope(lib, n=-1) == INVALID
    assert _rope(lib, H=0) == INVALID
    assert _rope(lib, d=514, xs=4096, ys=4096) == UNSUPPORTED
    assert _rope(lib, xs=255) == INVALID
    assert _rope(lib, ys=255) == INVALID
    assert _rope(lib, tr=2) == INVALID
    assert _rope(lib, dtype=7) == INVALID
    for rot in (0, -2, 3, 66):
        assert _rope(lib, rope=sta.Rope(rot)) == INVALID
    for kw in (dict(base=1.0), dict(base=math.nan), dict(mscale=0.0), dict(mscale=math.inf), dict(scaling="linear", factor=0.0),
               dict(scaling="blend", factor=2.0), dict(scaling="blend", factor=2.0, orig_len=100, low_turns=4, high_turns=4),
               dict(freqs=[math.nan] * 32)):
        assert _rope(lib, **kw) == INVALID, kw
    r = sta.Rope(64)
    r.struct.layout = 2
    assert _rope(lib, rope=r) == INVALID
    assert _rope(lib, n=1, x=None) == INVALID
    assert _rope(lib, n=1, pos=None) == INVALID
    assert _rope(lib, n=1, x=P + 1) == UNSUPPORTED
    assert _rope(lib, n=1, y=P + 2, x=P, dtype=sta.STA_F32) == UNSUPPORTED
    assert _rope(lib, n=1, pos=P + 2) == UNSUPPORTED
    assert _rope(lib, n=2, xs=256, ys=512) == INVALID  # in place with two strides
    with pytest.raises(ValueError):
        sta.Rope(64, scaling="none at all")
    with pytest.raises(ValueError):
        sta.Rope(64, freqs=[1.0])


def _append(lib, q=P, k=P, v=P, qs=512, ks=128, vs=128, qo=2 * P, kp=3 * P, vp=4 * P, page=16, n_pages=4, n=0, n_req=2, Hq=8,
            Hkv=2, d=64, dtype=sta.STA_BF16, pip=P, pidx=P, qip=P, kip=P, pos=None, rope=None):
    return lib.sta_rope_append_paged(q, k, v, qs, ks, vs, qo, kp, vp, page, n_pages, pip, pidx, qip, kip, pos,
                                     C.byref(rope.struct) if rope else None, n, n_req, Hq, Hkv, d, dtype, None)


def test_append_refusals(lib):
    assert _append(lib) == OK
    assert _append(lib, rope=sta.Rope(64)) == OK
    assert _append(lib, rope=sta.Rope(128)) == INVALID
    assert _append(lib, n=-1) == INVALID
    assert _append(lib, n_req=0) == INVALID
    assert _append(lib, page=0) == INVALID
    assert _append(lib, n_pages=0) == INVALID
    assert _append(lib, Hkv=0) == INVALID
    assert _append(lib, Hq=0) == INVALID  # with a q
    assert _append(lib, Hq=0, q=None, qo=None) == OK
    assert _append(lib, q=None, qo=None) == INVALID  # without one
    assert _append(lib, d=600, qs=9999, ks=9999, vs=9999) == UNSUPPORTED
    assert _append(lib, dtype=sta.STA_F32) == UNSUPPORTED
    assert _append(lib, qs=511) == INVALID
    assert _append(lib, ks=127) == INVALID
    assert _append(lib, vs=127) == INVALID
    for name in ("k", "v", "kp", "vp", "pip", "pidx", "qip", "kip", "qo"):
        assert _append(lib, n=1, **{name: None}) == INVALID, name
    assert _append(lib, n=1, k=P + 1) == UNSUPPORTED
    assert _append(lib, n=1, qip=P + 2) == UNSUPPORTED
    assert _append(lib, n=1, qo=P, qs=640) == INVALID  # in place in rows of a wider tensor


def _chunk(lib, q_indptr=(0, 3, 4), kv_indptr=(0, 30, 50), Hq=8, Hkv=2, d=64, page=16, n_pages=8, q_stride=0, scale=0.1,
           dtype=sta.STA_BF16, splits=0, pattern=None, ws=None, ws_bytes=0, q=P, n_req=None, o=P, kv_null=False, lse=P):
    qi, ki = (C.c_int32 * len(q_indptr))(*q_indptr), (C.c_int32 * len(kv_indptr))(*kv_indptr)
    n = C.c_size_t(ws_bytes)
    st = lib.sta_chunk_fwd_paged(q, q_stride, P, P, page, n_pages, P, P, P, qi, P, None if kv_null else ki,
                                 len(q_indptr) - 1 if n_req is None else n_req, Hq, Hkv, d, dtype, scale,
                                 C.byref(pattern) if pattern is not None else None, splits, o, lse, ws, C.byref(n), None)
    return st, n.value


def test_chunk_refusals(lib):
    assert _chunk(lib)[0] == OK and _chunk(lib)[1] >= 256
    assert _chunk(lib, q_indptr=(0, 0, 0), ws=P, ws_bytes=1 << 30)[0] == OK  # no new token: nothing launched
    assert _chunk(lib, q_indptr=(1, 3, 4))[0] == INVALID
    assert _chunk(lib, q_indptr=(0, 3, 2))[0] == INVALID
    assert _chunk(lib, kv_indptr=(0, 30, 20))[0] == INVALID
    assert _chunk(lib, kv_indptr=(2, 30, 40))[0] == INVALID
    assert _chunk(lib, kv_null=True)[0] == INVALID
    assert _chunk(lib, n_req=0)[0] == INVALID
    assert _chunk(lib, Hq=9)[0] == INVALID
    assert _chunk(lib, Hq=258)[0] == UNSUPPORTED  # 129 query heads per KV head
    assert _chunk(lib, d=96)[0] == UNSUPPORTED
    assert _chunk(lib, dtype=sta.STA_F32)[0] == UNSUPPORTED
    assert _chunk(lib, page=0)[0] == INVALID
    assert _chunk(lib, n_pages=0)[0] == INVALID
    assert _chunk(lib, n_pages=1 << 20, page=1 << 11)[0] == UNSUPPORTED  # 2^31 cache rows
    assert _chunk(lib, scale=0.0)[0] == INVALID
    assert _chunk(lib, scale=math.nan)[0] == INVALID
    assert _chunk(lib, splits=-1)[0] == INVALID
    assert _chunk(lib, splits=1025)[0] == INVALID
    assert _chunk(lib, q_stride=511)[0] == UNSUPPORTED  # not a multiple of 8
    assert _chunk(lib, q_stride=504)[0] == INVALID      # shorter than a row
    dense = sta._MaskSrc()
    dense.kind = sta.STA_MASK_DENSE_U8
    assert _chunk(lib, pattern=dense)[0] == INVALID
    assert _chunk(lib, ws=P, ws_bytes=1)[0] == WORKSPACE
    assert _chunk(lib, ws=P + 16, ws_bytes=1 << 30)[0] == UNSUPPORTED
    assert _chunk(lib, ws=P, ws_bytes=1 << 30, q=None)[0] == INVALID
    assert _chunk(lib, ws=P, ws_bytes=1 << 30, o=None)[0] == INVALID
    assert _chunk(lib, ws=P, ws_bytes=1 << 30, q=P + 8)[0] == UNSUPPORTED
    assert _chunk(lib, ws=P, ws_bytes=1 << 30, lse=P + 2)[0] == UNSUPPORTED


def test_chunk_workspace_grows_with_the_splits(lib):
    # s chunks of (new tokens x query heads) rows, d floats and an LSE each
    st, n = _chunk(lib, splits=5)
    rows = 5 * 4 * 8
    assert st == OK and n >= rows * (64 + 1) * 4
    assert _chunk(lib, splits=1)[1] == 256


def test_chunk_workspace_of_many_requests(lib):
    # planned 1024 requests at a time, over one workspace: that of the largest part
    def need(n_req, kv, splits):
        return sta.chunk_workspace_bytes(np.arange(n_req + 1), np.arange(n_req + 1) * kv, n_req, 8, 2, 64, num_splits=splits)

    assert need(1024, 300, 2) == need(2048, 300, 2) == need(3000, 300, 2) > need(1000, 300, 2)
    assert need(3000, 300, 1) == 256
    assert need(1, 1, 0) == 256  # one key: nothing to cut
    assert need(1, 1 << 20, 0) > 256  # one long sequence: cut over the SMs


def _bufs(n=2, at=P):
    return (C.c_void_p * max(n, 1))(*[at + 4096 * i for i in range(n)])


def test_pages_refusals(lib):
    n = C.c_size_t(0)
    copy = lambda bufs=_bufs(), nb=2, pb=256, np_=8, s=P, d=P, k=0: lib.sta_pages_copy(bufs, nb, pb, np_, s, d, k, None)  # noqa: E731
    assert copy() == OK
    assert copy(k=-1) == INVALID
    assert copy(np_=0) == INVALID
    assert copy(nb=-1) == INVALID
    assert copy(bufs=None) == INVALID
    assert copy(pb=0) == INVALID
    assert copy(pb=24) == UNSUPPORTED
    assert copy(bufs=_bufs(at=P + 8)) == UNSUPPORTED
    assert copy(k=3, s=None) == INVALID
    assert copy(k=3, d=P + 2) == UNSUPPORTED

    def grow(ref=P, np_=8, pip=P, pidx=P, a=P, b=P, n_req=2, page=16, ws=None, nb=0):
        n.value = nb
        return lib.sta_pages_grow(ref, np_, pip, pidx, a, b, n_req, page, None, ws, C.byref(n), None)

    assert grow() == OK and n.value >= 8 * 4
    assert grow(np_=0) == INVALID
    assert grow(np_=(1 << 30) + 1) == INVALID
    assert grow(n_req=0) == INVALID
    assert grow(page=0) == INVALID
    assert grow(ws=P, nb=1) == WORKSPACE
    assert grow(ws=P + 4, nb=4096) == UNSUPPORTED
    for name in ("ref", "pip", "pidx", "a", "b"):
        assert grow(ws=P, nb=4096, **{name: None}) == INVALID, name
    assert grow(ws=P, nb=4096, ref=P + 2) == UNSUPPORTED
    assert lib.sta_pages_grow(P, 8, P, P, P, P, 2, 16, None, None, None, None) == INVALID

    def fork(bufs=_bufs(), nb=2, pb=256, ref=P, np_=8, pip=P, pidx=P, kv=P, n_req=4, page=16, par=P, ch=P, k=2, ws=None, wb=0):
        n.value = wb
        return lib.sta_pages_fork(bufs, nb, pb, ref, np_, pip, pidx, kv, n_req, page, par, ch, k, None, ws, C.byref(n), None)

    assert fork() == OK and n.value >= 4 * (3 * 2 + 4)
    assert fork(k=5) == INVALID  # more forks than requests
    assert fork(k=-1) == INVALID
    assert fork(pb=8) == UNSUPPORTED
    assert fork(nb=0, bufs=None) == OK  # lists only
    assert fork(ws=P, wb=16) == WORKSPACE
    for name in ("ref", "pip", "pidx", "kv", "par", "ch"):
        assert fork(ws=P, wb=1 << 20, **{name: None}) == INVALID, name

    free = lambda ref=P, r=P, k=0, n_req=2: lib.sta_pages_free(ref, 8, P, P, P, n_req, 16, r, k, None)  # noqa: E731
    assert free() == OK
    assert free(k=-1) == INVALID
    assert free(n_req=0) == INVALID
    assert free(k=1, r=None) == INVALID
    assert free(k=1, ref=None) == INVALID
    assert free(k=1, ref=P + 1) == UNSUPPORTED

    def compact(ref=P, np_=8, pip=P, pidx=P, kv=P, mp=P, ws=None, wb=0, pb=256):
        n.value = wb
        return lib.sta_pages_compact(_bufs(), 2, pb, ref, np_, pip, pidx, kv, 2, 16, mp, None, ws, C.byref(n), None)

    assert compact() == OK and n.value >= 2 * 4 * 5 + 4
    assert compact(pb=20) == UNSUPPORTED
    assert compact(ws=P, wb=8) == WORKSPACE
    for name in ("ref", "pip", "pidx", "kv", "mp"):
        assert compact(ws=P, wb=1 << 20, **{name: None}) == INVALID, name


def test_binding_refusals_on_the_host():
    import torch

    z = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    pos = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        sta.sta_rope(z, pos, sta.Rope(64))  # on the host
    with pytest.raises(ValueError):
        sta.sta_rope(z[:, :, ::2], pos, sta.Rope(32))
    with pytest.raises(ValueError):
        sta.sta_pages_copy([], pos, pos)
    with pytest.raises(ValueError):
        sta.sta_pages_copy([z], pos, pos)
    i = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: sta.sta_pages_free(i, i, i, i, pos, 16), lambda: sta.sta_pages_grow(i, i, i, i, i, 16),
                 lambda: sta.sta_pages_compact([], i, i, i, i, 16), lambda: sta.sta_pages_fork([], i, i, i, i, pos, pos, 16)):
        with pytest.raises(ValueError):
            call()
    pages = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sta.sta_chunk_fwd_paged(z, pages, pages, i, i, i, [0, 1, 2], i, [0, 5, 9])
    with pytest.raises(ValueError):
        sta.sta_rope_append_paged(z, z[:, :2], z[:, :2], pages, pages, i, i, i, i)


# ---- the plain forms


def test_rope_plain_form_closed_cases():
    g = np.random.default_rng(0)
    x = g.standard_normal((5, 2, 8))
    pos = np.array([0, 1, 7, 1000, -3])
    f = freqs(8, base=100.0)
    assert np.allclose(f, [1.0, 100 ** -0.25, 0.1, 100 ** -0.75])
    for il in (False, True):
        y, _ = rope_ref(x, pos, f, il)
        assert np.array_equal(y[0], x[0])  # position 0 turns nothing
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        back, _ = rope_ref(y, pos, f, il, transpose=True)
        assert np.allclose(back, x)
        # the transposed turn is the gradient: <T x, z> = <x, T' z>
        z = g.standard_normal(x.shape)
        assert np.isclose((y * z).sum(), (x * rope_ref(z, pos, f, il, transpose=True)[0]).sum())
        # scores depend on the distance of two positions alone
        q0, _ = rope_ref(z, np.full(5, 12), f, il)
        k5, _ = rope_ref(x, np.full(5, 5), f, il)
        q17, _ = rope_ref(z, np.full(5, 17), f, il)
        assert np.allclose((q17 * k5).sum(-1), (q0 * x).sum(-1))
    b = freqs(64, base=10000.0, scaling="blend", factor=8.0, orig_len=4096, low_turns=1, high_turns=32)
    plain = freqs(64)
    turns = 4096 * plain / (2 * math.pi)
    assert np.allclose(b[turns >= 32], plain[turns >= 32]) and np.allclose(b[turns <= 1], plain[turns <= 1] / 8)
    assert np.allclose(freqs(64, scaling="linear", factor=4.0), plain / 4)


def test_chunk_plain_form_closed_cases():
    g = np.random.default_rng(1)
    q, k, v = g.standard_normal((3, 4, 8)), g.standard_normal((7, 2, 8)), g.standard_normal((7, 2, 8))
    o, lse, _, _ = chunk_ref(q, k, v, np.array([0, 1, 6]), 0.3)
    assert np.allclose(o[0, 3], v[0, 1])  # one key: its value
    assert np.allclose(lse[0, 0], 0.3 * q[0, 0] @ k[0, 0])
    o, lse, _, _ = chunk_ref(np.zeros_like(q), k, v, np.array([-1, 2, 6]), 0.3)
    assert (o[0] == 0).all() and np.isneginf(lse[0]).all()  # before the sequence: no key
    assert np.allclose(o[1, 0], v[:3, 0].mean(0)) and np.allclose(lse[1], math.log(3))
    o, lse, _, _ = chunk_ref(np.zeros_like(q), k, v, np.array([4, 5, 6]), 0.3, win_lo=-1, n_global=2)
    assert np.allclose(o[2, 0], v[[0, 1, 5, 6], 0].mean(0))


def test_pool_plain_form():
    import copy

    pool = Pool(3, [5, 0, 17, 32, 0, 0], 8, 6, 24)
    start = copy.deepcopy(pool)
    live = sum(c > 0 for c in pool.ref)
    assert live == 1 + 3 + 4
    buf = np.arange(24.0)
    assert pool.fork([buf], [2, 3], [1, 4]) == [1, 0]
    assert sum(pool.ref) == live + (2 + 1) + 4
    for r, n in ((1, 17), (4, 32)):
        pool.kv[r] = n
    vals = lambda: [[buf[p] for p in pool.idx[pool.ptr[r]:pool.ptr[r] + pool.need(pool.kv[r])]] for r in range(6)]  # noqa: E731
    before = vals()
    assert before[1] == before[2] and before[3] == before[4]
    goes, status = pool.compact([buf])
    assert vals() == before and status[0] == live + 1
    assert all(c > 0 for c in pool.ref[:status[0]]) and not any(pool.ref[status[0]:])
    pool.free([2, 3, 1, 4, 0, 0])
    assert sum(pool.ref) == 0 and set(pool.idx) == {-1}
    assert start.ref != pool.ref

"""CPU checks of the attention over shared prefixes: refusals on the host, and when a prefix is taken apart."""

import ctypes as C
import math

import numpy as np
import pytest

import split_kv_decode_bsr_gb300 as sta
from split_kv_decode_bsr_gb300 import build as sta_build

P = 1 << 20  # an aligned pointer value that nothing dereferences
OK, INVALID, UNSUPPORTED, WORKSPACE = sta.STA_OK, sta.STA_ERR_INVALID_ARG, sta.STA_ERR_UNSUPPORTED, sta.STA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    sta_build.build()
    return sta.lib()


def _i32(x):
    return None if x is None else (C.c_int32 * len(x))(*x)


def _call(lib, q_indptr=(0, 1, 2, 5), kv_indptr=(0, 2066, 4152, 4672), groups=(0, 2, 3), prefix=(2048, 0), n_groups=None, Hq=8, Hkv=2,
          d=64, page=16, n_pages=400, q_stride=0, scale=0.1, dtype=sta.STA_BF16, splits=0, ws=None, ws_bytes=0, q=P, o=P, lse=P,
          n_req=None):
    n = C.c_size_t(ws_bytes)
    st = lib.sta_prefix_fwd_paged(q, q_stride, P, P, page, n_pages, P, P, P, _i32(q_indptr), P, _i32(kv_indptr),
                                  len(q_indptr) - 1 if n_req is None else n_req, _i32(groups), _i32(prefix),
                                  len(groups or (0, 0)) - 1 if n_groups is None else n_groups, Hq, Hkv, d, dtype, scale, splits, o, lse,
                                  ws, C.byref(n), None)
    return st, n.value


def test_prefix_refusals(lib):
    st, size = _call(lib)
    assert st == OK and size > 256
    assert _call(lib, q_indptr=(0, 0, 0, 0), ws=P, ws_bytes=1 << 30)[0] == OK  # no new token: nothing launched
    for groups in (None, (1, 2, 3), (0, 2, 4), (0, 2, 2), (0, 3, 2, 3)[:3]):
        assert _call(lib, groups=groups)[0] == INVALID, groups
    assert _call(lib, groups=(0, 3, 2, 3), prefix=(0, 0, 0))[0] == INVALID
    assert _call(lib, groups=(0, 2, 2, 3), prefix=(2048, 64, 0))[0] == OK  # an empty group
    assert _call(lib, prefix=None)[0] == INVALID
    assert _call(lib, n_groups=0)[0] == INVALID
    assert _call(lib, prefix=(-16, 0))[0] == INVALID
    assert _call(lib, prefix=(500, 0))[0] == INVALID  # no whole pages
    assert _call(lib, prefix=(2080, 0))[0] == INVALID  # longer than what the first request has
    assert _call(lib, prefix=(2064, 0))[0] == OK  # up to its new token
    assert _call(lib, prefix=(2048, 512))[0] == OK
    assert _call(lib, prefix=(2048, 528))[0] == INVALID  # the last request's new tokens reach into it
    assert _call(lib, q_indptr=(0, 0, 1, 4), prefix=(2080, 0))[0] == OK  # a request without new tokens does not count
    assert _call(lib, q_indptr=(1, 1, 2, 5))[0] == INVALID
    assert _call(lib, kv_indptr=(0, 2066, 500, 4672))[0] == INVALID
    assert _call(lib, n_req=0)[0] == INVALID
    assert _call(lib, Hq=9)[0] == INVALID
    assert _call(lib, Hq=258)[0] == UNSUPPORTED
    assert _call(lib, d=96)[0] == UNSUPPORTED
    assert _call(lib, dtype=sta.STA_F32)[0] == UNSUPPORTED
    assert _call(lib, page=0)[0] == INVALID
    assert _call(lib, scale=math.nan)[0] == INVALID
    assert _call(lib, splits=1025)[0] == INVALID
    assert _call(lib, q_stride=511)[0] == UNSUPPORTED
    assert _call(lib, ws=P, ws_bytes=size - 1) == (WORKSPACE, size)
    assert _call(lib, ws=P + 16, ws_bytes=1 << 30)[0] == UNSUPPORTED
    assert _call(lib, ws=P, ws_bytes=1 << 30, q=None)[0] == INVALID
    assert _call(lib, ws=P, ws_bytes=1 << 30, o=None)[0] == INVALID
    assert _call(lib, ws=P, ws_bytes=1 << 30, q=P + 8)[0] == UNSUPPORTED
    assert _call(lib, ws=P, ws_bytes=1 << 30, lse=P + 2)[0] == UNSUPPORTED


def _need(new, own, sizes, prefix, Hq=32, Hkv=8, d=128, page=16, splits=0):
    mine = np.repeat(np.arange(len(sizes)), sizes)
    q, kv = np.concatenate([[0], np.cumsum(new)]), np.concatenate([[0], np.cumsum(np.array(prefix)[mine] + own)])
    args = (q.astype(np.int32), kv.astype(np.int32), len(new))
    shared = sta.prefix_workspace_bytes(*args, np.concatenate([[0], np.cumsum(sizes)]), prefix, Hq, Hkv, d, page, splits)
    return shared, sta.chunk_workspace_bytes(*args, Hq, Hkv, d, page, num_splits=splits)


def test_what_is_shared():
    one = np.ones(64, np.int32)
    # a row of partials, d floats and an LSE, for the prefix and one for each request's own part
    rows = 64 * 32
    assert _need(one, one * 100, [64], [8192], splits=1)[0] >= 2 * rows * (128 + 1) * 4 > _need(one, one * 100, [64], [8192], splits=1)[1]
    # no prefix, requests alone in their groups, or one with new tokens: the chunk attention's plan
    for sizes, prefix in (([64], [0]), ([1] * 64, [8192] * 64)):
        a, b = _need(one, one * 100, sizes, prefix)
        assert a == b
    new = np.zeros(64, np.int32)
    new[5] = 1
    a, b = _need(new, one * 100, [64], [8192])
    assert a == b
    # more requests than one launch plans
    assert _need(np.ones(3000, np.int32), np.full(3000, 40), [3000], [2048], splits=1)[0] > 256


def test_binding_refusals_on_the_host():
    import torch

    z = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    i, pages = torch.zeros(3, dtype=torch.int32), torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    args = (z, pages, pages, i, i, i, [0, 1, 2], i, [0, 17, 34])
    for groups, prefix in (([0, 2], [16]), ([0], []), ([0, 2], [16, 16]), ([], [])):
        with pytest.raises(ValueError):
            sta.sta_prefix_fwd_paged(*args, groups, prefix)

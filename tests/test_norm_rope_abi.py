"""CPU checks of the norm calls: refusals on the host, before anything is launched, and the plain forms that
the GPU tests compare with against closed cases and differences."""

import ctypes as C
import math

import numpy as np
import pytest

import split_kv_decode_bsr_gb300 as sta
from _norm import norm_bwd_ref, norm_ref
from _serving import freqs
from split_kv_decode_bsr_gb300 import build as sta_build

P = 1 << 20  # an aligned pointer value that nothing dereferences
OK, INVALID, UNSUPPORTED, WORKSPACE = sta.STA_OK, sta.STA_ERR_INVALID_ARG, sta.STA_ERR_UNSUPPORTED, sta.STA_ERR_WORKSPACE
NO_ROPE = object()


@pytest.fixture(scope="module")
def lib():
    sta_build.build()
    return sta.lib()


def _rope(rope):
    return None if rope is NO_ROPE else C.byref((rope or sta.Rope(64)).struct)


def _fwd(lib, q=P, k=2 * P, qs=256, ks=128, qo=3 * P, ko=4 * P, qos=256, kos=128, qw=P, kw=P, eps=1e-6, pos=P, rope=None, n=0,
         Hq=4, Hk=2, d=64, dtype=sta.STA_BF16):
    return lib.sta_norm_rope(q, k, qs, ks, qo, ko, qos, kos, qw, kw, eps, pos, _rope(rope), n, Hq, Hk, d, dtype, None)


def test_norm_rope_refusals(lib):
    assert _fwd(lib) == OK  # no tokens: nothing launched
    assert _fwd(lib, q=None, k=None, qo=None, ko=None, pos=None) == OK
    assert _fwd(lib, rope=NO_ROPE, pos=None) == OK
    assert _fwd(lib, n=-1) == INVALID
    assert _fwd(lib, Hq=0) == INVALID  # with a q
    assert _fwd(lib, Hk=0) == INVALID
    assert _fwd(lib, Hk=0, k=None, ko=None) == OK
    assert _fwd(lib, Hq=0, q=None, qo=None) == OK
    assert _fwd(lib, Hq=0, q=None, qo=None, Hk=0, k=None, ko=None) == INVALID
    assert _fwd(lib, Hq=65537, qs=1 << 23, qos=1 << 23) == INVALID
    assert _fwd(lib, Hk=-1) == INVALID
    assert _fwd(lib, d=1, rope=NO_ROPE) == INVALID
    assert _fwd(lib, d=514, qs=4096, ks=4096, qos=4096, kos=4096) == UNSUPPORTED
    for name, least in (("qs", 256), ("ks", 128), ("qos", 256), ("kos", 128)):
        assert _fwd(lib, **{name: least - 1}) == INVALID, name
    for eps in (0.0, -1e-6, math.nan, math.inf):
        assert _fwd(lib, eps=eps) == INVALID
    assert _fwd(lib, dtype=7) == INVALID
    assert _fwd(lib, rope=sta.Rope(66)) == INVALID
    assert _fwd(lib, rope=sta.Rope(64, base=1.0)) == INVALID
    for name in ("q", "k", "qo", "ko", "pos"):
        assert _fwd(lib, n=1, **{name: None}) == INVALID, name
    for name in ("q", "k", "qo", "ko"):
        assert _fwd(lib, n=1, **{name: 5 * P + 1}) == UNSUPPORTED, name
        assert _fwd(lib, n=1, dtype=sta.STA_F32, **{name: 5 * P + 2}) == UNSUPPORTED, name
    for name in ("qw", "kw", "pos"):
        assert _fwd(lib, n=1, **{name: P + 2}) == UNSUPPORTED, name
    assert _fwd(lib, n=2, qo=P, qos=512) == INVALID  # in place with two strides


def _bwd(lib, dqo=P, dko=2 * P, yqs=256, yks=128, q=3 * P, k=4 * P, qs=256, ks=128, dq=5 * P, dk=6 * P, dqs=256, dks=128, qw=P,
         kw=P, dqw=P, dkw=P, eps=1e-6, pos=P, rope=None, n=1, Hq=4, Hk=2, d=64, dtype=sta.STA_BF16, ws=P, wb=1 << 30):
    size = C.c_size_t(wb)
    st = lib.sta_norm_rope_bwd(dqo, dko, yqs, yks, q, k, qs, ks, dq, dk, dqs, dks, qw, kw, dqw, dkw, eps, pos, _rope(rope), n, Hq,
                               Hk, d, dtype, ws, C.byref(size), None)
    return st, size.value


def test_norm_rope_bwd_refusals(lib):
    st, size = _bwd(lib, ws=None)
    assert st == OK and size >= 152 * 2 * 64 * 4
    assert _bwd(lib, ws=None, n=1 << 20, Hq=40, qs=1 << 20, dqs=1 << 20, yqs=1 << 20)[1] == size  # by d alone
    assert _bwd(lib, wb=size - 1) == (WORKSPACE, size)
    assert _bwd(lib, ws=P + 16)[0] == UNSUPPORTED
    assert lib.sta_norm_rope_bwd(P, P, 256, 128, P, P, 256, 128, P, P, 256, 128, P, P, P, P, 1e-6, P, None, 0, 4, 2, 64, 0, P, None,
                                 None) == INVALID
    assert _bwd(lib, n=0, dqw=None, dkw=None)[0] == OK  # nothing to write: nothing launched
    assert _bwd(lib, n=-1)[0] == INVALID
    assert _bwd(lib, eps=0.0)[0] == INVALID
    assert _bwd(lib, dtype=7)[0] == INVALID
    assert _bwd(lib, rope=sta.Rope(66))[0] == INVALID
    assert _bwd(lib, Hk=0)[0] == INVALID
    assert _bwd(lib, Hk=0, k=None, dk=None, dko=None)[0] == INVALID  # a weight's gradient of a tensor that is not there
    assert _bwd(lib, n=0, Hk=0, k=None, dk=None, dko=None, dkw=None, dqw=None)[0] == OK
    for name, least in (("yqs", 256), ("yks", 128), ("qs", 256), ("ks", 128), ("dqs", 256), ("dks", 128)):
        assert _bwd(lib, **{name: least - 1})[0] == INVALID, name
    for name in ("dqo", "dko", "q", "k", "dq", "dk", "pos"):
        assert _bwd(lib, **{name: None})[0] == INVALID, name
        assert _bwd(lib, **{name: 7 * P + 1})[0] == UNSUPPORTED, name
    for name in ("qw", "kw", "dqw", "dkw"):
        assert _bwd(lib, **{name: P + 2})[0] == UNSUPPORTED, name
    assert _bwd(lib, dq=P, dqs=512)[0] == INVALID  # over dq_out with another stride
    assert _bwd(lib, dk=4 * P, dks=512)[0] == INVALID  # over k


def _append(lib, q=P, k=P, v=P, qs=512, ks=128, vs=128, qo=2 * P, kp=3 * P, vp=4 * P, page=16, n_pages=4, n=0, n_req=2, Hq=8,
            Hkv=2, d=64, dtype=sta.STA_BF16, pip=P, pidx=P, qip=P, kip=P, pos=None, qw=P, kw=P, eps=1e-6, rope=None):
    return lib.sta_norm_rope_append_paged(q, k, v, qs, ks, vs, qo, kp, vp, page, n_pages, pip, pidx, qip, kip, pos, qw, kw, eps,
                                          _rope(rope), n, n_req, Hq, Hkv, d, dtype, None)


def test_norm_append_refusals(lib):
    assert _append(lib) == OK
    assert _append(lib, rope=NO_ROPE) == OK
    assert _append(lib, qw=None, kw=None) == OK
    assert _append(lib, rope=sta.Rope(128)) == INVALID
    for name in ("n", "n_req", "page", "n_pages", "Hkv"):
        assert _append(lib, **{name: -1}) == INVALID, name
    assert _append(lib, Hkv=0) == INVALID
    assert _append(lib, Hq=0) == INVALID  # with a q
    assert _append(lib, Hq=0, q=None, qo=None) == OK
    assert _append(lib, q=None, qo=None) == INVALID  # without one
    assert _append(lib, eps=0.0) == INVALID
    assert _append(lib, d=600, qs=9999, ks=9999, vs=9999) == UNSUPPORTED
    assert _append(lib, dtype=sta.STA_F32) == UNSUPPORTED
    for name, least in (("qs", 512), ("ks", 128), ("vs", 128)):
        assert _append(lib, **{name: least - 1}) == INVALID, name
    for name in ("k", "v", "kp", "vp", "pip", "pidx", "qip", "kip", "qo"):
        assert _append(lib, n=1, **{name: None}) == INVALID, name
    assert _append(lib, n=1, k=P + 1) == UNSUPPORTED
    for name in ("qip", "pos", "qw", "kw"):
        assert _append(lib, n=1, **{name: P + 2}) == UNSUPPORTED, name
    assert _append(lib, n=1, qo=P, qs=640) == INVALID  # in place in rows of a wider tensor


def test_binding_refusals_on_the_host():
    import torch

    z = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    pos = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: sta.sta_norm_rope(z, z, pos, sta.Rope(64)),  # on the host
                 lambda: sta.sta_norm_rope(None, None, pos, sta.Rope(64)),
                 lambda: sta.sta_norm_rope(z[0], None, pos, sta.Rope(64)),
                 lambda: sta.sta_norm_rope_bwd(z, z, z, z, pos, sta.Rope(64)),
                 lambda: sta.sta_norm_rope_append_paged(z, z[:, :2], z[:, :2], z[None], z[None], pos, pos, pos, pos)):
        with pytest.raises(ValueError):
            call()


# ---- the plain forms


def test_norm_plain_form_closed_cases():
    g = np.random.default_rng(0)
    x, pos, f = g.standard_normal((5, 2, 8)), np.array([0, 1, 7, 1000, -3]), freqs(6, base=100.0)
    for il in (False, True):
        y, _ = norm_ref(3.0 * x, None, 1e-30, pos, f, il)
        assert np.allclose((y ** 2).mean(-1), 1.0)  # of unit size at any scale and position
        assert np.allclose(norm_ref(x, None, 1e-30, pos, f, il)[0], y)
        w = g.standard_normal(8)
        assert np.allclose(norm_ref(x, w, 0.5, pos, np.zeros(0), il)[0], x / np.sqrt((x ** 2).mean(-1, keepdims=True) + 0.5) * w)
    assert (norm_ref(np.zeros((1, 1, 8)), None, 1e-6, pos[:1], f, False)[0] == 0).all()


def test_norm_gradient_plain_form_against_differences():
    g = np.random.default_rng(1)
    x, dy, w = g.standard_normal((4, 3, 10)), g.standard_normal((4, 3, 10)), g.standard_normal(10)
    pos, f, eps = np.array([0, 5, 70, 4000]), freqs(6), 1e-2
    for il in (False, True):
        loss = lambda a, b: (norm_ref(a, b, eps, pos, f, il, 1.25)[0] * dy).sum()  # noqa: E731
        dx, dw, _, _ = norm_bwd_ref(dy, x, w, eps, pos, f, il, 1.25)
        h = 1e-5  # central differences in 64 bits: off by h^2 of third derivatives of some units, and 1e-16 / h
        for at in np.ndindex(*x.shape):
            e = np.zeros_like(x)
            e[at] = h
            assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[at]) < 1e-7
        for p in range(10):
            e = np.zeros(10)
            e[p] = h
            assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[p]) < 1e-7

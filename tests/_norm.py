"""Plain 64-bit forms of the norms of query and key heads with rotary positions, and bounds on their errors."""

import numpy as np

from _serving import rope_ref

U = 2.0 ** -24  # half a step of fp32, relative


def _eta(d):
    """Relative error of a normed element before its turn: the fp32 sum of d squares is off by d + 8 roundings at
    most, which the root halves; rsqrtf by 2^-22; the mean, eps and the products by half a step each."""
    return ((d + 8) / 2 + 8) * U


def _spread(a, rot, interleaved):
    """|a| + |b| of each element's pair where it turns, else 0."""
    i = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    j = i + 1 if interleaved else i + rot // 2
    out = np.zeros_like(a)
    out[..., i] = out[..., j] = np.abs(a[..., i]) + np.abs(a[..., j])
    return out


def norm_ref(x, w, eps, pos, f, interleaved, mscale=1.0):
    """x [n, H, d] float64, w [d] or None: the result, and the bound on fp32 arithmetic before the last rounding."""
    d, rot = x.shape[-1], 2 * len(f)
    xn = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * (1.0 if w is None else w)
    y, err = rope_ref(xn, pos, f, interleaved, mscale)
    part = np.abs(xn)
    part[..., :rot] = _spread(xn, rot, interleaved)[..., :rot] * mscale
    return y, err + _eta(d) * part


def norm_bwd_ref(dy, x, w, eps, pos, f, interleaved, mscale=1.0, chain=200):
    """dx, dw and the bounds on fp32 arithmetic before their last rounding. chain: fp32 additions that a term of dw
    goes through (a thread's heads, 5 of a warp, 8 of a CTA's warps, then the CTAs' sums)."""
    d = x.shape[-1]
    w = np.ones(d) if w is None else w
    g, err_g = rope_ref(dy, pos, f, interleaved, mscale, transpose=True)
    r = 1 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    s = (g * w * x).sum(-1, keepdims=True)
    c = r ** 3 * s / d
    dx, dw = r * g * w - x * c, (g * x * r).sum((0, 1))
    eta = _eta(d)
    err_s = (err_g * np.abs(w * x)).sum(-1, keepdims=True) + (d + 8) * U * np.abs(g * w * x).sum(-1, keepdims=True)
    tol = np.abs(r * w) * err_g + (eta + 4 * U) * np.abs(r * g * w) + np.abs(x) * ((3 * eta + 8 * U) * np.abs(c) + r ** 3 / d * err_s)
    dw_tol = (np.abs(x * r) * err_g + (eta + (3 + chain) * U) * np.abs(g * x * r)).sum((0, 1))
    return dx, dw, tol, dw_tol

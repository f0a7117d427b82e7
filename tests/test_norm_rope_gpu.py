"""Norms of query and key heads with rotary positions on the GPU, against plain 64-bit forms: the pass itself,
its gradient, and the write of normed keys into pages."""

import numpy as np
import pytest

from _norm import norm_bwd_ref, norm_ref
from _serving import BF16_HALF_STEP, F32_HALF_STEP, PagedCase, freqs

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


def _np(t):
    return t.double().cpu().numpy()


def _close(got, ref, tol, step, what):
    """Within the bound of its fp32 arithmetic and one rounding."""
    off = np.abs(_np(got) - ref) - (step * np.abs(ref) + tol * (1 + step) + 1e-38)
    assert off.max(initial=0) <= 0, f"{what}: {off.max():.3e} past its bound"


class Case:
    """q and k in one packed tensor of `pad` more elements, positions of both signs, weights around 1."""

    def __init__(self, dev, n, Hq, Hk, d, rot, interleaved, dtype, pad=0, weights=True, max_pos=4096, seed=0, scale=1.0, eps=1e-6,
                 **rope):
        import torch

        import split_kv_decode_bsr_gb300 as sta

        g = np.random.default_rng(seed)
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.step = BF16_HALF_STEP if dtype == "bf16" else F32_HALF_STEP
        to = lambda a: torch.from_numpy(a.astype(np.float32)).to(dev)  # noqa: E731
        self.wide = to(scale * g.standard_normal((n, (Hq + Hk) * d + pad))).to(self.dt)
        self.split(Hq, Hk, d)
        pos = g.integers(-max_pos, max_pos, n).astype(np.int32)
        pos[:2] = [0, max_pos - 1][:min(n, 2)]
        self.pos = torch.from_numpy(pos).to(dev)
        self.qw, self.kw = (to(1 + 0.3 * g.standard_normal(d)) for _ in range(2)) if weights else (None, None)
        self.eps, self.il = eps, interleaved
        self.mscale = rope.pop("mscale", 1.0)
        self.rope = sta.Rope(rot, interleaved=interleaved, mscale=self.mscale, **rope) if rot else None
        self.f = freqs(rot, **rope) if rot else np.zeros(0)
        self.dy = [to(g.standard_normal((n, H, d))).to(self.dt) if H else None for H in (Hq, Hk)]

    def split(self, Hq, Hk, d):
        self.q = self.wide[:, :Hq * d].unflatten(1, (Hq, d)) if Hq else None
        self.k = self.wide[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d)) if Hk else None

    def args(self):
        return self.pos if self.rope else None, self.rope

    def kw_args(self):
        return dict(q_weight=self.qw, k_weight=self.kw, eps=self.eps)

    def parts(self):
        return [(x, w, dy) for x, w, dy in ((self.q, self.qw, self.dy[0]), (self.k, self.kw, self.dy[1]))]

    def ref(self, x, w, at=slice(None)):
        return norm_ref(_np(x[at]), None if w is None else _np(w), self.eps, self.pos[at].cpu().numpy(), self.f, self.il,
                        np.float32(self.mscale))

    def check_forward(self, got, at=slice(None)):
        for y, (x, w, _) in zip(got, self.parts()):
            if x is None:
                assert y is None
            else:
                assert y.shape == x.shape and y.dtype == x.dtype
                _close(y[at], *self.ref(x, w, at), self.step, "y")


SHAPES = [(1, 1, 0, 2, 2, 0), (3, 5, 2, 128, 128, 0), (70, 32, 8, 128, 64, 8), (33, 3, 3, 80, 40, 16), (17, 2, 1, 96, 30, 3),
          (5, 7, 2, 63, 6, 0), (9, 1, 1, 512, 512, 1), (4, 2, 3, 512, 512, 8), (4, 1, 1, 512, 16, 0), (300, 2, 0, 64, 64, 24),
          (6, 0, 4, 64, 32, 0), (2, 3, 1, 256, 0, 0), (1, 3, 1, 7, 0, 5), (50, 1, 1, 2, 2, 0), (50, 6, 2, 128, 42, 8),
          (7, 2, 2, 64, 62, 0), (5, 1, 3, 256, 2, 16), (3, 2, 1, 512, 510, 0), (9, 3, 1, 40, 36, 8), (90, 5, 1, 32, 10, 0)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,Hq,Hk,d,rot,pad", SHAPES)
def test_norm_rope(dev, n, Hq, Hk, d, rot, pad, interleaved, dtype):
    import split_kv_decode_bsr_gb300 as sta

    c = Case(dev, n, Hq, Hk, d, rot, interleaved, dtype, pad, seed=n)
    got = sta.sta_norm_rope(c.q, c.k, *c.args(), **c.kw_args())
    c.check_forward(got)
    # in place in the packed tensor: the same numbers, and nothing else of it touched (a row's alignment may differ from
    # the results' above, and with it the order of a head's sum)
    wide = c.wide.clone()
    want = Case(dev, n, Hq, Hk, d, rot, interleaved, dtype, pad, seed=n)
    got = sta.sta_norm_rope(c.q, c.k, *c.args(), **c.kw_args(), q_out=c.q, k_out=c.k)
    assert got[0] is c.q and got[1] is c.k
    want.check_forward(got)
    assert (c.wide[:, (Hq + Hk) * d:] == wide[:, (Hq + Hk) * d:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,Hq,Hk,d,rot,pad", SHAPES)
def test_norm_rope_gradients(dev, n, Hq, Hk, d, rot, pad, interleaved, dtype):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = Case(dev, n, Hq, Hk, d, rot, interleaved, dtype, pad, seed=n, mscale=1.25 if rot else 1.0, eps=1e-3)
    got = sta.sta_norm_rope_bwd(*c.dy, c.q, c.k, *c.args(), **c.kw_args())
    for i, (x, w, dy) in enumerate(c.parts()):
        if x is None:
            assert got[i] is None and got[2 + i] is None
            continue
        dx, dw, tol, dw_tol = norm_bwd_ref(_np(dy), _np(x), _np(w), c.eps, c.pos.cpu().numpy(), c.f, c.il, np.float32(c.mscale))
        assert got[i].shape == x.shape and got[i].dtype == x.dtype and got[2 + i].dtype == torch.float32
        _close(got[i], dx, tol, c.step, "dx")
        _close(got[2 + i], dw, dw_tol, F32_HALF_STEP, "dw")
    # the same bits again, in place over the results' gradients
    again = sta.sta_norm_rope_bwd(*c.dy, c.q, c.k, *c.args(), **c.kw_args(), dq=c.dy[0], dk=c.dy[1])
    for a, b in zip(again, got):
        assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_rope_gradient_against_differences(dev, dtype):
    # <(f(x + h z) - f(x - h z)) / 2h, dy> of the kernel's own results against <z, dx>: off by the results' bounds over 2h, by
    # what the 64-bit form's own difference is off its gradient, and by the gradient's bound
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = Case(dev, 40, 3, 0, 64, 48, True, dtype, eps=1e-2, mscale=1.25)
    x, dy, h = c.q.float(), c.dy[0], 2.0 ** -4
    z = torch.randn(x.shape, device=dev).to(c.dt)
    ends = [(x + s * h * z.float()).to(c.dt) for s in (1, -1)]  # rounded: the difference goes by what they hold
    dz = (_np(ends[0]) - _np(ends[1])) / (2 * h)
    f = [sta.sta_norm_rope(e, None, *c.args(), q_weight=c.qw, eps=c.eps)[0] for e in ends]
    refs = [c.ref(e, c.qw) for e in ends]
    mid = (ends[0].float() + ends[1].float()).div(2).to(torch.float32)
    w = _np(dy)
    diff = ((_np(f[0]) - _np(f[1])) * w).sum() / (2 * h)
    allowed = sum(((c.step * np.abs(r) + t * (1 + c.step)) * np.abs(w)).sum() for r, t in refs) / (2 * h)
    # the gradient at the middle, in 32 bits: the middle of two bf16 numbers is exact there
    dx = sta.sta_norm_rope_bwd(dy.float(), None, mid, None, *c.args(), q_weight=c.qw, eps=c.eps)[0]
    g, _, tol, _ = norm_bwd_ref(w, _np(mid), _np(c.qw), c.eps, c.pos.cpu().numpy(), c.f, True, np.float32(1.25))
    curve = abs(((refs[0][0] - refs[1][0]) * w).sum() / (2 * h) - (dz * g).sum())
    allowed += curve + ((tol + F32_HALF_STEP * np.abs(g)) * np.abs(dz)).sum()
    assert abs(diff - (dz * _np(dx)).sum()) <= allowed


@pytest.mark.parametrize("kw", [dict(base=500000.0), dict(scaling="blend", factor=32.0, orig_len=8192.0, low_turns=1.0,
                                                          high_turns=4.0, mscale=1.35)])
def test_norm_rope_far_positions(dev, kw):
    # positions to 2^20: the 64-bit angles of the plain form are exact to 1e-10 there
    import split_kv_decode_bsr_gb300 as sta

    c = Case(dev, 64, 3, 2, 32, 32, False, "f32", max_pos=1 << 20, **kw)
    c.check_forward(sta.sta_norm_rope(c.q, c.k, *c.args(), **c.kw_args()))


@pytest.mark.parametrize("interleaved,rot", [(False, 42), (False, 64), (True, 42), (True, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_rope_what_is_infinite_past_the_rotation_stays_there(dev, interleaved, rot, dtype):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = Case(dev, 5, 3, 2, 128, rot, interleaved, dtype, seed=rot)
    c.dy[0][2, 1, rot] = float("inf")
    dqw = sta.sta_norm_rope_bwd(*c.dy, c.q, c.k, *c.args(), **c.kw_args())[2]
    assert torch.isinf(dqw[rot]) and torch.isfinite(dqw).sum() == 127
    c.qw[rot] = float("inf")
    y = sta.sta_norm_rope(c.q, c.k, *c.args(), **c.kw_args())[0]
    assert torch.isinf(y[..., rot]).all() and torch.isfinite(y).sum() == 5 * 3 * 127


def test_norm_rope_a_refused_call_raises_and_leaves_the_device_as_it_was(dev):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = Case(dev, 5, 3, 2, 64, 64, False, "bf16")
    for call in (lambda **kw: sta.sta_norm_rope(c.q, c.k, *c.args(), **kw),
                 lambda **kw: sta.sta_norm_rope_bwd(*c.dy, c.q, c.k, *c.args(), **kw)):
        for kw in (dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf"))):
            with pytest.raises(sta.StaError):
                call(**kw)
        with pytest.raises(ValueError):
            call(q_weight=c.qw[:32])
        with pytest.raises(ValueError):
            call(q_weight=c.qw.cpu())
    with pytest.raises(sta.StaError):  # more turns than the head has
        sta.sta_norm_rope(c.q, c.k, c.pos, sta.Rope(66))
    torch.cuda.synchronize()
    c.check_forward(sta.sta_norm_rope(c.q, c.k, *c.args(), **c.kw_args()))


def test_norm_rope_no_weights_zero_rows_and_sizes(dev):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    for scale in (1e-12, 1e12):  # below eps, and squares near 1e26
        c = Case(dev, 9, 2, 2, 64, 64, False, "f32", weights=False, scale=scale)
        c.wide[3] = 0.0
        got = sta.sta_norm_rope(c.q, c.k, *c.args(), **c.kw_args())
        c.check_forward(got)
        assert (got[0][3] == 0).all()
    grads = sta.sta_norm_rope_bwd(*c.dy, c.q, c.k, *c.args(), **c.kw_args())
    assert all(torch.isfinite(t).all() for t in grads) and grads[2].shape == (64,)
    # a row that is no number stays one, and its neighbours do not see it
    c.wide[4, 5] = float("nan")
    y = sta.sta_norm_rope(c.q, c.k, *c.args(), **c.kw_args())[0]
    assert torch.isnan(y[4, 0]).all() and torch.isfinite(y[4, 1]).all() and torch.isfinite(y[5]).all()
    e = torch.empty(0, 2, 64, device=dev)
    none = torch.empty(0, dtype=torch.int32, device=dev)
    assert sta.sta_norm_rope(e, None, none, sta.Rope(64))[0].shape == (0, 2, 64)
    dq, dk, dqw, dkw = sta.sta_norm_rope_bwd(e, None, e, None, none, sta.Rope(64))
    assert dq.shape == (0, 2, 64) and dk is None and dkw is None and (dqw == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_rope_many_tokens(dev, dtype):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    n, Hq, Hk, d = 20011, 6, 2, 128  # several tokens a block, many steps of a block, a partial last one
    c = Case(dev, n, Hq, Hk, d, d, False, dtype, max_pos=1 << 20)
    got = sta.sta_norm_rope(c.q, c.k, *c.args(), **c.kw_args())
    pick = torch.from_numpy(np.r_[0:40, n // 2:n // 2 + 40, n - 40:n])
    c.check_forward(got, pick)
    got = sta.sta_norm_rope_bwd(*c.dy, c.q, c.k, *c.args(), **c.kw_args())
    for i, (x, w, dy) in enumerate(c.parts()):
        dx, _, tol, _ = norm_bwd_ref(_np(dy[pick]), _np(x[pick]), _np(w), c.eps, c.pos[pick].cpu().numpy(), c.f, c.il)
        _close(got[i][pick], dx, tol, c.step, "dx")
        # a thread adds the heads of its places: at most n H / 8 / 600 of them and a step's rest, then the joins
        _, dw, _, dw_tol = norm_bwd_ref(_np(dy), _np(x), _np(w), c.eps, c.pos.cpu().numpy(), c.f, c.il, chain=400)
        _close(got[2 + i], dw, dw_tol, F32_HALF_STEP, "dw")
    again = sta.sta_norm_rope_bwd(*c.dy, c.q, c.k, *c.args(), **c.kw_args())
    assert all(torch.equal(a, b) for a, b in zip(again, got))


def test_norm_rope_tokens_far_apart(dev):
    # offsets past 32 bits, in elements and bytes: the same numbers as side by side
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = Case(dev, 3, 2, 0, 64, 64, False, "bf16")
    far = torch.empty(3 << 31, device=dev, dtype=torch.bfloat16)
    at = lambda first: far[first:].as_strided((3, 2, 64), (1 << 31, 64, 1))  # noqa: E731
    q, dy = at(0).copy_(c.q), at(1024).copy_(c.dy[0])
    want = sta.sta_norm_rope(c.q.contiguous(), None, *c.args(), q_weight=c.qw)[0]
    assert torch.equal(sta.sta_norm_rope(q, None, *c.args(), q_weight=c.qw, q_out=at(4096))[0], want)
    want = sta.sta_norm_rope_bwd(c.dy[0], None, c.q.contiguous(), None, *c.args(), q_weight=c.qw)
    got = sta.sta_norm_rope_bwd(dy, None, q, None, *c.args(), q_weight=c.qw, dq=at(8192))
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])


def test_norm_rope_streams_and_graphs(dev):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = Case(dev, 100, 4, 2, 64, 64, False, "bf16")
    want = sta.sta_norm_rope(c.q, c.k, *c.args(), **c.kw_args())
    grads = sta.sta_norm_rope_bwd(*c.dy, c.q, c.k, *c.args(), **c.kw_args())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = sta.sta_norm_rope(c.q, c.k, *c.args(), **c.kw_args(), stream=s)
    back = sta.sta_norm_rope_bwd(*c.dy, c.q, c.k, *c.args(), **c.kw_args(), stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*got, *back), (*want, *grads)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = sta.sta_norm_rope(c.q, c.k, *c.args(), **c.kw_args())
        back = sta.sta_norm_rope_bwd(*c.dy, c.q, c.k, *c.args(), **c.kw_args())
    for scale in (1.0, -0.5):
        c.wide.mul_(scale)
        for t in (*got, *back):
            t.zero_()
        g.replay()
        want = sta.sta_norm_rope(c.q, c.k, *c.args(), **c.kw_args())
        grads = sta.sta_norm_rope_bwd(*c.dy, c.q, c.k, *c.args(), **c.kw_args())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*got, *back), (*want, *grads)))


def test_norm_rope_as_an_autograd_function(dev):
    # as a model's layer uses the two: gradients into one packed tensor, under captured and eager graphs
    import torch

    import split_kv_decode_bsr_gb300 as sta

    n, Hq, Hk, d = 37, 4, 2, 64
    pos, rope = torch.arange(n, device=dev, dtype=torch.int32), sta.Rope(d)

    class NormRope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, packed, qw, kw):
            ctx.save_for_backward(packed, qw, kw)
            q, k = packed.view(n, Hq + Hk, d).split([Hq, Hk], 1)
            return sta.sta_norm_rope(q, k, pos, rope, qw, kw)

        @staticmethod
        def backward(ctx, gq, gk):
            packed, qw, kw = ctx.saved_tensors
            q, k = packed.view(n, Hq + Hk, d).split([Hq, Hk], 1)
            grad = torch.empty_like(packed)
            dq, dk = grad.view(n, Hq + Hk, d).split([Hq, Hk], 1)
            _, _, dqw, dkw = sta.sta_norm_rope_bwd(gq.contiguous(), gk.contiguous(), q, k, pos, rope, qw, kw, dq=dq, dk=dk)
            return grad, dqw, dkw

    packed = torch.randn(n, (Hq + Hk) * d, device=dev, requires_grad=True)
    qw, kw = (torch.rand(d, device=dev).add_(0.5).requires_grad_() for _ in range(2))
    wq, wk = torch.randn(n, Hq, d, device=dev), torch.randn(n, Hk, d, device=dev)
    q, k = NormRope.apply(packed, qw, kw)
    ((q * wq).sum() + (k * wk).sum()).backward()
    x = _np(packed.detach()).reshape(n, Hq + Hk, d)
    for y, w, part, dwt, sl in ((wq, qw, packed.grad, qw.grad, slice(0, Hq)), (wk, kw, packed.grad, kw.grad, slice(Hq, None))):
        dx, dw, tol, dw_tol = norm_bwd_ref(_np(y), x[:, sl], _np(w.detach()), 1e-6, np.arange(n), freqs(d), False)
        _close(part.view(n, Hq + Hk, d)[:, sl], dx, tol, F32_HALF_STEP, "dx")
        _close(dwt, dw, dw_tol, F32_HALF_STEP, "dw")


# ---- new tokens into pages


@pytest.mark.parametrize("P", [1, 7, 16, 100])
@pytest.mark.parametrize("interleaved,rot,d,Hq,Hkv", [(False, 128, 128, 8, 2), (True, 32, 64, 3, 3), (False, 0, 64, 0, 1),
                                                      (True, 20, 72, 5, 5), (False, 30, 60, 4, 1), (False, 50, 96, 4, 2)])
def test_norm_append(dev, P, interleaved, rot, d, Hq, Hkv):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    new, kv = [1, 0, 37, 5, 1, 9], [1, 40, 37, 105, 64, 4]  # the last sequence is shorter than its chunk
    c = PagedCase(P + d, new, kv, max(Hq, 1), Hkv, d, P, spare_entries=1, pad_rows=3)
    x = c.dev(dev)
    N, T = c.q.shape[0], int(c.q_indptr[-1])
    packed = torch.randn(N, (Hq + 2 * Hkv) * d + 4, device=dev).to(torch.bfloat16)
    q, k, v = (t.unflatten(1, (t.shape[1] // d, d)) if t.shape[1] else None
               for t in packed[:, :-4].split([Hq * d, Hkv * d, Hkv * d], dim=1))
    qw, kw = torch.rand(d, device=dev) + 0.5, torch.rand(d, device=dev) + 0.5
    q_out = torch.full((N, Hq, d), 9.0, device=dev, dtype=torch.bfloat16) if Hq else None
    k0, v0 = x["k_pages"].clone(), x["v_pages"].clone()
    got = sta.sta_norm_rope_append_paged(q, k, v, x["k_pages"], x["v_pages"], x["page_indptr_dev"], x["page_indices_dev"],
                                         x["q_indptr_dev"], x["kv_indptr_dev"],
                                         rope=sta.Rope(rot, interleaved=interleaved) if rot else None, q_weight=qw, k_weight=kw,
                                         eps=1e-5, q_out=q_out)
    req = np.repeat(np.arange(len(new)), new)
    pos = np.concatenate([kv[r] - new[r] + np.arange(new[r]) for r in range(len(new))])
    f = freqs(rot) if rot else np.zeros(0)
    if Hq:
        assert got is q_out
        _close(q_out[:T], *norm_ref(_np(q[:T]), _np(qw), 1e-5, pos, f, interleaved), BF16_HALF_STEP, "q")
        assert (q_out[T:] == 9.0).all()  # padding: left as it was
    kr, tol = norm_ref(_np(k[:T]), _np(kw), 1e-5, pos, f, interleaved)
    live = pos >= 0
    rows = np.array([c.rows(r, np.array([p]))[0] for r, p in zip(req[live], pos[live])])
    kn, vn = x["k_pages"].view(-1, Hkv, d), x["v_pages"].view(-1, Hkv, d)
    _close(kn[rows], kr[live], tol[live], BF16_HALF_STEP, "k")
    assert torch.equal(vn[rows], v[:T][torch.from_numpy(live).to(dev)])
    rest = np.setdiff1d(np.arange(kn.shape[0]), rows)  # everything else: bit for bit as before
    for a, b in ((kn, k0.view(-1, Hkv, d)), (vn, v0.view(-1, Hkv, d))):
        assert torch.equal(a[rest].view(torch.int16), b[rest].view(torch.int16))


@pytest.mark.parametrize("n_req", [1, 2, 127, 128, 129, 700])
def test_norm_append_finds_each_request(dev, n_req):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    g = np.random.default_rng(n_req)
    new = g.integers(0, 4, n_req)
    new[0] = 2
    kv = new + g.integers(0, 20, n_req)
    c = PagedCase(n_req, new, kv, 1, 1, 64, 8)
    x = c.dev(dev)
    n = int(new.sum())
    k, v = (torch.randn(n, 1, 64, device=dev).to(torch.bfloat16) for _ in range(2))
    q = sta.sta_norm_rope_append_paged(k, k, v, x["k_pages"], x["v_pages"], x["page_indptr_dev"], x["page_indices_dev"],
                                       x["q_indptr_dev"], x["kv_indptr_dev"], rope=sta.Rope(64))
    pos = np.concatenate([kv[r] - new[r] + np.arange(new[r]) for r in range(n_req)]).astype(np.int32)
    rows = np.concatenate([c.rows(r, kv[r] - new[r] + np.arange(new[r])) for r in range(n_req)])
    same, _ = sta.sta_norm_rope(k, None, torch.from_numpy(pos).to(dev), sta.Rope(64))
    assert torch.equal(q, same)
    assert torch.equal(x["k_pages"].view(-1, 1, 64)[rows], same) and torch.equal(x["v_pages"].view(-1, 1, 64)[rows], v)


def test_norm_append_positions_and_bad_pages(dev):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = PagedCase(5, [4, 2], [10, 2], 2, 1, 64, 8)
    x = c.dev(dev)
    k, v = torch.randn(6, 1, 64, device=dev).to(torch.bfloat16), torch.randn(6, 1, 64, device=dev).to(torch.bfloat16)
    pos = torch.from_numpy(np.array([900, 3, 3, 70000, 1, 0], np.int32)).to(dev)
    q = sta.sta_norm_rope_append_paged(x["q"], k, v, x["k_pages"], x["v_pages"], x["page_indptr_dev"], x["page_indices_dev"],
                                       x["q_indptr_dev"], x["kv_indptr_dev"], rope=sta.Rope(64), positions=pos)
    want_q, want_k = sta.sta_norm_rope(x["q"], k, pos, sta.Rope(64))
    rows = np.r_[c.rows(0, np.arange(6, 10)), c.rows(1, np.arange(2))]
    assert torch.equal(q, want_q) and torch.equal(x["k_pages"].view(-1, 1, 64)[rows], want_k)
    for bad, code in ((99, 0x110), (-1, 0x110), (None, 0x604)):
        c = PagedCase(6, [3], [20], 1, 1, 64, 8)
        x = c.dev(dev)
        if bad is None:
            x["page_indptr_dev"][1] = 2  # a list one entry short
        else:
            x["page_indices_dev"][2] = bad
        k0 = x["k_pages"].clone()
        sta.sta_norm_rope_append_paged(None, k[:3], v[:3], x["k_pages"], x["v_pages"], x["page_indptr_dev"],
                                       x["page_indices_dev"], x["q_indptr_dev"], x["kv_indptr_dev"])
        assert sta.sta_device_error(reset=True) == code
        assert torch.equal(k0.view(torch.int16), x["k_pages"].view(torch.int16))


def test_norm_append_into_far_pages(dev):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = PagedCase(77, [1, 30, 5], [90, 30, 41], 4, 8, 128, 16)
    x, N = c.dev(dev), c.q.shape[0]
    k, v = (torch.randn(N, 8, 128, device=dev).to(torch.bfloat16) for _ in "kv")
    pages = lambda big: dict(x, k_pages=big[0], v_pages=big[1])  # noqa: E731

    def append(x, indices):
        sta.sta_norm_rope_append_paged(None, k, v, x["k_pages"], x["v_pages"], x["page_indptr_dev"], indices, x["q_indptr_dev"],
                                       x["kv_indptr_dev"], rope=sta.Rope(128))
        return x["k_pages"], x["v_pages"]

    n = x["k_pages"].shape[0]
    big = [torch.empty(135000, 16, 8, 128, device=dev, dtype=torch.bfloat16) for _ in "kv"]  # 4.4 GB each
    for b, a in zip(big, (x["k_pages"], x["v_pages"])):
        b[-n:] = a
    got = append(pages(big), x["page_indices_dev"] + 135000 - n)
    for a, b in zip(got, append(x, x["page_indices_dev"])):
        assert torch.equal(a[-n:].view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("n,Hq,Hk,d,rot,dtype", [(200, 31, 1, 256, 256, "f32"), (90, 25, 7, 256, 256, "f32"), (130, 27, 5, 256, 128, "bf16"),
                                                 (300, 42, 21, 128, 64, "bf16"), (170, 29, 3, 256, 0, "bf16")])
def test_norm_rope_gradients_stay_in_their_workspace(dev, n, Hq, Hk, d, rot, dtype):
    # q's and k's shares of the CTAs end in one half: together they still have a row of scratch each
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = Case(dev, n, Hq, Hk, d, rot, False, dtype, seed=n, eps=1e-3)
    need = 304 * d * 4
    ws = torch.full((need + 8 * d * 4,), 255, dtype=torch.uint8, device=dev)
    with pytest.raises(ValueError):
        sta.sta_norm_rope_bwd(*c.dy, c.q, c.k, *c.args(), **c.kw_args(), workspace=ws[:need - 1])
    got = sta.sta_norm_rope_bwd(*c.dy, c.q, c.k, *c.args(), **c.kw_args(), workspace=ws[:need])
    assert (ws[need:] == 255).all()
    for i, (x, w, dy) in enumerate(c.parts()):
        dx, dw, tol, dw_tol = norm_bwd_ref(_np(dy), _np(x), _np(w), c.eps, c.pos.cpu().numpy(), c.f, c.il)
        _close(got[i], dx, tol, c.step, "dx")
        _close(got[2 + i], dw, dw_tol, F32_HALF_STEP, "dw")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,Hq", [(48, 16), (3000, 8)])
def test_norm_rope_by_weights_that_the_last_call_wrote(dev, n, Hq, dtype):
    # each step's weights are the gradient of the step before, in one place; a kernel may start before the one that writes them
    # has ended
    import ctypes as C

    import torch

    import split_kv_decode_bsr_gb300 as sta

    d = 128
    c = Case(dev, n, Hq, 0, d, d, False, dtype)
    w, x = torch.empty(d, device=dev), torch.empty(n, Hq, d, device=dev, dtype=c.dt)
    ws, size = torch.empty(304 * d * 4, dtype=torch.uint8, device=dev), C.c_size_t(304 * d * 4)
    dx, P = torch.empty_like(x), lambda t: C.c_void_p(t.data_ptr())  # noqa: E731
    code = sta.STA_BF16 if dtype == "bf16" else sta.STA_F32

    def chain(wait):
        x.copy_(c.q)
        w.copy_(c.qw)
        for i in range(20):
            sta.sta_norm_rope(x, None, *c.args(), q_weight=w, q_out=x)
            if wait:
                torch.cuda.synchronize()
            assert sta.lib().sta_norm_rope_bwd(P(c.dy[0]), None, Hq * d, 0, P(x), None, Hq * d, 0, P(dx), None, Hq * d, 0, None, None,
                                               P(w), None, 1e-6, P(c.pos), C.byref(c.rope.struct), n, Hq, 0, d, code, P(ws),
                                               C.byref(size), C.c_void_p(torch.cuda.current_stream().cuda_stream)) == sta.STA_OK
            if wait:
                torch.cuda.synchronize()
        return x.clone(), w.clone()

    want = chain(True)
    assert torch.isfinite(want[0]).all() and torch.isfinite(want[1]).all()
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(chain(False), want))

"""Serving over a paged KV cache on the GPU, against plain 64-bit forms: rotary positions, the write
of new tokens into pages, the attention of chunks, page bookkeeping, and a run of them together."""

import math

import numpy as np
import pytest

from _serving import BF16_HALF_STEP, F32_HALF_STEP, PagedCase, Pool, check_chunk, freqs, rope_ref

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


# ---- rotary positions


def _rope_case(dev, n, H, d, rot, interleaved, dtype, pad=0, transpose=False, max_pos=4096, seed=0, in_place=False, **kw):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    g = np.random.default_rng(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    wide = torch.from_numpy(g.standard_normal((n, H * d + pad)).astype(np.float32)).to(dt)
    x = wide.to(dev)[:, :H * d].unflatten(1, (H, d))
    pos = g.integers(-max_pos, max_pos, n).astype(np.int32)
    pos[: 2] = [0, max_pos - 1][: min(n, 2)]
    mscale = kw.pop("mscale", 1.0)
    rope = sta.Rope(rot, interleaved=interleaved, mscale=mscale, **kw)
    f = np.array(kw["freqs"]) if "freqs" in kw else freqs(rot, **kw)
    ref, err = rope_ref(_np(x), pos, f, interleaved, np.float32(mscale), transpose)
    y = sta.sta_rope(x, torch.from_numpy(pos).to(dev), rope, transpose=transpose, y=x if in_place else None)
    step = BF16_HALF_STEP if dtype == "bf16" else F32_HALF_STEP
    off = np.abs(_np(y) - ref) - (step * np.abs(ref) + err * (1 + step))
    assert off.max() <= 0, f"{off.max():.3e} past its bound"
    assert np.array_equal(_np(y)[..., rot:], _np(wide)[:, :H * d].reshape(n, H, d)[..., rot:])  # the rest is copied


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,H,d,rot,pad", [(1, 1, 2, 2, 0), (3, 5, 128, 128, 0), (70, 40, 128, 64, 8), (33, 3, 80, 40, 16),
                                           (17, 2, 96, 30, 3), (5, 7, 63, 6, 0), (9, 1, 512, 512, 1), (1000, 2, 64, 64, 24)])
def test_rope(dev, n, H, d, rot, pad, interleaved, dtype):
    _rope_case(dev, n, H, d, rot, interleaved, dtype, pad=pad, seed=n)
    _rope_case(dev, n, H, d, rot, interleaved, dtype, pad=pad, seed=n + 1, transpose=True, in_place=True)


@pytest.mark.parametrize("kw", [dict(base=500000.0), dict(scaling="linear", factor=8.0),
                                dict(scaling="blend", factor=32.0, orig_len=8192.0, low_turns=1.0, high_turns=4.0, mscale=1.35),
                                dict(freqs=[7.5, -0.25, 0.0, 1e-9, -1e-30, 3.0, 0.5, 2 * math.pi])])
def test_rope_far_positions_and_scaling(dev, kw):
    # positions to 2^31 - 1: an fp32 angle would be off by whole turns. (64-bit angles of the plain
    # form are off by 2^-53 of them: 3e-7 radians at 2^31 radians, so 1e-6 is allowed on top)
    import torch

    import split_kv_decode_bsr_gb300 as sta

    rot = 16
    x = torch.randn(64, 3, rot, device=dev)
    pos = np.random.default_rng(0).integers(-(1 << 31), (1 << 31) - 1, 64).astype(np.int32)
    pos[:3] = [(1 << 31) - 1, -(1 << 31), 1 << 20]
    kw = dict(kw)
    mscale = kw.pop("mscale", 1.0)
    f = np.array(kw["freqs"]) if "freqs" in kw else freqs(rot, **kw)
    ref, err = rope_ref(_np(x), pos, f, False, np.float32(mscale))
    y = sta.sta_rope(x, torch.from_numpy(pos).to(dev), sta.Rope(rot, mscale=mscale, **kw))
    assert (np.abs(_np(y) - ref) <= F32_HALF_STEP * np.abs(ref) + err + 1e-5 * np.abs(f).max()).all()


def test_rope_many_tokens_sampled(dev):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    n, H, d = 20011, 8, 128  # several tokens a block, a partial last one
    x = torch.randn(n, H, d, device=dev).to(torch.bfloat16)
    pos = torch.randint(0, 1 << 20, (n,), device=dev, dtype=torch.int32)
    y = sta.sta_rope(x, pos, sta.Rope(d))
    pick = np.r_[0:40, n // 2:n // 2 + 40, n - 40:n]
    ref, err = rope_ref(_np(x[pick]), pos[pick].cpu().numpy(), freqs(d), False)
    assert (np.abs(_np(y[pick]) - ref) <= BF16_HALF_STEP * np.abs(ref) + err * (1 + BF16_HALF_STEP)).all()


def test_rope_gradient_is_the_transposed_turn(dev):
    # against the plain form's own differences: <rope(x + e z) - rope(x - e z), w> / 2e = <z, rope'(w)>
    import torch

    import split_kv_decode_bsr_gb300 as sta

    rope = sta.Rope(48, interleaved=True, mscale=1.25)
    pos = torch.arange(0, 4000, 97, device=dev, dtype=torch.int32)
    x, z, w = (torch.randn(pos.numel(), 3, 64, device=dev) for _ in range(3))
    grad = sta.sta_rope(w, pos, rope, transpose=True)
    f = lambda t: (sta.sta_rope(t, pos, rope).double() * w.double()).sum()  # noqa: E731
    e = 0.5  # the map is linear: any step will do
    diff = float((f(x + e * z) - f(x - e * z)) / (2 * e))
    n = float(z.norm()) * float(w.norm())
    assert abs(diff - float((z.double() * grad.double()).sum())) <= 1e-5 * n


def test_rope_leaves_what_lies_between_tokens(dev):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    wide = torch.full((6, 100), 7.0, device=dev, dtype=torch.bfloat16)
    y = wide[:, :64].unflatten(1, (2, 32))
    sta.sta_rope(torch.randn(6, 2, 32, device=dev).to(torch.bfloat16), torch.arange(6, device=dev, dtype=torch.int32),
                 sta.Rope(32), y=y)
    assert (wide[:, 64:] == 7.0).all()
    empty = torch.empty(0, 2, 32, device=dev)
    assert sta.sta_rope(empty, torch.empty(0, dtype=torch.int32, device=dev), sta.Rope(32)).shape == (0, 2, 32)


# ---- new tokens into pages


@pytest.mark.parametrize("P", [1, 7, 16, 100])
@pytest.mark.parametrize("interleaved,rot,d,Hq,Hkv", [(False, 128, 128, 8, 2), (True, 32, 64, 3, 3), (False, 0, 64, 0, 1),
                                                      (True, 20, 72, 5, 5), (False, 30, 60, 4, 1)])
def test_append(dev, P, interleaved, rot, d, Hq, Hkv):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    new, kv = [1, 0, 37, 5, 1, 9], [1, 40, 37, 105, 64, 4]  # the last sequence is shorter than its chunk
    c = PagedCase(P + d, new, kv, max(Hq, 1), Hkv, d, P, spare_entries=1, pad_rows=3)
    x = c.dev(dev)
    N, T = c.q.shape[0], int(c.q_indptr[-1])
    packed = torch.randn(N, (Hq + 2 * Hkv) * d + 4, device=dev).to(torch.bfloat16)
    q, k, v = (t.unflatten(1, (t.shape[1] // d, d)) if t.shape[1] else None
               for t in packed[:, :-4].split([Hq * d, Hkv * d, Hkv * d], dim=1))
    q_out = torch.full((N, Hq, d), 9.0, device=dev, dtype=torch.bfloat16) if Hq else None
    k0, v0 = x["k_pages"].clone(), x["v_pages"].clone()
    got = sta.sta_rope_append_paged(q, k, v, x["k_pages"], x["v_pages"], x["page_indptr_dev"], x["page_indices_dev"],
                                    x["q_indptr_dev"], x["kv_indptr_dev"], rope=sta.Rope(rot, interleaved=interleaved) if rot
                                    else None, q_out=q_out)
    req = np.repeat(np.arange(len(new)), new)
    pos = np.concatenate([kv[r] - new[r] + np.arange(new[r]) for r in range(len(new))])
    f = freqs(rot) if rot else np.zeros(0)
    if Hq:
        assert got is q_out
        ref, err = rope_ref(_np(q[:T]), pos, f, interleaved)
        assert (np.abs(_np(q_out[:T]) - ref) <= BF16_HALF_STEP * np.abs(ref) + err * (1 + BF16_HALF_STEP)).all()
        assert (q_out[T:] == 9.0).all()  # padding: left as it was
    kr, err = rope_ref(_np(k[:T]), pos, f, interleaved)
    tol = BF16_HALF_STEP * np.abs(kr) + err * (1 + BF16_HALF_STEP)
    live = pos >= 0
    rows = np.array([c.rows(r, np.array([p]))[0] for r, p in zip(req[live], pos[live])])
    kn, vn = x["k_pages"].view(-1, Hkv, d), x["v_pages"].view(-1, Hkv, d)
    assert (np.abs(_np(kn[rows]) - kr[live]) <= tol[live]).all()
    assert torch.equal(vn[rows], v[:T][torch.from_numpy(live).to(dev)])
    rest = np.setdiff1d(np.arange(kn.shape[0]), rows)  # everything else: bit for bit as before
    for a, b in ((kn, k0.view(-1, Hkv, d)), (vn, v0.view(-1, Hkv, d))):
        assert torch.equal(a[rest].view(torch.int16), b[rest].view(torch.int16))


def test_append_positions_of_the_callers_own(dev):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = PagedCase(5, [4, 2], [10, 2], 2, 1, 64, 8)
    x = c.dev(dev)
    k, v = torch.randn(6, 1, 64, device=dev).to(torch.bfloat16), torch.randn(6, 1, 64, device=dev).to(torch.bfloat16)
    pos = np.array([900, 3, 3, 70000, 1, 0], np.int32)
    q = sta.sta_rope_append_paged(x["q"], k, v, x["k_pages"], x["v_pages"], x["page_indptr_dev"], x["page_indices_dev"],
                                  x["q_indptr_dev"], x["kv_indptr_dev"], rope=sta.Rope(64), positions=torch.from_numpy(pos).to(dev))
    same = sta.sta_rope(x["q"], torch.from_numpy(pos).to(dev), sta.Rope(64))
    assert torch.equal(q, same)
    rows = np.r_[c.rows(0, np.arange(6, 10)), c.rows(1, np.arange(2))]
    assert torch.equal(x["k_pages"].view(-1, 1, 64)[rows], sta.sta_rope(k, torch.from_numpy(pos).to(dev), sta.Rope(64)))


def test_append_bad_pages_are_reported_and_not_written(dev):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    for bad, code in ((99, 0x110), (-1, 0x110), (None, 0x604)):
        c = PagedCase(6, [3], [20], 1, 1, 64, 8)
        x = c.dev(dev)
        if bad is None:
            x["page_indptr_dev"][1] = 2  # a list one entry short
        else:
            x["page_indices_dev"][2] = bad
        k0 = x["k_pages"].clone()
        k = torch.randn(3, 1, 64, device=dev).to(torch.bfloat16)
        sta.sta_rope_append_paged(None, k, k, x["k_pages"], x["v_pages"], x["page_indptr_dev"], x["page_indices_dev"],
                                  x["q_indptr_dev"], x["kv_indptr_dev"])
        assert sta.sta_device_error(reset=True) == code
        assert torch.equal(k0.view(torch.int16), x["k_pages"].view(torch.int16))


# ---- attention of a chunk


def _chunk_case(dev, c, scale=None, pattern=None, **kw):
    import split_kv_decode_bsr_gb300 as sta

    scale = 1 / math.sqrt(c.d) if scale is None else scale
    pat = None
    p = {}
    if pattern:
        pat = sta.MaskSource.pattern(**pattern)
        p = dict(causal=bool(pat.causal), win_lo=pat.win_lo, win_hi=pat.win_hi, n_global=pat.n_global_cols)
    o, lse = sta.sta_chunk_fwd_paged(**c.dev(dev), scale=scale, pattern=pat, **kw)
    check_chunk(o, lse, c.ref(scale, **p), int(c.q_indptr[-1]), f"{vars(c)['P']} {pattern} {kw}")
    return o, lse


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (4, 4, 64), (7, 1, 128), (12, 4, 64), (16, 1, 64), (32, 2, 128), (130, 2, 64)])
@pytest.mark.parametrize("P", [1, 8, 16, 100, 128])
def test_chunk_ragged(dev, Hq, Hkv, d, P):
    new, kv = [1, 0, 5, 1, 33, 17, 2], [1, 300, 5, 257, 140, 128, 700]
    _chunk_case(dev, PagedCase(Hq + P, new, kv, Hq, Hkv, d, P, spare_entries=2, pad_rows=2))


@pytest.mark.parametrize("P", [12, 48, 64, 256])
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_long(dev, P, d):
    # several query tiles a request, several key tiles, borders off every tile's
    _chunk_case(dev, PagedCase(P, [300, 77, 129], [300, 1000, 1111], 4, 2, d, P))


@pytest.mark.parametrize("P", [3, 9, 31, 33, 39, 41, 60, 127, 129, 300])
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_pages_off_the_swizzle(dev, P, d):
    """Pages that no box of whole 8-row groups tiles, on both sides of the size where their runs go by TMA."""
    _chunk_case(dev, PagedCase(P + d, [1, 70, 0, 40], [1 + 3 * P, 70 + 2 * P, 5, 40], 6, 2, d, P, spare_entries=1))


@pytest.mark.parametrize("pattern", [dict(causal=True, win_lo=0), dict(causal=True, win_lo=-63), dict(causal=True, win_lo=-200, n_global_cols=5),
                                     dict(causal=True, win_lo=-30, n_global_cols=300), dict(causal=False),
                                     dict(causal=False, win_lo=-40, win_hi=40), dict(causal=False, win_lo=3, win_hi=9),
                                     dict(causal=True, win_lo=5), dict(causal=True, win_hi=-20), dict(causal=False, win_lo=1, win_hi=0, n_global_cols=2),
                                     dict(causal=True, win_lo=-500, win_hi=-300, n_global_cols=130)])
def test_chunk_patterns(dev, pattern):
    # windows that end before the token, lie past it or are empty leave rows without a key
    _chunk_case(dev, PagedCase(11, [40, 1, 260, 3], [40, 390, 700, 3], 6, 2, 64, 16), pattern=pattern)


@pytest.mark.parametrize("splits", [1, 2, 3, 7, 64])
def test_chunk_any_split_count(dev, splits):
    c = PagedCase(12, [1, 70, 0, 3], [900, 641, 20, 5], 8, 2, 128, 16)
    _chunk_case(dev, c, num_splits=splits)
    _chunk_case(dev, c, num_splits=splits, pattern=dict(causal=True, win_lo=-100, n_global_cols=16))


def test_chunk_shorter_sequence_than_chunk(dev):
    # the first rows come before the sequence: no key, O = 0, LSE = -inf; an empty sequence: all rows
    o, lse = _chunk_case(dev, PagedCase(13, [10, 4, 200], [3, 0, 150], 4, 2, 64, 16))
    assert lse.isneginf().any()


def test_chunk_rows_behind_the_last_sequence_stay(dev):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = PagedCase(14, [3, 140], [50, 150], 8, 2, 64, 16, pad_rows=40)
    n = int(c.q_indptr[-1])
    o = torch.full((n + 40, 8, 64), 5.0, device=dev, dtype=torch.bfloat16)
    lse = torch.full((n + 40, 8), 5.0, device=dev)
    x = c.dev(dev)
    x["q"][n:] = float("nan")
    for s in (1, 3):
        sta.sta_chunk_fwd_paged(**x, o=o, lse=lse, num_splits=s)
        assert (o[n:] == 5.0).all() and (lse[n:] == 5.0).all()
        check_chunk(o, lse, c.ref(1 / 8), n)


def test_chunk_large_scores(dev):
    # scores of several hundred: one key takes all, and exponents reach the edge of fp32
    _chunk_case(dev, PagedCase(15, [50, 1], [300, 500], 4, 2, 64, 16, value=4.0), scale=3.0)


@pytest.mark.parametrize("splits", [1, 3])
def test_chunk_nan_query_stays_nan(dev, splits):
    """A NaN in one head's query shows in that row's output and LSE, and nowhere else. (The second of
    them is at position 5 - 40 + 19 of its sequence: it sees no key, and has no score to be NaN.)"""
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = PagedCase(15, [1, 40, 200], [700, 5, 300], 8, 2, 64, 16)
    x = c.dev(dev)
    clean, clean_lse = sta.sta_chunk_fwd_paged(**x, num_splits=splits)
    bad = [(0, 3), (20, 0), (240, 7)]
    for t, h in bad:
        x["q"][t, h, 5] = float("nan")
    o, lse = sta.sta_chunk_fwd_paged(**x, num_splits=splits)
    for t, h in bad[::2]:
        assert torch.isnan(o[t, h]).all() and torch.isnan(lse[t, h])
        o[t, h], lse[t, h] = clean[t, h], clean_lse[t, h]
    assert torch.equal(o, clean) and torch.equal(lse, clean_lse)


def test_chunk_strided_queries(dev):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = PagedCase(16, [30, 1], [60, 9], 4, 2, 64, 16)
    x = c.dev(dev)
    wide = torch.zeros(31, 4 * 64 + 72, device=dev, dtype=torch.bfloat16)
    wide[:, :256] = x["q"].flatten(1)
    o, lse = sta.sta_chunk_fwd_paged(**{**x, "q": wide[:, :256].unflatten(1, (4, 64))})
    o2, lse2 = sta.sta_chunk_fwd_paged(**x)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check_chunk(o, lse, c.ref(1 / 8), 31)


def test_chunk_single_tokens_equal_the_paged_decode(dev):
    import split_kv_decode_bsr_gb300 as sta

    kv = [1, 17, 640, 3000, 129]
    c = PagedCase(17, [1] * 5, kv, 8, 2, 128, 16)
    x = c.dev(dev)
    o, lse = sta.sta_chunk_fwd_paged(**x)
    o2, lse2 = sta.sta_decode_splitkv_paged(x["q"], x["k_pages"], x["v_pages"], x["page_indptr_dev"], x["page_indices_dev"],
                                            x["kv_indptr_dev"], c.kv_indptr)
    ref = c.ref(1 / math.sqrt(128))
    check_chunk(o, lse, ref, 5)
    check_chunk(o2, lse2, ref, 5)


def test_chunk_many_requests(dev):
    # more requests than one launch plans, single tokens and short chunks, all lengths from 0 on
    import torch

    import split_kv_decode_bsr_gb300 as sta

    g = np.random.default_rng(23)
    R = 1300
    new = g.integers(0, 3, R)
    kv = np.maximum(new, g.integers(0, 60, R))
    c = PagedCase(23, new, kv, 2, 1, 64, 16)
    ref = c.ref(1 / 8)
    for splits in (0, 2):
        o, lse = sta.sta_chunk_fwd_paged(**c.dev(dev), num_splits=splits)
        check_chunk(o, lse, ref, int(c.q_indptr[-1]), f"{splits}")
    # the lists' numbers and lengths of an empty batch
    x = c.dev(dev)
    zero = torch.zeros(R + 1, dtype=torch.int32, device=dev)
    x.update(kv_indptr_dev=zero, kv_indptr_host=np.zeros(R + 1, np.int32), page_indptr_dev=zero,
             page_indices_dev=torch.empty(0, dtype=torch.int32, device=dev))
    o, lse = sta.sta_chunk_fwd_paged(**x)
    assert (o == 0).all() and lse.isneginf().all()


def test_chunk_several_prompts(dev):
    # query tiles of several prompts in one launch order
    _chunk_case(dev, PagedCase(24, [700, 1, 333, 500, 2, 64], [700, 900, 800, 510, 3, 64], 6, 2, 64, 32))


def test_chunk_group_of_128_heads(dev):
    _chunk_case(dev, PagedCase(25, [3, 1, 2], [40, 500, 2], 128, 1, 128, 16))


def test_chunk_output_at_odd_places(dev):
    # o on a 16-byte boundary that is not a 32-byte one; lse on a 4-byte one
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = PagedCase(26, [5, 40], [300, 50], 4, 2, 64, 16)
    room = torch.full((45 * 4 * 64 + 8 + 8,), 3.0, device=dev, dtype=torch.bfloat16)
    o = room[8:-8].view(45, 4, 64)
    lroom = torch.full((45 * 4 + 2,), 3.0, device=dev)
    lse = lroom[1:-1].view(45, 4)
    sta.sta_chunk_fwd_paged(**c.dev(dev), o=o, lse=lse)
    check_chunk(o, lse, c.ref(1 / 8), 45)
    assert (room[:8] == 3.0).all() and (room[-8:] == 3.0).all() and lroom[0] == 3.0 and lroom[-1] == 3.0


def test_chunk_cache_past_32_bits(dev):
    # pages at the end of a cache of more than 4 GiB a tensor: byte offsets past 2^32
    import torch

    import split_kv_decode_bsr_gb300 as sta

    n_pages, P, Hkv, d = 40000, 64, 8, 128
    kc = torch.zeros(n_pages, P, Hkv, d, device=dev, dtype=torch.bfloat16)
    vc = torch.zeros_like(kc)
    assert kc.numel() * 2 > 1 << 32
    for P_case in (64, 100):
        c = PagedCase(27, [3, 20], [200, 150], 16, 8, 128, P_case)
        x = c.dev(dev)
        at = n_pages * P // P_case - c.n_pages  # the case's pages, at the end of the cache
        k, v = (t.flatten()[: (n_pages * P // P_case) * P_case * Hkv * d].view(-1, P_case, Hkv, d) for t in (kc, vc))
        k[at:].copy_(x["k_pages"]), v[at:].copy_(x["v_pages"])
        x["page_indices_dev"] += at
        x.update(k_pages=k, v_pages=v)
        o, lse = sta.sta_chunk_fwd_paged(**x)
        check_chunk(o, lse, c.ref(1 / math.sqrt(128)), 23, f"{P_case}")
        new = torch.randn(23, 8, 128, device=dev).to(torch.bfloat16)
        sta.sta_rope_append_paged(None, new, new, k, v, x["page_indptr_dev"], x["page_indices_dev"], x["q_indptr_dev"],
                                  x["kv_indptr_dev"])
        rows = np.r_[c.rows(0, np.arange(197, 200)), c.rows(1, np.arange(130, 150))] + at * P_case
        assert torch.equal(k.reshape(-1, 8, 128)[torch.from_numpy(rows).to(dev)], new)


def test_chunk_is_bitwise_repeatable(dev):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = PagedCase(28, [200, 1, 1, 77], [900, 3000, 20, 77], 8, 2, 128, 16)
    x = c.dev(dev)
    first = sta.sta_chunk_fwd_paged(**x)
    for _ in range(5):
        again = sta.sta_chunk_fwd_paged(**x)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_chunk_two_calls_at_once(dev):
    # two streams, two workspaces, one cache
    import torch

    import split_kv_decode_bsr_gb300 as sta

    a, b = PagedCase(29, [300, 1], [900, 4000], 8, 2, 128, 16), PagedCase(30, [1, 9, 64], [2500, 30, 640], 8, 2, 128, 16)
    xa, xb = a.dev(dev), b.dev(dev)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(4):
        outs.append((sta.sta_chunk_fwd_paged(**xa, stream=s), sta.sta_chunk_fwd_paged(**xb, stream=t)))
    torch.cuda.synchronize()
    ra, rb = a.ref(1 / math.sqrt(128)), b.ref(1 / math.sqrt(128))
    for (oa, la), (ob, lb) in outs:
        check_chunk(oa, la, ra, 301)
        check_chunk(ob, lb, rb, 74)


def test_chunk_bad_pages_are_reported(dev):
    import split_kv_decode_bsr_gb300 as sta

    for bad in (99, -5, None):
        c = PagedCase(18, [3], [40], 4, 2, 64, 8)
        x = c.dev(dev)
        x["k_pages"].nan_to_num_(0.0), x["v_pages"].nan_to_num_(0.0)
        if bad is None:
            x["page_indptr_dev"][1] = 3
        else:
            x["page_indices_dev"][2] = bad
        sta.sta_chunk_fwd_paged(**x)
        assert sta.sta_device_error(reset=True) == 0x110


def test_chunk_replayed_with_other_lengths(dev):
    # a captured call goes by the device's lengths, lists and values: they may change between replays
    import torch

    import split_kv_decode_bsr_gb300 as sta

    big = PagedCase(19, [4, 100, 1], [900, 400, 2000], 8, 2, 64, 16, spare_entries=0)
    small = PagedCase(20, [2, 100, 0], [30, 120, 1500], 8, 2, 64, 16, spare_entries=0)
    x = big.dev(dev)
    for splits in (0, 3):
        o, lse = (torch.zeros(105, 8, 64, device=dev, dtype=torch.bfloat16), torch.zeros(105, 8, device=dev))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            sta.sta_chunk_fwd_paged(**x, num_splits=splits, o=o, lse=lse)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sta.sta_chunk_fwd_paged(**x, num_splits=splits, o=o, lse=lse)
        g.replay()
        check_chunk(o, lse, big.ref(1 / 8), 105, "as captured")
        y = small.dev(dev)
        keep = {k: v.clone() for k, v in x.items() if torch.is_tensor(v)}
        o.fill_(5.0), lse.fill_(5.0)
        n = int(small.q_indptr[-1])
        x["q"][:n] = y["q"][:n]
        for k in ("k_pages", "v_pages"):
            x[k][: small.n_pages] = y[k]
        x["page_indices_dev"][: y["page_indices_dev"].numel()] = y["page_indices_dev"]
        for k in ("page_indptr_dev", "q_indptr_dev", "kv_indptr_dev"):
            x[k].copy_(y[k])
        g.replay()
        check_chunk(o, lse, small.ref(1 / 8), n, "other lengths")
        assert (o[n:] == 5.0).all() and (lse[n:] == 5.0).all()
        for k, v in keep.items():
            x[k].copy_(v)


def test_chunk_more_new_tokens_than_planned_is_reported(dev):
    import split_kv_decode_bsr_gb300 as sta

    c = PagedCase(21, [400, 1], [400, 10], 4, 2, 64, 16)
    x = c.dev(dev)
    x["q_indptr_host"] = np.array([0, 1, 401], np.int32)  # 1 and 400 on the host, 400 and 1 on the device
    sta.sta_chunk_fwd_paged(**x)
    assert sta.sta_device_error(reset=True) == 0x606


def test_chunk_on_another_stream(dev):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = PagedCase(22, [5, 60], [500, 600], 8, 2, 128, 16)
    x = c.dev(dev)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o, lse = sta.sta_chunk_fwd_paged(**x, num_splits=4, stream=s)
    o2, lse2 = sta.sta_chunk_fwd_paged(**x, num_splits=4, stream=s.cuda_stream)
    s.synchronize()
    check_chunk(o, lse, c.ref(1 / math.sqrt(128)), 65)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)  # bitwise the same twice


# ---- page bookkeeping


def _pool_dev(pool, dev, extra=()):
    import torch

    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    kv = np.concatenate([[0], np.cumsum(pool.kv)])
    return i32(pool.ref), i32(pool.ptr), i32(pool.idx), i32(kv)


def _buffers(pool, dev, n, elems, seed=0):
    import torch

    host = [np.random.default_rng(seed + b).integers(0, 1 << 15, (pool.n_pages, elems)).astype(np.int16) for b in range(n)]
    return host, [torch.from_numpy(h.copy()).to(dev) for h in host]


def _same(pool, ref, idx, host=(), bufs=()):
    assert ref.tolist() == pool.ref and idx.tolist() == pool.idx
    for h, b in zip(host, bufs):
        assert np.array_equal(b.cpu().numpy(), h)


SHAPES = [(1, [5], 4, 8, 9), (16, [40, 0, 16, 1, 100, 33, 0, 7], 8, 9, 60), (3, [0, 50, 21, 0, 9] * 60, 30, 20, 5000),
          (5, [int(x) for x in np.random.default_rng(1).integers(0, 90, 1100)], 3, 40, 40000)]


@pytest.mark.parametrize("P,lens,elems,room,n_pages", SHAPES)
def test_pages_grow_and_free(dev, P, lens, elems, room, n_pages):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    pool = Pool(len(lens), lens, P, room, n_pages)
    ref, ptr, idx, kv = _pool_dev(pool, dev)
    g = np.random.default_rng(2)
    leave = g.permutation(len(lens))[: (len(lens) + 1) // 2].tolist()
    reqs = torch.tensor(leave + leave[:2], dtype=torch.int32, device=dev)  # some named twice
    sta.sta_pages_free(ref, ptr, idx, kv, reqs, P)
    pool.free(leave)
    _same(pool, ref, idx)
    for r in leave:
        pool.kv[r] = 0
    after = torch.tensor(np.concatenate([[0], np.cumsum(pool.kv)]), dtype=torch.int32, device=dev)
    new = [int(min(x + g.integers(0, 3 * P + 1), room * P)) for x in pool.kv]
    grown = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=dev)
    status = sta.sta_pages_grow(ref, ptr, idx, after, grown, P)
    assert status.tolist() == pool.grow(new)
    _same(pool, ref, idx)


@pytest.mark.parametrize("P,lens,elems,room,n_pages", SHAPES[1:])
@pytest.mark.parametrize("n_bufs", [0, 1, 3])
def test_pages_fork(dev, P, lens, elems, room, n_pages, n_bufs):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    pool = Pool(len(lens) + 1, lens, P, room, n_pages)
    ref, ptr, idx, kv = _pool_dev(pool, dev)
    host, bufs = _buffers(pool, dev, n_bufs, 8 * elems)
    child = [r for r, n in enumerate(lens) if n == 0]
    g = np.random.default_rng(3)
    parent = [int(g.choice([r for r, n in enumerate(lens) if n])) for _ in child]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    status = sta.sta_pages_fork(bufs, ref, ptr, idx, kv, i32(parent), i32(child), P)
    assert status.tolist() == pool.fork(host, parent, child)
    _same(pool, ref, idx, host, bufs)


@pytest.mark.parametrize("P,lens,elems,room,n_pages", SHAPES)
def test_pages_compact(dev, P, lens, elems, room, n_pages):
    import split_kv_decode_bsr_gb300 as sta

    for seed in (0, 1):
        pool = Pool(seed + 40, lens, P, room, n_pages)
        if seed:  # a page that no list names moves too
            free = [p for p in range(n_pages) if not pool.ref[p]]
            pool.ref[free[-1]] = 2
        ref, ptr, idx, kv = _pool_dev(pool, dev)
        host, bufs = _buffers(pool, dev, 2, 8 * elems)
        page_map, status = sta.sta_pages_compact(bufs, ref, ptr, idx, kv, P)
        goes, want = pool.compact(host)
        assert status.tolist() == want and page_map.tolist() == goes
        _same(pool, ref, idx, host, bufs)


def test_pages_more_forks_than_one_round(dev):
    """1,300 forks of three parents, whose partly filled last pages are copied until no page is left."""
    import torch

    import split_kv_decode_bsr_gb300 as sta

    lens = [7, 4, 10] + [0] * 1300
    pool = Pool(80, lens, 4, 3, 6 + 1000)
    ref, ptr, idx, kv = _pool_dev(pool, dev)
    host, bufs = _buffers(pool, dev, 1, 8)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    parent, child = [k % 7 % 3 for k in range(1300)], list(np.random.default_rng(4).permutation(1300) + 3)
    status = sta.sta_pages_fork(bufs, ref, ptr, idx, kv, i32(parent), i32(child), 4)
    assert status.tolist() == pool.fork(host, parent, [int(c) for c in child])
    _same(pool, ref, idx, host, bufs)


@pytest.mark.parametrize("P", [1, 16])
def test_pages_of_long_sequences(dev, P):
    """Lists of thousands of pages, shared by many warps: freed, grown, forked, compacted."""
    import torch

    import split_kv_decode_bsr_gb300 as sta

    lens, room = [9000, 0, 20011, 0, 0, 5], 22000
    pool = Pool(70, lens, P, room, 110000 // P + 6)
    ref, ptr, idx, kv = _pool_dev(pool, dev)
    host, bufs = _buffers(pool, dev, 1, 8)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    cum = lambda a: i32([0] + np.cumsum(a).tolist())  # noqa: E731
    assert sta.sta_pages_fork(bufs, ref, ptr, idx, kv, i32([2, 5]), i32([1, 3]), P).tolist() == pool.fork(host, [2, 5], [1, 3])
    _same(pool, ref, idx, host, bufs)
    pool.kv[1], pool.kv[3] = lens[2], lens[5]
    sta.sta_pages_free(ref, ptr, idx, cum(pool.kv), i32([0, 2]), P)
    pool.free([0, 2])
    _same(pool, ref, idx)
    pool.kv[0] = pool.kv[2] = 0
    new = [0, 20500, 0, 5, 21999, 18000]
    assert sta.sta_pages_grow(ref, ptr, idx, cum(pool.kv), cum(new), P).tolist() == pool.grow(new)
    _same(pool, ref, idx)
    pool.kv = new
    sta.sta_pages_free(ref, ptr, idx, cum(new), i32([4]), P)
    pool.free([4])
    pool.kv[4] = 0
    page_map, status = sta.sta_pages_compact(bufs, ref, ptr, idx, cum(pool.kv), P)
    goes, want = pool.compact(host)
    assert status.tolist() == want and page_map.tolist() == goes
    _same(pool, ref, idx, host, bufs)


def test_pages_counts_at_an_odd_place(dev):
    # ref on a 4-byte boundary, and a pool that ends inside a run of 16 pages
    import torch

    import split_kv_decode_bsr_gb300 as sta

    pool = Pool(77, [int(x) for x in np.random.default_rng(9).integers(0, 60, 90)], 7, 12, 1237)
    ref, ptr, idx, kv = _pool_dev(pool, dev)
    room = torch.full((pool.n_pages + 6,), 9, dtype=torch.int32, device=dev)
    room[3:-3] = ref
    ref = room[3:-3]
    host, bufs = _buffers(pool, dev, 1, 16)
    _, status = sta.sta_pages_compact(bufs, ref, ptr, idx, kv, 7)
    assert status.tolist() == pool.compact(host)[1]
    _same(pool, ref, idx, host, bufs)
    new = [min(x + 9, 84) for x in pool.kv]
    grown = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=dev)
    assert sta.sta_pages_grow(ref, ptr, idx, kv, grown, 7).tolist() == pool.grow(new)
    _same(pool, ref, idx)
    assert (room[:3] == 9).all() and (room[-3:] == 9).all()


def test_pages_calls_captured_together(dev):
    # one graph holds a step's bookkeeping; replayed on other lists and counts it does other work
    import torch

    import split_kv_decode_bsr_gb300 as sta

    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)  # noqa: E731
    lens = [[40, 0, 16, 1, 100, 33, 0, 7], [9, 64, 0, 80, 16, 0, 3, 50]]
    forks = [([0, 4], [1, 6]), ([3, 1], [2, 5])]
    leave = [[2, 7], [0, 6]]
    pools = [Pool(50 + i, n, 16, 9, 60) for i, n in enumerate(lens)]
    state = [t.clone() for t in _pool_dev(pools[0], dev)]
    ref, ptr, idx, kv = state
    _, bufs = _buffers(pools[0], dev, 2, 64)
    par, ch, out = i32(forks[0][0]), i32(forks[0][1]), i32(leave[0])

    def step():
        a = sta.sta_pages_fork(bufs, ref, ptr, idx, kv, par, ch, 16)
        sta.sta_pages_free(ref, ptr, idx, kv, out, 16)
        return a

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        status = step()
    for i, pool in enumerate(pools):
        host, fresh = _buffers(pool, dev, 2, 64, seed=i)
        for t, n in zip(state, _pool_dev(pool, dev)):
            t.copy_(n)
        for b, f in zip(bufs, fresh):
            b.copy_(f)
        par.copy_(i32(forks[i][0])), ch.copy_(i32(forks[i][1])), out.copy_(i32(leave[i]))
        g.replay()
        assert status.tolist() == pool.fork(host, *forks[i])
        pool.free(leave[i])
        _same(pool, ref, idx, host, bufs)


def test_pages_compact_full_and_empty_pools(dev):
    import split_kv_decode_bsr_gb300 as sta

    for lens, n_pages in (([64, 64], 8), ([0, 0], 8)):
        pool = Pool(0, lens, 16, 4, n_pages)
        ref, ptr, idx, kv = _pool_dev(pool, dev)
        page_map, status = sta.sta_pages_compact([], ref, ptr, idx, kv, 16)
        goes, want = pool.compact([])
        assert status.tolist() == want and page_map.tolist() == goes
        _same(pool, ref, idx)


def test_pages_run_out(dev):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    pool = Pool(5, [20, 30, 0, 0, 9], 8, 8, 10)  # 3 + 4 + 2 of 10 pages used
    ref, ptr, idx, kv = _pool_dev(pool, dev)
    host, bufs = _buffers(pool, dev, 1, 64)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    status = sta.sta_pages_fork(bufs, ref, ptr, idx, kv, i32([0, 1]), i32([2, 3]), 8)
    assert status.tolist() == [1, 1] == pool.fork(host, [0, 1], [2, 3])
    _same(pool, ref, idx, host, bufs)
    new = [40, 30, 0, 0, 60]
    status = sta.sta_pages_grow(ref, ptr, idx, kv, i32(np.concatenate([[0], np.cumsum(new)])), 8)
    assert status.tolist() == pool.grow(new)
    _same(pool, ref, idx)


def test_pages_bad_arguments_on_the_device_are_reported(dev):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731

    def fresh():
        pool = Pool(6, [20, 30, 0, 0], 8, 5, 30)
        return (pool, *_pool_dev(pool, dev))

    for parent, child, code in (([4], [2], 0x602), ([0], [-1], 0x602), ([0], [0], 0x602), ([0], [1], 0x605)):
        pool, ref, ptr, idx, kv = fresh()
        assert sta.sta_pages_fork([], ref, ptr, idx, kv, i32(parent), i32(child), 8).tolist() == [0, 0]
        assert sta.sta_device_error(reset=True) == code
        _same(pool, ref, idx)
    pool, ref, ptr, idx, kv = fresh()  # of two forks onto one child the first counts
    sta.sta_pages_fork([], ref, ptr, idx, kv, i32([0, 1]), i32([2, 2]), 8)
    pool.fork([], [0], [2])
    assert sta.sta_device_error(reset=True) == 0x605
    _same(pool, ref, idx)
    pool, ref, ptr, idx, kv = fresh()
    sta.sta_pages_free(ref, ptr, idx, kv, i32([9, 1, -1]), 8)
    pool.free([1])
    assert sta.sta_device_error(reset=True) == 0x602
    _same(pool, ref, idx)
    pool, ref, ptr, idx, kv = fresh()  # a list without room gets nothing, the others do
    new = [5 * 8 + 1, 33, 9, 0]
    assert sta.sta_pages_grow(ref, ptr, idx, kv, i32(np.concatenate([[0], np.cumsum(new)])), 8).tolist() == pool.grow(new)
    assert sta.sta_device_error(reset=True) == 0x604
    _same(pool, ref, idx)
    pool, ref, ptr, idx, kv = fresh()  # a page freed behind the lists' back
    page = pool.idx[0]
    ref[page] = 0
    sta.sta_pages_free(ref, ptr, idx, kv, i32([0]), 8)
    assert sta.sta_device_error(reset=True) == 0x603
    assert int(ref[page]) == 0
    pool, ref, ptr, idx, kv = fresh()
    idx[1] = 77
    before = idx.clone()
    sta.sta_pages_compact([], ref, ptr, idx, kv, 8)
    assert sta.sta_device_error(reset=True) == 0x601
    assert int(idx[1]) == int(before[1])
    sta.sta_pages_copy([torch.zeros(4, 16, device=dev)], i32([0, 9]), i32([1, 2]))
    assert sta.sta_device_error(reset=True) == 0x601


@pytest.mark.parametrize("page_elems,n_bufs", [(8, 1), (8 * 1025, 2), (40000, 300)])
def test_pages_copy(dev, page_elems, n_bufs):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    n_pages = 12
    bufs = [torch.randint(0, 100, (n_pages, page_elems), device=dev, dtype=torch.int16) for _ in range(n_bufs)]
    want = [b.clone() for b in bufs]
    src, dst = [3, 3, -1, 7, 5, 2], [0, 4, 1, -1, 5, 11]
    for b in want:
        b[0], b[4], b[11] = b[3].clone(), b[3].clone(), b[2].clone()
    sta.sta_pages_copy(bufs, torch.tensor(src, dtype=torch.int32, device=dev), torch.tensor(dst, dtype=torch.int32, device=dev))
    assert all(torch.equal(a, b) for a, b in zip(bufs, want))


# ---- together, as a serving loop uses them


def test_serving_loop(dev):
    """Prompts enter the cache, a sequence is forked, tokens follow one by one, a sequence leaves, the pool
    is compacted, decoding goes on; every step's attention against the plain form of its whole sequences."""
    import torch

    import split_kv_decode_bsr_gb300 as sta

    Hq, Hkv, d, P, n_pages, R, room = 8, 2, 64, 16, 64, 5, 12
    g = torch.Generator(device=dev).manual_seed(0)
    k_pages = torch.full((n_pages, P, Hkv, d), float("nan"), device=dev, dtype=torch.bfloat16)
    v_pages = k_pages.clone()
    ref = torch.zeros(n_pages, device=dev, dtype=torch.int32)
    ptr = torch.arange(0, (R + 1) * room, room, device=dev, dtype=torch.int32)
    idx = torch.full((R * room,), -1, device=dev, dtype=torch.int32)
    rope = sta.Rope(d, base=1e4)
    f = freqs(d)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)  # noqa: E731
    indptr = lambda a: np.concatenate([[0], np.cumsum(a)]).astype(np.int32)  # noqa: E731
    lens = [0] * R
    hist = [([], []) for _ in range(R)]  # each sequence's turned keys and values, in 64 bits

    def step(new):
        kv = [a + b for a, b in zip(lens, new)]
        status = sta.sta_pages_grow(ref, ptr, idx, i32(indptr(lens)), i32(indptr(kv)), P)
        assert int(status[1]) == 0
        n = sum(new)
        packed = torch.randn(n, (Hq + 2 * Hkv) * d, device=dev, generator=g).to(torch.bfloat16)
        q, k, v = (t.unflatten(1, (-1, d)) for t in packed.split([Hq * d, Hkv * d, Hkv * d], dim=1))
        qi, ki = indptr(new), indptr(kv)
        qd, kd = i32(qi), i32(ki)
        qr = sta.sta_rope_append_paged(q, k, v, k_pages, v_pages, ptr, idx, qd, kd, rope=rope)
        o, lse = sta.sta_chunk_fwd_paged(qr, k_pages, v_pages, ptr, idx, qd, qi, kd, ki)
        from _serving import chunk_ref

        for r in range(R):
            a, b = qi[r], qi[r + 1]
            pos = np.arange(lens[r], kv[r])
            kr = torch.from_numpy(rope_ref(_np(k[a:b]), pos, f, False)[0]).to(torch.bfloat16).double().numpy()
            hist[r][0].append(kr), hist[r][1].append(_np(v[a:b]))
            if b == a:
                continue
            ref_ = chunk_ref(_np(qr[a:b]), np.concatenate(hist[r][0]), np.concatenate(hist[r][1]), pos, 1 / 8)
            # keys turned here and there may round apart by a step where the value lies at a border
            loose = (ref_[0], ref_[1], ref_[2] + 2e-3, ref_[3] + 2e-3)
            check_chunk(o[a:b], lse[a:b], loose, b - a, f"step of {new}, request {r}")
            lens[r] = kv[r]

    step([37, 0, 80, 1, 0])
    sta.sta_pages_fork([k_pages, v_pages], ref, ptr, idx, i32(indptr(lens)), i32([2, 0]), i32([1, 4]), P)
    for a, c in ((2, 1), (0, 4)):
        lens[c] = lens[a]
        hist[c] = (list(hist[a][0]), list(hist[a][1]))
    for new in ([1, 1, 1, 1, 1], [1, 3, 0, 40, 1], [1, 1, 1, 1, 1]):
        step(new)
    sta.sta_pages_free(ref, ptr, idx, i32(indptr(lens)), i32([2]), P)
    lens[2], hist[2] = 0, ([], [])
    _, status = sta.sta_pages_compact([k_pages, v_pages], ref, ptr, idx, i32(indptr(lens)), P)
    assert int((ref > 0).sum()) == int(status[0]) and bool((ref[: int(status[0])] > 0).all())
    for new in ([1, 1, 0, 1, 1], [0, 20, 30, 1, 1]):
        step(new)

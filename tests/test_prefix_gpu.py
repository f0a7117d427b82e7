"""Attention of requests that share their first pages, on the GPU, against the plain 64-bit form of the chunk attention."""

import math

import numpy as np
import pytest

from _prefix import SharedCase
from _serving import check_chunk

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


def _run(dev, c, scale=None, splits=(0, 1, 3)):
    """As the library chooses; with every prefix taken apart, in one piece and in three (own parts of few rows then in
    so many runs)."""
    import split_kv_decode_bsr_gb300 as sta

    scale = 1 / math.sqrt(c.d) if scale is None else scale
    ref = c.ref(scale)
    for n in splits:
        o, lse = sta.sta_prefix_fwd_paged(**c.dev(dev), scale=scale, num_splits=n)
        check_chunk(o, lse, ref, int(c.q_indptr[-1]), f"{c.P} {n}")


def _whole_pages(tokens, P):
    return [t // P * P for t in tokens]


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 128), (4, 4, 64), (7, 1, 128), (9, 3, 64), (16, 1, 64), (130, 2, 64), (24, 12, 64)])
@pytest.mark.parametrize("P", [1, 8, 16, 48, 100, 128])
def test_prefix_ragged(dev, Hq, Hkv, d, P):
    # groups of three, one, four and two requests; own parts of one token to many, chunks that end in the middle of tiles
    prefix = _whole_pages([1200, 900, 1100, 777], P)
    new = [1, 1, 5, 1, 0, 1, 33, 2, 1, 1]
    own = [1, 140, 5, 20, 9, 129, 40, 300, 128, 16]
    c = SharedCase(P + d, [3, 1, 4, 2], prefix, new, own, Hq, Hkv, d, P, pad_rows=2)
    _run(dev, c, splits=(0, 1, 3, 40))


@pytest.mark.parametrize("n", [2, 15, 16, 17, 33, 70])
def test_prefix_of_one_group(dev, n):
    # its rows one, two or more query tiles, the last one partly filled, single or in a pair
    c = SharedCase(n, [n], [640], [1] * n, [1 + 37 * i % 50 for i in range(n)], 32, 4, 64, 16)
    _run(dev, c)
    c = SharedCase(n, [n], [640], [1 + i % 3 for i in range(n)], [3 + 37 * i % 50 for i in range(n)], 6, 2, 128, 64)
    _run(dev, c)


def test_prefix_rows_are_those_of_the_chunk_attention_where_nothing_is_shared(dev):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    for sizes, prefix in (([2, 3], [0, 0]), ([1] * 5, [320] * 5)):
        c = SharedCase(3, sizes, prefix, [1, 4, 1, 1, 9], [30, 40, 1, 70, 9], 8, 2, 64, 16)
        x = c.dev(dev)
        o, lse = sta.sta_prefix_fwd_paged(**x)
        x.pop("group_indptr_host"), x.pop("prefix_host")
        want = sta.sta_chunk_fwd_paged(**x)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_prefix_long_chunks(dev):
    # whole query tiles of each request
    c = SharedCase(11, [3], [256], [150, 64, 257], [150, 70, 300], 8, 2, 64, 16)
    _run(dev, c)
    c = SharedCase(12, [8], [1920], [40, 41, 40, 42, 40, 39, 38, 40], [40, 41, 50, 42, 60, 40, 150, 129], 8, 2, 64, 64)
    _run(dev, c, splits=(0, 1, 5))


@pytest.mark.parametrize("d", [64, 128])
def test_prefix_many_rows_to_merge(dev, d):
    # more rows than the merge has warps for at once; pieces of both kinds and requests without a prefix between them
    c = SharedCase(22, [3, 1, 2], [320, 0, 192], [90, 1, 120, 60, 70, 3], [95, 30, 120, 80, 70, 200], 48, 6, d, 32)
    _run(dev, c, splits=(0, 1, 3))


def test_prefix_many_requests_in_several_launches(dev):
    # 1500 requests in groups of 1 to 400, which the launches' parts cut
    sizes = [400, 1, 300, 2, 397, 400]
    n = sum(sizes)
    g = np.random.default_rng(4)
    c = SharedCase(13, sizes, [128, 64, 256, 128, 0, 192], g.integers(0, 3, n), 3 + g.integers(0, 9, n), 2, 1, 64, 16)
    _run(dev, c)


def test_prefix_strides_padding_outputs_and_workspace(dev):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = SharedCase(14, [4], [512], [1, 2, 1, 3], [5, 6, 130, 9], 8, 2, 128, 16, pad_rows=5)
    x, n = c.dev(dev), int(c.q_indptr[-1])
    scale = 0.07
    ref = c.ref(scale)
    wide = torch.full((n + 5, 8 * 128 + 72), float("nan"), device=dev, dtype=torch.bfloat16)
    wide[:, :1024] = x["q"].flatten(1)
    x["q"] = wide[:, :1024].unflatten(1, (8, 128))
    o, lse = torch.full((n + 5, 8, 128), 5.0, device=dev, dtype=torch.bfloat16), torch.full((n + 5, 8), 5.0, device=dev)
    need = sta.prefix_workspace_bytes(c.q_indptr, c.kv_indptr, 4, c.group_indptr, c.prefix, 8, 2, 128, 16, num_splits=2)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=dev)
    got = sta.sta_prefix_fwd_paged(**x, scale=scale, num_splits=2, o=o, lse=lse, workspace=ws[:need])
    assert got[0] is o and got[1] is lse
    check_chunk(o, lse, ref, n)
    assert (o[n:] == 5.0).all() and (lse[n:] == 5.0).all() and (ws[need:] == 255).all()
    with pytest.raises(ValueError):
        sta.sta_prefix_fwd_paged(**x, num_splits=2, workspace=ws[:256])


@pytest.mark.parametrize("P", [16, 100])
def test_prefix_in_far_pages(dev, P):
    # offsets past 32 bits in the cache: the same numbers as at its start
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = SharedCase(18, [40], [1200 // P * P], [1] * 39 + [20], [3 + 5 * i % 70 for i in range(39)] + [55], 32, 8, 128, P)
    x = c.dev(dev)
    want = [sta.sta_prefix_fwd_paged(**x, num_splits=s) for s in (0, 2)]
    n, far = x["k_pages"].shape[0], (1 << 31) // (P * 8 * 128) + 1000
    for name in ("k_pages", "v_pages"):
        big = torch.empty(far + n, P, 8, 128, device=dev, dtype=torch.bfloat16)  # 4.3 GB and more
        big[far:] = x[name]
        x[name] = big
    x["page_indices_dev"] = x["page_indices_dev"] + far
    for s, (o, lse) in zip((0, 2), want):
        got = sta.sta_prefix_fwd_paged(**x, num_splits=s)
        assert torch.equal(got[0], o) and torch.equal(got[1], lse)


def test_prefix_streams_and_repeats(dev):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = SharedCase(15, [20, 12], [2048, 1024], [1] * 32, [1 + 13 * i % 90 for i in range(32)], 16, 4, 128, 16)
    x = c.dev(dev)
    want = sta.sta_prefix_fwd_paged(**x)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):  # two calls at once
        one, two = sta.sta_prefix_fwd_paged(**x, stream=a), sta.sta_prefix_fwd_paged(**x, stream=b)
        torch.cuda.synchronize()
        for got in (one, two):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("splits", [0, 2])
def test_prefix_calls_that_read_what_the_last_one_wrote(dev, splits):
    # each call's queries are the last one's results, in two buffers by turns or in one; its kernels may start before the
    # last one's have ended
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = SharedCase(17, [40, 24], [1024, 512], [1] * 60 + [3] * 4, [4 + 11 * i % 60 for i in range(64)], 16, 8, 128, 16)
    x = c.dev(dev)
    q = x.pop("q")
    ws = torch.empty(sta.prefix_workspace_bytes(c.q_indptr, c.kv_indptr, 64, c.group_indptr, c.prefix, 16, 8, 128, 16,
                                                num_splits=splits), dtype=torch.uint8, device=dev)

    def chain(buffers, wait):
        at = buffers[0].copy_(q)
        for i in range(12):
            at, _ = sta.sta_prefix_fwd_paged(q=at, **x, scale=3.0, num_splits=splits, o=buffers[(i + 1) % len(buffers)], workspace=ws)
            if wait:
                torch.cuda.synchronize()
        return at.clone()

    two = [torch.empty_like(q) for _ in range(2)]
    want = chain(two, True)
    for _ in range(5):
        assert torch.equal(chain(two, False), want)
        assert torch.equal(chain(two[:1], False), want)


def test_prefix_host_values_of_any_kind(dev):
    import array

    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = SharedCase(20, [3, 2], [256, 128], [1, 2, 1, 1, 4], [5, 20, 9, 30, 7], 4, 2, 64, 16)
    x, names = c.dev(dev), ("q_indptr_host", "kv_indptr_host", "group_indptr_host", "prefix_host")
    host = {n: np.asarray(x.pop(n)) for n in names}
    want = sta.sta_prefix_fwd_paged(**x, **host, num_splits=1)
    strided = lambda a: np.repeat(a, 2)[::2]  # noqa: E731
    for kind in (list, tuple, torch.from_numpy, lambda a: torch.from_numpy(a).long(), lambda a: a.astype(np.int64), strided,
                 lambda a: array.array("i", a.tolist()), lambda a: memoryview(a)):
        got = sta.sta_prefix_fwd_paged(**x, **{n: kind(a) for n, a in host.items()}, num_splits=1)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for name in names:
        for bad in (lambda a: a[:-1], lambda a: np.concatenate([a, a[-1:]]), lambda a: np.stack([a, a]), lambda a: a[:0]):
            with pytest.raises((ValueError, sta.StaError)):
                sta.sta_prefix_fwd_paged(**x, **dict(host, **{name: bad(host[name])}))
        with pytest.raises(TypeError):
            sta.sta_prefix_fwd_paged(**x, **dict(host, **{name: torch.from_numpy(host[name]).to(dev)}))


@pytest.mark.parametrize("P", [16, 20])
@pytest.mark.parametrize("d", [64, 128])
def test_prefix_steps_one_after_the_other(dev, d, P):
    # norms and the cache write, then the attention of what was written, whose results are the next step's queries; each of the
    # kernels may start before the one before it has ended
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = SharedCase(d, [30, 1, 20], [640, 0, 960], [1] * 49 + [4, 2], [5 + 9 * i % 70 for i in range(51)], 8, 4, d, P)
    x = c.dev(dev)
    q, groups = x.pop("q"), {n: x.pop(n) for n in ("group_indptr_host", "prefix_host")}
    hosts = {n: x.pop(n) for n in ("q_indptr_host", "kv_indptr_host")}
    k, v = (torch.randn(q.shape[0], 4, d, device=dev).to(torch.bfloat16) for _ in "kv")
    rope, w = sta.Rope(d), torch.rand(d, device=dev) + 0.5

    def steps(wait):
        at, cache = q, dict(x, k_pages=x["k_pages"].clone(), v_pages=x["v_pages"].clone())
        for i in range(10):
            at = sta.sta_norm_rope_append_paged(at, k.roll(i, 0), v.roll(i, 1), cache["k_pages"], cache["v_pages"],
                                                *(cache[n] for n in ("page_indptr_dev", "page_indices_dev", "q_indptr_dev",
                                                                     "kv_indptr_dev")), rope=rope, q_weight=w, k_weight=w)
            if wait:
                torch.cuda.synchronize()
            at, _ = sta.sta_prefix_fwd_paged(q=at, **cache, **hosts, **groups, num_splits=i % 3)
            if wait:
                torch.cuda.synchronize()
        return at

    want = steps(True)
    for _ in range(5):
        assert torch.equal(steps(False), want)


@pytest.mark.parametrize("splits", [0, 1, 4])
def test_prefix_captured_and_replayed_with_other_lengths(dev, splits):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    # planned for up to 60 own tokens a request, two of them new; lists with room for them
    n, prefix = 6, 512
    full = SharedCase(16, [n], [prefix], [2] * n, [60] * n, 8, 2, 64, 16)
    x = full.dev(dev)
    q = torch.zeros(2 * n, 8, 64, device=dev, dtype=torch.bfloat16)
    x["q"] = q
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = sta.sta_prefix_fwd_paged(**x, num_splits=splits)
    for seed, new, own in ((1, [2] * n, [60] * n), (2, [1, 2, 0, 1, 0, 2], [1, 2, 0, 33, 17, 48]), (3, [1] * n, [20] * n),
                           (4, [0, 0, 0, 1, 0, 0], [0, 7, 0, 9, 0, 0])):
        c = SharedCase(16 + seed, [n], [prefix], new, own, 8, 2, 64, 16)
        # the same lists and pages, filled anew
        for r in range(n):
            at = torch.from_numpy(full.rows(r, np.arange(c.kv[r])))
            for name, seq in (("k_pages", c.k_seq), ("v_pages", c.v_seq)):
                x[name].view(-1, 2, 64)[at.to(dev)] = seq[r].to(dev)
        rows = int(c.q_indptr[-1])
        q.zero_()
        q[:rows] = c.q.to(dev)
        x["q_indptr_dev"].copy_(torch.from_numpy(c.q_indptr))
        x["kv_indptr_dev"].copy_(torch.from_numpy(c.kv_indptr))
        o.fill_(5.0)
        lse.fill_(5.0)
        g.replay()
        torch.cuda.synchronize()
        assert sta.sta_device_error() == 0
        check_chunk(o, lse, c.ref(1 / 8.0), rows, f"replay {seed}")
        assert (o[rows:] == 5.0).all() and (lse[rows:] == 5.0).all()


def test_prefix_damaged_lists_and_lengths_are_reported(dev):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = SharedCase(17, [4], [512], [1] * 4, [5, 6, 30, 9], 8, 2, 64, 16)
    good = sta.sta_prefix_fwd_paged(**c.dev(dev), num_splits=2)
    torch.cuda.synchronize()
    assert sta.sta_device_error() == 0

    def broken(change):
        x = c.dev(dev)
        change(x)
        got = sta.sta_prefix_fwd_paged(**x, num_splits=2)
        torch.cuda.synchronize()
        return got, sta.sta_device_error(reset=True)

    last = int(c.page_indptr[2]) + 512 // 16 - 1
    (o, _), code = broken(lambda x: x["page_indices_dev"].__setitem__(last, int(c.page_indices[c.page_indptr[1]])))
    assert code == 0x609  # request 2 has another last shared page
    assert torch.equal(o[[0, 1, 3]], good[0][[0, 1, 3]])
    for bad in (-1, c.n_pages):
        _, code = broken(lambda x: x["page_indices_dev"].__setitem__(3, bad))  # a page of the prefix
        assert code == 0x110
    # request 1 shorter than the prefix on the device alone
    short = c.kv_indptr.copy()
    short[2:] -= 6 + 200
    (o, _), code = broken(lambda x: x["kv_indptr_dev"].copy_(torch.from_numpy(short)))
    assert code == 0x608
    assert torch.equal(o[[0, 2, 3]], good[0][[0, 2, 3]])


def test_prefix_a_query_that_is_no_number(dev):
    import torch

    import split_kv_decode_bsr_gb300 as sta

    c = SharedCase(18, [3], [512], [1, 2, 1], [5, 20, 9], 4, 2, 64, 16)
    x = c.dev(dev)
    want = sta.sta_prefix_fwd_paged(**x, num_splits=2)
    x["q"][2, 1, 7] = float("nan")
    got = sta.sta_prefix_fwd_paged(**x, num_splits=2)
    dead = torch.zeros(4, 4, dtype=torch.bool, device=dev)
    dead[2, 1] = True
    assert torch.isnan(got[0][dead]).all() and torch.isnan(got[1][dead]).all()
    assert torch.equal(got[0][~dead], want[0][~dead]) and torch.equal(got[1][~dead], want[1][~dead])


def test_prefix_scores_far_apart(dev):
    # scores of some hundreds: all of a row's weight in the prefix, or all of it behind it
    c = SharedCase(19, [8], [384], [1] * 8, [1 + 9 * i for i in range(8)], 8, 2, 64, 16, value=8.0)
    _run(dev, c, scale=0.5)


def test_a_forked_batch_is_served_together(dev):
    # one prompt written and attended, forked seven times, then three steps of one token each: grow, norm and write, attend
    import torch

    import split_kv_decode_bsr_gb300 as sta
    from _norm import norm_ref
    from _serving import BF16_HALF_STEP, chunk_ref, freqs

    n, Hq, Hkv, d, P, L = 8, 8, 2, 64, 16, 1000
    i32 = dict(dtype=torch.int32, device=dev)
    g = torch.Generator(device=dev).manual_seed(5)
    rand = lambda *s: torch.randn(s, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    room, n_pages = 70, 140
    ref, idx = torch.zeros(n_pages, **i32), torch.full((room * n,), -1, **i32)
    ptr = torch.arange(0, room * n + 1, room, **i32)
    kp, vp = (torch.full((n_pages, P, Hkv, d), float("nan"), device=dev, dtype=torch.bfloat16) for _ in "kv")
    qw, kw = torch.rand(d, device=dev) + 0.5, torch.rand(d, device=dev) + 0.5
    rope, f = sta.Rope(d), freqs(d)
    lens = np.zeros(n, np.int64)
    keys, vals = [np.zeros((0, Hkv, d)) for _ in range(n)], [np.zeros((0, Hkv, d)) for _ in range(n)]
    indptr = lambda a: np.concatenate([[0], np.cumsum(a)]).astype(np.int32)  # noqa: E731
    to = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731

    def step(new, shared):
        nonlocal lens
        after = lens + new
        assert sta.sta_pages_grow(ref, ptr, idx, to(indptr(lens)), to(indptr(after)), P).tolist()[1] == 0
        m = int(new.sum())
        q, k, v = rand(m, Hq, d), rand(m, Hkv, d), rand(m, Hkv, d)
        qi, ki = indptr(new), indptr(after)
        qn = sta.sta_norm_rope_append_paged(q, k, v, kp, vp, ptr, idx, to(qi), to(ki), rope, qw, kw)
        if shared:
            o, lse = sta.sta_prefix_fwd_paged(qn, kp, vp, ptr, idx, to(qi), qi, to(ki), ki, [0, n], [shared],
                                              num_splits=2)
        else:
            o, lse = sta.sta_chunk_fwd_paged(qn, kp, vp, ptr, idx, to(qi), qi, to(ki), ki)
        for r in range(n):
            a, b = qi[r], qi[r + 1]
            pos = np.arange(lens[r], after[r])
            want, tol = norm_ref(k[a:b].double().cpu().numpy(), kw.double().cpu().numpy(), 1e-6, pos, f, False)
            rows = to(np.array([int(idx[room * r + t // P]) * P + t % P for t in pos], np.int64))
            got = kp.view(-1, Hkv, d)[rows].double().cpu().numpy()
            assert (np.abs(got - want) <= BF16_HALF_STEP * np.abs(want) + tol * (1 + BF16_HALF_STEP)).all()
            keys[r] = np.concatenate([keys[r], got])
            vals[r] = np.concatenate([vals[r], v[a:b].double().cpu().numpy()])
            at = slice(-3, None)  # of a long prompt the last tokens
            x = chunk_ref(qn[a:b][at].double().cpu().numpy(), keys[r], vals[r], pos[at], 1 / math.sqrt(d))
            if b > a:
                check_chunk(o[a:b][at], lse[a:b][at], x, len(pos[at]), f"request {r}")
        lens = after

    step(np.array([L] + [0] * (n - 1)), 0)
    bufs = [kp, vp]
    status = sta.sta_pages_fork(bufs, ref, ptr, idx, to(indptr(lens)), torch.zeros(n - 1, **i32), torch.arange(1, n, **i32), P)
    assert status.tolist() == [n - 1, 0]
    lens = np.full(n, L)
    for r in range(1, n):
        keys[r], vals[r] = keys[0].copy(), vals[0].copy()
    for _ in range(3):
        step(np.ones(n, np.int64), L // P * P)
    assert sta.sta_device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 1, 128), (16, 2, 128), (4, 1, 64), (8, 2, 64), (12, 3, 128), (8, 4, 128)])
@pytest.mark.parametrize("own", [(40, 40, 40, 200), (17, 100, 33, 260), (1, 16, 1, 16, 1, 16, 700)])
def test_prefix_short_own_parts_before_long_ones(dev, Hq, Hkv, d, own):
    # several warps a head: some have no tile of the short pieces, and come first to the long ones, past the ring's first turn
    import torch

    import split_kv_decode_bsr_gb300 as sta

    n = 8 * len(own)
    c = SharedCase(23, [n], [512], [1] * n, list(own) * 8, Hq, Hkv, d, 16)
    x, scale = c.dev(dev), 1 / math.sqrt(d)
    ref, cold = c.ref(scale), torch.empty(1 << 28, dtype=torch.uint8, device=dev)
    for splits in (0, 1, 2):
        first = None
        for _ in range(4):
            cold.fill_(1)  # K and V come from memory, the lists too
            got = sta.sta_prefix_fwd_paged(**x, scale=scale, num_splits=splits)
            check_chunk(*got, ref, n, f"{splits}")
            first = first or got
            assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])

"""Operators around a paged KV cache whose sequences share their beginnings, measured over their range of sizes.

Root-mean-square norms of query and key heads with the rotary positions in the same pass (forward, the
gradient, and fused with the write of new tokens into the cache's pages), and the attention of a batch whose
requests share a long prefix, computed once for each group of them. Each case is a dict of plain values; `run`
makes one pass, in plain torch operations or, where `own` is true, through the library's calls.
"""

import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
BASE, ORIG, LOW, HIGH = 500000.0, 8192.0, 1.0, 32.0
MOST_ROWS = 8192 * 40 * 128 * 2  # bytes of queries and keys in the largest norm
MOST_PAIRS = 1.9e9               # (query head, key) pairs of the largest attention


def listed():
    return [
        # a training step's 8192 tokens: one layer's queries and keys out of a packed projection
        dict(name="norm_rope_train", op="norm", dtype="bf16", n=8192, hq=32, hk=8, d=128, rot=128, interleaved=False,
             scaling="blend", factor=32.0, max_pos=1 << 17, pad=1024, eps=1e-6),
        # a decode step of 48 sequences that keep no cache of their own: latency
        dict(name="norm_rope_step", op="norm", dtype="bf16", n=48, hq=16, hk=2, d=64, rot=64, interleaved=True,
             scaling="none", factor=1.0, max_pos=32768, pad=128, eps=1e-5),
        # heads that turn in part, in 32 bits, odd lengths
        dict(name="norm_rope_part_f32", op="norm", dtype="f32", n=1999, hq=12, hk=3, d=80, rot=40, interleaved=False,
             scaling="linear", factor=4.0, max_pos=8192, pad=0, eps=1e-6),
        # the backward pass of the training step
        dict(name="norm_grad_train", op="grad", dtype="bf16", n=8192, hq=32, hk=8, d=128, rot=128, interleaved=False,
             scaling="blend", factor=32.0, max_pos=1 << 17, pad=1024, eps=1e-6),
        # the backward pass of a small model in 32 bits, a part of each head turning in neighbouring pairs
        dict(name="norm_grad_part_f32", op="grad", dtype="f32", n=1999, hq=12, hk=4, d=64, rot=32, interleaved=True,
             scaling="none", factor=1.0, max_pos=8192, pad=64, eps=1e-6),
        # one decode step: 64 sequences of one new token each enter the cache
        dict(name="norm_append_64", op="append", mix=1, n_req=64, hq=32, hkv=8, d=128, page=16, new="one", new_max=1,
             past_min=512, past_max=32767, rot=128, interleaved=False, eps=1e-6),
        # prompts of odd lengths enter a cache of 100-token pages
        dict(name="norm_append_prompts", op="append", mix=2, n_req=24, hq=32, hkv=4, d=128, page=100, new="log",
             new_max=4096, past_min=0, past_max=5000, rot=64, interleaved=True, eps=1e-6),
        # a few answers to one short prompt: latency
        dict(name="prefix_small", op="prefix", mix=3, groups=1, n_req=4, hq=16, hkv=2, d=64, page=16, prefix_min=512,
             prefix_max=512, new="one", new_max=1, past_min=0, past_max=90),
        # one decode step of 64 requests behind one system prompt of 8192 tokens
        dict(name="prefix_single_64", op="prefix", mix=4, groups=1, n_req=64, hq=32, hkv=8, d=128, page=16,
             prefix_min=8192, prefix_max=8192, new="one", new_max=1, past_min=16, past_max=1024),
        # 120 answers forked from one long document
        dict(name="prefix_forks_120", op="prefix", mix=5, groups=1, n_req=120, hq=32, hkv=8, d=128, page=64,
             prefix_min=32768, prefix_max=32768, new="one", new_max=1, past_min=0, past_max=4000),
        # several documents, drafted tokens checked against each, odd head group and pages
        dict(name="prefix_groups_drafts", op="prefix", mix=6, groups=7, n_req=33, hq=28, hkv=4, d=128, page=100,
             prefix_min=900, prefix_max=20000, new="log", new_max=8, past_min=0, past_max=3000),
        # questions of odd lengths behind one document, all their tokens at once: bound by the matrix products
        dict(name="prefix_chunks", op="prefix", mix=7, groups=1, n_req=32, hq=32, hkv=8, d=128, page=16,
             prefix_min=12000, prefix_max=12000, new="log", new_max=1024, past_min=0, past_max=200),
    ]


def _log_int(rng, lo, hi):
    return int(min(hi, max(lo, math.floor(math.exp(rng.uniform(math.log(max(lo, 0.7)), math.log(hi + 0.99)))))))


def draw(rng):
    op = rng.choice(["norm", "grad", "append", "prefix", "prefix", "prefix"])
    mix = rng.randrange(1 << 30)
    if op in ("norm", "grad"):
        d = rng.choice([32, 64, 80, 96, 128, 256])
        c = dict(op=op, dtype=rng.choice(["bf16", "f32"]), n=_log_int(rng, 1, 16384), hq=rng.randint(1, 40),
                 hk=rng.randint(1, 8), d=d, rot=2 * rng.randint(1, d // 2) if rng.random() < 0.5 else d,
                 interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "blend"]),
                 factor=rng.choice([1.5, 4.0, 32.0]), max_pos=_log_int(rng, 100, 1 << 20), pad=8 * rng.randint(0, 40),
                 eps=rng.choice([1e-6, 1e-5, 1e-3]))
        c["n"] = max(1, min(c["n"], MOST_ROWS // ((c["hq"] + c["hk"]) * d * (2 if c["dtype"] == "bf16" else 4))))
        return c
    if op == "append":
        d = rng.choice([64, 128])
        hkv = rng.randint(1, 8)
        return dict(op=op, mix=mix, n_req=_log_int(rng, 1, 64), hq=hkv * rng.randint(1, 8), hkv=hkv, d=d,
                    page=rng.choice([1, 5, 16, 64, 100, 256]), new=rng.choice(["one", "log"]),
                    new_max=_log_int(rng, 1, 600), past_min=0, past_max=_log_int(rng, 1, 6000),
                    rot=rng.choice([d // 4, d // 2, d]), interleaved=rng.random() < 0.5, eps=rng.choice([1e-6, 1e-5]))
    hkv = rng.choice([1, 2, 3, 4, 8])
    group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
    n_req = _log_int(rng, 1, 128)
    prefix = _log_int(rng, 64, 32768)
    c = dict(op=op, mix=mix, groups=_log_int(rng, 1, min(n_req, 12)), n_req=n_req, hq=hkv * group, hkv=hkv,
             d=rng.choice([64, 128]), page=rng.choice([1, 8, 16, 17, 48, 64, 100, 128]), prefix_min=prefix // rng.choice([1, 1, 4]),
             prefix_max=prefix, new=rng.choice(["one", "log", "log"]), new_max=_log_int(rng, 1, 1024), past_min=0,
             past_max=_log_int(rng, 1, 4000))
    while n_req * c["hq"] * c["new_max"] * (c["new_max"] + c["past_max"] + c["prefix_max"]) > MOST_PAIRS:
        c["new_max"] = max(1, c["new_max"] // 2)
        if c["new_max"] == 1:
            break
    return c


# ---------------------------------------------------------------------------
# what a case's numbers stand for: lengths and groups, from the case alone


def _spread(g, lo, hi, n):
    """n whole numbers in [lo, hi], spread over their logarithm."""
    x = np.floor(np.exp(g.uniform(math.log(lo + 1.0), math.log(hi + 1.0 + 1e-9), n))).astype(np.int64) - 1
    return np.clip(x, lo, max(hi, lo))


def _lens(case):
    """Each request's own past tokens (behind its prefix) and its new ones."""
    g = np.random.default_rng(case["mix"])
    n, m = case["n_req"], case["new_max"]
    past = _spread(g, case["past_min"], case["past_max"], n)
    new = np.ones(n, np.int64) if case["new"] == "one" else _spread(g, 1, m, n)
    return past, new


def _groups(case):
    """group_indptr over the requests, and each group's shared tokens, in whole pages."""
    g = np.random.default_rng(case["mix"] + 1)
    n, k = case["n_req"], case["groups"]
    cuts = np.sort(g.choice(np.arange(1, n), k - 1, replace=False)) if k > 1 else np.zeros(0, np.int64)
    shared = _spread(g, case["prefix_min"], case["prefix_max"], k)
    return np.concatenate([[0], cuts, [n]]).astype(np.int32), (shared // case["page"] * case["page"]).astype(np.int32)


def _indptr(x):
    return np.concatenate([[0], np.cumsum(x)]).astype(np.int32)


def _pages_of(lens, page):
    return (lens + page - 1) // page


def _rope_of(case):
    return dict(rot=case["rot"], interleaved=case["interleaved"], scaling=case.get("scaling", "none"),
                factor=case.get("factor", 1.0), mscale=1.25 if case.get("scaling") == "blend" else 1.0)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    op = case["op"]
    randn = lambda *shape: torch.randn(shape, generator=g, device=dev)  # noqa: E731
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    st = dict(case=case)
    if op != "prefix":
        d = case["d"]
        st.update(rope=_rope_of(case), eps=case["eps"], q_weight=1.0 + 0.2 * randn(d), k_weight=1.0 + 0.2 * randn(d))
    if op in ("norm", "grad"):
        n, hq, hk, dt = case["n"], case["hq"], case["hk"], DT[case["dtype"]]
        wide = (2.0 * randn(n, (hq + hk) * d + case["pad"])).to(dt)  # one projection's output
        st.update(q=wide[:, :hq * d].unflatten(1, (hq, d)), k=wide[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)),
                  pos=torch.randint(0, case["max_pos"], (n,), generator=g, device=dev, dtype=torch.int32))
        if op == "grad":
            st.update(dq=randn(n, hq, d).to(dt), dk=randn(n, hk, d).to(dt))
        return st
    past, new = _lens(case)
    page, n_req, hq, hkv, d = case["page"], case["n_req"], case["hq"], case["hkv"], case["d"]
    n = int(new.sum())
    if op == "append":
        kv = past + new
        held = _pages_of(kv, page)
        n_pages = int(held.sum()) + 3
        order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
        packed = randn(n, (hq + 2 * hkv) * d).to(torch.bfloat16)  # one projection's output
        q, k, v = packed.split([hq * d, hkv * d, hkv * d], dim=1)
        st.update(q=q.unflatten(1, (hq, d)), k=k.unflatten(1, (hkv, d)), v=v.unflatten(1, (hkv, d)),
                  page_indices=order[:int(held.sum())].contiguous())
    else:
        ptr, shared = _groups(case)
        mine = np.repeat(np.arange(case["groups"]), np.diff(ptr))  # each request's group
        kv = shared[mine] + past + new
        first, rest = shared // page, _pages_of(past + new, page)  # pages of a group's prefix, of a request's own
        n_pages = int(first.sum() + rest.sum()) + 3
        order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
        held = first[mine] + rest
        f0, r0 = _indptr(first), int(first.sum()) + _indptr(rest)
        at = np.concatenate([np.concatenate([np.arange(f0[a], f0[a + 1]), np.arange(r0[r], r0[r + 1])])
                             for r, a in enumerate(mine)])
        st.update(q=randn(n, hq, d).to(torch.bfloat16), page_indices=order[to(at.astype(np.int64))],
                  group_indptr_host=ptr, prefix_host=shared, scale=1.0 / math.sqrt(d))
    st.update(page=page, page_indptr=to(_indptr(held)), q_indptr=to(_indptr(new)), kv_indptr=to(_indptr(kv)),
              q_indptr_host=_indptr(new), kv_indptr_host=_indptr(kv), k_pages=randn(n_pages, page, hkv, d).to(torch.bfloat16),
              v_pages=randn(n_pages, page, hkv, d).to(torch.bfloat16))
    return st


def run(st):
    op = st["case"]["op"]
    if own:
        return {"norm": _own_norm, "grad": _own_grad, "append": _own_append, "prefix": _own_prefix}[op](st)
    return {"norm": _plain_norm, "grad": _plain_grad, "append": _plain_append, "prefix": _plain_prefix}[op](st)


# ---------------------------------------------------------------------------
# the library's calls


def _params(r):
    import split_kv_decode_bsr_gb300 as sta

    return sta.Rope(r["rot"], base=BASE, interleaved=r["interleaved"], scaling=r["scaling"], factor=r["factor"],
                    orig_len=ORIG, low_turns=LOW, high_turns=HIGH, mscale=r["mscale"])


def _own_norm(st):
    import split_kv_decode_bsr_gb300 as sta

    return sta.sta_norm_rope(st["q"], st["k"], st["pos"], _params(st["rope"]), q_weight=st["q_weight"],
                             k_weight=st["k_weight"], eps=st["eps"])


def _own_grad(st):
    import split_kv_decode_bsr_gb300 as sta

    return sta.sta_norm_rope_bwd(st["dq"], st["dk"], st["q"], st["k"], st["pos"], _params(st["rope"]),
                                 q_weight=st["q_weight"], k_weight=st["k_weight"], eps=st["eps"])


def _own_append(st):
    import split_kv_decode_bsr_gb300 as sta

    q = sta.sta_norm_rope_append_paged(st["q"], st["k"], st["v"], st["k_pages"], st["v_pages"], st["page_indptr"],
                                       st["page_indices"], st["q_indptr"], st["kv_indptr"], rope=_params(st["rope"]),
                                       q_weight=st["q_weight"], k_weight=st["k_weight"], eps=st["eps"])
    return q, st["k_pages"], st["v_pages"]


def _own_prefix(st):
    import split_kv_decode_bsr_gb300 as sta

    return sta.sta_prefix_fwd_paged(st["q"], st["k_pages"], st["v_pages"], st["page_indptr"], st["page_indices"],
                                    st["q_indptr"], st["q_indptr_host"], st["kv_indptr"], st["kv_indptr_host"],
                                    st["group_indptr_host"], st["prefix_host"], scale=st["scale"])


# ---------------------------------------------------------------------------
# plain forms


def _cos_sin(pos, r):
    """[n, 1, rot / 2] each; angles in 64 bits, since far positions need them."""
    rot = r["rot"]
    f = BASE ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if r["scaling"] == "linear":
        f = f / r["factor"]
    if r["scaling"] == "blend":
        w = np.clip((ORIG * f / (2 * math.pi) - LOW) / (HIGH - LOW), 0.0, 1.0)
        f = w * f + (1 - w) * f / r["factor"]
    ang = pos.double()[:, None] * torch.from_numpy(f).to(pos.device)[None, :]
    return (torch.cos(ang) * r["mscale"]).float()[:, None], (torch.sin(ang) * r["mscale"]).float()[:, None]


def _turn(x, cos, sin, r):
    rot = r["rot"]
    y = x.clone()
    if r["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2:rot]
        y[..., : rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    return y


def _rms(x, eps):
    return torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)


def _plain_norm(st):
    cos, sin = _cos_sin(st["pos"], st["rope"])
    q, k = st["q"].float(), st["k"].float()
    return (_turn(q * _rms(q, st["eps"]) * st["q_weight"], cos, sin, st["rope"]).to(st["q"].dtype),
            _turn(k * _rms(k, st["eps"]) * st["k_weight"], cos, sin, st["rope"]).to(st["k"].dtype))


def _norm_back(dy, x, w, cos, sin, st):
    """Gradients of x and of w, sums over all rows in 64 bits."""
    g = _turn(dy.float(), cos, -sin, st["rope"])
    r = _rms(x.float(), st["eps"])
    xhat = x.float() * r
    gw = g * w
    dx = r * (gw - xhat * (gw * xhat).mean(-1, keepdim=True))
    return dx.to(x.dtype), (g * xhat).sum((0, 1), dtype=torch.float64).float()


def _plain_grad(st):
    cos, sin = _cos_sin(st["pos"], st["rope"])
    dq, dqw = _norm_back(st["dq"], st["q"], st["q_weight"], cos, sin, st)
    dk, dkw = _norm_back(st["dk"], st["k"], st["k_weight"], cos, sin, st)
    return dq, dk, dqw, dkw


def _plain_append(st):
    qp, kp, page = st["q_indptr"].long(), st["kv_indptr"].long(), st["page"]
    t = torch.arange(st["q"].shape[0], device=qp.device)
    r = torch.searchsorted(qp, t, right=True) - 1
    pos = (kp[r + 1] - kp[r]) - (qp[r + 1] - qp[r]) + (t - qp[r])
    row = st["page_indices"].long()[st["page_indptr"].long()[r] + pos // page] * page + pos % page
    cos, sin = _cos_sin(pos, st["rope"])
    q, k = st["q"].float(), st["k"].float()
    q = _turn(q * _rms(q, st["eps"]) * st["q_weight"], cos, sin, st["rope"])
    k = _turn(k * _rms(k, st["eps"]) * st["k_weight"], cos, sin, st["rope"])
    st["k_pages"].flatten(0, 1)[row] = k.to(torch.bfloat16)
    st["v_pages"].flatten(0, 1)[row] = st["v"]
    return q.to(torch.bfloat16), st["k_pages"], st["v_pages"]


def _keys(pages, st, entry, lens, L, skip):
    """[B, hkv, L, d] in 32 bits: tokens skip .. skip + L - 1 of lists that start at `entry`, `lens` of them there."""
    page = st["page"]
    j = torch.arange(L, device=entry.device)
    at = (entry[:, None] + (skip[:, None] + j) // page).clamp(max=st["page_indices"].numel() - 1)
    slot = st["page_indices"].long()[at] * page + (skip[:, None] + j) % page
    return pages.flatten(0, 1)[torch.where(j < lens[:, None], slot, 0)].float().permute(0, 2, 1, 3)


def _part(q, rows, live, see, K, V, scale):
    """Attention of q's rows [B, T] over K, V [B, hkv, L, d]: maxima, sums and products of each, by row of q."""
    n, hq, d = q.shape
    B, T = rows.shape
    hkv = K.shape[1]
    Q = q[rows].float().reshape(B, T, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    s = torch.matmul(Q.reshape(B, hkv, -1, d), K.transpose(2, 3)).mul_(scale).reshape(B, hkv, hq // hkv, T, -1)
    s.masked_fill_(~see[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True) if s.shape[-1] else s.new_full((*s.shape[:-1], 1), -math.inf)
    s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    o = torch.matmul(s.reshape(B, hkv, -1, s.shape[-1]), V).reshape(B, hkv, hq // hkv, T, d)
    out = torch.cat([m, s.sum(-1, keepdim=True), o], -1).permute(0, 3, 1, 2, 4).reshape(B, T, hq, d + 2)
    by_row = q.new_zeros((n, hq, d + 2), dtype=torch.float32)
    by_row[rows[live]] = out[live]
    return by_row[..., 0], by_row[..., 1], by_row[..., 2:]


def _plain_prefix(st):
    q, dev = st["q"], st["q"].device
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev).long()  # noqa: E731
    qh, kh, gp, shared = st["q_indptr_host"], st["kv_indptr_host"], st["group_indptr_host"], st["prefix_host"]
    mine = np.repeat(np.arange(shared.size), np.diff(gp))
    qp, ptr, last = st["q_indptr"].long(), st["page_indptr"].long(), q.shape[0] - 1
    # each group's prefix, seen by all of its tokens
    T = int(np.diff(qh[gp]).max())
    t, n_t = torch.arange(T, device=dev), to(np.diff(qh[gp]))
    P, L = to(shared), int(shared.max())
    live = t < n_t[:, None]
    see = (torch.arange(L, device=dev) < P[:, None])[:, None].expand(-1, T, -1)
    zero, lead = torch.zeros_like(P), ptr[to(gp[:-1])]
    m0, l0, o0 = _part(q, (to(qh[gp[:-1]])[:, None] + t).clamp(max=last), live, see,
                       _keys(st["k_pages"], st, lead, P, L, zero), _keys(st["v_pages"], st, lead, P, L, zero), st["scale"])
    # each request's own tokens behind it, causal
    own_len, ql, skip = to(np.diff(kh) - shared[mine]), to(np.diff(qh)), to(shared[mine])
    T, L = int(np.diff(qh).max()), int((np.diff(kh) - shared[mine]).max())
    t, j = torch.arange(T, device=dev), torch.arange(L, device=dev)
    see = j <= ((own_len - ql)[:, None] + t)[..., None]
    see &= j < own_len[:, None, None]
    m1, l1, o1 = _part(q, (qp[:-1, None] + t).clamp(max=last), t < ql[:, None], see,
                       _keys(st["k_pages"], st, ptr[:-1], own_len, L, skip),
                       _keys(st["v_pages"], st, ptr[:-1], own_len, L, skip), st["scale"])
    m = torch.maximum(m0, m1)
    w0, w1 = torch.exp(m0 - m), torch.exp(m1 - m)
    tot = w0 * l0 + w1 * l1
    return ((w0[..., None] * o0 + w1[..., None] * o1) / tot[..., None]).to(q.dtype), m + torch.log(tot)


# ---------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    op = case["op"]
    if op in ("norm", "grad"):
        size = {"bf16": 2, "f32": 4}[case["dtype"]]
        elems = case["n"] * (case["hq"] + case["hk"]) * case["d"]
        times, flops = (2, 4) if op == "norm" else (3, 12)
        return {"bytes": times * size * elems + 4 * case["n"] + 8 * times // 2 * case["d"],
                "flops": flops * elems + 3 * case["n"] * (case["hq"] + case["hk"]) * case["rot"]}
    past, new = _lens(case)
    n, hq, hkv, d = int(new.sum()), case["hq"], case["hkv"], case["d"]
    if op == "append":
        return {"bytes": 2 * 2 * n * (hq + 2 * hkv) * d, "flops": n * (hq + hkv) * (4 * d + 3 * case["rot"])}
    ptr, shared = _groups(case)
    mine = np.repeat(np.arange(case["groups"]), np.diff(ptr))
    pairs = int((new * (shared[mine] + past) + new * (new + 1) // 2).sum())
    seen = int(shared.sum() + (past + new).sum())  # tokens of the cache, a shared one once
    return {"bytes": 2 * 2 * n * hq * d + 4 * n * hq + 2 * 2 * seen * hkv * d, "flops": 4 * d * hq * pairs}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits


def _exact_norm_turn(x, w, pos, r, eps):
    x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + eps) * w
    rot, half = r["rot"], r["rot"] // 2
    speed = [BASE ** (-2.0 * p / rot) for p in range(half)]
    if r["scaling"] == "linear":
        speed = [f / r["factor"] for f in speed]
    elif r["scaling"] == "blend":
        keep = [min(max((ORIG * f / (2 * math.pi) - LOW) / (HIGH - LOW), 0.0), 1.0) for f in speed]
        speed = [f * a + f / r["factor"] * (1.0 - a) for f, a in zip(speed, keep)]
    angle = pos.double()[:, None] * torch.tensor(speed, dtype=torch.float64, device=pos.device)
    turn = torch.polar(torch.full_like(angle, r["mscale"]), angle)[:, None]
    if r["interleaved"]:
        z = torch.view_as_complex(x[..., :rot].unflatten(-1, (half, 2)).contiguous()) * turn
        return torch.cat([torch.view_as_real(z).flatten(-2), x[..., rot:]], -1)
    z = torch.complex(x[..., :half], x[..., half:rot]) * turn
    return torch.cat([z.real, z.imag, x[..., rot:]], -1)


def exact(case, seed):
    op = case["op"]
    st = prepare(case, seed)
    if op != "prefix":
        w = [st["q_weight"].double(), st["k_weight"].double()]
    if op == "norm":
        return tuple(_exact_norm_turn(x.double(), v, st["pos"], st["rope"], st["eps"]) for x, v in zip((st["q"], st["k"]), w))
    if op == "grad":
        leaves = [st["q"].double(), st["k"].double(), *w]
        leaves = [t.detach().clone().requires_grad_() for t in leaves]
        total = 0.0
        for x, v, dy in ((leaves[0], leaves[2], st["dq"]), (leaves[1], leaves[3], st["dk"])):
            total = total + (_exact_norm_turn(x, v, st["pos"], st["rope"], st["eps"]) * dy.double()).sum()
        return torch.autograd.grad(total, leaves)
    past, new = _lens(case)
    page = case["page"]
    idx, ptr = st["page_indices"], st["page_indptr"].tolist()
    if op == "append":
        at = [(r, t) for r in range(case["n_req"]) for t in range(int(past[r]), int(past[r] + new[r]))]
        lists = idx.tolist()
        rows = [lists[ptr[r] + t // page] * page + t % page for r, t in at]
        pos = torch.tensor([t for _, t in at], device=idx.device)
        q, k = (_exact_norm_turn(x.double(), v, pos, st["rope"], st["eps"]) for x, v in zip((st["q"], st["k"]), w))
        kc, vc = st["k_pages"].double(), st["v_pages"].double()
        kc.view(-1, *kc.shape[2:])[rows], vc.view(-1, *vc.shape[2:])[rows] = k, st["v"].double()
        return q, kc, vc
    q, grp, at = st["q"].double(), case["hq"] // case["hkv"], 0
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    kv = np.diff(st["kv_indptr_host"])
    for r in range(case["n_req"]):
        L, m = int(kv[r]), int(new[r])
        pages = idx[ptr[r]:ptr[r + 1]].long()
        k = st["k_pages"][pages].flatten(0, 1)[:L].double()
        v = st["v_pages"][pages].flatten(0, 1)[:L].double()
        hide = torch.arange(L, device=q.device)[None, :] > torch.arange(L - m, L, device=q.device)[:, None]
        for h in range(case["hq"]):
            s = (q[at:at + m, h] @ k[:, h // grp].T) * st["scale"]
            s[hide] = -math.inf
            lse[at:at + m, h] = torch.logsumexp(s, -1)
            out[at:at + m, h] = torch.softmax(s, -1) @ v[:, h // grp]
        at += m
    return out, lse

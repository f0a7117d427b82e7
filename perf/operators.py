"""Operators of serving over a paged KV cache, measured over their range of sizes.

Rotary positions (alone, and fused with the write of new tokens into the cache's pages), the
attention of a chunk of new tokens over the cache, and the cache's page bookkeeping (growing,
forking, compacting and freeing). Each case is a dict of plain values; `run` makes one pass, in
plain torch operations or, where `own` is true, through the library's calls.
"""

import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one layer's query and key heads of a 16384-token prompt, rotated with frequencies blended
        # for a context 32 times the trained one, positions spread over it
        dict(name="rope_long_bf16", op="rope", dtype="bf16", n=16384, heads=40, d=128, rot=128, interleaved=False,
             scaling="blend", factor=32.0, max_pos=1 << 20, transpose=False, pad=0),
        # the gradient of a part-of-head interleaved rotation, rows of a wider packed tensor
        dict(name="rope_grad_f32", op="rope", dtype="f32", n=1999, heads=12, d=64, rot=32, interleaved=True,
             scaling="linear", factor=4.0, max_pos=8192, transpose=True, pad=128),
        # one decode step: 64 sequences of one new token each enter the cache
        dict(name="append_decode_64", op="append", mix=1, n_req=64, hq=32, hkv=8, d=128, page=16, new="one", new_max=1,
             past_min=512, past_max=32767, rot=128, interleaved=False),
        # prompts of odd lengths enter a cache of 100-token pages
        dict(name="append_prompts", op="append", mix=2, n_req=6, hq=32, hkv=8, d=128, page=100, new="log", new_max=4096,
             past_min=0, past_max=5000, rot=64, interleaved=True),
        # a few draft tokens checked against short contexts: latency
        dict(name="chunk_small", op="chunk", mix=3, n_req=2, hq=16, hkv=2, d=64, page=16, new="log", new_max=4,
             past_min=100, past_max=700, window=0, sinks=0),
        # one decode step of 64 ragged requests, one token each
        dict(name="chunk_single_64", op="chunk", mix=1, n_req=64, hq=32, hkv=8, d=128, page=16, new="one", new_max=1,
             past_min=511, past_max=32767, window=0, sinks=0),
        # a mixed step with a causal window and always-visible first tokens, ragged chunks, odd head group and pages
        dict(name="chunk_window_mixed", op="chunk", mix=4, n_req=9, hq=28, hkv=4, d=128, page=100, new="log",
             new_max=2048, past_min=0, past_max=14336, window=256, sinks=16),
        # a whole prompt of 8192 tokens: bound by the matrix products
        dict(name="chunk_prompt_8192", op="chunk", mix=5, n_req=1, hq=32, hkv=8, d=128, page=64, new="max", new_max=8192,
             past_min=0, past_max=0, window=0, sinks=0),
        # one step's bookkeeping: finished sequences leave, the others grow by a few tokens
        dict(name="pages_turnover", op="turn", mix=6, n_pages=32768, n_req=256, page=16, past_min=64, past_max=2048,
             leave=32, grow_max=24),
        # a sampled answer forked four ways
        dict(name="pages_fork_4", op="fork", mix=7, n_pages=512, n_req=16, page=16, hkv=8, d=128, bufs=2, past_min=50,
             past_max=400, forks=4),
        # many branches over the caches of several layers
        dict(name="pages_fork_120", op="fork", mix=8, n_pages=3100, n_req=240, page=17, hkv=8, d=128, bufs=16,
             past_min=1, past_max=700, forks=120),
        # a pool left full of holes closed up
        dict(name="pages_compact", op="compact", mix=9, n_pages=8192, n_req=96, page=16, hkv=8, d=128, bufs=8,
             past_min=16, past_max=1400),
    ]


def _log_int(rng, lo, hi):
    return int(min(hi, max(lo, math.floor(math.exp(rng.uniform(math.log(max(lo, 0.7)), math.log(hi + 0.99)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "chunk", "chunk", "turn", "fork", "compact"])
    mix = rng.randrange(1 << 30)
    if op == "rope":
        d = rng.choice([32, 64, 80, 96, 128, 256])
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), n=_log_int(rng, 1, 16384), heads=rng.randint(1, 40), d=d,
                    rot=2 * rng.randint(1, d // 2) if rng.random() < 0.5 else d, interleaved=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "blend"]), factor=rng.choice([1.5, 4.0, 32.0]),
                    max_pos=_log_int(rng, 100, 1 << 20), transpose=rng.random() < 0.5, pad=8 * rng.randint(0, 40))
    if op == "append":
        d = rng.choice([64, 128])
        hkv = rng.randint(1, 8)
        return dict(op=op, mix=mix, n_req=_log_int(rng, 1, 64), hq=hkv * rng.randint(1, 8), hkv=hkv, d=d,
                    page=rng.choice([1, 5, 16, 64, 100, 256]), new=rng.choice(["one", "log"]),
                    new_max=_log_int(rng, 1, 400), past_min=0, past_max=_log_int(rng, 1, 6000),
                    rot=rng.choice([0, d // 2, d]), interleaved=rng.random() < 0.5)
    if op == "chunk":
        hkv = rng.choice([1, 2, 3, 4, 8])
        group = rng.choice([1, 2, 3, 4, 5, 7, 8, 12, 16])
        c = dict(op=op, mix=mix, n_req=_log_int(rng, 1, 64), hq=hkv * group, hkv=hkv, d=rng.choice([64, 128]),
                 page=rng.choice([1, 8, 16, 17, 48, 64, 100, 128]), new=rng.choice(["one", "log", "log"]),
                 new_max=_log_int(rng, 1, 4096), past_min=0, past_max=_log_int(rng, 1, 20000),
                 window=rng.choice([0, 0, 64, 300, 1024]), sinks=rng.choice([0, 0, 1, 16, 200]))
        while c["n_req"] * c["hq"] * c["new_max"] * (c["new_max"] + c["past_max"]) > 1.05e9:
            if c["n_req"] > 1:
                c["n_req"] = c["n_req"] // 2
            else:
                c["new_max"] = max(1, c["new_max"] // 2)
        return c
    if op == "turn":
        n_req = _log_int(rng, 2, 512)
        return dict(op=op, mix=mix, n_pages=n_req * 320, n_req=n_req, page=rng.choice([1, 8, 16, 100]), past_min=0,
                    past_max=_log_int(rng, 10, 250), leave=rng.randint(0, n_req // 2), grow_max=rng.randint(1, 60))
    hkv, d, page = rng.choice([1, 2, 8]), rng.choice([64, 128]), rng.choice([8, 16, 17, 33])
    n_req = _log_int(rng, 4, 160)
    c = dict(op=op, mix=mix, n_pages=n_req * 40 + 37, n_req=n_req, page=page, hkv=hkv, d=d, bufs=rng.randint(1, 6),
             past_min=rng.randint(0, 20), past_max=_log_int(rng, 20, 16 * page))
    if op == "fork":
        c["forks"] = rng.randint(1, n_req // 2)
    return c


# ---------------------------------------------------------------------------
# what a case's numbers stand for: lengths and page tables, from the case alone


def _lens(case):
    g = np.random.default_rng(case["mix"])
    n, lo, hi = case["n_req"], max(case["past_min"], 0), case["past_max"]
    past = np.floor(np.exp(g.uniform(math.log(lo + 1.0), math.log(hi + 1.0 + 1e-9), n))).astype(np.int64) - 1
    past = np.clip(past, lo, max(hi, lo))
    m = case.get("new_max", 1)
    kind = case.get("new", "one")
    if kind == "one":
        new = np.ones(n, np.int64)
    elif kind == "max":
        new = np.full(n, m, np.int64)
    else:
        new = np.clip(np.floor(np.exp(g.uniform(0.0, math.log(m + 0.99), n))).astype(np.int64), 1, m)
    return past, new


def _indptr(x):
    return np.concatenate([[0], np.cumsum(x)]).astype(np.int32)


def _pages_of(lens, page):
    return (lens + page - 1) // page


def _freqs(rot, base, scaling, factor, orig_len, low, high):
    """Radians a token for each pair, in 64 bits."""
    f = base ** (-np.arange(0, rot, 2, dtype=np.float64) / rot) if rot else np.zeros(0)
    if scaling == "linear":
        f = f / factor
    if scaling == "blend":
        g = np.clip((orig_len * f / (2 * math.pi) - low) / (high - low), 0.0, 1.0)
        f = g * f + (1 - g) * f / factor
    return f


BASE, ORIG, LOW, HIGH = 500000.0, 8192.0, 1.0, 32.0


def _rope_of(case):
    return dict(rot=case["rot"], interleaved=case["interleaved"], scaling=case.get("scaling", "none"),
                factor=case.get("factor", 1.0), mscale=1.25 if case.get("scaling") == "blend" else 1.0)


def prepare(case, seed):
    import random

    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    op = case["op"]
    randn = lambda *shape: torch.randn(shape, generator=g, device=dev)  # noqa: E731
    if op == "rope":
        n, h, d = case["n"], case["heads"], case["d"]
        wide = randn(n, h * d + case["pad"]).to(DT[case["dtype"]])
        return dict(case=case, x=wide[:, :h * d].unflatten(1, (h, d)),
                    pos=torch.randint(0, case["max_pos"], (n,), generator=g, device=dev, dtype=torch.int32),
                    rope=_rope_of(case), transpose=case["transpose"])
    past, new = _lens(case)
    page, n_req = case["page"], case["n_req"]
    st = dict(case=case, page=page)
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    if op in ("append", "chunk"):
        kv = past + new
        held = _pages_of(kv, page)
        n_pages = int(held.sum()) + 3
        order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        n = int(new.sum())
        st.update(page_indptr=to(_indptr(held)), page_indices=order[:max(int(held.sum()), 1)].contiguous(),
                  q_indptr=to(_indptr(new)), kv_indptr=to(_indptr(kv)), q_indptr_host=_indptr(new),
                  kv_indptr_host=_indptr(kv), k_pages=randn(n_pages, page, hkv, d).to(torch.bfloat16),
                  v_pages=randn(n_pages, page, hkv, d).to(torch.bfloat16))
        if op == "append":
            packed = randn(n, (hq + 2 * hkv) * d).to(torch.bfloat16)  # one projection's output
            q, k, v = packed.split([hq * d, hkv * d, hkv * d], dim=1)
            st.update(q=q.unflatten(1, (hq, d)), k=k.unflatten(1, (hkv, d)), v=v.unflatten(1, (hkv, d)),
                      rope=_rope_of(case) if case["rot"] else None)
        else:
            st.update(q=randn(n, hq, d).to(torch.bfloat16), window=case["window"], sinks=case["sinks"],
                      scale=1.0 / math.sqrt(d))
        return st
    # page bookkeeping: a pool of pages, lists with room for twice what a sequence holds, in a seeded order
    rng = random.Random(int(seed))
    kv = past
    if op == "fork":
        kv = np.concatenate([kv[: n_req - case["forks"]], np.zeros(case["forks"], np.int64)])
    held = _pages_of(kv, page)
    room = np.full(n_req, int(_pages_of(np.array([case["past_max"] + case.get("grow_max", 0)]), page)[0]) + 1, np.int64)
    ptr = _indptr(room)
    perm = torch.randperm(case["n_pages"], generator=g, device=dev).to(torch.int32)
    idx = torch.full((int(ptr[-1]),), -1, dtype=torch.int32, device=dev)
    at = np.concatenate([np.arange(ptr[r], ptr[r] + held[r]) for r in range(n_req)]) if held.sum() else np.zeros(0, np.int64)
    idx[to(at.astype(np.int64))] = perm[: at.size]
    ref = torch.zeros(case["n_pages"], dtype=torch.int32, device=dev)
    ref[perm[: at.size].long()] = 1
    st.update(page_indptr=to(ptr), page_indices=idx, ref=ref, kv_indptr=to(_indptr(kv)))
    if op == "turn":
        leave = sorted(rng.sample(range(n_req), case["leave"]))
        after = kv.copy()
        after[leave] = 0
        grown = after + np.array([0 if r in set(leave) else rng.randint(0, case["grow_max"]) for r in range(n_req)])
        st.update(leave=to(np.array(leave, np.int32)), after=to(_indptr(after)), grown=to(_indptr(grown)))
        return st
    shape = (case["n_pages"], page, case["hkv"], case["d"])
    st["bufs"] = [randn(*shape).to(torch.bfloat16) for _ in range(case["bufs"])]
    if op == "fork":
        n_parents = n_req - case["forks"]
        st.update(parent=to(np.array([rng.randrange(n_parents) for _ in range(case["forks"])], np.int32)),
                  child=to(np.arange(n_parents, n_req).astype(np.int32)))
    return st


def run(st):
    op = st["case"]["op"]
    if own:
        return {"rope": _own_rope, "append": _own_append, "chunk": _own_chunk, "turn": _own_turn, "fork": _own_fork,
                "compact": _own_compact}[op](st)
    return {"rope": _plain_rope, "append": _plain_append, "chunk": _plain_chunk, "turn": _plain_turn,
            "fork": _plain_fork, "compact": _plain_compact}[op](st)


# ---------------------------------------------------------------------------
# the library's calls


def _params(r):
    import split_kv_decode_bsr_gb300 as sta

    return sta.Rope(r["rot"], base=BASE, interleaved=r["interleaved"], scaling=r["scaling"], factor=r["factor"],
                    orig_len=ORIG, low_turns=LOW, high_turns=HIGH, mscale=r["mscale"])


def _own_rope(st):
    import split_kv_decode_bsr_gb300 as sta

    return sta.sta_rope(st["x"], st["pos"], _params(st["rope"]), transpose=st["transpose"])


def _own_append(st):
    import split_kv_decode_bsr_gb300 as sta

    q = sta.sta_rope_append_paged(st["q"], st["k"], st["v"], st["k_pages"], st["v_pages"], st["page_indptr"],
                                  st["page_indices"], st["q_indptr"], st["kv_indptr"],
                                  rope=_params(st["rope"]) if st["rope"] else None)
    return q, st["k_pages"], st["v_pages"]


def _own_chunk(st):
    import split_kv_decode_bsr_gb300 as sta

    pattern = sta.MaskSource.pattern(causal=True, win_lo=1 - st["window"], n_global_cols=st["sinks"]) if st["window"] else None
    return sta.sta_chunk_fwd_paged(st["q"], st["k_pages"], st["v_pages"], st["page_indptr"], st["page_indices"],
                                   st["q_indptr"], st["q_indptr_host"], st["kv_indptr"], st["kv_indptr_host"],
                                   scale=st["scale"], pattern=pattern)


def _own_turn(st):
    import split_kv_decode_bsr_gb300 as sta

    ref, idx = st["ref"].clone(), st["page_indices"].clone()
    sta.sta_pages_free(ref, st["page_indptr"], idx, st["kv_indptr"], st["leave"], st["page"])
    status = sta.sta_pages_grow(ref, st["page_indptr"], idx, st["after"], st["grown"], st["page"])
    return ref, idx, status


def _own_fork(st):
    import split_kv_decode_bsr_gb300 as sta

    ref, idx = st["ref"].clone(), st["page_indices"].clone()
    status = sta.sta_pages_fork(st["bufs"], ref, st["page_indptr"], idx, st["kv_indptr"], st["parent"], st["child"],
                                st["page"])
    return ref, idx, status, st["bufs"]


def _own_compact(st):
    import split_kv_decode_bsr_gb300 as sta

    ref, idx = st["ref"].clone(), st["page_indices"].clone()
    page_map, status = sta.sta_pages_compact(st["bufs"], ref, st["page_indptr"], idx, st["kv_indptr"], st["page"])
    return ref, idx, page_map, status, st["bufs"]


# ---------------------------------------------------------------------------
# plain forms


def _plain_rotate(x, pos, r, transpose=False):
    """x [n, h, d] in 32 bits; angles in 64, since far positions need them."""
    rot = r["rot"]
    f = torch.from_numpy(_freqs(rot, BASE, r["scaling"], r["factor"], ORIG, LOW, HIGH)).to(x.device)
    ang = pos.double()[:, None] * f[None, :]
    cos, sin = (torch.cos(ang) * r["mscale"]).float()[:, None], (torch.sin(ang) * r["mscale"]).float()[:, None]
    if transpose:
        sin = -sin
    y = x.clone()
    if r["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2:rot]
        y[..., : rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    return y


def _plain_rope(st):
    return _plain_rotate(st["x"].float(), st["pos"], st["rope"], st["transpose"]).to(st["x"].dtype)


def _token_places(st):
    """For every new token: its position in its sequence and the cache row it goes to."""
    qp, kp, page = st["q_indptr"].long(), st["kv_indptr"].long(), st["page"]
    t = torch.arange(st["q"].shape[0], device=qp.device)
    r = torch.searchsorted(qp, t, right=True) - 1
    pos = (kp[r + 1] - kp[r]) - (qp[r + 1] - qp[r]) + (t - qp[r])
    entry = st["page_indices"].long()[st["page_indptr"].long()[r] + pos // page]
    return pos, entry * page + pos % page


def _plain_append(st):
    pos, row = _token_places(st)
    q, k = st["q"].float(), st["k"].float()
    if st["rope"]:
        q, k = _plain_rotate(q, pos, st["rope"]), _plain_rotate(k, pos, st["rope"])
    st["k_pages"].flatten(0, 1)[row] = k.to(st["k_pages"].dtype)
    st["v_pages"].flatten(0, 1)[row] = st["v"]
    return q.to(st["q"].dtype), st["k_pages"], st["v_pages"]


def _visible(pos, kl, Lk, window, sinks, dev):
    """[R, Lq, Lk]: key j of the sequence is seen by the query at position pos."""
    j = torch.arange(Lk, device=dev)
    see = (j <= pos[..., None]) & (j < kl[:, None, None])
    if window:
        see &= (j > pos[..., None] - window) | (j < sinks)
    return see


def _plain_chunk(st):
    q, dev, page = st["q"], st["q"].device, st["page"]
    n, hq, d = q.shape
    hkv = st["k_pages"].shape[2]
    grp = hq // hkv
    qp, kp, pp = st["q_indptr"].long(), st["kv_indptr"].long(), st["page_indptr"].long()
    R = qp.numel() - 1
    ql, kl = qp[1:] - qp[:-1], kp[1:] - kp[:-1]
    Lq, Lk = int(np.diff(st["q_indptr_host"]).max()), int(np.diff(st["kv_indptr_host"]).max())
    i, j = torch.arange(Lq, device=dev), torch.arange(Lk, device=dev)
    rows = (qp[:-1, None] + i).clamp(max=n - 1)
    entry = (pp[:-1, None] + j // page).clamp(max=st["page_indices"].numel() - 1)
    slot = st["page_indices"].long()[entry] * page + j % page
    slot = torch.where(j < kl[:, None], slot, slot[:, :1])
    K = st["k_pages"].flatten(0, 1)[slot].float().permute(0, 2, 3, 1)  # [R, hkv, d, Lk]
    V = st["v_pages"].flatten(0, 1)[slot].float().permute(0, 2, 1, 3)  # [R, hkv, Lk, d]
    Q = q[rows].float().reshape(R, Lq, hkv, grp, d).permute(0, 2, 3, 1, 4).reshape(R, hkv, grp * Lq, d)
    see = _visible(kl[:, None] - ql[:, None] + i, kl, Lk, st["window"], st["sinks"], dev)[:, None, None]
    s = torch.matmul(Q, K).mul_(st["scale"]).reshape(R, hkv, grp, Lq, Lk)
    s.masked_fill_(~see, -math.inf)
    m = s.amax(-1, keepdim=True)
    s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    tot = s.sum(-1, keepdim=True)
    o = torch.matmul(s.reshape(R, hkv, grp * Lq, Lk), V).reshape(R, hkv, grp, Lq, d) / torch.where(tot > 0, tot, 1.0)
    lse = (m + torch.log(tot))[..., 0]
    live = i < ql[:, None]
    out = torch.empty_like(q)
    out[rows[live]] = o.permute(0, 3, 1, 2, 4).reshape(R, Lq, hq, d)[live].to(q.dtype)
    lse_out = torch.empty((n, hq), dtype=torch.float32, device=dev)
    lse_out[rows[live]] = lse.permute(0, 3, 1, 2).reshape(R, Lq, hq)[live]
    return out, lse_out


def _held(ptr, kv_indptr, page, n_entries):
    """[n_entries] list entry e's request, and whether that request holds it."""
    ptr, kp = ptr.long(), kv_indptr.long()
    e = torch.arange(n_entries, device=ptr.device)
    r = torch.searchsorted(ptr, e, right=True) - 1
    return r, (e - ptr[r]) < (kp[r + 1] - kp[r] + page - 1) // page


def _plain_turn(st):
    ref, idx, page = st["ref"].clone(), st["page_indices"].clone(), st["page"]
    ptr = st["page_indptr"].long()
    r, held = _held(ptr, st["kv_indptr"], page, idx.numel())
    gone = torch.zeros(ptr.numel() - 1, dtype=torch.bool, device=ptr.device)
    gone[st["leave"].long()] = True
    drop = held & gone[r]
    ref.index_add_(0, idx[drop].long(), torch.full_like(idx[drop], -1))
    idx[drop] = -1
    _, was = _held(ptr, st["after"], page, idx.numel())
    _, now = _held(ptr, st["grown"], page, idx.numel())
    want = torch.nonzero(now & ~was)[:, 0]
    free = torch.nonzero(ref == 0)[:, 0]
    n = min(want.numel(), free.numel())
    idx[want[:n]] = free[:n].int()
    idx[want[n:]] = -1
    ref[free[:n]] = 1
    status = torch.tensor([n, want.numel() - n], dtype=torch.int32, device=ref.device)
    return ref, idx, status


def _plain_fork(st):
    ref, idx, page = st["ref"].clone(), st["page_indices"].clone(), st["page"]
    ptr, kp, dev = st["page_indptr"].long(), st["kv_indptr"].long(), ref.device
    par, ch = st["parent"].long(), st["child"].long()
    ln = kp[par + 1] - kp[par]
    k = torch.arange(int((ptr[1:] - ptr[:-1]).max()), device=dev)
    whole = k < (ln // page)[:, None]
    src, dst = (ptr[par][:, None] + k)[whole], (ptr[ch][:, None] + k)[whole]
    shared = idx[src]
    idx[dst] = shared
    ref.index_add_(0, shared.long(), torch.ones_like(shared))
    part = torch.nonzero(ln % page)[:, 0]
    free = torch.nonzero(st["ref"] == 0)[:, 0]
    n = min(part.numel(), free.numel())
    last = (ln // page)[part]
    old = idx[ptr[par[part]] + last].long()
    new = torch.full_like(old, -1)
    new[:n] = free[:n]
    idx[ptr[ch[part]] + last] = new.int()
    ref[free[:n]] = 1
    bufs = [b.index_copy_(0, new[:n], b[old[:n]]) for b in st["bufs"]]
    status = torch.tensor([n, part.numel() - n], dtype=torch.int32, device=dev)
    return ref, idx, status, bufs


def _plain_compact(st):
    ref, idx, page = st["ref"].clone(), st["page_indices"].clone(), st["page"]
    n, dev = ref.numel(), ref.device
    live = ref > 0
    used = int(live.sum())
    p = torch.arange(n, device=dev)
    src, dst = p[live & (p >= used)], p[~live & (p < used)]
    page_map = torch.where(live, p, -1).int()
    page_map[src] = dst.int()
    _, held = _held(st["page_indptr"], st["kv_indptr"], page, idx.numel())
    idx[held] = page_map[idx[held].long()]
    ref[dst] = ref[src]
    ref[src] = 0
    bufs = [b.index_copy_(0, dst, b[src]) for b in st["bufs"]]
    status = torch.tensor([used, src.numel()], dtype=torch.int32, device=dev)
    return ref, idx, page_map, status, bufs


# ---------------------------------------------------------------------------
# what a pass cannot do without


def _pairs(case):
    past, new = _lens(case)
    total, seen = 0, 0
    for p, m in zip(past.tolist(), new.tolist()):
        pos = np.arange(p, p + m)
        if case["window"]:
            lo = np.maximum(pos + 1 - case["window"], 0)
            total += int((pos + 1 - lo + np.minimum(case["sinks"], lo)).sum())
            seen += min(p + m, int(p + m - lo[0] + min(case["sinks"], lo[0])))
        else:
            total += int((pos + 1).sum())
            seen += p + m
    return total, seen


def work(case):
    op = case["op"]
    if op == "rope":
        size = {"bf16": 2, "f32": 4}[case["dtype"]]
        return {"bytes": 2 * case["n"] * case["heads"] * case["d"] * size + 4 * case["n"],
                "flops": 3 * case["n"] * case["heads"] * case["rot"]}
    past, new = _lens(case)
    if op == "append":
        n, hq, hkv, d = int(new.sum()), case["hq"], case["hkv"], case["d"]
        return {"bytes": 2 * 2 * n * (hq + 2 * hkv) * d, "flops": 3 * n * (hq + hkv) * case["rot"]}
    if op == "chunk":
        n, hq, hkv, d = int(new.sum()), case["hq"], case["hkv"], case["d"]
        pairs, seen = _pairs(case)
        return {"bytes": 2 * 2 * n * hq * d + 4 * n * hq + 2 * 2 * seen * hkv * d, "flops": 4 * d * hq * pairs}
    tables = 8 * case["n_pages"] + 8 * case["n_req"] * int(_pages_of(np.array([case["past_max"]]), case["page"])[0] + 1)
    if op == "turn":
        return {"bytes": tables, "flops": case["n_pages"]}
    page_bytes = case["page"] * case["hkv"] * case["d"] * 2
    if op == "fork":
        moved = case["forks"]
    else:
        used = int(_pages_of(past, case["page"]).sum())
        moved = used * (case["n_pages"] - used) // case["n_pages"]  # live pages past the used ones, as many as holes
    return {"bytes": tables + 2 * moved * page_bytes * case["bufs"], "flops": case["n_pages"]}


# ---------------------------------------------------------------------------
# the definitions, in 64 bits


def _exact_rotation(x, pos, r, transpose):
    x = x.double()
    rot, half = r["rot"], r["rot"] // 2
    y = x.clone()
    for p in range(half):
        f = BASE ** (-2.0 * p / rot)
        if r["scaling"] == "linear":
            f /= r["factor"]
        elif r["scaling"] == "blend":
            w = min(max((ORIG * f / (2 * math.pi) - LOW) / (HIGH - LOW), 0.0), 1.0)
            f = f * w + f / r["factor"] * (1.0 - w)
        turn = torch.polar(torch.full_like(pos, r["mscale"], dtype=torch.float64), pos.double() * f)
        turn = (turn.conj() if transpose else turn)[:, None]
        i, k = (2 * p, 2 * p + 1) if r["interleaved"] else (p, p + half)
        z = torch.complex(x[..., i], x[..., k]) * turn
        y[..., i], y[..., k] = z.real, z.imag
    return y


def exact(case, seed):
    op = case["op"]
    st = prepare(case, seed)
    if op == "rope":
        return _exact_rotation(st["x"], st["pos"], st["rope"], st["transpose"])
    past, new = _lens(case)
    page = case["page"]
    if op == "append":
        idx, ptr = st["page_indices"].tolist(), st["page_indptr"].tolist()
        rows = [idx[ptr[r] + t // page] * page + t % page for r in range(case["n_req"])
                for t in range(int(past[r]), int(past[r] + new[r]))]
        pos = torch.tensor([t for r in range(case["n_req"]) for t in range(int(past[r]), int(past[r] + new[r]))],
                           device=st["q"].device)
        q, k = st["q"].double(), st["k"].double()
        if st["rope"]:
            q, k = _exact_rotation(q, pos, st["rope"], False), _exact_rotation(k, pos, st["rope"], False)
        kc, vc = st["k_pages"].double(), st["v_pages"].double()
        kc.view(-1, *kc.shape[2:])[rows], vc.view(-1, *vc.shape[2:])[rows] = k, st["v"].double()
        return q, kc, vc
    if op == "chunk":
        q, grp = st["q"].double(), case["hq"] // case["hkv"]
        idx, ptr, at = st["page_indices"].long(), st["page_indptr"].tolist(), 0
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
        for r in range(case["n_req"]):
            L, m = int(past[r] + new[r]), int(new[r])
            pages = idx[ptr[r]:ptr[r + 1]]
            k = st["k_pages"][pages].flatten(0, 1)[:L].double()
            v = st["v_pages"][pages].flatten(0, 1)[:L].double()
            i = torch.arange(L - m, L, device=q.device)[:, None]
            j = torch.arange(L, device=q.device)[None, :]
            hide = j > i
            if case["window"]:
                hide = hide | ((i - j >= case["window"]) & (j >= case["sinks"]))
            for h in range(case["hq"]):
                s = (q[at:at + m, h] @ k[:, h // grp].T) * st["scale"]
                s[hide] = -math.inf
                lse[at:at + m, h] = torch.logsumexp(s, -1)
                out[at:at + m, h] = torch.softmax(s, -1) @ v[:, h // grp]
            at += m
        return out, lse
    # page bookkeeping, entry by entry
    dev, ptr, kv = st["ref"].device, st["page_indptr"].tolist(), np.diff(st["kv_indptr"].tolist()).tolist()
    ref, idx = st["ref"].tolist(), st["page_indices"].tolist()
    need = lambda tokens: -(-tokens // page)  # noqa: E731
    ints = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)  # noqa: E731
    if op == "turn":
        for r in st["leave"].tolist():
            for e in range(ptr[r], ptr[r] + need(kv[r])):
                ref[idx[e]] -= 1
                idx[e] = -1
        free, missing, got = (p for p, c in enumerate(list(ref)) if c == 0), 0, 0
        was, now = np.diff(st["after"].tolist()).tolist(), np.diff(st["grown"].tolist()).tolist()
        for r in range(case["n_req"]):
            for e in range(ptr[r] + need(was[r]), ptr[r] + need(now[r])):
                idx[e] = next(free, -1)
                if idx[e] >= 0:
                    ref[idx[e]], got = 1, got + 1
                else:
                    missing += 1
        return ints(ref), ints(idx), ints([got, missing])
    bufs = [b.double() for b in st["bufs"]]
    if op == "fork":
        free, missing, got = (p for p, c in enumerate(list(ref)) if c == 0), 0, 0
        for a, c in zip(st["parent"].tolist(), st["child"].tolist()):
            for e in range(need(kv[a])):
                old = idx[ptr[a] + e]
                if (e + 1) * page <= kv[a]:
                    idx[ptr[c] + e] = old
                    ref[old] += 1
                    continue
                new = idx[ptr[c] + e] = next(free, -1)
                if new < 0:
                    missing += 1
                    continue
                ref[new], got = 1, got + 1
                for b in bufs:
                    b[new] = b[old]
        return ints(ref), ints(idx), ints([got, missing]), bufs
    used = sum(c > 0 for c in ref)
    holes = [p for p in range(used) if ref[p] == 0]
    late = [p for p in range(used, len(ref)) if ref[p] > 0]
    goes = [p if c > 0 else -1 for p, c in enumerate(ref)]
    for a, c in zip(late, holes):
        goes[a], ref[c], ref[a] = c, ref[a], 0
    for r in range(case["n_req"]):
        for e in range(ptr[r], ptr[r] + need(kv[r])):
            idx[e] = goes[idx[e]]
    for b in bufs:
        b[holes] = b[late]
    return ints(ref), ints(idx), ints(goes), ints([used, len(late)]), bufs

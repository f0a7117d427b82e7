"""Plain 64-bit forms of the serving operators over a paged cache, and their test inputs."""

import math

import numpy as np

BF16_HALF_STEP = 2.0 ** -8  # finfo(bfloat16).eps / 2, relative
F32_HALF_STEP = 2.0 ** -24


# ---- rotary positions


def freqs(rot, base=10000.0, scaling="none", factor=1.0, orig_len=0.0, low_turns=1.0, high_turns=32.0):
    f = base ** (-2.0 * np.arange(rot // 2) / rot)
    if scaling == "linear":
        f = f / factor
    elif scaling == "blend":
        g = np.clip((orig_len * f / (2 * math.pi) - low_turns) / (high_turns - low_turns), 0.0, 1.0)
        f = g * f + (1 - g) * f / factor
    return f


def rope_ref(x, pos, f, interleaved, mscale=1.0, transpose=False):
    """x [n, H, d] float64, pos [n]: the result, and the bound on fp32 arithmetic before the last rounding.

    The bound: the angle is off by at most pi 2^-25 (its fp32 half turns), cosine and sine by 2 units
    in the last place (2^-23), the magnitude, the products and the sum by half a unit each: below
    4e-7 (|a| + |b|) mscale."""
    rot = 2 * len(f)
    ang = pos.astype(np.float64)[:, None] * f[None, :]
    c, s = np.cos(ang)[:, None] * mscale, np.sin(ang)[:, None] * mscale * (-1.0 if transpose else 1.0)
    i = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    j = i + 1 if interleaved else i + rot // 2
    y, err = x.copy(), np.zeros_like(x)
    a, b = x[..., i], x[..., j]
    y[..., i], y[..., j] = a * c - b * s, a * s + b * c
    err[..., i] = err[..., j] = 4e-7 * mscale * (np.abs(a) + np.abs(b))
    return y, err


# ---- attention of a chunk over a paged cache


def visible(pos, length, causal, win_lo, win_hi, n_global):
    """[len(pos), length]: token at position i sees key j."""
    i, j = pos[:, None].astype(np.int64), np.arange(length, dtype=np.int64)[None, :]
    see = ((j - i >= win_lo) & (j - i <= win_hi)) | (j < n_global)
    return see & (j <= i) if causal else see


def chunk_ref(q, k, v, pos, scale, causal=True, win_lo=-(1 << 40), win_hi=1 << 40, n_global=0):
    """One request: q [n, Hq, d], k, v [L, Hkv, d] float64 -> o, lse and the bounds on their errors.

    P is rounded to bf16 before the product with V: off by half a step of each term, hence
    2^-8 sum p |v|; O is rounded once, 2^-8 |o|. Scores are fp32 sums of d exact products, off by
    (d + 2) 2^-24 sum |q k| scale, which shifts exponents (relative error of P and of its sum) and
    the LSE directly; 1e-5 covers the exponential, the sum and the logarithm."""
    n, Hq, d = q.shape
    L, Hkv, _ = k.shape
    see = visible(pos, L, causal, win_lo, win_hi, n_global)
    o, lse = np.zeros_like(q), np.full((n, Hq), -np.inf)
    o_tol, lse_tol = np.zeros_like(q), np.zeros((n, Hq))
    for h in range(Hq):
        kk, vv = k[:, h // (Hq // Hkv)], v[:, h // (Hq // Hkv)]
        s = np.where(see, q[:, h] @ kk.T * scale, -np.inf)
        for t in range(n):
            if not see[t].any():
                continue
            m = s[t].max()
            p = np.exp(s[t] - m)
            tot = p.sum()
            p /= tot
            o[t, h] = p @ vv
            lse[t, h] = m + math.log(tot)
            ds = (d + 2) * 2.0 ** -24 * scale * float(np.max(np.abs(q[t, h]) @ np.abs(kk[see[t]]).T)) + 1e-5
            spread = p @ np.abs(vv)
            o_tol[t, h] = (BF16_HALF_STEP + 2 * ds) * spread + BF16_HALF_STEP * np.abs(o[t, h])
            lse_tol[t, h] = ds + 2.0 ** -23 * abs(lse[t, h])
    return o, lse, o_tol, lse_tol


class PagedCase:
    """Requests of new[r] new tokens at the end of kv[r]-token sequences, in a cache of pages in a
    seeded order. What pages hold behind their sequences, and spare pages, is NaN."""

    def __init__(self, seed, new, kv, Hq, Hkv, d, page_size, spare_entries=0, pad_rows=0, value=1.0):
        import torch

        g = np.random.default_rng(seed)
        self.new, self.kv, self.Hq, self.Hkv, self.d, self.P = np.array(new), np.array(kv), Hq, Hkv, d, page_size
        self.q_indptr = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.kv_indptr = np.concatenate([[0], np.cumsum(kv)]).astype(np.int32)
        held = -(-self.kv // page_size)
        self.page_indptr = np.concatenate([[0], np.cumsum(held + spare_entries)]).astype(np.int32)
        self.n_pages = int(held.sum()) + 2
        perm = g.permutation(self.n_pages).astype(np.int32)
        self.page_indices = np.full(max(int(self.page_indptr[-1]), 1), -1, np.int32)
        at = 0
        for r, h in enumerate(held):
            self.page_indices[self.page_indptr[r]:self.page_indptr[r] + h] = perm[at:at + h]
            at += h
        bf = lambda a: torch.from_numpy(a.astype(np.float32) * value).to(torch.bfloat16)  # noqa: E731
        N = int(self.q_indptr[-1]) + pad_rows
        self.q = bf(g.standard_normal((N, Hq, d)))
        self.k_seq = [bf(g.standard_normal((int(x), Hkv, d))) for x in kv]
        self.v_seq = [bf(g.standard_normal((int(x), Hkv, d))) for x in kv]
        self.k_pages = torch.full((self.n_pages, page_size, Hkv, d), float("nan"), dtype=torch.bfloat16)
        self.v_pages = self.k_pages.clone()
        for r in range(len(kv)):
            if kv[r]:
                rows = torch.from_numpy(self.rows(r, np.arange(kv[r])))
                self.k_pages.view(-1, Hkv, d)[rows] = self.k_seq[r]
                self.v_pages.view(-1, Hkv, d)[rows] = self.v_seq[r]

    def rows(self, r, t):
        """Cache rows of tokens t of request r."""
        return self.page_indices[self.page_indptr[r] + t // self.P].astype(np.int64) * self.P + t % self.P

    def ref(self, scale, **pattern):
        N = self.q.shape[0]
        o, lse = np.zeros((N, self.Hq, self.d)), np.zeros((N, self.Hq))
        o_tol, lse_tol = np.zeros_like(o), np.zeros_like(lse)
        for r in range(len(self.new)):
            a, b = self.q_indptr[r], self.q_indptr[r + 1]
            pos = self.kv[r] - self.new[r] + np.arange(self.new[r])
            o[a:b], lse[a:b], o_tol[a:b], lse_tol[a:b] = chunk_ref(
                self.q[a:b].double().numpy(), self.k_seq[r].double().numpy(), self.v_seq[r].double().numpy(), pos, scale,
                **pattern)
        return o, lse, o_tol, lse_tol

    def dev(self, dev):
        import torch

        to = lambda a: torch.from_numpy(a).to(dev)  # noqa: E731
        return dict(q=self.q.to(dev), k_pages=self.k_pages.to(dev), v_pages=self.v_pages.to(dev),
                    page_indptr_dev=to(self.page_indptr), page_indices_dev=to(self.page_indices),
                    q_indptr_dev=to(self.q_indptr), q_indptr_host=self.q_indptr, kv_indptr_dev=to(self.kv_indptr),
                    kv_indptr_host=self.kv_indptr)


def check_chunk(o, lse, ref, n, what=""):
    """The first n rows against the reference within its bounds."""
    o_ref, lse_ref, o_tol, lse_tol = (x[:n] for x in ref)
    o, lse = o[:n].double().cpu().numpy(), lse[:n].double().cpu().numpy()
    dead = np.isneginf(lse_ref)
    assert np.array_equal(np.isneginf(lse), dead), f"{what}: rows without a key"
    assert (o[dead] == 0).all(), f"{what}: rows without a key must be 0"
    assert np.isfinite(o).all(), f"{what}: O not finite"
    off = np.abs(o - o_ref) - o_tol
    assert (off <= 1e-30).all(), f"{what}: O off by {np.abs(o - o_ref).max():.3e}, {off.max():.3e} past its bound"
    off = np.abs(lse[~dead] - lse_ref[~dead]) - lse_tol[~dead]
    assert off.size == 0 or off.max() <= 0, f"{what}: LSE {off.max():.3e} past its bound"


# ---- page bookkeeping, entry by entry


class Pool:
    """ref, lists and lengths as Python lists; the operators as loops."""

    def __init__(self, seed, lens, page_size, room, n_pages):
        g = np.random.default_rng(seed)
        self.P, self.n_pages, self.kv = page_size, n_pages, list(lens)
        self.ptr = [room * r for r in range(len(lens) + 1)]
        self.idx, self.ref = [-1] * (room * len(lens)), [0] * n_pages
        free = g.permutation(n_pages).tolist()
        for r in range(len(lens)):
            for e in range(self.need(lens[r])):
                p = free.pop()
                self.idx[self.ptr[r] + e], self.ref[p] = p, 1

    def need(self, tokens):
        return -(-tokens // self.P)

    def room(self, r):
        return self.ptr[r + 1] - self.ptr[r]

    def grow(self, new_lens):
        free = iter([p for p in range(self.n_pages) if self.ref[p] == 0])
        got = missing = 0
        for r, (a, b) in enumerate(zip(self.kv, new_lens)):
            if self.need(b) > self.room(r):
                continue
            for e in range(self.need(a), self.need(b)):
                p = next(free, -1)
                self.idx[self.ptr[r] + e] = p
                if p >= 0:
                    self.ref[p] = 1
                    got += 1
                else:
                    missing += 1
        return [got, missing]

    def fork(self, bufs, parent, child):
        free = iter([p for p in range(self.n_pages) if self.ref[p] == 0])
        got = missing = 0
        for i, (a, c) in enumerate(zip(parent, child)):
            n = self.need(self.kv[a])
            if c in child[:i] or self.kv[c] > 0 or n > self.room(c):
                continue
            for e in range(n):
                old = self.idx[self.ptr[a] + e]
                if (e + 1) * self.P <= self.kv[a]:
                    self.idx[self.ptr[c] + e] = old
                    self.ref[old] += 1
                    continue
                p = self.idx[self.ptr[c] + e] = next(free, -1)
                if p < 0:
                    missing += 1
                    continue
                self.ref[p] = 1
                got += 1
                for b in bufs:
                    b[p] = b[old]
        return [got, missing]

    def free(self, reqs):
        for r in dict.fromkeys(reqs):
            for e in range(self.need(self.kv[r])):
                p = self.idx[self.ptr[r] + e]
                if p >= 0:
                    self.ref[p] -= 1
                self.idx[self.ptr[r] + e] = -1

    def compact(self, bufs):
        used = sum(c > 0 for c in self.ref)
        holes = [p for p in range(used) if self.ref[p] == 0]
        late = [p for p in range(used, self.n_pages) if self.ref[p] > 0]
        goes = [p if c > 0 else -1 for p, c in enumerate(self.ref)]
        for a, c in zip(late, holes):
            goes[a], self.ref[c], self.ref[a] = c, self.ref[a], 0
            for b in bufs:
                b[c] = b[a]
        for r in range(len(self.kv)):
            for e in range(self.need(self.kv[r])):
                if self.idx[self.ptr[r] + e] >= 0:
                    self.idx[self.ptr[r] + e] = goes[self.idx[self.ptr[r] + e]]
        return goes, [used, len(late)]

"""Paged K/V cases and their plain 64-bit computation on the CPU: what the GPU
tests of host_transfer_amd.kv compare with.

Everything here is written from the formulas of include/ibp_kv.h, a token at a
time where that is the plainest, on float64 copies of the 16-bit inputs.
"""
import math

import torch

U32 = 2.0 ** -24  # half a step of fp32, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


class Case:
    """A pool of pages, a ragged batch and its queries, on the CPU."""

    def __init__(self, lens, *, dtype=torch.bfloat16, h=2, group=2, d=64, page=16, seed=0, extra=2,
                 fill=None, tail_rows=0, head_major=False, fused=True):
        """lens: (new tokens, all tokens) of each sequence.  fill: value of every key and value
        that no sequence holds.  tail_rows: rows behind the last sequence."""
        g = torch.Generator().manual_seed(seed)
        self.lens, self.dtype, self.h, self.group, self.d, self.page = lens, dtype, h, group, d, page
        need = [-(-kv // page) for _, kv in lens]
        self.n_pages = sum(need) + extra
        order = torch.randperm(self.n_pages, generator=g).int()
        self.table = torch.full((len(lens), max(need + [1]) + 1), -1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        shape = (self.n_pages, page, h, d)
        scale = torch.exp(torch.empty(h, d).uniform_(math.log(0.2), math.log(2.0), generator=g))
        self.k = (torch.randn(shape, generator=g) * scale).to(dtype)
        self.v = torch.randn(shape, generator=g).to(dtype)
        if fill is not None:
            used = torch.zeros(self.n_pages, page, dtype=torch.bool)
            for s, (_, kv) in enumerate(lens):
                for j in range(kv):
                    used[int(self.table[s, j // page]), j % page] = True
            self.k[~used] = fill
            self.v[~used] = fill
        self.q_start = torch.tensor([0] + [q for q, _ in lens], dtype=torch.int32).cumsum(0).int()
        self.kv_len = torch.tensor([kv for _, kv in lens], dtype=torch.int32)
        self.n = int(self.q_start[-1]) + tail_rows
        wide = torch.randn((self.n, h * group + (2 if fused else 0), d), generator=g).to(dtype)
        self.wide_q = wide
        self.q = wide[:, :h * group]
        self.head_major = head_major

    @property
    def max_q(self):
        return max([q for q, _ in self.lens] + [0])

    @property
    def max_kv(self):
        return max([kv for _, kv in self.lens] + [0])

    def pools(self):
        """GPU pools; head_major: (page, head, token, channel) memory seen as (page, token, ...)."""
        out = []
        for x in (self.k, self.v):
            x = x.cuda()
            if self.head_major:
                x = x.transpose(1, 2).contiguous().transpose(1, 2)
            out.append(x)
        return out

    def rows(self):
        """(row, sequence, position) of every row that a sequence holds."""
        for s, (q, kv) in enumerate(self.lens):
            for i in range(q):
                yield int(self.q_start[s]) + i, s, kv - q + i

    def keys(self, s, upto=None):
        """(positions, pool rows) of sequence s that are there."""
        kv = self.lens[s][1] if upto is None else min(upto, self.lens[s][1])
        pos = torch.arange(kv)
        ids = self.table[s].long()[pos // self.page] if kv else pos
        there = (ids >= 0) & (ids < self.n_pages)
        return pos[there], (ids * self.page + pos % self.page)[there]


def attention(c, scale, *, causal=True, window=0, sel=None):
    """(out, lse, tolerance of out, tolerance of lse), float64, and which rows sequences hold.  sel: (n, h, n_select) pages of each row and key head.

    Tolerances, u = half a step of the dtype: a weight exp(s - max) carries the error of s (a dot
    product of d terms in fp32, times the scale, and the rounded exponent: (d + 8) U32 times the sum
    of the magnitudes, twice for numerator and denominator) and its rounding to the dtype (u,
    and in fp16 at least half of the smallest subnormal); the sums over n keys carry n U32; the
    output is rounded once."""
    hq = c.h * c.group
    out = torch.full((c.n, hq, c.d), math.nan, dtype=torch.float64)
    lse = torch.full((c.n, hq), math.nan, dtype=torch.float64)
    tol, tol_lse = out.clone(), lse.clone()
    held = torch.zeros(c.n, dtype=torch.bool)
    u, tiny = half_step(c.dtype), torch.finfo(c.dtype).smallest_normal * torch.finfo(c.dtype).eps / 2
    k64, v64 = c.k.double().view(-1, c.h, c.d), c.v.double().view(-1, c.h, c.d)
    for r, s, pos in c.rows():
        held[r] = True
        p_all, rows_all = c.keys(s)
        for h in range(c.h):
            see = torch.ones_like(p_all, dtype=torch.bool)
            if causal:
                see = p_all <= pos
                if window:
                    see &= p_all > pos - window
            if sel is not None:
                pages = sel[r, h][sel[r, h] >= 0]
                see &= torch.isin(p_all // c.page, pages.long())
            rows = rows_all[see]
            kk, vv = k64[rows, h], v64[rows, h]
            for e in range(c.group):
                x = c.q[r, h * c.group + e].double()
                a = h * c.group + e
                n = len(rows)
                if n == 0:
                    out[r, a], lse[r, a], tol[r, a], tol_lse[r, a] = 0.0, -math.inf, 0.0, 0.0
                    continue
                sc = (kk @ x) * scale
                mag = (kk.abs() @ x.abs()) * abs(scale)
                delta = float(mag.nan_to_num(0, 0, 0).max()) * (c.d + 8) * U32 + 8 * U32
                lse[r, a] = torch.logsumexp(sc, 0)
                w = torch.exp(sc - lse[r, a])
                out[r, a] = w @ vv
                av = w @ vv.abs()
                most = torch.exp(sc - sc.max()).sum()
                tol[r, a] = (u * out[r, a].abs() + (u + 2 * delta + (n + 8) * U32) * av +
                             (tiny * vv.abs().sum(0) / most) + tiny)
                tol_lse[r, a] = delta + (n + 8) * U32 + 4 * U32 * lse[r, a].abs()
    return out, lse, tol, tol_lse, held


def check_attention(c, got_out, got_lse, ref, what=""):
    out, lse, tol, tol_lse, held = ref
    g, gl = got_out.cpu().double()[held], got_lse.cpu().double()[held]
    w, wl, t, tl = out[held], lse[held], tol[held], tol_lse[held]
    odd = ~torch.isfinite(w)
    assert (torch.isnan(g) == torch.isnan(w)).all(), f"{what}: NaN in other places"
    assert (g[odd & ~torch.isnan(w)] == w[odd & ~torch.isnan(w)]).all(), f"{what}: infinities differ"
    err = ((g - w).abs() / t.clamp(min=1e-300))[~odd]
    assert err.numel() == 0 or (g - w).abs()[~odd].le(t[~odd]).all(), \
        f"{what}: out off by {float(err.max()):.2f} tolerances"
    assert (torch.isnan(gl) == torch.isnan(wl)).all(), f"{what}: lse is NaN in other places"
    none = wl == -math.inf
    assert (gl[none] == -math.inf).all() and (g[none] == 0).all(), f"{what}: empty rows"
    fin = torch.isfinite(wl)
    errl = (gl - wl).abs()[fin]
    assert errl.numel() == 0 or errl.le(tl[fin]).all(), \
        f"{what}: lse off by {float((errl / tl[fin]).max()):.2f} tolerances"


def page_bounds(c):
    """{page id: (low, high)} of every page with a new token, in the dtype (no rounding)."""
    out = {}
    for s, (q, kv) in enumerate(c.lens):
        for p in range(max(kv - q, 0) // c.page, -(-kv // c.page) if q else 0):
            i = int(c.table[s, p])
            if not 0 <= i < c.n_pages:
                continue
            x = c.k[i, :min(c.page, kv - p * c.page)]
            out[i] = (x.amin(0), x.amax(0))
    return out


def all_bounds(c):
    """(n_pages, h, 2, d) bounds of all pages, of their tokens below kv_len."""
    b = torch.zeros(c.n_pages, c.h, 2, c.d, dtype=c.dtype)
    for s, (_, kv) in enumerate(c.lens):
        for p in range(-(-kv // c.page)):
            i = int(c.table[s, p])
            if 0 <= i < c.n_pages:
                x = c.k[i, :min(c.page, kv - p * c.page)]
                b[i, :, 0], b[i, :, 1] = x.amin(0), x.amax(0)
    return b


def select(c, bounds, n_first, n_last, n_select):
    """sel (n, h, n_select) by sorting (-score, page)."""
    sel = torch.full((c.n, c.h, n_select), -7, dtype=torch.int32)
    for r, s, pos in c.rows():
        sel[r] = -1
        if pos < 0:
            continue
        last = pos // c.page
        forced = [p for p in range(last + 1) if p < n_first or p > last - n_last]
        for h in range(c.h):
            if last + 1 <= n_select:
                pick = list(range(last + 1))
            else:
                cand = []
                for p in range(n_first, last + 1 - n_last):
                    i = int(c.table[s, p])
                    score = -math.inf
                    if 0 <= i < bounds.shape[0]:
                        x = c.q[r, h * c.group:(h + 1) * c.group].double()
                        lo, hi = bounds[i, h].double()
                        v = torch.maximum(x * lo, x * hi).sum(-1).amax()
                        score = float(v)
                    # NaN above everything, then by value, then the lower page
                    cand.append((0 if math.isnan(score) else 1,
                                 0.0 if math.isnan(score) else -score, p))
                cand.sort()
                pick = sorted(forced + [p for _, _, p in cand[:n_select - len(forced)]])
            sel[r, h, :len(pick)] = torch.tensor(pick, dtype=torch.int32)
    return sel


def norm_rotate(x, pos, rope, inter, w, eps):
    """x (n, heads, d) float64 -> the normalised and rotated heads, float64."""
    y = x.clone()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    if rope is None:
        return y
    half = rope.shape[1] // 2
    z = y.clone()
    for t in range(x.shape[0]):
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
            co, si = float(rope[pos[t], i]), float(rope[pos[t], half + i])
            z[t, :, a] = y[t, :, a] * co - y[t, :, b] * si
            z[t, :, b] = y[t, :, b] * co + y[t, :, a] * si
    return z


def rope_table(n_pos, r):
    inv = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)
    a = torch.arange(n_pos, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()

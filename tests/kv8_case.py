"""8-bit paged K/V cases and their plain 64-bit computation on the CPU: what the GPU tests of
host_transfer_amd.kv8 compare with.

Written from the formulas of include/ibp_kv8.h on float64 copies of the 16-bit inputs; attention over
a cache is kv_case.attention over the values that the codes stand for."""
import math

import torch

from tests import kv_case as K

E4M3 = torch.float8_e4m3fn


def grid(x):
    """The e4m3 number next to each x (float64, |x| <= 464), ties to the even one."""
    step = grid_step(x)
    return torch.round(x / step) * step


def grid_step(x):
    """Distance of the e4m3 numbers around x."""
    return torch.exp2(torch.frexp(x.abs())[1].clamp(min=-5).double() - 4)


def codes_of(x):
    """The codes of e4m3 numbers (float64)."""
    return x.float().to(E4M3)


def exponent(most):
    """The least e in [1, 254] with most <= 448 * 2^(e - 127), by trying them."""
    for e in range(1, 255):
        if most <= 448 * 2.0 ** (e - 127):
            return e
    return 254


class Case8(K.Case):
    """A K.Case whose pools are held in 8 bits: k8, v8 (codes), ke, ve (exponents); its k and v are the
    values that those stand for, in float64."""

    def __init__(self, lens, *, block=None, strange=False, **kw):
        super().__init__(lens, **kw)
        self.block = block or self.page
        self.ke, self.k8 = self._quantise(self.k, kw.get("seed", 0))
        self.ve, self.v8 = self._quantise(self.v, kw.get("seed", 0) + 1)
        if strange:  # each block's exponent some powers off, so that blocks differ widely
            g = torch.Generator().manual_seed(7)
            self.ve += torch.randint(-3, 4, self.ve.shape, generator=g).to(torch.uint8)
        self.renew()

    def renew(self):
        """k and v from the codes and exponents."""
        self.k, self.v = self.values(self.k8, self.ke), self.values(self.v8, self.ve)

    def _quantise(self, x, seed):
        nb = self.page // self.block
        x = x.double().unflatten(1, (nb, self.block))
        most = torch.where(torch.isfinite(x), x.abs(), 0.0).amax((2, 4))
        e = torch.tensor([exponent(float(m)) for m in most.flatten()], dtype=torch.uint8).view(most.shape)
        s = torch.exp2(e.double() - 127)[:, :, None, :, None]
        return e, torch.where(torch.isfinite(x), grid(torch.where(torch.isfinite(x), x, 0.0) / s),
                              math.nan).flatten(1, 2).float().to(E4M3)

    def values(self, codes, exps):
        s = torch.exp2(exps.double().clamp(1, 254) - 127).repeat_interleave(self.block, 1)[..., None]
        return codes.double() * s

    def pools8(self, head_major=None):
        """GPU codes and exponents: k, v, k_exp, v_exp."""
        out = []
        for x in (self.k8, self.v8):
            x = x.view(torch.uint8).cuda()
            if self.head_major if head_major is None else head_major:
                x = x.transpose(1, 2).contiguous().transpose(1, 2)
            out.append(x.view(E4M3))
        return out + [self.ke.cuda(), self.ve.cuda()]


def append(c, new_k, new_v, placed):
    """The cache after the new rows new_k, new_v (n, h, d; float64, normed and rotated): codes and
    exponents of k and v as {name: (value grid, exponents, written)}: `written` marks the new tokens,
    whose codes follow from values in 64 bits.  placed: which rows are placed."""
    out = {}
    for name, codes, exps, x in (("k", c.k8, c.ke, new_k), ("v", c.v8, c.ve, new_v)):
        val, e_out = codes.double().clone(), exps.clone()
        exact = torch.full(val.shape, math.nan, dtype=torch.float64)  # of the new tokens: value / scale
        written = torch.zeros(val.shape[:2], dtype=torch.bool)
        for s, (q, kv) in enumerate(c.lens):
            r0 = int(c.q_start[s])
            first = kv - q
            begin, end = max(first, 0), min(first + min(q, c.max_rows), min(kv, c.most_kv))
            for base in range(begin // c.block * c.block, max(end, 0), c.block):
                page = int(c.table[s, base // c.page])
                if begin >= end or not 0 <= page < c.n_pages:
                    continue
                a, b, at = max(base, begin), min(base + c.block, end), base % c.page
                rows = [r0 + j - first for j in range(a, b)]
                ok = [r for r in rows if placed[r]]
                for h in range(c.h):
                    y = x[ok, h]
                    most = float(torch.where(torch.isfinite(y), y.abs(), 0.0).max()) if ok else 0.0
                    e = exponent(most)
                    was = min(max(int(exps[page, at // c.block, h]), 1), 254)
                    if a > base:
                        e = max(e, was)
                        old = val[page, at:at + a - base, h]
                        val[page, at:at + a - base, h] = grid(old * 2.0 ** (was - e))
                    e_out[page, at // c.block, h] = e
                    for j, r in zip(range(a, b), rows):
                        if placed[r]:
                            z = x[r, h] * 2.0 ** (127 - e)
                            exact[page, at + j - base, h] = torch.where(torch.isfinite(z), z, math.nan)
                            val[page, at + j - base, h] = grid(exact[page, at + j - base, h])
                for j, r in zip(range(a, b), rows):
                    written[page, at + j - base] |= bool(placed[r])
        out[name] = (val, e_out, written, exact)
    return out

"""Plain 64-bit implementations of a generation step's operators -- the norms of queries
and keys with the rotation, 4-bit rows, pages handed out and taken back -- with
bounds on what rounding may do (as in grouped.py: half a step of bf16 is 2^-8 of the
value, of fp32 2^-24, of e2m1 2^-2, and below 1 a quarter of the block's power of two).
"""
from __future__ import annotations

import math

import torch

from grouped import D, F64, U16, U32, Cache, rotate

U4 = 2.0 ** -2
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ norms

def norm(x, w, eps, pos=None, base=10000.0):
    """RMS norm of each head of rows x [n, heads, 64] with weight w [64], turned by the
    angles of `pos` (None or base 0: not turned).  Returns the values and their bound."""
    x, w = x.to(F64), w.to(F64)
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w
    # 64 squares summed (half of it on the root), eps, the root (2 ulp), two products.
    err = 44 * U32 * y.abs()
    if pos is None or not base:
        return y, err + U16 * y.abs()
    out = rotate(y, pos, base)
    pair = y[..., :32].abs() + y[..., 32:].abs()
    return out, 50 * U32 * torch.cat((pair, pair), -1) + U16 * out.abs()


def norm_grads(dr, x, w, eps, pos=None, base=10000.0):
    """Gradients w.r.t. x and w of norm() from dr, and their bounds (fp32 sums of n terms:
    n 2^-24 of the magnitudes at most)."""
    dr, x, w = dr.to(F64), x.to(F64), w.to(F64)
    turned = pos is not None and base
    dy = rotate(dr, pos, base, back=True) if turned else dr
    pair = dr[..., :32].abs() + dr[..., 32:].abs()
    size = torch.cat((pair, pair), -1) if turned else dr.abs()  # |dy| and its rounding's scale
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    xn = x * r
    g = dy * w
    along = (g * xn).mean(-1, keepdim=True)
    dx = r * (g - xn * along)
    gsize = size * w.abs()
    mag = (gsize * xn.abs()).mean(-1, keepdim=True)
    # dy 4 roundings, xn 44, the mean's 64 terms and products, r again and the last steps.
    dx_err = r * (60 * U32 * gsize + xn.abs() * 170 * U32 * mag) + 48 * U32 * dx.abs() + U16 * dx.abs()
    n = x.shape[0] * x.shape[1]
    dw = (dy * xn).sum((0, 1))
    dw_err = (n + 64) * U32 * (size * xn.abs()).sum((0, 1))
    return dx, dw, dx_err, dw_err


# ------------------------------------------------------------------ 4 bits

def quantise4(x):
    """(values, exponents [..., 2]) of rows x [..., 64] (64 bits) as the 4-bit cache holds
    them, by the definition; NaN and 128 (scale byte 255) for a half that holds an
    infinity or NaN."""
    x = x.unflatten(-1, (2, 32))
    a = x.abs().amax(-1)
    bad = ~torch.isfinite(x).all(-1)
    e = (torch.floor(torch.log2(a / 6)) - 1).clamp(-100, 125)
    for _ in range(3):
        e = torch.where((a > 6 * torch.exp2(e)) & (e < 125), e + 1, e)
    e = torch.where(bad, 128, e)
    y = (x.abs() * torch.exp2(-e)[..., None]).clamp(max=6)
    got = torch.zeros_like(y)
    for i in range(1, 8):  # past the middle, or on it where the upper code is even
        mid = (GRID[i - 1] + GRID[i]) / 2
        got = torch.where((y > mid) | ((y == mid) & (i % 2 == 0)), GRID[i], got)
    got = (torch.copysign(got, x) * torch.exp2(e)[..., None]).masked_fill(bad[..., None], math.nan)
    return got.flatten(-2), e


def byte_of(d):
    """Byte and low bit of dim d in a row of 32 bytes."""
    return 4 * (d % 32 // 4) + 2 * (d // 32) + d % 4 // 2, 4 * (d % 2)


def decode4(pages, scale):
    """Rows [..., 32] bytes, [..., 2] scale bytes -> 64-bit values [..., 64]."""
    grid = torch.tensor(GRID + tuple(-g for g in GRID), dtype=F64, device=pages.device)
    byte, low = torch.tensor([byte_of(d) for d in range(D)], device=pages.device).T
    x = grid[(pages[..., byte].long() >> low) & 15]
    e = scale.to(F64) - 127
    two = torch.where(e == 128, math.nan, torch.exp2(e))
    return x * two.repeat_interleave(32, -1)


class Cache4(Cache):
    """grouped.Cache in 4 bits.  Unused slots hold NaN (scale byte 255)."""

    def __init__(self, lens, Hkv, page, seed=0, device="cuda", **kw):
        super().__init__(lens, Hkv, page, True, seed, device, **kw)
        shape = (self.n_pages, Hkv, page)
        self.k = torch.full((*shape, 32), 0x77, dtype=torch.uint8, device=device)
        self.v = self.k.clone()
        self.ks = torch.full((*shape, 2), 255, dtype=torch.uint8, device=device)
        self.vs = self.ks.clone()

    def fill_random(self, seed):
        """Random codes and scales in every sequence's positions (and nowhere else)."""
        g = torch.Generator("cpu").manual_seed(seed)
        for s, n in enumerate(self.lens):
            for pool, scale in ((self.k, self.ks), (self.v, self.vs)):
                page, slot = (t.to(pool.device) for t in self.where(s, torch.arange(n)))
                pool[page, :, slot] = torch.randint(0, 256, (n, self.Hkv, 32), generator=g).to(
                    torch.uint8).to(pool.device)
                scale[page, :, slot] = torch.randint(123, 128, (n, self.Hkv, 2), generator=g).to(
                    torch.uint8).to(pool.device)
        return self

    def rows(self, s, n=None, first=0):
        n = self.lens[s] if n is None else n
        page, slot = (t.to(self.k.device) for t in self.where(s, first + torch.arange(n)))
        return [decode4(pool[page, :, slot], scale[page, :, slot])
                for pool, scale in ((self.k, self.ks), (self.v, self.vs))]

    def value_scales(self, s, n=None):
        """The scale bytes [n, Hkv, 2] of the rows of v."""
        page, slot = self.where(s, torch.arange(self.lens[s] if n is None else n))
        return self.vs[page.to(self.vs.device), :, slot.to(self.vs.device)]


def half_weights(q, k, scale_bytes, scale):
    """What weights held in halves add to attention()'s bound, [H, 64], for a query q [H, 64]
    over k [m, Hkv, 64] and value rows with the scale bytes [m, Hkv, 2]: a weight is p_j 2^e_j
    over its largest seen so far or more, so that a half, whose smallest step is 2^-24,
    is off by at most 2^-25 of the largest p_j 2^e_j (beside 2^-11 of itself), times a
    magnitude of at most 6, for each of m keys.  (Where the key with the weight holds a zero,
    that is all there is.)"""
    H, Hkv = q.shape[0], k.shape[1]
    s = scale * torch.einsum("hgd,mhd->hgm", q.to(F64).view(Hkv, H // Hkv, D), k.to(F64))
    p = torch.exp(s - torch.logsumexp(s, -1, keepdim=True))
    two = torch.exp2(scale_bytes.to(F64) - 127).permute(1, 2, 0)  # [Hkv, half, m]
    most = (p[:, :, None] * two[:, None]).amax(-1)  # [Hkv, G, half]
    return (6 * k.shape[0] * 2.0 ** -25 * most).reshape(H, 2).repeat_interleave(32, -1)


# ------------------------------------------------------------------ pages

class Pages:
    """Pages, tables and lengths on the host, handed out and taken back one by one."""

    def __init__(self, nseq, max_pages, n_pages, page, order):
        self.page, self.n_pages = page, n_pages
        self.lens = [0] * nseq
        self.table = [[-1] * max_pages for _ in range(nseq)]
        self.free = list(order)

    def reserve(self, new, room):
        """(cu_seqlens, start_pos, positions, slots) of the new rows."""
        cu, start, pos, slots = [0], list(self.lens), [], []
        for s, m in enumerate(new):
            for p in range(self.lens[s], self.lens[s] + m):
                if p % self.page == 0:
                    self.table[s][p // self.page] = self.free.pop()
                pos.append(p)
                slots.append(self.table[s][p // self.page] * self.page + p % self.page)
            self.lens[s] += m
            cu.append(cu[-1] + m)
        more = [-1] * (room - len(pos))
        return cu, start, pos + more, slots + more

    def release(self, finished):
        for s, f in enumerate(finished):
            if f:
                for i in range(-(-self.lens[s] // self.page)):
                    self.free.append(self.table[s][i])
                    self.table[s][i] = -1
                self.lens[s] = 0

"""Plain 64-bit implementations of the grouped-head and paged-cache operators,
with bounds on what rounding may do to each output.

Every bound counts roundings of the types in use: half a step of bf16 is 2^-8
of the value (u16), of e4m3 2^-4 (u8), of fp32 2^-24 (u32).  A sum of n fp32
terms is off by at most n u32 times the sum of magnitudes.
"""
from __future__ import annotations

import math

import torch

U8, U16, U32 = 2.0 ** -4, 2.0 ** -8, 2.0 ** -24
D = 64
F64 = torch.float64


def rotate(x, pos, base=10000.0, back=False):
    """RoPE (rotate-half) of rows x [n, heads, 64] at positions pos [n], in 64 bits."""
    theta = base ** (-torch.arange(32, dtype=F64, device=x.device) / 32)
    a = pos.to(F64)[:, None] * theta
    c, s = a.cos()[:, None], a.sin()[:, None]
    s = -s if back else s
    x = x.to(F64)
    lo, hi = x[..., :32], x[..., 32:]
    return torch.cat((lo * c - hi * s, hi * c + lo * s), -1)


def rotate_bound(x):
    """Bound on an fp32 rotation's error: the table entry's rounding (u32), two
    products and a sum (each u32), against the pair's magnitudes."""
    a = x.to(F64).abs()
    pair = a[..., :32] + a[..., 32:]
    return 4 * U32 * torch.cat((pair, pair), -1)


def quantise(x):
    """(e4m3 values, exponents) of rows x [..., 64] (64 bits), by the definition; NaN
    and 128 (scale byte 255) for a row that holds an infinity or NaN."""
    a = x.abs().amax(-1)
    bad = ~torch.isfinite(x).all(-1)
    e = (torch.floor(torch.log2(a / 448)) - 1).clamp(-100, 127)
    for _ in range(3):
        e = torch.where(a > 448 * torch.exp2(e), e + 1, e)
    e = torch.where(bad, 128, e)
    x = x.masked_fill(bad[..., None], math.nan)
    y = x * torch.exp2(-e)[..., None]
    # e4m3: 3 bits after the leading one down to 2^-6, steps of 2^-9 below.
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, e


def positions(cu, dev):
    n = [int(b) - int(a) for a, b in zip(cu[:-1], cu[1:])]
    return torch.cat([torch.arange(x, device=dev) for x in n]) if sum(n) else \
        torch.zeros(0, dtype=torch.int64, device=dev)


def attention(q, k, v, scale, first=None):
    """Causal attention of one sequence: q [n, H, 64] (the last n positions),
    k, v [m, Hkv, 64], in 64 bits.  Returns out, lse [H, n] and their bounds, for
    a kernel that rounds the weights to bf16 and sums in fp32."""
    n, H, _ = q.shape
    m, Hkv, _ = k.shape
    G = H // Hkv
    q, k, v = (t.to(F64) for t in (q, k, v))
    q = q.view(n, Hkv, G, D)
    row = torch.arange(n, device=q.device) + (m - n)
    hidden = torch.arange(m, device=q.device)[None, :] > row[:, None]
    s = scale * torch.einsum("nhgd,mhd->hgnm", q, k)
    size = scale * torch.einsum("nhgd,mhd->hgnm", q.abs(), k.abs())
    s = s.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None])
    out = torch.einsum("hgnm,mhd->nhgd", p, v)
    # A score: 64 products summed, the scale, the conversion to a power of two.
    s_err = (size.masked_fill(hidden, 0).amax(-1) * 68 + lse.abs() * 4) * U32
    lse_err = s_err + (64 + m) * U32 + 4 * U32 * lse.abs()
    # Weights: their own exponent's error, 2^-22 of the exponential, bf16.
    w_err = U16 + 2 * s_err + (16 + m) * U32
    mag = torch.einsum("hgnm,mhd->nhgd", p, v.abs())
    out_err = mag * w_err.permute(2, 0, 1)[..., None] + out.abs() * U16
    return (out.reshape(n, H, D), lse.reshape(H, n), out_err.reshape(n, H, D),
            lse_err.reshape(H, n))


def attention_grads(q, k, v, out, do, lse, scale):
    """Gradients of one sequence w.r.t. q, k (as multiplied: rotated) and v, in
    64 bits, from the given out [n, H, 64] and lse [H, n]; and bounds for a kernel
    that rounds the weights and dS to bf16."""
    n, H, _ = q.shape
    Hkv = k.shape[1]
    G = H // Hkv
    q, out, do = (t.to(F64).view(n, Hkv, G, D) for t in (q, out, do))
    k, v = k.to(F64), v.to(F64)
    lse = lse.to(F64).view(Hkv, G, n)
    hidden = torch.ones((n, n), dtype=torch.bool, device=q.device).triu(1)
    s = scale * torch.einsum("nhgd,mhd->hgnm", q, k)
    size = scale * torch.einsum("nhgd,mhd->hgnm", q.abs(), k.abs())
    p = torch.exp(s - lse[..., None]).masked_fill(hidden, 0)
    p_rel = (size * 68 + lse.abs()[..., None] * 8 + 16) * U32
    delta = (do * out).sum(-1).permute(1, 2, 0)[..., None]
    delta_size = (do * out).abs().sum(-1).permute(1, 2, 0)[..., None]
    dp = torch.einsum("nhgd,mhd->hgnm", do, v)
    dp_size = torch.einsum("nhgd,mhd->hgnm", do.abs(), v.abs())
    ds = p * (dp - delta)
    ds_err = ds.abs() * (U16 + p_rel) + p * 68 * U32 * (dp_size + delta_size)
    sums = 4 * n * U32  # fp32 sums over the rows and heads
    dv = torch.einsum("hgnm,nhgd->mhd", p, do)
    dv_mag = torch.einsum("hgnm,nhgd->mhd", p * (U16 + p_rel + sums * G), do.abs())
    dq = scale * torch.einsum("hgnm,mhd->nhgd", ds, k)
    dq_mag = scale * torch.einsum("hgnm,mhd->nhgd", ds_err + ds.abs() * sums, k.abs())
    dk = scale * torch.einsum("hgnm,nhgd->mhd", ds, q)
    dk_mag = scale * torch.einsum("hgnm,nhgd->mhd", ds_err + ds.abs() * sums * G, q.abs())
    return ((dq.reshape(n, H, D), dk, dv),
            (dq_mag.reshape(n, H, D), dk_mag, dv_mag + dv.abs() * U16))


def unrotate_bound(x, err, roundings):
    """Bound on R^T x where x carries `err` and is rounded to bf16 `roundings`
    times (before and after the rotation)."""
    e = err + (roundings - 1) * U16 * x.abs()
    pair = e[..., :32] + e[..., 32:]
    y = x.abs()
    mag = y[..., :32] + y[..., 32:]
    return torch.cat((pair, pair), -1) + torch.cat((mag, mag), -1) * (U16 + 8 * U32)


def within(got, want, err, what):
    """Every element of got within err of want (equal where want is infinite, NaN
    where it is NaN)."""
    got, want = got.to(F64), want.to(F64)
    fin = torch.isfinite(want)
    assert torch.equal(torch.nan_to_num(got[~fin], nan=7.0), torch.nan_to_num(want[~fin], nan=7.0))
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    d = (got - want).abs()[fin]
    e = err.expand_as(want)[fin] + 1e-30
    worst = float((d / e).max()) if d.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound"
    return worst


class Cache:
    """A paged cache with its pages handed out in a shuffled order; room for
    `lens[s]` positions of each sequence.  Unused table entries are -1, unused
    slots hold `fill` (NaN by default: nothing may read them)."""

    def __init__(self, lens, Hkv, page, e4m3, seed=0, device="cuda", fill=float("nan"), spare=2,
                 extra_columns=1):
        g = torch.Generator("cpu").manual_seed(seed)
        used = [-(-n // page) for n in lens]
        self.n_pages = sum(used) + spare
        perm = torch.randperm(self.n_pages, generator=g).to(torch.int32)
        self.max_pages = max(used + [1]) + extra_columns
        table = torch.full((len(lens), self.max_pages), -1, dtype=torch.int32)
        at = 0
        for s, u in enumerate(used):
            table[s, :u] = perm[at:at + u]
            at += u
        self.table = table.to(device)
        self.page, self.Hkv, self.e4m3, self.lens = page, Hkv, e4m3, list(lens)
        shape = (self.n_pages, Hkv, page, D)
        if e4m3:
            self.k = torch.full(shape, fill, device=device).to(torch.float8_e4m3fn)
            self.v = self.k.clone()
            self.ks = torch.full(shape[:3], 255, dtype=torch.uint8, device=device)
            self.vs = self.ks.clone()
        else:
            self.k = torch.full(shape, fill, device=device, dtype=torch.bfloat16)
            self.v = self.k.clone()
            self.ks = self.vs = None

    def fill_random(self, seed):
        """Random rows in every sequence's positions (and nowhere else)."""
        g = torch.Generator("cpu").manual_seed(seed)
        for s, n in enumerate(self.lens):
            for pool, scale in ((self.k, self.ks), (self.v, self.vs)):
                x = torch.randn((n, self.Hkv, D), generator=g)
                page, slot = self.where(s, torch.arange(n))
                page, slot = page.to(pool.device), slot.to(pool.device)
                if self.e4m3:
                    q8 = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn).to(pool.device)
                    pool.view(torch.uint8)[page, :, slot] = q8.view(torch.uint8)
                    e = torch.randint(117, 123, (n, self.Hkv), generator=g)
                    scale[page, :, slot] = e.to(torch.uint8).to(pool.device)
                else:
                    pool[page, :, slot] = x.bfloat16().to(pool.device)
        return self

    def where(self, s, pos):
        t = self.table[s].cpu().long()
        return t[pos // self.page], pos % self.page

    def rows(self, s, n=None, first=0):
        """k, v rows [n, Hkv, 64] of sequence s in 64 bits."""
        n = self.lens[s] if n is None else n
        page, slot = self.where(s, first + torch.arange(n))
        got = []
        for pool, scale in ((self.k, self.ks), (self.v, self.vs)):
            page, slot = page.to(pool.device), slot.to(pool.device)
            if self.e4m3:
                x = pool.view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).to(F64)
                byte = scale[page, :, slot].to(F64)
                x = x * torch.exp2(byte - 127)[..., None]
                x = x.masked_fill((byte == 255)[..., None], math.nan)
            else:
                x = pool[page, :, slot].to(F64)
            got.append(x)
        return got

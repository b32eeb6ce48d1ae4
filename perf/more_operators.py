"""The workloads by which the operators around the paged cache are measured.

Five operators of one generation step, in its order: pages, positions and slots
for the step's new rows (``reserve``), the norms of queries and keys for each
head with the rotation in the same pass (``norm``) and its gradients
(``norm_grad``), rows into a cache held in 4 bits and back (``store``), and
attention of one new token over that cache (``decode``).  Heads are 64 wide;
query head h uses key/value head h // (H // Hkv); RoPE is rotate-half with base
10000.  A 4-bit row is 64 e2m1 values, two to a byte (the even one in the low
half), with a power of two for each half of the row; word w of its 8 holds
values 4 w .. 4 w + 3 and then 32 + 4 w .. 32 + 4 w + 3, which the first are
rotated with.

With ``own`` false, ``run`` computes the operators with elementary torch
operations in fp32; with ``own`` true it calls the library.
"""
from __future__ import annotations

import math
import random

import torch

own = False

D = 64
BASE = 10000.0
SCALE = 0.125
EPS = 1e-5
LONGEST = 16384


# ---------------------------------------------------------------------- cases
def _reserve_case(nseq, cached, nmin, nmax, idle, page, lens, **more):
    """cached: the longest cached length; nmin .. nmax: new rows; idle: the share without any."""
    return dict(op="reserve", nseq=nseq, cached=cached, nmin=nmin, nmax=nmax, idle=idle, page=page,
                lens=lens, **more)


def _norm_case(op, nseq, lmin, lmax, lens, H, Hkv, step=False, **more):
    return dict(op=op, nseq=nseq, lmin=lmin, lmax=lmax, lens=lens, H=H, Hkv=Hkv, step=step, **more)


def _cache_case(op, nseq, lmin, lmax, lens, H, Hkv, page, step=False, **more):
    return dict(op=op, nseq=nseq, lmin=lmin, lmax=lmax, lens=lens, H=H, Hkv=Hkv, page=page,
                step=step, **more)


def listed():
    return [
        # One step of generation: a token for each of 64 running sequences.  A few KB: latency.
        _reserve_case(64, 4000, 1, 1, 0.0, 64, 1, name="reserve_step"),
        # A burst of 4096 requests with prompts (or parts of them) of 1 to 2048 tokens, small pages.
        _reserve_case(4096, 2048, 1, 2048, 0.1, 16, 2, name="reserve_burst"),
        # The queries and keys of one step of generation for 64 sequences.
        _norm_case("norm", 64, 200, 4000, 3, 12, 4, step=True, name="norm_step"),
        # 32 packed prompts of 64 to 2048 tokens.
        _norm_case("norm", 32, 64, 2048, 4, 12, 4, name="norm_prompts"),
        # A large packed batch of long contexts.
        _norm_case("norm", 8, 5000, 16384, 5, 32, 8, name="norm_long"),
        # Training on 8 sequences of 1024 tokens (the GPT-2-small shape, heads shared by three).
        _norm_case("norm_grad", 8, 1024, 1024, 6, 12, 4, name="norm_grad_1k"),
        # Training on long contexts with more heads.
        _norm_case("norm_grad", 4, 16384, 16384, 7, 32, 8, name="norm_grad_16k"),
        # One step's rows, at the ends of 64 sequences, into the cache and back.
        _cache_case("store", 64, 200, 4000, 8, 12, 4, 64, step=True, name="store_step"),
        # Whole prompts into a cache of small pages, read back for the next part's attention.
        _cache_case("store", 32, 64, 2048, 9, 32, 8, 16, name="store_prompts"),
        # One user's next token, a short cache: latency.
        _cache_case("decode", 1, 777, 777, 10, 12, 4, 16, name="decode_one_short"),
        # A serving batch of very different lengths.
        _cache_case("decode", 64, 1, 16384, 11, 32, 8, 64, name="decode_ragged"),
        # 64 long contexts: the cache's bytes are what counts.
        _cache_case("decode", 64, 15000, 16384, 12, 32, 8, 128, name="decode_16k"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("reserve", "norm", "norm_grad", "store", "decode"))
    lens = rng.randrange(1 << 30)
    page = rng.choice((16, 32, 64, 128, 256))
    if op == "reserve":
        nseq, nmax = _log_int(rng, 1, 4096), _log_int(rng, 1, 2048)
        return _reserve_case(nseq, _log_int(rng, 1, 4096), _log_int(rng, 1, nmax), nmax,
                             rng.choice((0.0, 0.1, 0.5)), page, lens)
    Hkv = rng.choice((1, 2, 3, 4, 6, 8, 12))
    G = rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 12, 16))
    while G * Hkv > 32:
        G = rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 12, 16))
    lmax = _log_int(rng, 1, LONGEST)
    lmin = _log_int(rng, 1, lmax)
    if op in ("norm", "norm_grad"):
        most = max(1, min(96, 4 * 16384 * 40 // (lmax * (G + 1) * Hkv)))
        return _norm_case(op, _log_int(rng, 1, most), lmin, lmax, lens, G * Hkv, Hkv,
                          step=op == "norm" and rng.random() < 0.4)
    most = max(1, min(96, 16 * 16384 * 8 // (lmax * Hkv)))
    return _cache_case(op, _log_int(rng, 1, most), lmin, lmax, lens, G * Hkv, Hkv, page,
                       step=op == "store" and rng.random() < 0.4)


def _lengths(case):
    """The sequences' lengths: part of the case, spread over the logarithm of their range."""
    rng = random.Random(case["lens"])
    n = [_log_int(rng, case["lmin"], case["lmax"]) for _ in range(case["nseq"])]
    n[rng.randrange(len(n))] = case["lmax"]
    return n


def _requests(case):
    """Cached lengths and new rows of each sequence, and the pages taken in all."""
    rng, ps = random.Random(case["lens"]), case["page"]
    old = [0 if rng.random() < 0.3 else _log_int(rng, 1, case["cached"])
           for _ in range(case["nseq"])]
    new = [0 if rng.random() < case["idle"] else _log_int(rng, case["nmin"], case["nmax"])
           for _ in old]
    if not any(new):
        new[0] = case["nmax"]
    return old, new, sum(-(-(a + b) // ps) - -(-a // ps) for a, b in zip(old, new))


def work(case):
    op = case["op"]
    if op == "reserve":
        _, new, taken = _requests(case)
        rows, n = sum(new), case["nseq"]
        # lengths and free pages in; table entries, row starts, lengths, positions, slots out
        return {"bytes": 4 * (2 * n + taken) + 4 * (taken + 3 * n + 2 * rows), "flops": 4 * rows}
    n, H, Hkv = _lengths(case), case["H"], case["Hkv"]
    tok = sum(n)
    row = 2 * (D // 2 + 2)  # one cached token of one head: K and V, each with two scale bytes
    if op == "norm":
        r = case["nseq"] if case["step"] else tok
        return {"bytes": r * ((H + Hkv) * 4 * D + 4), "flops": r * (H + Hkv) * 8 * D}
    if op == "norm_grad":  # gradients and inputs in, gradients out
        return {"bytes": tok * ((H + Hkv) * 6 * D + 4), "flops": tok * (H + Hkv) * 20 * D}
    if op == "store":  # rows in, cache out; cache in, rows out
        r = case["nseq"] if case["step"] else tok
        return {"bytes": r * Hkv * 2 * (4 * D + row), "flops": r * Hkv * 8 * D}
    return {"bytes": tok * Hkv * row + case["nseq"] * H * (4 * D + 4), "flops": tok * H * 4 * D}


# --------------------------------------------------------------------- inputs
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cu(n):
    return torch.cat((_ints([0]), torch.cumsum(_ints(n), 0).to(torch.int32)))


def _prepare_reserve(case, g):
    old, new, taken = _requests(case)
    ps, nseq = case["page"], case["nseq"]
    used = [-(-x // ps) for x in old]
    n_pages = sum(used) + taken + 5
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    width = max(-(-(a + b) // ps) for a, b in zip(old, new)) + 1
    table = torch.full((nseq, width), -1, dtype=torch.int32)
    at = 0
    for i, u in enumerate(used):
        table[i, :u] = torch.arange(at, at + u, dtype=torch.int32)
        at += u
    table = table.cuda()
    table = torch.where(table >= 0, perm[table.clamp(min=0).long()], -1).to(torch.int32)
    free = torch.full((n_pages,), -1, dtype=torch.int32, device="cuda")
    free[:n_pages - sum(used)] = perm[sum(used):]
    rows = sum(new)
    return dict(seq_lens=_ints(old), new_lens=_ints(new), table=table.contiguous(), free=free,
                n_free=_ints([n_pages - sum(used)]), n_pages=n_pages, rows=rows, taken=taken,
                room=-(-rows // 64) * 64, max_seqlen=width * ps,
                seq_lens_out=_ints([0] * nseq), n_free_out=_ints([0]))


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    op = case["op"]
    if op == "reserve":
        return dict(_prepare_reserve(case, g), case=case)
    n, H, Hkv = _lengths(case), case["H"], case["Hkv"]
    st = dict(case=case, n=n, max_seqlen=max(n))
    if op in ("norm", "norm_grad"):
        if case["step"]:
            st["pos"] = _ints([x - 1 for x in n])
        else:
            st["pos"] = torch.cat([torch.arange(x, dtype=torch.int32, device="cuda") for x in n])
        N = st["pos"].numel()
        # The projection's output: q, k and v of a token side by side.
        qkv = _randn(g, N, H + 2 * Hkv, D).mul_(2).bfloat16()
        st["q"], st["k"] = qkv[:, :H], qkv[:, H:H + Hkv]
        st["wq"], st["wk"] = ((1 + 0.3 * _randn(g, D)).bfloat16() for _ in range(2))
        if op == "norm_grad":
            st["dqr"], st["dkr"] = (_randn(g, N, h, D).bfloat16() for h in (H, Hkv))
        return st
    # A cache whose pages were handed out in no order, with some to spare.
    ps = case["page"]
    used = [-(-x // ps) for x in n]
    n_pages = sum(used) + 3
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    at = torch.full((len(n), max(used)), -1, dtype=torch.int64)
    start = 0
    for i, u in enumerate(used):
        at[i, :u] = torch.arange(start, start + u)
        start += u
    at = at.cuda()
    st["table"] = torch.where(at >= 0, perm[at.clamp(min=0)], -1).to(torch.int32).contiguous()
    st["values"] = _values()
    for name in ("k", "v"):
        # (a page at a time in the pool's order: 16 at once)
        pages = torch.empty((n_pages, Hkv, ps, D // 2), dtype=torch.uint8, device="cuda")
        scale = torch.empty((n_pages, Hkv, ps, 2), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 22) // (Hkv * ps))
        for i in range(0, n_pages, step):
            x = _randn(g, min(step, n_pages - i), Hkv, ps, D).bfloat16().float()
            pages[i:i + step], scale[i:i + step] = _encode(x)
        st[name + "_pages"], st[name + "_scale"] = pages, scale
    if op == "store":
        rows = [1] * len(n) if case["step"] else n
        st["cu"] = _cu(rows)
        st["start"] = _ints([x - 1 for x in n] if case["step"] else [0] * len(n))
        st["rows"] = sum(rows)
        st["k"], st["v"] = (_randn(g, st["rows"], Hkv, D).bfloat16() for _ in range(2))
    else:
        st["lens"] = _ints(n)
        st["q"] = _randn(g, len(n), H, D).bfloat16()
    return st


# ----------------------------------------------------------- the plain forms
def _values():
    """The two values of each byte, [256, 2] fp32."""
    one = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    one = torch.cat((one, -one))
    byte = torch.arange(256, device="cuda")
    return torch.stack((one[byte & 15], one[byte >> 4]), -1)


def _encode(x):
    """Rows x [..., 64] fp32 as e2m1 bytes [..., 32] and scale bytes [..., 2]: for each 32
    values the smallest e from -100 on with max |x| <= 6 * 2^e, to the nearest, ties to even."""
    x = x.unflatten(-1, (2, 32))
    m, e = torch.frexp(x.abs().amax(-1))  # max = m 2^e, 0.5 <= m < 1; 6 = 0.75 * 2^3
    e = torch.where(m == 0, -100, e - 3 + (m > 0.75).to(torch.int32)).clamp(-100, 125)
    y = torch.ldexp(x, -e[..., None])
    a = y.abs().clamp(max=6)
    # Steps of 0.5 below 2, of 1 below 4, of 2 from there on; codes 0..4, 4..6, 6..7.
    code = torch.where(a < 2, torch.round(a * 2),
                       torch.where(a < 4, torch.round(a) + 2, torch.round(a / 2) + 4))
    code = code.to(torch.uint8) | (torch.signbit(y).to(torch.uint8) << 3)
    code = code[..., 0::2] | (code[..., 1::2] << 4)  # [..., half, 16 bytes]
    code = code.unflatten(-1, (8, 2)).transpose(-3, -2).flatten(-3)
    return code, (e + 127).to(torch.uint8)


def _decoded(st, pages, scale):
    """The values of e2m1 rows: bytes [..., 32] and scale bytes [..., 2] to fp32 [..., 64]."""
    x = st["values"][pages.to(torch.int32)].unflatten(-2, (8, 2, 2))  # [..., word, half, 2, 2]
    two = torch.exp2(scale.float() - 127)[..., None, :, None, None]
    return (x * two).transpose(-4, -3).flatten(-4)


def _cos_sin(pos):
    """cos, sin of the angles of positions `pos`, formed in 64 bits (far positions)."""
    theta = BASE ** (-torch.arange(32, device=pos.device, dtype=torch.float64) / 32)
    a = pos.double()[:, None] * theta
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _rotate(x, c, s):
    a, b = x[..., :32], x[..., 32:]
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def _rstd(x):
    return torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _norm(st):
    c, s = _cos_sin(st["pos"])

    def one(x, w):
        x = x.float()
        return _rotate(x * _rstd(x) * w.float(), c, s).bfloat16()

    return one(st["q"], st["wq"]), one(st["k"], st["wk"])


def _norm_grad(st):
    c, s = _cos_sin(st["pos"])

    def one(dr, x, w):
        x = x.float()
        r = _rstd(x)
        xn, dy = x * r, _rotate(dr.float(), c, -s)
        dw = (dy * xn).sum((0, 1), dtype=torch.float64).float()
        g = dy * w.float()
        return (r * (g - xn * (g * xn).mean(-1, keepdim=True))).bfloat16(), dw

    dq, dwq = one(st["dqr"], st["q"], st["wq"])
    dk, dwk = one(st["dkr"], st["k"], st["wk"])
    return dq, dk, dwq, dwk


def _rows(cu, nseq, rows):
    """The sequence of each packed row, and its place in it."""
    cu = cu.long()
    seq = torch.repeat_interleave(torch.arange(nseq, device=cu.device), cu[1:] - cu[:-1],
                                  output_size=rows)
    return seq, torch.arange(rows, device=cu.device) - cu[seq]


def _reserve(st):
    ps, nseq, dev = st["case"]["page"], st["case"]["nseq"], st["table"].device
    old, new, table = st["seq_lens"], st["new_lens"], st["table"]
    had, want = (old + ps - 1) // ps, (old + new + ps - 1) // ps
    cu = torch.cat((torch.zeros(1, dtype=torch.int32, device=dev),
                    torch.cumsum(new, 0, dtype=torch.int32)))
    pages = torch.cat((torch.zeros(1, dtype=torch.int32, device=dev),
                       torch.cumsum(want - had, 0, dtype=torch.int32)))
    # The pages taken, in the order of the sequences, from the end of the free ones.
    seq, j = _rows(pages, nseq, st["taken"])
    at = st["n_free"].long() - 1 - torch.arange(st["taken"], device=dev)
    table[seq, had[seq] + j] = st["free"][at]
    seq, i = _rows(cu, nseq, st["rows"])
    pos = old[seq] + i
    positions = torch.full((st["room"],), -1, dtype=torch.int32, device=dev)
    slots = positions.clone()
    positions[:st["rows"]] = pos.to(torch.int32)
    slots[:st["rows"]] = (table[seq, pos // ps] * ps + pos % ps).to(torch.int32)
    return cu, old.clone(), positions, slots, table, old + new, st["n_free"] - pages[-1:]


def _places(st):
    c = st["case"]
    seq, at = _rows(st["cu"], c["nseq"], st["rows"])
    pos = at + st["start"].long()[seq]
    return st["table"].long()[seq, pos // c["page"]], pos % c["page"]


def _store(st):
    page, slot = _places(st)

    def one(name):
        pages, scale = st[name + "_pages"], st[name + "_scale"]
        pages[page, :, slot], scale[page, :, slot] = _encode(st[name].float())
        return _decoded(st, pages[page, :, slot], scale[page, :, slot]).bfloat16()

    return one("k"), one("v")


def _decode(st):
    c = st["case"]
    B, H, Hkv, ps = c["nseq"], c["H"], c["Hkv"], c["page"]
    n = st["lens"].long()
    pos = torch.arange(st["max_seqlen"], device=n.device)
    page = st["table"].long()[:, pos // ps].clamp(min=0)
    slot = (pos % ps).expand(B, -1)

    def rows(name):  # [B, positions, Hkv, 64]
        return _decoded(st, st[name + "_pages"][page, :, slot], st[name + "_scale"][page, :, slot])

    s = torch.matmul(st["q"].float().view(B, Hkv, H // Hkv, D), rows("k").permute(0, 2, 3, 1))
    s = s.mul_(SCALE).masked_fill_((pos >= n[:, None])[:, None, None, :], -math.inf)
    lse = torch.logsumexp(s, -1, keepdim=True)
    o = torch.matmul(torch.exp(s - lse), rows("v").permute(0, 2, 1, 3))
    return o.reshape(B, H, D).bfloat16(), lse.reshape(B, H)


# ------------------------------------------------------------------- one pass
NAMES = dict(reserve=("cu_seqlens", "start_pos", "positions", "slots", "table", "seq_lens",
                      "n_free"),
             norm=("qr", "kr"), norm_grad=("dq", "dk", "dwq", "dwk"), store=("k", "v"),
             decode=("out", "lse"))


def run(state):
    st, op = state, state["case"]["op"]
    if not own:
        got = dict(reserve=_reserve, norm=_norm, norm_grad=_norm_grad, store=_store,
                   decode=_decode)[op](st)
    else:
        from causal_self_attention_gb300 import ne_attn as na
        if op == "reserve":
            got = na.ne_kv_reserve(st["new_lens"], st["seq_lens"], st["table"], st["free"],
                                   st["n_free"], st["room"], st["case"]["page"], st["max_seqlen"],
                                   seq_lens_out=st["seq_lens_out"], n_free_out=st["n_free_out"])
            got = (*got, st["table"], st["seq_lens_out"], st["n_free_out"])
        elif op == "norm":
            got = na.ne_qk_norm_rope_fwd(st["q"], st["k"], st["wq"], st["wk"], st["pos"],
                                         st["max_seqlen"], eps=EPS, rope_base=BASE)
        elif op == "norm_grad":
            got = na.ne_qk_norm_rope_bwd(st["dqr"], st["dkr"], st["q"], st["k"], st["wq"],
                                         st["wk"], st["pos"], st["max_seqlen"], eps=EPS,
                                         rope_base=BASE)
        elif op == "store":  # what is held in 4 bits comes back as the values it stands for
            na.ne_kv_append(st["k"], st["v"], st["cu"], st["start"], st["k_pages"],
                            st["v_pages"], st["table"], st["max_seqlen"], st["k_scale"],
                            st["v_scale"], rope_base=0.0)
            got = na.ne_kv_read(st["k_pages"], st["v_pages"], st["table"], st["cu"], st["start"],
                                st["rows"], st["k_scale"], st["v_scale"])
        else:
            got = na.ne_attn_decode_paged(st["q"], st["k_pages"], st["v_pages"], st["table"],
                                          st["lens"], st["max_seqlen"], st["k_scale"],
                                          st["v_scale"], rope_base=0.0, scale=SCALE)
    return dict(zip(NAMES[op], got))


# ------------------------------------------- the operators' values in 64 bits
def _turn(x, pos, sign=1.0):
    """Rows x [n, heads, 64] in 64 bits turned by the angles of positions pos."""
    i = torch.arange(64, device=x.device)
    angle = pos.double()[:, None] * torch.exp((i % 32).double() * (-math.log(BASE) / 32))
    swapped = torch.where(i < 32, -x.roll(-32, -1), x.roll(32, -1))
    return x * angle.cos()[:, None] + sign * swapped * angle.sin()[:, None]


def _nearest(x):
    """Rows x [..., 64] in 64 bits as the 4-bit cache holds them: each 32 values on the grid
    of 2^e times 0, 0.5, 1, 1.5, 2, 3, 4, 6, found by comparing with every point of it."""
    x = x.unflatten(-1, (2, 32))
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top / 6)).clamp(-100, 125)
    e = torch.where((top <= 6 * torch.pow(2.0, e - 1)) & (e > -100), e - 1, e)
    a = x.abs() / torch.pow(2.0, e)
    grid = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
    got = torch.zeros_like(a)
    for k in range(1, 8):  # past the middle, or on it where the upper neighbour's code is even
        mid = (grid[k - 1] + grid[k]) / 2
        got = torch.where((a > mid) | ((a == mid) & (k % 2 == 0)), grid[k], got)
    return (torch.copysign(got, x) * torch.pow(2.0, e)).flatten(-2)


def _sequence(st, name, s):
    """The cached rows of sequence s, all heads, in 64 bits: [n, Hkv, 64]."""
    ps, n, Hkv = st["case"]["page"], st["n"][s], st["case"]["Hkv"]
    ids = st["table"][s, :-(-n // ps)].long()
    byte = st[name + "_pages"][ids].long()
    code = torch.stack((byte % 16, byte // 16), -1).flatten(-2)  # words of 4 + 4 values
    d = torch.arange(D, device=code.device)
    code = code[..., d % 32 // 4 * 8 + d // 32 * 4 + d % 4]
    size = code % 8
    x = torch.where(size < 2, size / 2.0, torch.pow(2.0, size // 2 - 1.0) * (1 + size % 2 / 2.0))
    x = torch.where(code >= 8, -x, x).double()
    two = torch.pow(2.0, st[name + "_scale"][ids].double() - 127)
    x = x * two.repeat_interleave(32, -1)
    return x.transpose(1, 2).reshape(-1, Hkv, D)[:n]


def exact(case, seed):
    op = case["op"]
    if op == "reserve":
        return None
    st = prepare(case, seed)
    n, H, Hkv = st["n"], case["H"], case["Hkv"]
    G = H // Hkv
    if op == "norm":
        got = {}
        for name, w in (("q", "wq"), ("k", "wk")):
            x = st[name].double()
            x = x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * st[w].double()
            got[name + "r"] = _turn(x, st["pos"])
        return got
    if op == "norm_grad":
        got = {}
        for name in ("q", "k"):
            w, pos = st["w" + name].double(), st["pos"]
            step = max(1, (1 << 24) // (st[name].shape[1] * D))
            dx, dw = [], torch.zeros(D, dtype=torch.float64, device="cuda")
            for i in range(0, pos.numel(), step):
                x = st[name][i:i + step].double()
                dy = _turn(st["d" + name + "r"][i:i + step].double(), pos[i:i + step], -1.0)
                size = (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt()
                dw += (dy * x / size).sum((0, 1))
                along = (dy * w * x).sum(-1, keepdim=True) / D
                dx.append(dy * w / size - x * along / size.pow(3))
            got["d" + name], got["dw" + name] = torch.cat(dx), dw
        return got
    if op == "store":
        return {x: _nearest(st[x].double()) for x in ("k", "v")}
    out = torch.zeros((len(n), H, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((len(n), H), dtype=torch.float64, device="cuda")
    for s in range(len(n)):
        q = st["q"][s].double()
        k, v = (_sequence(st, x, s) for x in ("k", "v"))
        for h in range(Hkv):
            z = SCALE * (q[h * G:(h + 1) * G] @ k[:, h].T)
            top = z.amax(1, keepdim=True)
            w = torch.exp(z - top)
            lse[s, h * G:(h + 1) * G] = (top + w.sum(1, keepdim=True).log())[:, 0]
            out[s, h * G:(h + 1) * G] = (w @ v[:, h]) / w.sum(1, keepdim=True)
    return dict(out=out, lse=lse)

"""The workloads by which the grouped-head and paged-cache operators are measured.

Five operators: writing rows into a paged key/value cache (``append``), reading
them back (``read``), attention of one new token over the cache (``decode``),
attention over packed prompts with shared key/value heads (``prompt``) and its
gradients (``train``).  Heads are 64 wide; query head h uses key/value head
h // (H // Hkv); RoPE is rotate-half with base 10000.

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


# ---------------------------------------------------------------------- cases
def _case(op, nseq, lmin, lmax, lens, H, Hkv, page=0, fp8=False, **more):
    return dict(op=op, nseq=nseq, lmin=lmin, lmax=lmax, lens=lens, H=H, Hkv=Hkv, page=page,
                fp8=fp8, **more)


def listed():
    return [
        # One step of generation for 64 running sequences: 64 new rows, each at the end of its
        # own sequence.  A few KB: its launch is what counts.
        _case("append", 64, 200, 4000, 1, 12, 4, 64, False, step=True,
              name="append_step_bf16"),
        # The prompts of a packed batch (64 to 2048 tokens) written into an 8-bit cache of small
        # pages, the keys rotated on the way.
        _case("append", 32, 64, 2048, 2, 12, 4, 16, True, step=False, name="append_prompts_e4m3"),
        # Three short sequences of a model without shared heads read back from a bf16 cache.
        _case("read", 3, 1, 1000, 3, 12, 12, 32, False, name="read_short_bf16"),
        # Long 8-bit sequences read back, for example to move them to another cache.
        _case("read", 8, 5000, 16384, 4, 32, 8, 64, True, name="read_long_e4m3"),
        # One user's next token, a short cache: latency.
        _case("decode", 1, 777, 777, 5, 12, 4, 16, False, name="decode_one_short_bf16"),
        # A serving batch of very different lengths on an 8-bit cache.
        _case("decode", 64, 1, 16384, 6, 32, 8, 64, True, name="decode_ragged_e4m3"),
        # 16 long contexts on a bf16 cache: the cache's bytes are what counts.
        _case("decode", 16, 15000, 16384, 7, 32, 8, 128, False, name="decode_16k_bf16"),
        # A handful of short prompts, some a few tokens long.
        _case("prompt", 7, 1, 200, 8, 12, 4, name="prompt_short"),
        # 32 packed prompts of 64 to 2048 tokens.
        _case("prompt", 32, 64, 2048, 9, 12, 4, name="prompt_packed"),
        # One long byte-level context.
        _case("prompt", 1, 16384, 16384, 10, 12, 2, name="prompt_16k"),
        # Training on 8 sequences of 1024 tokens (the GPT-2-small shape, heads shared by three).
        _case("train", 8, 1024, 1024, 11, 12, 4, name="train_1k"),
        # Training on one long context.
        _case("train", 1, 16384, 16384, 12, 12, 2, name="train_16k"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("append", "read", "decode", "prompt", "train"))
    Hkv = rng.choice((1, 2, 3, 4, 6, 8, 12))
    G = rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 12, 16))
    while G * Hkv > 32:
        G = rng.choice((1, 2, 3, 4, 5, 6, 7, 8, 12, 16))
    lens = rng.randrange(1 << 30)
    if op in ("prompt", "train"):
        # Scores of the plain form: nseq * H * lmax^2 stays under those of the longest listed case.
        lmax = _log_int(rng, 1, 16384)
        most = max(1, min(48, int(12 * 16384 ** 2 / (G * Hkv * lmax ** 2))))
        while G > 1 and G * Hkv * lmax ** 2 > 12 * 16384 ** 2:
            G -= 1
        if G * Hkv * lmax ** 2 > 12 * 16384 ** 2:
            Hkv = 1
        nseq = _log_int(rng, 1, most)
        return _case(op, nseq, _log_int(rng, 1, lmax), lmax, lens, G * Hkv, Hkv)
    lmax = _log_int(rng, 1, 16384)
    most = max(1, min(96, 16 * 16384 * 8 // (lmax * Hkv)))
    nseq = _log_int(rng, 1, most)
    page, fp8 = rng.choice((16, 32, 64, 128, 256)), rng.random() < 0.5
    lmin = _log_int(rng, 1, lmax)
    if op == "append":
        return _case(op, nseq, lmin, lmax, lens, G * Hkv, Hkv, page, fp8, step=rng.random() < 0.4)
    return _case(op, nseq, lmin, lmax, lens, G * Hkv, Hkv, page, fp8)


def _lengths(case):
    """The sequences' lengths: part of the case, spread over the logarithm of their range."""
    rng = random.Random(case["lens"])
    n = [_log_int(rng, case["lmin"], case["lmax"]) for _ in range(case["nseq"])]
    n[rng.randrange(len(n))] = case["lmax"]
    return n


def work(case):
    n, H, Hkv = _lengths(case), case["H"], case["Hkv"]
    tok = sum(n)
    pairs = sum(x * (x + 1) // 2 for x in n)
    row = 2 * D + 2 if case["fp8"] else 4 * D  # one cached token of one head: K and V
    op = case["op"]
    if op == "append":
        r = case["nseq"] if case["step"] else tok
        return {"bytes": r * Hkv * (4 * D + row), "flops": r * Hkv * 3 * D}
    if op == "read":
        return {"bytes": tok * Hkv * (4 * D + row), "flops": tok * Hkv * 2 * D}
    if op == "decode":
        return {"bytes": tok * Hkv * row + case["nseq"] * H * (4 * D + 4),
                "flops": tok * H * 4 * D}
    if op == "prompt":  # q, k, v in; out, q', k', lse out
        return {"bytes": tok * (H * (6 * D + 4) + Hkv * 6 * D), "flops": pairs * H * 4 * D}
    # q', k', v, out, dout, lse in; dq, dk, dv out
    return {"bytes": tok * (H * (8 * D + 4) + Hkv * 8 * D), "flops": pairs * H * 10 * D}


# --------------------------------------------------------------------- inputs
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cu(n):
    return _ints([0] + [sum(n[:i + 1]) for i in range(len(n))])


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    n, H, Hkv, op = _lengths(case), case["H"], case["Hkv"], case["op"]
    st = dict(case=case, n=n, max_seqlen=max(n))
    if op in ("prompt", "train"):
        tok = sum(n)
        st["cu"] = _cu(n)
        q, k, v = (_randn(g, tok, h, D).bfloat16() for h in (H, Hkv, Hkv))
        if op == "prompt":
            st.update(q=q, k=k, v=v)
            return st
        # What the forward of the training step left for its backward.
        out, lse, qr, kr = _prompt(dict(st, q=q, k=k, v=v))
        st.update(qr=qr, kr=kr, v=v, out=out, lse=lse, dout=_randn(g, tok, H, D).bfloat16())
        return st
    # A cache whose pages were handed out in no order, with some to spare.
    ps = case["page"]
    used = [-(-x // ps) for x in n]
    n_pages = sum(used) + 3
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    width = max(used)
    at = torch.zeros((len(n), width), dtype=torch.int64)
    start = 0
    for i, u in enumerate(used):
        at[i, :u] = torch.arange(start, start + u)
        at[i, u:] = -1
        start += u
    at = at.cuda()
    st["table"] = torch.where(at >= 0, perm[at.clamp(min=0)], -1).to(torch.int32).contiguous()
    for name in ("k", "v"):
        x = _randn(g, n_pages, Hkv, ps, D)
        if case["fp8"]:
            e = torch.randint(118, 122, (n_pages, Hkv, ps), generator=g, device="cuda")
            st[name + "_pages"] = (x * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
            st[name + "_scale"] = e.to(torch.uint8)
        else:
            st[name + "_pages"] = x.bfloat16()
            st[name + "_scale"] = None
    if op == "append":
        rows = [1] * len(n) if case["step"] else n
        st["cu"] = _cu(rows)
        st["start"] = _ints([x - 1 for x in n] if case["step"] else [0] * len(n))
        st["rows"] = sum(rows)
        st["k"], st["v"] = (_randn(g, st["rows"], Hkv, D).bfloat16() for _ in range(2))
    elif op == "read":
        st["cu"], st["rows"] = _cu(n), sum(n)
        st["start"] = _ints([0] * len(n))
    else:
        st["lens"] = _ints(n)
        st["q"] = _randn(g, len(n), H, D).bfloat16()
    return st


# ----------------------------------------------------------- the plain forms
def _cos_sin(pos):
    """cos, sin of the angles of positions `pos`, formed in 64 bits (far positions)."""
    theta = BASE ** (-torch.arange(32, device=pos.device, dtype=torch.float64) / 32)
    a = pos.double()[:, None] * theta
    return a.cos().float(), a.sin().float()


def _rotate(x, pos, back=False):
    """RoPE of rows x [N, heads, 64] (fp32) at positions pos [N]."""
    c, s = (t[:, None, :] for t in _cos_sin(pos))
    if back:
        s = -s
    a, b = x[..., :32], x[..., 32:]
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def _rows(cu, nseq, rows):
    """The sequence of each packed row, and its place in it."""
    cu = cu.long()
    seq = torch.repeat_interleave(torch.arange(nseq, device=cu.device), cu[1:] - cu[:-1],
                                  output_size=rows)
    return seq, torch.arange(rows, device=cu.device) - cu[seq]


def _exponent(x):
    """The smallest e from -100 on with max |x| <= 448 * 2^e over the last axis."""
    m, e = torch.frexp(x.abs().amax(-1))  # max = m 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    return torch.where(m == 0, -100, e - 9 + (m > 0.875).to(torch.int32)).clamp(-100, 127)


def _append(st):
    c = st["case"]
    seq, at = _rows(st["cu"], c["nseq"], st["rows"])
    pos = at + st["start"].long()[seq]
    page, slot = st["table"].long()[seq, pos // c["page"]], pos % c["page"]
    for name, x in (("k", _rotate(st["k"].float(), pos)), ("v", st["v"].float())):
        pages = st[name + "_pages"]
        if c["fp8"]:
            e = _exponent(x)
            x8 = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn)
            pages.view(torch.uint8)[page, :, slot] = x8.view(torch.uint8)
            st[name + "_scale"][page, :, slot] = (e + 127).to(torch.uint8)
        else:
            pages[page, :, slot] = x.bfloat16()


def _pages(st, name, page, slot):
    """Rows of the cache in fp32: [..., Hkv, 64] for page, slot of any one shape."""
    x = st[name + "_pages"]
    if not st["case"]["fp8"]:
        return x[page, :, slot].float()
    e = st[name + "_scale"][page, :, slot].float() - 127
    return x.view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).float() * \
        torch.exp2(e)[..., None]


def _read(st):
    c = st["case"]
    seq, at = _rows(st["cu"], c["nseq"], st["rows"])
    pos = at + st["start"].long()[seq]
    page, slot = st["table"].long()[seq, pos // c["page"]], pos % c["page"]
    return _pages(st, "k", page, slot).bfloat16(), _pages(st, "v", page, slot).bfloat16()


def _decode(st):
    c = st["case"]
    B, H, Hkv = c["nseq"], c["H"], c["Hkv"]
    n = st["lens"].long()
    pos = torch.arange(st["max_seqlen"], device=n.device)
    page = st["table"].long()[:, pos // c["page"]].clamp(min=0)
    slot = (pos % c["page"]).expand(B, -1)
    q = _rotate(st["q"].float(), n - 1).bfloat16().float()  # the operator's q' is bf16
    k = _pages(st, "k", page, slot).permute(0, 2, 3, 1)
    s = torch.matmul(q.view(B, Hkv, H // Hkv, D), k) * SCALE
    s.masked_fill_((pos >= n[:, None])[:, None, None, :], -math.inf)
    lse = torch.logsumexp(s, -1, keepdim=True)
    o = torch.matmul(torch.exp(s - lse), _pages(st, "v", page, slot).permute(0, 2, 1, 3))
    return o.reshape(B, H, D).bfloat16(), lse.reshape(B, H)


def _padded(x, cu, T, heads):
    """Packed rows as [nseq, Hkv, heads of each, T, 64] in fp32 (rows past an end: any row)."""
    at = (cu.long()[:-1, None] + torch.arange(T, device=x.device)).clamp(max=x.shape[0] - 1)
    x = x.float()[at]
    return x.view(*at.shape, heads, -1, D).permute(0, 2, 3, 1, 4)


def _hidden(st):
    """[nseq, 1, 1, T, T]: later keys, and every key of rows past a sequence's end."""
    cu, t = st["cu"].long(), torch.arange(st["max_seqlen"], device="cuda")
    end = t >= (cu[1:] - cu[:-1])[:, None]
    return ((t[None, :] > t[:, None])[None] | end[:, :, None])[:, None, None]


def _prompt(st):
    c = st["case"]
    H, Hkv, T = c["H"], c["Hkv"], st["max_seqlen"]
    seq, pos = _rows(st["cu"], c["nseq"], st["q"].shape[0])
    qr, kr = (_rotate(st[x].float(), pos).bfloat16() for x in ("q", "k"))
    s = torch.matmul(_padded(qr, st["cu"], T, Hkv), _padded(kr, st["cu"], T, Hkv).mT)
    s.mul_(SCALE).masked_fill_(_hidden(st), -math.inf)
    lse = torch.logsumexp(s, -1)
    o = torch.matmul(s.sub_(lse[..., None]).exp_(), _padded(st["v"], st["cu"], T, Hkv))
    o = o.flatten(1, 2)[seq, :, pos]
    return o.bfloat16(), lse.flatten(1, 2)[seq, :, pos].T.contiguous(), qr, kr


def _train(st):
    c = st["case"]
    H, Hkv, T, cu = c["H"], c["Hkv"], st["max_seqlen"], st["cu"]
    seq, pos = _rows(cu, c["nseq"], st["qr"].shape[0])
    q, k, v, do = (_padded(st[x], cu, T, Hkv) for x in ("qr", "kr", "v", "dout"))
    lse = _padded(st["lse"].T[..., None].expand(-1, -1, D), cu, T, Hkv)[..., :1]
    delta = (do * _padded(st["out"], cu, T, Hkv)).sum(-1, keepdim=True)
    p = torch.matmul(q, k.mT).mul_(SCALE).sub_(lse).masked_fill_(_hidden(st), -math.inf).exp_()
    dv = torch.matmul(p.mT, do).sum(2)
    ds = torch.matmul(do, v.mT).sub_(delta).mul_(p).mul_(SCALE)
    dq = torch.matmul(ds, k).flatten(1, 2)[seq, :, pos]
    dk = torch.matmul(ds.mT, q).sum(2)[seq, :, pos]
    return (_rotate(dq, pos, back=True).bfloat16(), _rotate(dk, pos, back=True).bfloat16(),
            dv[seq, :, pos].bfloat16())


# ------------------------------------------------------------------- one pass
def _cache(st):
    """The cache after a call, as the values that its pages and scales stand for."""
    got = dict(k=st["k_pages"], v=st["v_pages"])
    if st["case"]["fp8"]:
        got.update(k_scale=st["k_scale"].view(torch.float8_e8m0fnu),
                   v_scale=st["v_scale"].view(torch.float8_e8m0fnu))
    return got


def run(state):
    st, op = state, state["case"]["op"]
    if not own:
        if op == "append":
            _append(st)
            return _cache(st)
        got = dict(read=_read, decode=_decode, prompt=_prompt, train=_train)[op](st)
    else:
        from causal_self_attention_gb300 import ne_attn as na
        if op == "append":
            na.ne_kv_append(st["k"], st["v"], st["cu"], st["start"], st["k_pages"],
                            st["v_pages"], st["table"], st["max_seqlen"], st["k_scale"],
                            st["v_scale"], rope_base=BASE)
            return _cache(st)
        if op == "read":
            got = na.ne_kv_read(st["k_pages"], st["v_pages"], st["table"], st["cu"], st["start"],
                                st["rows"], st["k_scale"], st["v_scale"])
        elif op == "decode":
            got = na.ne_attn_decode_paged(st["q"], st["k_pages"], st["v_pages"], st["table"],
                                          st["lens"], st["max_seqlen"], st["k_scale"],
                                          st["v_scale"], rope_base=BASE, scale=SCALE)
        elif op == "prompt":
            got = na.ne_attn_gqa_varlen_fwd(st["q"], st["k"], st["v"], st["cu"],
                                            st["max_seqlen"], rope_base=BASE, scale=SCALE)
        else:
            got = na.ne_attn_gqa_varlen_bwd(st["qr"], st["kr"], st["v"], st["out"], st["dout"],
                                            st["lse"], st["cu"], st["max_seqlen"],
                                            rope_base=BASE, scale=SCALE)
    names = dict(read=("k", "v"), decode=("out", "lse"), prompt=("out", "lse", "qr", "kr"),
                 train=("dq", "dk", "dv"))[op]
    return dict(zip(names, got))


# ------------------------------------------- the operators' values in 64 bits
def _turn(x, first, sign=1.0):
    """Rows x [n, heads, 64] in 64 bits turned by the angles of positions first, first + 1, ..."""
    i = torch.arange(64, device=x.device)
    angle = (first + torch.arange(x.shape[0], device=x.device, dtype=torch.float64))[:, None] \
        * torch.pow(torch.tensor(BASE, dtype=torch.float64, device=x.device), -(i % 32) / 32.0)
    swapped = torch.where(i < 32, -x.roll(-32, -1), x.roll(32, -1))
    return x * angle.cos()[:, None] + sign * swapped * angle.sin()[:, None]


def _bf16(x):
    """64-bit values rounded to bf16 (once: not by way of 32 bits), in 64 bits."""
    m, e = torch.frexp(x)
    return torch.ldexp(torch.round(m * 256), e.double() - 8)


def _sequence(st, name, s):
    """The cached rows of sequence s, all heads, in 64 bits: [n, Hkv, 64]."""
    ps, n = st["case"]["page"], st["n"][s]
    ids = st["table"][s, :-(-n // ps)].long()
    x = st[name + "_pages"][ids].double()
    if st["case"]["fp8"]:
        x = x * torch.pow(2.0, st[name + "_scale"][ids].double() - 127)[..., None]
    return x.transpose(1, 2).reshape(-1, st["case"]["Hkv"], D)[:n]


def exact(case, seed):
    st = prepare(case, seed)
    op, n, H, Hkv = case["op"], st["n"], case["H"], case["Hkv"]
    G = H // Hkv
    if op == "append":
        got, cu, start, ps = {}, st["cu"].tolist(), st["start"].tolist(), case["page"]
        for name in ("k", "v"):
            pages = st[name + "_pages"].double()
            two = torch.pow(2.0, st[name + "_scale"].double() - 127) if case["fp8"] else None
            for s in range(len(n)):
                x = st[name][cu[s]:cu[s + 1]].double()
                x = _turn(x, start[s]) if name == "k" else x
                at = start[s] + torch.arange(x.shape[0], device="cuda")
                ids = st["table"][s].long()[at // ps]
                if case["fp8"]:  # 64-bit values before their rounding to e4m3
                    amax = x.abs().amax(-1)
                    e = torch.ceil(torch.log2(amax / 448)).clamp(-100, 127)
                    e = torch.where(amax <= 448 * torch.pow(2.0, e - 1), e - 1, e)
                    two[ids, :, at % ps] = torch.pow(2.0, e)
                    x = x / torch.pow(2.0, e)[..., None]
                pages[ids, :, at % ps] = x
            got[name] = pages
            if case["fp8"]:
                got[name + "_scale"] = two
        return got
    if op == "read":
        return {x: torch.cat([_sequence(st, x, s) for s in range(len(n))]) for x in ("k", "v")}
    if op == "decode":
        out = torch.zeros((len(n), H, D), dtype=torch.float64, device="cuda")
        lse = torch.zeros((len(n), H), dtype=torch.float64, device="cuda")
        for s in range(len(n)):
            q = _bf16(_turn(st["q"][s:s + 1].double(), n[s] - 1))[0]
            k, v = (_sequence(st, x, s) for x in ("k", "v"))
            for g in range(Hkv):
                z = SCALE * (q[g * G:(g + 1) * G] @ k[:, g].T)
                top = z.amax(1, keepdim=True)
                w = torch.exp(z - top)
                lse[s, g * G:(g + 1) * G] = (top + w.sum(1, keepdim=True).log())[:, 0]
                out[s, g * G:(g + 1) * G] = (w @ v[:, g]) / w.sum(1, keepdim=True)
        return dict(out=out, lse=lse)
    cu, tok = st["cu"].tolist(), sum(n)
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    if op == "prompt":
        got = dict(out=new(tok, H, D), lse=new(H, tok), qr=new(tok, H, D), kr=new(tok, Hkv, D))
    else:
        got = dict(dq=new(tok, H, D), dk=new(tok, Hkv, D), dv=new(tok, Hkv, D))
    for s in range(len(n)):
        r = slice(cu[s], cu[s + 1])
        later = torch.ones((n[s], n[s]), dtype=torch.bool, device="cuda").triu(1)
        if op == "prompt":
            got["qr"][r], got["kr"][r] = (_turn(st[x][r].double(), 0) for x in ("q", "k"))
            q, k, v = _bf16(got["qr"][r]), _bf16(got["kr"][r]), st["v"][r].double()
        else:
            q, k, v, o, do = (st[x][r].double() for x in ("qr", "kr", "v", "out", "dout"))
        for h in range(H):
            z = (SCALE * (q[:, h] @ k[:, h // G].T)).masked_fill_(later, -math.inf)
            if op == "prompt":
                top = z.amax(1, keepdim=True)
                z = z.sub_(top).exp_()
                total = z.sum(1, keepdim=True)
                got["lse"][h, r] = (top + total.log())[:, 0]
                got["out"][r, h] = (z @ v[:, h // G]) / total
                continue
            z = z.sub_(st["lse"][h, r].double()[:, None]).exp_()
            got["dv"][r, h // G] += z.T @ do[:, h]
            z *= do[:, h] @ v[:, h // G].T - (do[:, h] * o[:, h]).sum(1, keepdim=True)
            got["dq"][r, h] = SCALE * (z @ k[:, h // G])
            got["dk"][r, h // G] += SCALE * (z.T @ q[:, h])
        if op == "train":
            got["dq"][r], got["dk"][r] = (_turn(got[x][r], 0, -1.0) for x in ("dq", "dk"))
    return got

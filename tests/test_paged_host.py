"""The grouped-head and paged-cache operators without a GPU: host argument
checks (every one returns before anything touches a device), the placement of
rows in the pages, the binding's checks, and the plain 64-bit implementations
that the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

import grouped
from grouped import D, F64, Cache


@pytest.fixture(scope="module")
def lib():
    from causal_self_attention_gb300 import build, ne_attn
    build.build()
    return ne_attn.lib()


P = ctypes.c_void_p
FAKE = P(0x10000)  # never dereferenced: every call below fails its host check first
INVALID, UNSUPPORTED, MISALIGNED = 1, 2, 3


def _append(lib, **kw):
    a = dict(k=FAKE, v=FAKE, cu=FAKE, start=FAKE, nseq=2, n_tot=10, Hkv=2, D=64, base=1e4, ty=1,
             kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, table=FAKE, mp=4, np=8, ps=16, ms=64)
    a.update(kw)
    return lib.ne_kv_append(*a.values(), None)


def _read(lib, **kw):
    a = dict(ty=1, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, table=FAKE, mp=4, np=8, ps=16, ms=64,
             cu=FAKE, start=FAKE, nseq=2, n_tot=10, Hkv=2, D=64, k=FAKE, v=FAKE)
    a.update(kw)
    return lib.ne_kv_read(*a.values(), None)


def _decode(lib, ws=None, ws_bytes=0, **kw):
    a = dict(q=FAKE, ty=1, kp=FAKE, vp=FAKE, ks=FAKE, vs=FAKE, table=FAKE, mp=4, np=8, ps=16,
             ms=64, lens=FAKE, B=2, H=4, Hkv=2, D=64, base=1e4, scale=0.125, out=FAKE, lse=FAKE)
    a.update(kw)
    return lib.ne_attn_decode_paged(*a.values(), ws, ws_bytes, None)


CACHE_REFUSALS = [
    (dict(kp=None), INVALID), (dict(vp=None), INVALID), (dict(table=None), INVALID),
    (dict(ks=None), INVALID), (dict(vs=None), INVALID), (dict(D=128), UNSUPPORTED),
    (dict(ty=2), UNSUPPORTED), (dict(ty=-1), UNSUPPORTED), (dict(ps=8), UNSUPPORTED),
    (dict(ps=48), UNSUPPORTED), (dict(ps=512), UNSUPPORTED), (dict(ps=0), UNSUPPORTED),
    (dict(ps=-16), UNSUPPORTED), (dict(mp=0), INVALID), (dict(np=0), INVALID),
    (dict(ms=0), INVALID), (dict(ms=65), INVALID),  # more than max_pages pages hold
    (dict(np=1 << 26), INVALID),                    # pool rows beyond 31 bits
    (dict(mp=1 << 30, ms=65535 * 128 + 1), INVALID),
    (dict(kp=P(0x10008)), MISALIGNED), (dict(vp=P(0x10004)), MISALIGNED),
    (dict(ks=P(0x10008)), MISALIGNED), (dict(vs=P(0x10001)), MISALIGNED),
    (dict(table=P(0x10002)), MISALIGNED),
]


@pytest.mark.parametrize("kw,code", CACHE_REFUSALS)
def test_cache_refusals(lib, kw, code):
    for call in (_append, _read, _decode):
        assert call(lib, **kw) == code


ROW_REFUSALS = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(cu=None), INVALID),
    (dict(start=None), INVALID), (dict(nseq=0), INVALID), (dict(n_tot=0), INVALID),
    (dict(n_tot=-1), INVALID), (dict(Hkv=0), INVALID), (dict(n_tot=1 << 30), INVALID),
    (dict(k=P(0x10008)), MISALIGNED), (dict(v=P(0x10002)), MISALIGNED),
    (dict(cu=P(0x10001)), MISALIGNED), (dict(start=P(0x10002)), MISALIGNED),
]


@pytest.mark.parametrize("kw,code", ROW_REFUSALS)
def test_row_refusals(lib, kw, code):
    for call in (_append, _read):
        assert call(lib, **kw) == code


def test_append_refuses_bad_rope_bases(lib):
    for base in (-1.0, math.nan, math.inf):
        assert _append(lib, base=base) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(lens=None), INVALID), (dict(out=None), INVALID),
    (dict(lse=None), INVALID), (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(H=3), INVALID),
    (dict(B=65536), INVALID), (dict(H=65536), INVALID), (dict(Hkv=0), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=math.nan), INVALID), (dict(base=-2.0), INVALID),
    (dict(base=math.inf), INVALID), (dict(q=P(0x10008)), MISALIGNED),
    (dict(out=P(0x10008)), MISALIGNED), (dict(lens=P(0x10002)), MISALIGNED),
    (dict(lse=P(0x10001)), MISALIGNED), (dict(ws=FAKE, ws_bytes=16), INVALID),
    (dict(ws=P(0x10008), ws_bytes=1 << 30), MISALIGNED),
])
def test_decode_refusals(lib, kw, code):
    assert _decode(lib, **kw) == code


def _gqa(lib, backward, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE)
    if backward:
        a.update(out=FAKE, do=FAKE, lse=FAKE)
    a.update(cu=FAKE, nseq=2, n=100, mx=64, H=4, Hkv=2, D=64, base=1e4, scale=0.125)
    a.update(dict(dq=FAKE, dk=FAKE, dv=FAKE, ws=None, wb=0) if backward else
             dict(out=FAKE, lse=FAKE, qr=FAKE, kr=FAKE))
    assert set(kw) <= set(a)
    a.update(kw)
    fn = lib.ne_attn_gqa_varlen_bwd if backward else lib.ne_attn_gqa_varlen_fwd
    return fn(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(cu=None), INVALID), (dict(H=3), INVALID),
    (dict(Hkv=0), INVALID), (dict(H=0), INVALID), (dict(Hkv=-2), INVALID), (dict(nseq=0), INVALID),
    (dict(nseq=65536), INVALID), (dict(n=0), INVALID), (dict(mx=0), INVALID),
    (dict(D=128), UNSUPPORTED), (dict(base=0.0), INVALID), (dict(base=math.nan), INVALID),
    (dict(scale=-1.0), INVALID), (dict(k=P(0x10004)), MISALIGNED),
    (dict(nseq=65535, mx=65535 * 128), INVALID),  # work items beyond 31 bits
])
def test_gqa_refusals(lib, kw, code):
    assert _gqa(lib, False, **kw) == code
    assert _gqa(lib, True, **kw) == code


def test_gqa_output_and_workspace_refusals(lib):
    assert _gqa(lib, False, qr=None) == INVALID
    assert _gqa(lib, False, kr=P(0x10008)) == MISALIGNED
    assert _gqa(lib, True, dk=None) == INVALID
    assert _gqa(lib, True, dv=P(0x10008)) == MISALIGNED
    assert _gqa(lib, True, ws=FAKE, wb=16) == INVALID
    assert _gqa(lib, True, ws=P(0x10010), wb=1 << 40) == MISALIGNED


def test_workspace_sizes(lib):
    from causal_self_attention_gb300 import ne_attn as na
    assert na.ne_attn_gqa_bwd_workspace_bytes(100, 64, 4, 3) == 0
    assert na.ne_attn_gqa_bwd_workspace_bytes(100, 64, 4, 2, 128) == 0
    assert na.ne_attn_gqa_bwd_workspace_bytes(0, 64, 4, 2) == 0
    assert na.ne_attn_gqa_bwd_workspace_bytes(8192, 1024, 12, 12) == \
        na.ne_attn_bwd_workspace_bytes(8192, 12)
    # dQ' and D of 12 heads; 8 x 1024 with 3 query heads per key/value head needs no split
    assert na.ne_attn_gqa_bwd_workspace_bytes(8192, 1024, 12, 4) == 8192 * 12 * 260
    # one short sequence: one query head per unit, fp32 dK' and dV of each
    assert na.ne_attn_gqa_bwd_workspace_bytes(1024, 1024, 12, 4) == \
        1024 * 12 * 260 + 2 * 3 * 1024 * 4 * 256
    assert na.ne_attn_decode_paged_workspace_bytes(2, 4, 3, 100) == 0
    assert na.ne_attn_decode_paged_workspace_bytes(0, 4, 2, 100) == 0
    assert na.ne_attn_decode_paged_workspace_bytes(2, 4, 2, 100) > 0


# --------------------------------------------------------------- placement

def _place(c, lens, start, pair, max_seqlen, table=None):
    from causal_self_attention_gb300 import ne_attn as na
    cu = torch.tensor([0] + [sum(lens[:i + 1]) for i in range(len(lens))], dtype=torch.int32)
    return na.ne_debug_kv_place(cu, torch.tensor(start, dtype=torch.int32),
                                c.table if table is None else table, c.Hkv, c.n_pages, c.page,
                                max_seqlen, pair)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_every_row_is_placed_where_the_table_says(lib, page):
    rows, start = [0, 3, 0, 0, 40, 1, 300, 0], [0, 14, 9, 0, 255, 16, 1, 5]
    c = Cache([r + s for r, s in zip(rows, start)], 3, page, False, seed=1, device="cpu")
    ms = 400 if page < 256 else 500
    r = 0
    for s, n in enumerate(rows):
        pages, slots = c.where(s, start[s] + torch.arange(n))
        for i in range(n):
            for h in range(3):
                code, src, slot, pos = _place(c, rows, start, r * 3 + h, ms)
                assert (code, src, pos) == (0, (r * 3 + h) * 64, start[s] + i)
                assert slot == (int(pages[i]) * 3 + h) * page + int(slots[i])
            r += 1
    for pair in (r * 3, r * 3 + 1, r * 3 + 1000):  # behind the last sequence
        assert _place(c, rows, start, pair, ms)[0] == -1


def test_bad_positions_pages_and_offsets_are_never_placed(lib):
    c = Cache([40, 40], 2, 16, False, seed=2, device="cpu")
    for page in (-1, c.n_pages, 2 ** 31 - 1, -2 ** 31):
        t = c.table.clone()
        t[1, 1] = page
        for i in range(40):
            code = _place(c, [0, 40], [0, 0], 2 * i, 40, t)[0]
            assert code == (2 if 16 <= i < 32 else 0)
    for start in (-1, 40, 2 ** 31 - 1, -2 ** 31):
        assert _place(c, [1, 0], [start, 0], 0, 40)[0] == 1
    assert _place(c, [1, 0], [39, 0], 0, 40)[0] == 0
    # cu_seqlens that is not nondecreasing: some sequence or none, nothing outside.
    from causal_self_attention_gb300 import ne_attn as na
    for cu in ([5, 2, 9], [0, 9, 3], [0, -4, 8], [-3, 2, 6], [0, 0, 0]):
        cu = torch.tensor(cu, dtype=torch.int32)
        for r in range(10):
            code, src, slot, pos = na.ne_debug_kv_place(
                cu, torch.zeros(2, dtype=torch.int32), c.table, 2, c.n_pages, 16, 40, 2 * r)
            assert code in (-1, 0, 1, 2)
            assert code != 0 or (0 <= slot < c.n_pages * 2 * 16 and src == 2 * r * 64)


def test_offsets_past_32_bits(lib):
    """A pool of 2^31 bytes and more: the row index times 64 leaves 32 bits."""
    from causal_self_attention_gb300 import ne_attn as na
    n_pages = (2 ** 31 - 512) // (8 * 256)
    table = torch.tensor([[n_pages - 1]], dtype=torch.int32)
    code, src, slot, pos = na.ne_debug_kv_place(
        torch.tensor([0, 256], dtype=torch.int32), torch.zeros(1, dtype=torch.int32), table, 8,
        n_pages, 256, 256, 255 * 8 + 7)
    assert code == 0 and slot == ((n_pages - 1) * 8 + 7) * 256 + 255
    code, src, _, _ = na.ne_debug_kv_place(
        torch.tensor([0, 2 ** 28], dtype=torch.int32), torch.tensor([-2 ** 28 + 5], dtype=torch.int32),
        table, 8, n_pages, 256, 256, (2 ** 28 - 1) * 8)
    assert code == 0 and src == (2 ** 28 - 1) * 8 * 64


# ------------------------------------------------------------- the binding

def test_binding_refuses_before_the_library(monkeypatch):
    from causal_self_attention_gb300 import ne_attn as na
    monkeypatch.setattr(na, "lib", lambda: pytest.fail("the library was called"))
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):  # CPU tensors
        na.ne_attn_gqa_varlen_fwd(bf(4, 4, 64), bf(4, 2, 64), bf(4, 2, 64), i(2), 4)
    with pytest.raises(ValueError):
        na.ne_kv_append(bf(1, 2, 64), bf(1, 2, 64), i(2), i(1), bf(2, 2, 16, 64), bf(2, 2, 16, 64),
                        i(1, 2), 16)
    with pytest.raises(ValueError):
        na.ne_kv_read(bf(2, 2, 16, 64), bf(2, 2, 16, 64), i(1, 2), i(2), i(1), 1)
    with pytest.raises(ValueError):
        na.ne_attn_decode_paged(bf(1, 4, 64), bf(2, 2, 16, 64), bf(2, 2, 16, 64), i(1, 2), i(1), 16)
    # The device checks aside (a stand-in for CUDA tensors), shapes and types.
    monkeypatch.setattr(na, "_need_on", lambda t, dtype, dev, name: t.dtype == dtype or
                        (_ for _ in ()).throw(ValueError(name)))
    monkeypatch.setattr(na, "_device", lambda t, name: -1)
    e4 = lambda *s: torch.zeros(s).to(torch.float8_e4m3fn)  # noqa: E731
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    bad = [
        lambda: na.ne_attn_gqa_varlen_fwd(bf(4, 3, 64), bf(4, 2, 64), bf(4, 2, 64), i(2), 4),
        lambda: na.ne_attn_gqa_varlen_fwd(bf(4, 4, 64), bf(5, 2, 64), bf(5, 2, 64), i(2), 4),
        lambda: na.ne_attn_gqa_varlen_fwd(bf(4, 4, 64), bf(4, 2, 64), bf(4, 1, 64), i(2), 4),
        lambda: na.ne_attn_gqa_varlen_fwd(bf(4, 4, 64), bf(4, 2, 64), bf(4, 2, 64), i(1), 4),
        lambda: na._paged(e4(2, 2, 16, 64), e4(2, 2, 16, 64), None, u8(2, 2, 16), i(1, 2), 1, -1),
        lambda: na._paged(e4(2, 2, 16, 64), e4(2, 2, 16, 64), u8(2, 2, 8), u8(2, 2, 16), i(1, 2), 1, -1),
        lambda: na._paged(bf(2, 2, 16, 64), bf(2, 2, 16, 64), u8(2, 2, 16), None, i(1, 2), 1, -1),
        lambda: na._paged(bf(2, 2, 16, 64), e4(2, 2, 16, 64), None, None, i(1, 2), 1, -1),
        lambda: na._paged(bf(2, 2, 16, 64), bf(3, 2, 16, 64), None, None, i(1, 2), 1, -1),
        lambda: na._paged(bf(2, 2, 16, 32), bf(2, 2, 16, 32), None, None, i(1, 2), 1, -1),
        lambda: na._paged(bf(2, 2, 16, 64), bf(2, 2, 16, 64), None, None, i(2, 2), 1, -1),
        lambda: na._paged(bf(2, 2, 16, 64).half(), bf(2, 2, 16, 64).half(), None, None, i(1, 2), 1, -1),
        lambda: na._row_places(i(3), i(1), -1),
        lambda: na._given(bf(2, 3), (2, 4), torch.bfloat16, -1, "out"),
    ]
    for n, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"refusal {n} did not happen")


# ------------------------------------------------- the plain implementations

def test_plain_quantisation_is_the_cast_of_the_type():
    g = torch.Generator().manual_seed(1)
    x = torch.randn((200, 64), generator=g, dtype=F64) * torch.exp2(
        torch.randint(-20, 20, (200, 1), generator=g).to(F64))
    x8, e = grouped.quantise(x)
    amax = x.abs().amax(-1)
    assert bool((amax <= 448 * torch.exp2(e)).all()) and bool((amax > 448 * torch.exp2(e - 1)).all())
    cast = (x.to(torch.bfloat16).to(F64) * torch.exp2(-e)[:, None]).float()
    x8, _ = grouped.quantise(x.to(torch.bfloat16).to(F64))
    assert torch.equal(x8, cast.to(torch.float8_e4m3fn).to(F64))
    assert grouped.quantise(torch.zeros((1, 64), dtype=F64))[1].item() == -100


@pytest.mark.parametrize("H,Hkv", [(4, 2), (3, 1), (2, 2)])
def test_plain_gradients_against_differences(H, Hkv):
    """The formulas that the kernels are held to, against centred differences of
    the forward: through the rotation, with heads shared."""
    g = torch.Generator().manual_seed(2)
    n, scale, h = 9, 0.125, 1e-6
    pos = torch.arange(n)
    q, k, v = (torch.randn((n, x, D), generator=g, dtype=F64) for x in (H, Hkv, Hkv))
    do = torch.randn((n, H, D), generator=g, dtype=F64)

    def forward(q, k, v):
        return grouped.attention(grouped.rotate(q, pos), grouped.rotate(k, pos), v, scale)

    out, lse, _, _ = forward(q, k, v)
    (dq, dk, dv), _ = grouped.attention_grads(grouped.rotate(q, pos), grouped.rotate(k, pos), v,
                                              out, do, lse, scale)
    grads = (grouped.rotate(dq, pos, back=True), grouped.rotate(dk, pos, back=True), dv)
    for i, x in enumerate((q, k, v)):
        for _ in range(12):
            at = tuple(int(torch.randint(0, s, (1,), generator=g)) for s in x.shape)
            args = [t.clone() for t in (q, k, v)]
            args[i][at] += h
            up = (forward(*args)[0] * do).sum()
            args[i][at] -= 2 * h
            down = (forward(*args)[0] * do).sum()
            # Second-order error h^2 and 64-bit rounding over h: below 1e-7 here.
            assert abs(float((up - down) / (2 * h) - grads[i][at])) < 1e-7 * (1 + H * n)

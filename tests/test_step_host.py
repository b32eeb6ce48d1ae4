"""A generation step's operators without a GPU: refusals of arguments (every one returns
before anything touches a device), the binding's checks, and the plain implementations
that the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

import step
from grouped import D, F64, rotate

P = ctypes.c_void_p
FAKE = P(0x10000)  # never dereferenced: every call below fails its host check first
INVALID, UNSUPPORTED, MISALIGNED = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from causal_self_attention_gb300 import build, ne_attn
    build.build()
    return ne_attn.lib()


def _call(fn, a, kw):
    assert set(kw) <= set(a)
    a.update(kw)
    return fn(*a.values(), None)


def _fwd(lib, **kw):
    return _call(lib.ne_qk_norm_rope_fwd, dict(
        q=FAKE, k=FAKE, qs=256, ks=128, qw=FAKE, kw=FAKE, pos=FAKE, n=10, H=4, Hkv=2, D=64, ms=64,
        eps=1e-5, base=1e4, qr=FAKE, kr=FAKE), kw)


def _bwd(lib, ws=None, ws_bytes=0, **kw):
    a = dict(dqr=FAKE, dkr=FAKE, q=FAKE, k=FAKE, qs=256, ks=128, qw=FAKE, kw=FAKE, pos=FAKE, n=10,
             H=4, Hkv=2, D=64, ms=64, eps=1e-5, base=1e4, dq=FAKE, dk=FAKE, dqs=256, dks=128,
             dqw=FAKE, dkw=FAKE, ws=ws, wb=ws_bytes)
    return _call(lib.ne_qk_norm_rope_bwd, a, kw)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(qw=None), INVALID),
    (dict(kw=None), INVALID), (dict(pos=None), INVALID), (dict(n=0), INVALID),
    (dict(n=-1), INVALID), (dict(H=0), INVALID), (dict(Hkv=0), INVALID), (dict(D=128), UNSUPPORTED),
    (dict(ms=0), INVALID), (dict(ms=65535 * 128 + 1), INVALID), (dict(n=1 << 29), INVALID),
    (dict(ms=2 ** 31 - 1), INVALID), (dict(H=2 ** 31 - 1, qs=64 * (2 ** 31 - 1)), INVALID),
    (dict(eps=-1e-5), INVALID), (dict(eps=math.nan), INVALID), (dict(base=-1.0), INVALID),
    (dict(base=math.inf), INVALID), (dict(qs=248), INVALID), (dict(ks=64), INVALID),
    (dict(qs=0), INVALID), (dict(qs=-256), INVALID), (dict(qs=(1 << 31) + 8), INVALID),
    (dict(qs=260), MISALIGNED), (dict(ks=129), MISALIGNED), (dict(q=P(0x10008)), MISALIGNED),
    (dict(k=P(0x10002)), MISALIGNED), (dict(qw=P(0x10004)), MISALIGNED),
    (dict(kw=P(0x10008)), MISALIGNED), (dict(pos=P(0x10002)), MISALIGNED),
])
def test_norm_refusals(lib, kw, code):
    assert _fwd(lib, **kw) == code
    assert _bwd(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [(dict(qr=None), INVALID), (dict(kr=None), INVALID),
                                     (dict(qr=P(0x10008)), MISALIGNED),
                                     (dict(kr=P(0x10002)), MISALIGNED)])
def test_norm_forward_refusals(lib, kw, code):
    assert _fwd(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dqr=None), INVALID), (dict(dkr=None), INVALID), (dict(dq=None), INVALID),
    (dict(dk=None), INVALID), (dict(dqw=None), INVALID), (dict(dkw=None), INVALID),
    (dict(dqs=192), INVALID), (dict(dks=0), INVALID), (dict(dqs=257), MISALIGNED),
    (dict(dq=P(0x10008)), MISALIGNED), (dict(dqr=P(0x10002)), MISALIGNED),
    (dict(dkw=P(0x10004)), MISALIGNED), (dict(ws=FAKE, ws_bytes=16), INVALID),
    (dict(ws=P(0x10008), ws_bytes=1 << 30), MISALIGNED),
])
def test_norm_backward_refusals(lib, kw, code):
    assert _bwd(lib, **kw) == code


def _reserve(lib, **kw):
    return _call(lib.ne_kv_reserve, dict(
        new=FAKE, lens=FAKE, nseq=3, table=FAKE, mp=4, free=FAKE, n_free=FAKE, np=8, ps=16, ms=64,
        n_tot=10, cu=FAKE, start=FAKE, pos=FAKE, slots=FAKE, lo=FAKE, fo=FAKE), kw)


def _release(lib, **kw):
    return _call(lib.ne_kv_release, dict(fin=FAKE, lens=FAKE, nseq=3, table=FAKE, mp=4, free=FAKE,
                                         n_free=FAKE, np=8, ps=16, ms=64), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(lens=None), INVALID), (dict(table=None), INVALID), (dict(free=None), INVALID),
    (dict(n_free=None), INVALID), (dict(nseq=0), INVALID), (dict(nseq=16385), INVALID),
    (dict(mp=0), INVALID), (dict(np=0), INVALID), (dict(ms=0), INVALID), (dict(ms=65), INVALID),
    (dict(ps=8), UNSUPPORTED), (dict(ps=48), UNSUPPORTED), (dict(ps=512), UNSUPPORTED),
    (dict(ps=-16), UNSUPPORTED), (dict(np=1 << 27), INVALID),
    (dict(mp=1 << 30, ms=65535 * 128 + 1), INVALID), (dict(lens=P(0x10002)), MISALIGNED),
    (dict(table=P(0x10001)), MISALIGNED), (dict(free=P(0x10002)), MISALIGNED),
    (dict(n_free=P(0x10002)), MISALIGNED),
])
def test_pages_refusals(lib, kw, code):
    assert _reserve(lib, **kw) == code
    assert _release(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(new=None), INVALID), (dict(lo=None), INVALID), (dict(fo=None), INVALID),
    (dict(n_tot=-1), INVALID), (dict(n_tot=(1 << 30) + 1), INVALID), (dict(new=P(0x10002)), MISALIGNED),
    (dict(cu=P(0x10002)), MISALIGNED), (dict(start=P(0x10001)), MISALIGNED),
    (dict(pos=P(0x10002)), MISALIGNED), (dict(slots=P(0x10002)), MISALIGNED),
    (dict(lo=P(0x10002)), MISALIGNED), (dict(fo=P(0x10002)), MISALIGNED),
])
def test_reserve_refusals(lib, kw, code):
    assert _reserve(lib, **kw) == code


def test_release_refusals(lib):
    assert _release(lib, fin=None) == INVALID


@pytest.mark.parametrize("ks", [None, P(0x10008)])
def test_four_bit_cache_refusals(lib, ks):
    """The scales of a 4-bit cache, as those of an 8-bit one."""
    code = INVALID if ks is None else MISALIGNED
    cache = (4, FAKE, FAKE, ks, FAKE, FAKE, 4, 8, 16, 64)
    assert lib.ne_kv_append(FAKE, FAKE, FAKE, FAKE, 2, 10, 2, 64, 0.0, 4, FAKE, FAKE, ks, FAKE, FAKE,
                            4, 8, 16, 64, None) == code
    assert lib.ne_kv_read(*cache, FAKE, FAKE, 2, 10, 2, 64, FAKE, FAKE, None) == code
    assert lib.ne_attn_decode_paged(FAKE, *cache, FAKE, 2, 4, 2, 64, 0.0, 0.125, FAKE, FAKE, None, 0,
                                    None) == code
    for ty in (2, 3, 5, -1):
        assert lib.ne_kv_read(ty, *cache[1:], FAKE, FAKE, 2, 10, 2, 64, FAKE, FAKE,
                              None) == UNSUPPORTED


def _rotated(lib, backward, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE)
    if backward:
        a.update(out=FAKE, do=FAKE, lse=FAKE)
    a.update(cu=FAKE, nseq=2, n=100, mx=64, H=4, Hkv=2, D=64, scale=0.125)
    a.update(dict(dq=FAKE, dk=FAKE, dv=FAKE, ws=None, wb=0) if backward else dict(out=FAKE, lse=FAKE))
    fn = lib.ne_attn_gqa_varlen_bwd_rotated if backward else lib.ne_attn_gqa_varlen_fwd_rotated
    return _call(fn, a, kw)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(cu=None), INVALID), (dict(H=3), INVALID), (dict(Hkv=0), INVALID),
    (dict(nseq=0), INVALID), (dict(nseq=65536), INVALID), (dict(n=0), INVALID),
    (dict(mx=0), INVALID), (dict(D=128), UNSUPPORTED), (dict(scale=0.0), INVALID),
    (dict(k=P(0x10004)), MISALIGNED), (dict(out=P(0x10008)), MISALIGNED),
])
def test_rotated_prompt_refusals(lib, kw, code):
    assert _rotated(lib, False, **kw) == code
    assert _rotated(lib, True, **kw) == code


def test_rotated_prompt_backward_refusals(lib):
    assert _rotated(lib, True, dk=None) == INVALID
    assert _rotated(lib, True, ws=FAKE, wb=16) == INVALID
    assert _rotated(lib, True, ws=P(0x10010), wb=1 << 40) == MISALIGNED


def test_status_string(lib):
    assert lib.ne_status_string(10) == b"NE_ERR_NO_PAGES"


def test_binding_refuses_before_the_library(monkeypatch):
    from causal_self_attention_gb300 import ne_attn as na
    monkeypatch.setattr(na, "lib", lambda: pytest.fail("the library was called"))
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    calls = [  # CPU tensors
        lambda: na.ne_qk_norm_rope_fwd(bf(4, 4, 64), bf(4, 2, 64), bf(64), bf(64), i(4), 4),
        lambda: na.ne_kv_reserve(i(2), i(2), i(2, 3), i(8), i(1), 4, 16, 48),
        lambda: na.ne_kv_release(u8(2), i(2), i(2, 3), i(8), i(1), 16, 48),
        lambda: na.ne_attn_gqa_varlen_fwd_rotated(bf(4, 4, 64), bf(4, 2, 64), bf(4, 2, 64), i(2), 4),
    ]
    for call in calls:
        with pytest.raises(ValueError):
            call()
    # The device checks aside (-1 stands for the device of CPU tensors), shapes and types.
    monkeypatch.setattr(na, "_device", lambda t, name: -1)
    wide = bf(4, 8, 64)
    assert na._rows_of(wide[:, 2:6], None, -1, "q") == 512
    assert na._rows_of(bf(1, 4, 64), None, -1, "q") == 256
    bad = [
        lambda: na._rows_of(bf(4, 64), None, -1, "q"),
        lambda: na._rows_of(bf(4, 2, 32), None, -1, "q"),
        lambda: na._rows_of(bf(4, 2, 64), (4, 3, 64), -1, "q"),
        lambda: na._rows_of(wide[:, ::2], None, -1, "q"),
        lambda: na._rows_of(bf(4, 64, 2).transpose(1, 2), None, -1, "q"),
        lambda: na._rows_of(bf(4, 2, 64).half(), None, -1, "q"),
        lambda: na._paged(u8(2, 2, 16, 64), u8(2, 2, 16, 64), u8(2, 2, 16, 2), u8(2, 2, 16, 2), i(1, 2), 1, -1),
        lambda: na._paged(u8(2, 2, 16, 32), u8(2, 2, 16, 32), None, None, i(1, 2), 1, -1),
        lambda: na._paged(u8(2, 2, 16, 32), u8(2, 2, 16, 32), u8(2, 2, 16), u8(2, 2, 16), i(1, 2), 1, -1),
    ]
    for n, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"refusal {n} did not happen")


def test_native_marshalling_hands_back_what_is_not_regular(lib):
    from causal_self_attention_gb300 import ne_attn as na
    na.lib()
    step, bf, i = na._step, torch.zeros((4, 2, 64), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    counts = dict(norm_fwd=10, norm_bwd=14, reserve=14, release=7, append=11, read=11, decode=12)
    for name, n in counts.items():
        call = getattr(step, name)
        for args in ((), (None,) * n, (bf,) * n, (i,) * n, (1,) * n, ("x",) * n, (None,) * (n + 1)):
            assert call(*args) is None  # CPU tensors, no tensors, too many
    for args in ((), (1,) * 8, ("x",) * 7):
        with pytest.raises(TypeError):
            step.bind(*args)


# ------------------------------------------------- the plain implementations

def test_plain_four_bit_rounding():
    """To the nearest of the grid, ties to the even code, the smallest scale that holds
    the largest value."""
    y = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.26, 4.9, -0.25, -2.5, -5.0],
                     dtype=F64)
    want = [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0, 0.5, 4.0, 0.0, -2.0, -4.0]
    x = torch.zeros((1, D), dtype=F64)
    x[0, :13] = y
    x[0, 32] = 6.01 * 2.0 ** -7
    got, e = step.quantise4(x)
    assert got[0, :13].tolist() == want and e.tolist() == [[0, -6]]
    assert step.quantise4(torch.zeros((1, D), dtype=F64))[1].tolist() == [[-100, -100]]
    big = torch.full((1, D), 3e38, dtype=F64)
    assert step.quantise4(big)[1].tolist() == [[125, 125]]
    assert float(step.quantise4(big)[0].max()) == 6 * 2.0 ** 125
    x[0, 40] = math.inf
    got, e = step.quantise4(x)
    assert e.tolist() == [[0, 128]] and bool(torch.isnan(got[0, 32:]).all())
    g = torch.Generator().manual_seed(1)
    x = torch.randn((300, D), generator=g, dtype=F64)
    got, e = step.quantise4(x)
    a = x.unflatten(-1, (2, 32)).abs().amax(-1)
    assert bool((a <= 6 * torch.exp2(e)).all()) and bool((a > 6 * torch.exp2(e - 1)).all())
    two = torch.exp2(e).repeat_interleave(32, -1)
    assert bool(((got - x).abs() <= torch.maximum(step.U4 * x.abs(), two / 4)).all())


def test_plain_order_of_a_row():
    """Every dim has four bits of its own; a byte holds neighbours."""
    seen = {step.byte_of(d) for d in range(D)}
    assert seen == {(b, s) for b in range(32) for s in (0, 4)}
    assert [step.byte_of(d)[0] for d in (0, 1, 2, 32, 34, 4, 63)] == [0, 0, 1, 2, 3, 4, 31]


@pytest.mark.parametrize("base", [10000.0, 0.0])
def test_plain_norm_gradients_against_differences(base):
    g = torch.Generator().manual_seed(2)
    n, H, eps, h = 5, 3, 1e-5, 1e-6
    pos = torch.tensor([0, 3, 9, 100, 2])
    x = torch.randn((n, H, D), generator=g, dtype=F64)
    w = 1 + 0.3 * torch.randn(D, generator=g, dtype=F64)
    dr = torch.randn((n, H, D), generator=g, dtype=F64)
    dx, dw, _, _ = step.norm_grads(dr, x, w, eps, pos, base)

    def loss(x, w):
        return (step.norm(x, w, eps, pos, base)[0] * dr).sum()

    for t, grad, which in ((x, dx, 0), (w, dw, 1)):
        for _ in range(20):
            at = tuple(int(torch.randint(0, s, (1,), generator=g)) for s in t.shape)
            args = [x.clone(), w.clone()]
            args[which][at] += h
            up = loss(*args)
            args[which][at] -= 2 * h
            # Second order in h, and 64-bit rounding over h.
            assert abs(float((up - loss(*args)) / (2 * h) - grad[at])) < 1e-7 * n * H


def test_plain_norm_is_the_rotation_of_the_norm():
    g = torch.Generator().manual_seed(3)
    x = torch.randn((4, 2, D), generator=g, dtype=F64)
    w = torch.ones(D, dtype=F64)
    pos = torch.tensor([1, 2, 3, 70])
    y, _ = step.norm(x, w, 0.0)
    assert torch.allclose(y.square().mean(-1), torch.ones(4, 2, dtype=F64))
    assert torch.allclose(step.norm(x, w, 0.0, pos)[0], rotate(y, pos))


def test_plain_pages():
    p = step.Pages(3, 4, 8, 16, range(8))
    cu, start, pos, slots = p.reserve([17, 0, 1], 20)
    assert (cu, start) == ([0, 17, 17, 18], [0, 0, 0])
    assert pos == list(range(17)) + [0, -1, -1] and p.table[0][:2] == [7, 6] and p.table[2][0] == 5
    assert slots[16:] == [6 * 16, 5 * 16, -1, -1] and p.lens == [17, 0, 1]
    p.release([1, 0, 0])
    assert p.free == [0, 1, 2, 3, 4, 7, 6] and p.table[0][:2] == [-1, -1] and p.lens == [0, 0, 1]

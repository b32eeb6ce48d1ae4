"""Scores of minus infinity: such a key has weight zero, wherever it stands, also
where a whole tile or a whole part of a sequence holds nothing else.  A row with
no other keys has no weights (NaN) and the log-sum-exp -inf."""
import pytest
import torch

from grouped import Cache, attention, within

pytestmark = pytest.mark.gpu
HUGE = 3e38  # times 16 overflows fp32


@pytest.fixture(scope="module")
def na():
    from causal_self_attention_gb300 import build, ne_attn
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ne_attn


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _randn(seed, *shape):
    g = torch.Generator("cpu").manual_seed(seed)
    return torch.randn(shape, generator=g).bfloat16().cuda()


def _qkv(seed, n, m, H, Hkv, bad):
    """Queries and keys that overlap in dims 31 and 63 only for the first `bad` keys and
    the queries from `bad` on: their products are -16 HUGE."""
    q, k, v = _randn(seed, n, H, 64), _randn(seed + 1, m, Hkv, 64), _randn(seed + 2, m, Hkv, 64)
    q[..., 31::32] = 0
    k[..., 31::32] = 0
    k[:bad, :, 31] = -HUGE
    return q, k, v


@pytest.mark.parametrize("H,Hkv", [(4, 2), (3, 1)])
@pytest.mark.parametrize("bad", [1, 127, 128, 150, 256, 300])
def test_prompt_whose_first_keys_have_infinite_scores(na, H, Hkv, bad):
    n = 500
    q, k, v = _qkv(1, n, n, H, Hkv, bad)
    q[bad:, :, 31] = 16
    cu = _i32([0, n])
    out, lse, qr, kr = na.ne_attn_gqa_varlen_fwd(q, k, v, cu, n)
    assert na.ne_attn_get_device_status() == 0
    s = torch.einsum("nhd,mhd->hnm", qr[bad:].float(), kr[:bad].float().repeat_interleave(H // Hkv, 1))
    assert bool((s == -float("inf")).all())
    for r in (slice(0, bad), slice(bad, n)):  # each part of the rows sees its own keys only
        o, l, oe, le = attention(qr[r], kr[r], v[r], 0.125)
        within(out[r], o, oe, "out")
        within(lse[:, r], l, le, "lse")


def test_prompt_with_nothing_but_infinite_scores(na):
    """Every key of some rows: no weights, and no other row's matter."""
    n = 400
    q, k, v = _qkv(11, n, n, 4, 2, n)
    q[200:300, :, 31] = 16
    cu = _i32([0, n])
    out, lse, qr, kr = na.ne_attn_gqa_varlen_fwd(q, k, v, cu, n)
    assert bool(torch.isnan(out[200:300]).all()) and bool((lse[:, 200:300] == -float("inf")).all())
    o, l, oe, le = attention(qr, kr, v, 0.125)
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[200:300] = False
    within(out[rest], o[rest], oe[rest], "out")
    within(lse[:, rest], l[:, rest], le[:, rest], "lse")


@pytest.mark.parametrize("n,bad", [(500, 128), (500, 300), (2300, 150), (2300, 2200)])
@pytest.mark.parametrize("form", ["fixed", "train", "packed", "rotated"])
def test_a_head_each_whose_first_keys_have_infinite_scores(na, form, n, bad):
    """The forwards without shared heads (from 2048 positions on they rotate their keys in
    a pass); the rotated operands as the training forward gives them."""
    q, k, v = _qkv(15, n, n, 3, 3, bad)
    q[bad:, :, 31] = 16
    _, _, qr, kr = na.ne_attn_fwd_train(q[None], k[None], v[None])
    if form == "packed":
        out, lse = na.ne_attn_varlen_fwd(q, k, v, _i32([0, n]), n)
    elif form == "rotated":
        out, lse = (t[0] for t in na.ne_attn_fwd_rotated(qr, kr, v[None]))
    else:
        fwd = na.ne_attn_fwd_train if form == "train" else na.ne_attn_fwd
        out, lse = (t[0] for t in fwd(q[None], k[None], v[None])[:2])
    assert na.ne_attn_get_device_status() == 0
    for r in (slice(0, bad), slice(bad, n)):
        o, l, oe, le = attention(qr[0][r], kr[0][r], v[r], 0.125)
        within(out[r], o, oe, "out")
        within(lse[:, r], l, le, "lse")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,bad", [(60, 40), (700, 100), (700, 650), (20000, 5000), (20000, 19990)])
@pytest.mark.parametrize("low", [False, True])
def test_decode_whose_first_keys_have_infinite_scores(na, e4m3, n, bad, low):
    """Parts of a sequence with no other keys among them; low: the others' scores
    near -600, so that a factor 2^(-score) would overflow."""
    H, Hkv = 6, 2
    q, k, v = _qkv(21, 1, n, H, Hkv, bad)
    q[..., 31] = 16
    if low:
        q[..., 0], k[..., 0] = 40, -120
    c = Cache([n], Hkv, 64, e4m3, seed=24)
    na.ne_kv_append(k, v, _i32([0, n]), _i32([0]), c.k, c.v, c.table, n, c.ks, c.vs, rope_base=0.0)
    out, lse = na.ne_attn_decode_paged(q, c.k, c.v, c.table, _i32([n]), n, c.ks, c.vs, rope_base=0.0)
    assert na.ne_attn_get_device_status() == 0
    kk, vv = c.rows(0)
    o, l, oe, le = attention(q, kk[bad:], vv[bad:], 0.125)
    within(out[0], o[0], oe[0], "out")
    within(lse[0], l[:, 0], le[:, 0], "lse")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [1, 60, 20000])
def test_decode_with_nothing_but_infinite_scores(na, e4m3, n):
    q, k, v = _qkv(31, 1, n, 6, 2, n)
    q[..., 31] = 16
    c = Cache([n], 2, 64, e4m3, seed=34)
    na.ne_kv_append(k, v, _i32([0, n]), _i32([0]), c.k, c.v, c.table, n, c.ks, c.vs, rope_base=0.0)
    out, lse = na.ne_attn_decode_paged(q, c.k, c.v, c.table, _i32([n]), n, c.ks, c.vs, rope_base=0.0)
    assert na.ne_attn_get_device_status() == 0
    assert bool(torch.isnan(out).all()) and bool((lse == -float("inf")).all())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("first,last", [(0, 5000), (15000, 20000), (9999, 10000)])
def test_decode_with_keys_of_nan_shows_them(na, e4m3, first, last):
    """A NaN score is no minus infinity: it shows, however many keys share it."""
    n = 20000
    q, k, v = _qkv(41, 1, n, 6, 2, 0)
    k[first:last] = float("nan")
    c = Cache([n], 2, 64, e4m3, seed=44)
    na.ne_kv_append(k, v, _i32([0, n]), _i32([0]), c.k, c.v, c.table, n, c.ks, c.vs, rope_base=0.0)
    out, lse = na.ne_attn_decode_paged(q, c.k, c.v, c.table, _i32([n]), n, c.ks, c.vs, rope_base=0.0)
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())

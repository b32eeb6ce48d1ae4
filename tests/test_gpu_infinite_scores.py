"""Scores of minus infinity: such a key has weight zero, wherever it stands, also
where a whole tile of a sequence holds nothing else.  A row with
no other keys has no weights (NaN) and the log-sum-exp -inf."""
import pytest
import torch

from grouped import attention, within

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

"""Decode attention over the 4-bit cache on random batches: scales of keys and values alike, in
ranges, apart, rising, falling, by blocks; zeros among the values, marked as the cache marks
them or not; large and small queries.  Against the plain 64-bit implementation."""
import random

import pytest
import torch

import step
from grouped import F64, attention, within
from step import Cache4
from test_gpu_paged import _decode, _i32

pytestmark = pytest.mark.gpu
LENS = (1, 5, 63, 64, 65, 200, 256, 257, 500, 700, 1500, 5000)


@pytest.fixture(scope="module")
def na():
    from causal_self_attention_gb300 import build, ne_attn
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ne_attn


def _bytes(rng, g, kind, center, n, Hkv):
    """Scale bytes [n, Hkv, 2] from `center` down."""
    i, shape = torch.arange(n), (n, Hkv, 2)
    if kind == "one":
        down = torch.zeros(shape, dtype=torch.long)
        down[rng.randrange(n)] = rng.choice((8, 30, 70))
    elif kind in ("near", "far"):
        down = torch.randint(0, 6 if kind == "near" else 60, shape, generator=g)
    else:
        along = {"same": 0 * i, "rise": 50 - 50 * i // n, "fall": 50 * i // n, "blocks": 20 * (i // 64 % 3)}
        down = along[kind][:, None, None].expand(shape)
    return (center - down).clamp(0, 252).to(torch.uint8).cuda()


def _zeros(rng, g, c, page, slot, n):
    """Some rows' values zero in one half or both, with the scale byte that the cache gives
    zeros or the one that they have."""
    zero = (torch.rand((n, c.Hkv), generator=g) < rng.choice((0.1, 0.9))).cuda()
    halves, marked = rng.choice(((0,), (1,), (0, 1))), rng.random() < 0.5
    values, scales = c.v[page, :, slot], c.vs[page, :, slot]
    for h in halves:
        for b in (b for b in range(32) if b % 4 // 2 == h):
            values[..., b] = values[..., b].masked_fill(zero, 0)
        if marked:
            scales[..., h] = scales[..., h].masked_fill(zero, 27)
    c.v[page, :, slot], c.vs[page, :, slot] = values, scales


def _batch(na, rng):
    Hkv, G = rng.choice((1, 2, 3)), rng.choice((1, 3, 4, 8, 9, 16))
    lens = [rng.choice(LENS) for _ in range(rng.choice((1, 1, 2, 5)))]
    seed = rng.randrange(1 << 30)
    g = torch.Generator("cpu").manual_seed(seed)
    c = Cache4(lens, Hkv, rng.choice((16, 32, 64, 128, 256)), seed=seed).fill_random(seed + 1)
    q_exp = rng.choice((0, 0, 0, -20, -110, 20))
    for s, n in enumerate(lens):
        page, slot = (t.cuda() for t in c.where(s, torch.arange(n)))
        keys = min(252, 127 - q_exp + rng.choice((0, -3, 2, 5)))  # (scores of a size, whatever q's)
        c.ks[page, :, slot] = _bytes(rng, g, rng.choice(("same", "near", "rise", "fall", "one")), keys, n, Hkv)
        kind = rng.choice(("same", "near", "far", "one", "rise", "fall", "blocks"))
        c.vs[page, :, slot] = _bytes(rng, g, kind, rng.choice((27, 33, 45, 60, 100, 127, 127, 200, 252)), n, Hkv)
        if rng.random() < 0.4:
            _zeros(rng, g, c, page, slot, n)
    size = 2.0 ** q_exp * rng.choice((1, 1, 30, 0.01))
    q = torch.randn((len(lens), G * Hkv, 64), generator=g, dtype=F64).clamp(-1.9, 1.9)
    q = (q * size).bfloat16().cuda()
    out, lse = _decode(na, c, q, _i32(lens), rng.choice((max(lens), c.max_pages * c.page)), 0.0)
    assert na.ne_attn_get_device_status() == 0
    for s, n in enumerate(lens):
        k, v = c.rows(s, n)
        o, l, oe, le = attention(q[s:s + 1], k, v, 0.125)
        # Weights below fp32's smallest normal number may be left out: a part's and a warp's
        # (2^-126 of all), a key's (2^-126 of 2^-8 of its warp's largest).
        lost = (2 * 2.0 ** -126 + n * 2.0 ** -134) * float(v.abs().amax())
        bound = oe[0] + step.half_weights(q[s], k, c.value_scales(s, n), 0.125) + lost
        within(out[s], o[0], bound, f"out of sequence {s} of seed {seed}")
        within(lse[s], l[:, 0], le[:, 0], f"lse of sequence {s} of seed {seed}")


@pytest.mark.parametrize("seed", range(20))
def test_random_batches(na, seed):
    rng = random.Random(seed)
    for _ in range(20):
        _batch(na, rng)

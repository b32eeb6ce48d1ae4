"""The paged cache in 4 bits -- writing rows, reading them back, decode attention over it
-- against the plain 64-bit implementations of step.py and grouped.py."""
import pytest
import torch

import step
from grouped import F64, U16, Cache, attention, rotate, rotate_bound, within
from step import Cache4, quantise4
from test_gpu_paged import BASE, LENS, _append, _cu, _decode, _i32, _randn
from test_gpu_paged import _check_append as check_append_e4m3

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def na():
    from causal_self_attention_gb300 import build, ne_attn
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ne_attn


# ------------------------------------------------------------ append and read

def _check_append(na, c, rows, start, base, seed):
    """Appends `rows[s]` rows at start[s]; checks them, and that nothing else moved."""
    tot = sum(rows)
    behind = 3  # rows behind the last sequence
    k, v = (_randn(seed + i, tot + behind, c.Hkv, 64) for i in range(2))
    before = [t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    _append(na, c, k, v, _cu(rows), _i32(start), base, max(s + r for s, r in zip(start, rows)))
    assert na.ne_attn_get_device_status() == 0
    at = 0
    touched = torch.zeros(c.k.shape[:3], dtype=torch.bool, device="cuda")
    for s, n in enumerate(rows):
        page, slot = c.where(s, start[s] + torch.arange(n))
        touched[page.cuda(), :, slot.cuda()] = True
        if n == 0:
            continue
        got_k, got_v = c.rows(s, n, start[s])
        kk, vv = k[at:at + n].to(F64), v[at:at + n].to(F64)
        at += n
        assert torch.equal(got_v, quantise4(vv)[0])
        if not base:
            assert torch.equal(got_k, quantise4(kk)[0])
            continue
        want = rotate(kk, start[s] + torch.arange(n, device="cuda"), base)
        # Half a step of the value, below 1 a quarter of the scale; a half whose largest
        # value sits at a border may take the next scale.
        two = torch.exp2(quantise4(want)[1]).repeat_interleave(32, -1)
        within(got_k, want, step.U4 * want.abs() + two / 2 + (1 + step.U4) * rotate_bound(kk), "k'")
    for t, b in zip((c.k, c.v, c.ks, c.vs), before):
        assert torch.equal(t[~touched], b[~touched])


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("base", [BASE, 0.0])
def test_append_prompts(na, page, base):
    lens = [1, 0, 15, 16, 17, 300, 64, 0, 129]
    _check_append(na, Cache4(lens, 3, page, seed=1), lens, [0] * len(lens), base, 11)


@pytest.mark.parametrize("Hkv", [1, 2, 5, 12])
def test_append_one_token_each_and_parts_of_prompts(na, Hkv):
    start = [0, 1, 15, 16, 17, 255, 256, 5000, 77]
    rows = [1] * 8 + [40]
    lens = [s + r for s, r in zip(start, rows)]
    _check_append(na, Cache4(lens, Hkv, 16, seed=2), rows, start, BASE, 12)


@pytest.mark.parametrize("Hkv,lens", [(2, [20000, 0, 13001]), (4, [9000, 9001]), (10, [7001])])
@pytest.mark.parametrize("e4m3", [False, True])
def test_append_and_read_many_rows(na, Hkv, lens, e4m3):
    """Rows enough to fill the GPU, with an even number of heads; e4m3's likewise."""
    if e4m3:
        c = Cache(lens, Hkv, 64, True, seed=9)
        check_append_e4m3(na, c, lens, [0] * len(lens), BASE, 14)
    else:
        c = Cache4(lens, Hkv, 64, seed=9)
        _check_append(na, c, lens, [0] * len(lens), BASE, 14)
    tot = sum(lens)
    k, v = na.ne_kv_read(c.k, c.v, c.table, _cu(lens), _i32([0] * len(lens)), tot, c.ks, c.vs)
    assert na.ne_attn_get_device_status() == 0
    at = 0
    for s, n in enumerate(lens):
        for got, want in zip((k, v), c.rows(s) if n else ()):
            assert torch.equal(got[at:at + n].to(F64), want)
        at += n


@pytest.mark.parametrize("page", [16, 256])
def test_pools_past_32_bits(na, page):
    """Pages at the end of pools of more than 4 GiB: written, read, attended to."""
    lens, Hkv, H = [700, 33], 4, 12
    c = Cache4(lens, Hkv, page, seed=10)
    many = (2 ** 27 + 2 ** 24) // (Hkv * page)
    c.table[c.table >= 0] += many - c.n_pages
    c.n_pages = many
    c.k, c.v = (torch.zeros((many, Hkv, page, 32), dtype=torch.uint8, device="cuda") for _ in range(2))
    c.ks, c.vs = (torch.zeros((many, Hkv, page, 2), dtype=torch.uint8, device="cuda")
                  for _ in range(2))
    tot = sum(lens)
    k, v = _randn(24, tot, Hkv, 64), _randn(25, tot, Hkv, 64)
    _append(na, c, k, v, _cu(lens), _i32([0, 0]), 0.0, 700)
    kk, vv = na.ne_kv_read(c.k, c.v, c.table, _cu(lens), _i32([0, 0]), tot, c.ks, c.vs)
    assert na.ne_attn_get_device_status() == 0
    for got, x in ((kk, k), (vv, v)):
        assert torch.equal(got.to(F64), quantise4(x.to(F64))[0])
    assert torch.equal(c.rows(0)[0], kk[:700].to(F64))
    _check_decode(na, c, H, lens, BASE, 26)


def test_append_many_sequences(na):
    rows = [(i * 7) % 4 for i in range(3000)]
    start = [(i * 13) % 50 for i in range(3000)]
    lens = [s + r for s, r in zip(start, rows)]
    _check_append(na, Cache4(lens, 1, 16, seed=3), rows, start, BASE, 13)


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1.0, 1e30, 1e38])
def test_append_quantises_over_the_range_of_bf16(na, scale):
    c = Cache4([64], 2, 64, seed=4)
    k, v = _randn(20, 64, 2, 64, scale=scale), _randn(21, 64, 2, 64, scale=scale)
    v[5] = 0  # an all-zero row: scales 2^-100
    for row, x in ((6, 6.0), (7, 6.0625), (8, 3.3e38)):  # on the border, past it, the largest
        v[row] = 0
        v[row, :, 0] = x
    # The second half has its own scale; ties go to the even code.
    v[9] = 0
    v[9, :, 32:45] = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -2.5, -3.5,
                                   -5], dtype=torch.bfloat16, device="cuda")
    _append(na, c, k, v, _cu([64]), _i32([0]), 0.0, 64)
    for got, x in zip(c.rows(0), (k, v)):
        # fp32 arithmetic below its smallest normal number: absolute 2^-126.
        want = quantise4(x.to(F64))[0]
        within(got, want, torch.full_like(got, 2.0 ** -126), "values")
    page, slot = c.where(0, torch.tensor([5, 6, 7, 8, 9]))
    assert c.vs[page.cuda(), 0, slot.cuda()].tolist() == [[27, 27], [127, 27], [128, 27], [252, 27],
                                                         [27, 127]]
    kk, vv = na.ne_kv_read(c.k, c.v, c.table, _cu([64]), _i32([0]), 64, c.ks, c.vs)
    for got, want, x in zip((kk, vv), c.rows(0), (k, v)):
        within(got, want, torch.zeros_like(want), "read back")
        assert not bool(torch.isinf(got).any())
        halves = torch.isfinite(x).unflatten(-1, (2, 32)).all(-1)
        assert torch.equal(torch.isfinite(got).unflatten(-1, (2, 32)).all(-1), halves)


def test_append_marks_halves_with_infinities_or_nan(na):
    c = Cache4([8], 2, 16, seed=5)
    k, v = _randn(22, 8, 2, 64), _randn(23, 8, 2, 64)
    k[1, 0, 3] = float("inf")   # rotated: both of its pair
    k[2, 1, 63] = float("nan")
    v[4, 0, 0] = float("-inf")  # the first half alone
    v[5, 1, 40] = float("nan")  # the second
    _append(na, c, k, v, _cu([8]), _i32([0]), BASE, 8)
    kk, vv = na.ne_kv_read(c.k, c.v, c.table, _cu([8]), _i32([0]), 8, c.ks, c.vs)
    bad_k = torch.zeros((8, 2, 64), dtype=torch.bool, device="cuda")
    bad_k[1, 0] = bad_k[2, 1] = True
    bad_v = torch.zeros_like(bad_k)
    bad_v[4, 0, :32] = bad_v[5, 1, 32:] = True
    assert torch.equal(torch.isnan(kk), bad_k) and torch.equal(torch.isnan(vv), bad_v)


@pytest.mark.parametrize("page", [16, 64, 256])
def test_read_ranges(na, page):
    lens = [1, 300, 17, 64, 500]
    c = Cache4(lens, 3, page, seed=6).fill_random(60)
    first, n = [0, 5, 16, 0, 255], [1, 295, 1, 64, 200]
    tot = sum(n)
    k = torch.full((tot + 4, 3, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    v = k.clone()
    na.ne_kv_read(c.k, c.v, c.table, _cu(n), _i32(first), tot + 4, c.ks, c.vs, k=k, v=v)
    assert na.ne_attn_get_device_status() == 0
    at = 0
    for s in range(5):
        for got, want in zip((k, v), c.rows(s, n[s], first[s])):
            assert torch.equal(got[at:at + n[s]].to(F64), want)
        at += n[s]
    assert bool((k[at:] == 7).all()) and bool((v[at:] == 7).all())


def test_read_every_byte_and_scale(na):
    """All 256 bytes, all scale bytes (values outside bf16's range round as bf16 does)."""
    c = Cache4([256], 1, 256, seed=7)
    page, slot = (t.cuda() for t in c.where(0, torch.arange(256)))
    byte = torch.arange(256, device="cuda").to(torch.uint8)
    c.k[page, 0, slot] = byte[:, None].expand(-1, 32)
    c.v[page, 0, slot] = byte[None, :32] * 8 + 7
    c.ks[page, 0, slot] = torch.stack((byte, 255 - byte), -1)
    c.vs[page, 0, slot] = 127
    k, v = na.ne_kv_read(c.k, c.v, c.table, _cu([256]), _i32([0]), 256, c.ks, c.vs)
    for got, want in zip((k, v), c.rows(0)):
        # (bf16 of 64-bit values: exact in range, 6 * 2^126 and more infinite.)
        within(got, want.float().bfloat16(), 2.0 ** -133 * torch.ones_like(want), "values")


def test_bad_positions_and_pages_are_reported_and_left_alone(na):
    lens = [40, 40, 40]
    c = Cache4(lens, 2, 16, seed=7)
    c.table[1, 1] = c.n_pages      # positions 16..31 of sequence 1
    c.table[2, 0] = -5
    k, v = _randn(30, 120, 2, 64), _randn(31, 120, 2, 64)
    clean = Cache4(lens, 2, 16, seed=7)
    _append(na, c, k, v, _cu(lens), _i32([0] * 3), BASE, 40)
    assert na.ne_attn_get_device_status() == 9
    _append(na, clean, k, v, _cu(lens), _i32([0] * 3), BASE, 40)
    assert na.ne_attn_get_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(c.rows(0), clean.rows(0)))
    out_k = torch.full((120, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    out_v = out_k.clone()
    na.ne_kv_read(c.k, c.v, c.table, _cu(lens), _i32([0] * 3), 120, c.ks, c.vs, k=out_k, v=out_v)
    assert na.ne_attn_get_device_status() == 9
    for out in (out_k, out_v):
        assert bool((out[56:72] == 3).all()) and bool((out[80:96] == 3).all())
        assert not bool((out[40:56] == 3).all()) and not bool((out[96:112] == 3).all())
    c = Cache4([40], 2, 16, seed=8)
    before = c.k.clone()
    for start in (-3, 38, 2 ** 31 - 2):
        _append(na, c, k[:3], v[:3], _cu([3]), _i32([start]), BASE, 38)
        assert na.ne_attn_get_device_status() == 7
    assert torch.equal(c.k, before)


# -------------------------------------------------------------- decode

def _check_decode(na, c, H, lens, base, seed, max_seqlen=None, qscale=1.0):
    q = _randn(seed, len(lens), H, 64, scale=qscale)
    out, lse = _decode(na, c, q, _i32(lens), max_seqlen or max(max(lens), 1), base)
    assert na.ne_attn_get_device_status() == 0
    for s, n in enumerate(lens):
        if n == 0:
            assert bool((out[s] == 0).all()) and bool((lse[s] == -float("inf")).all())
            continue
        _check_sequence(c, s, n, q[s:s + 1], out[s], lse[s], base)


def _check_sequence(c, s, n, q, out, lse, base=0.0):
    qq, slack = q.to(F64), torch.zeros(q.shape[1], dtype=F64, device=q.device)
    k, v = c.rows(s, n)
    if base:
        # q' as the operator rounds it, and the effect of a value at a rounding border
        # that fp32 puts on its other side (one bf16 step, two halves).
        exact = rotate(qq, torch.tensor([n - 1], device="cuda"), base)
        qq, off = exact.to(torch.float32).to(torch.bfloat16).to(F64), rotate_bound(q)
        if bool(((exact - off).to(torch.bfloat16) != (exact + off).to(torch.bfloat16)).any()):
            slack = 0.125 * 2 * U16 * torch.einsum(
                "hgd,mhd->hgm", qq[0].abs().view(c.Hkv, -1, 64), k.abs()).amax(-1).reshape(-1)
    o, l, oe, le = attention(qq, k, v, 0.125)
    G = q.shape[1] // c.Hkv
    oe = oe[0] + step.half_weights(qq[0], k, c.value_scales(s, n), 0.125) + \
        4 * slack[:, None] * v.abs().amax(0).repeat_interleave(G, 0)
    within(out, o[0], oe, f"out of sequence {s}")
    within(lse, l[:, 0], le[:, 0] + slack, f"lse of sequence {s}")


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("H,Hkv", [(6, 2), (5, 5)])
def test_decode_lengths_and_pages(na, page, H, Hkv):
    c = Cache4(LENS, Hkv, page, seed=40).fill_random(41)
    _check_decode(na, c, H, LENS, BASE, 42)
    _check_decode(na, c, H, LENS, 0.0, 43)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (12, 4), (8, 1), (9, 1), (16, 1), (17, 1), (32, 2),
                                   (40, 1), (32, 8), (21, 7), (12, 12)])
def test_decode_head_layouts(na, H, Hkv):
    lens = [333, 1, 77]
    c = Cache4(lens, Hkv, 32, seed=44).fill_random(45)
    _check_decode(na, c, H, lens, BASE, 46)


@pytest.mark.parametrize("page", [128, 256])
@pytest.mark.parametrize("H,Hkv", [(9, 1), (16, 1), (32, 2), (40, 1), (21, 7)])
def test_decode_head_layouts_of_large_pages(na, H, Hkv, page):
    lens = [333, 1, 1030, 0, 256]
    c = Cache4(lens, Hkv, page, seed=44).fill_random(45)
    _check_decode(na, c, H, lens, BASE, 46)


@pytest.mark.parametrize("H,Hkv,B,n", [(8, 2, 1, 20000), (8, 2, 3, 9001), (32, 2, 2, 5000)])
def test_decode_long(na, H, Hkv, B, n):
    lens = [n - 777 * i for i in range(B)]
    c = Cache4(lens, Hkv, 64, seed=47).fill_random(48)
    _check_decode(na, c, H, lens, BASE, 49)


@pytest.mark.parametrize("B", [300, 1100])
def test_decode_many_sequences(na, B):
    """More than a launch takes (512) among them."""
    lens = [(37 * i) % 200 for i in range(B)]
    c = Cache4(lens, 1, 16, seed=50).fill_random(51)
    _check_decode(na, c, 4, lens, BASE, 52)


def test_decode_with_a_bound_far_above_the_lengths(na):
    lens = [5, 700, 0, 64]
    c = Cache4(lens, 2, 16, seed=53, extra_columns=3000).fill_random(54)
    _check_decode(na, c, 4, lens, BASE, 55, max_seqlen=40000)


def test_decode_sharp_scores(na):
    """Scores far apart, and rising along the sequence, so that the running maximum keeps
    moving."""
    lens = [900, 129]
    c = Cache4(lens, 2, 64, seed=56).fill_random(57)
    _check_decode(na, c, 6, lens, 0.0, 58, qscale=30.0)
    for s, n in enumerate(lens):
        page, slot = (t.cuda() for t in c.where(s, torch.arange(n)))
        c.k[page, :, slot] = 0x66  # 4 throughout, scales 2^-8 .. 2^4: scores up to 8 * 4 * 2^4
        c.ks[page, :, slot] = (119 + torch.arange(n, device="cuda") * 13 // n).to(
            torch.uint8)[:, None, None].expand(n, 2, 2)
    q = torch.full((2, 6, 64), 0.5, dtype=torch.bfloat16, device="cuda")
    out, lse = _decode(na, c, q, _i32(lens), 900, 0.0)
    for s, n in enumerate(lens):
        _check_sequence(c, s, n, q[s:s + 1], out[s], lse[s])


@pytest.mark.parametrize("H", [4, 13])
@pytest.mark.parametrize("halves", [(True, False), (False, True), (True, True)])
def test_decode_values_of_very_different_scales(na, halves, H):
    """Rows whose scales differ by 2^40, in one half or in both: the small ones with the
    weight."""
    lens = [200]
    c = Cache4(lens, 1, 64, seed=61).fill_random(62)
    page, slot = (t.cuda() for t in c.where(0, torch.arange(200)))
    for h in (h for h in (0, 1) if halves[h]):
        c.vs[page, 0, slot, h] = torch.where(torch.arange(200) < 3, 150, 110).to(torch.uint8).cuda()
    _check_decode(na, c, H, lens, BASE, 63)
    # The keys with large values get almost no weight (scores near -60).
    c.k[page[:3], 0, slot[:3]] = 0xee  # -4, times 2^1
    c.ks[page[:3], 0, slot[:3]] = 128
    q = torch.ones((1, H, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = _decode(na, c, q, _i32(lens), 200, 0.0)
    _check_sequence(c, 0, 200, q, out[0], lse[0])


@pytest.mark.parametrize("H", [4, 16])
@pytest.mark.parametrize("up", [6, 9, 20, 40])
def test_decode_values_whose_scales_rise_along_the_sequence(na, up, H):
    """The weight on early keys with small values, and tiles of much larger ones behind
    them, each tile's scales alike: what the later keys add counts by its size, not by its
    weight."""
    lens = [320, 1500]
    c = Cache4(lens, 1, 64, seed=71).fill_random(72)
    for s, n in enumerate(lens):
        page, slot = (t.cuda() for t in c.where(s, torch.arange(n)))
        late = (torch.arange(n) >= 64).cuda()
        c.vs[page, 0, slot] = torch.where(late, 127 + up, 127).to(torch.uint8)[:, None].expand(n, 2)
        # Scores of 0 for the first keys, -0.125 * 64 * 2.25 = -18 (2^-26) for the others.
        c.k[page, 0, slot] = torch.where(late, 0xcc, 0x00).to(torch.uint8)[:, None].expand(n, 32)
        c.ks[page, 0, slot] = 127
    q = torch.full((2, H, 64), 1.125, dtype=torch.bfloat16, device="cuda")
    out, lse = _decode(na, c, q, _i32(lens), 1500, 0.0)
    for s, n in enumerate(lens):
        _check_sequence(c, s, n, q[s:s + 1], out[s], lse[s])


def test_decode_halves_of_a_key_with_scales_far_apart(na):
    """A score is the sum of its halves', each with its own scale."""
    lens = [150]
    c = Cache4(lens, 2, 16, seed=64).fill_random(65)
    page, slot = (t.cuda() for t in c.where(0, torch.arange(150)))
    c.ks[page, :, slot, 0] = 130
    c.ks[page, :, slot, 1] = 100
    _check_decode(na, c, 4, lens, 0.0, 66)
    c.ks[page, :, slot, 0] = 0  # 2^-127: nothing but the other half
    c.ks[page, :, slot, 1] = 127
    _check_decode(na, c, 4, lens, 0.0, 67)


def test_decode_bad_lengths_and_pages_give_zero_and_minus_infinity(na):
    lens = [600, 600, 600, 30]
    c = Cache4(lens, 2, 16, seed=64).fill_random(65)
    want_out, want_lse = (t.clone() for t in _decode(na, c, _randn(66, 4, 4, 64), _i32(lens), 600))
    good = c.table.clone()
    for bad, seq in ((c.n_pages, 0), (-1, 1), (2 ** 31 - 1, 2), (-2 ** 31, 0)):
        for col in (0, 20, 37):
            c.table.copy_(good)
            c.table[seq, col] = bad
            out, lse = _decode(na, c, _randn(66, 4, 4, 64), _i32(lens), 600)
            assert na.ne_attn_get_device_status() == 9
            for s in range(4):
                if s == seq:
                    assert bool((out[s] == 0).all()) and bool((lse[s] == -float("inf")).all())
                else:
                    assert torch.equal(out[s], want_out[s]) and torch.equal(lse[s], want_lse[s])
    c.table.copy_(good)
    for n in (-1, 601, 2 ** 31 - 1, -2 ** 31):
        out, lse = _decode(na, c, _randn(66, 4, 4, 64), _i32([600, n, 600, 30]), 600)
        assert na.ne_attn_get_device_status() == 7
        assert bool((out[1] == 0).all()) and bool((lse[1] == -float("inf")).all())


def test_decode_nan_of_an_attended_row_shows(na):
    """A half marked as not a number: those dims of v, or the whole score of k."""
    lens = [100, 100, 100]
    c = Cache4(lens, 1, 16, seed=67).fill_random(68)
    page, slot = (t.cuda() for t in c.where(1, torch.tensor([50])))
    c.vs[page, 0, slot, 1] = 255
    page, slot = (t.cuda() for t in c.where(2, torch.tensor([50])))
    c.ks[page, 0, slot, 0] = 255
    out, lse = _decode(na, c, _randn(69, 3, 3, 64), _i32(lens), 100)
    assert bool(torch.isfinite(out[0]).all()) and bool(torch.isfinite(lse[:2]).all())
    assert bool(torch.isfinite(out[1, :, :32]).all()) and bool(torch.isnan(out[1, :, 32:]).all())
    assert bool(torch.isnan(out[2]).all()) and bool(torch.isnan(lse[2]).all())


def test_decode_workspace_streams_and_graphs(na):
    lens, H = [700, 3, 0, 257], 6
    c = Cache4(lens, 2, 32, seed=80).fill_random(81)
    q, n = _randn(82, 4, H, 64), _i32(lens)
    want, wl = (t.clone() for t in _decode(na, c, q, n, 700))
    need = na.ne_attn_decode_paged_workspace_bytes(4, H, 2, 700)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for kw in (dict(workspace=ws), dict(workspace=ws, stream=side)):
        out, lse = _decode(na, c, q, n, 700, **kw)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        got = _decode(na, c, q, n, 700)
    n.copy_(_i32([10, 3, 0, 100]))
    eager = [t.clone() for t in _decode(na, c, q, n, 700)]
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, eager))
    assert na.ne_attn_get_device_status() == 0


def test_decode_of_what_was_stored(na):
    """Rows written in 4 bits: the attention's answer is that of the values read back in
    bf16, by the bf16 cache's kernel, within the bounds of either."""
    lens, H, Hkv = [400, 77], 8, 2
    tot = sum(lens)
    c, b = Cache4(lens, Hkv, 64, seed=90), Cache(lens, Hkv, 64, False, seed=90)
    k, v = _randn(91, tot, Hkv, 64), _randn(92, tot, Hkv, 64)
    _append(na, c, k, v, _cu(lens), _i32([0, 0]), BASE, 400)
    kk, vv = na.ne_kv_read(c.k, c.v, c.table, _cu(lens), _i32([0, 0]), tot, c.ks, c.vs)
    _append(na, b, kk, vv, _cu(lens), _i32([0, 0]), 0.0, 400)
    q = _randn(93, 2, H, 64)
    (o, l), (o2, l2) = _decode(na, c, q, _i32(lens), 400, 0.0), _decode(na, b, q, _i32(lens), 400, 0.0)
    for s, n in enumerate(lens):
        _, _, oe, le = attention(q[s:s + 1], *c.rows(s, n), 0.125)
        oe = oe[0] + step.half_weights(q[s], c.rows(s, n)[0], c.value_scales(s, n), 0.125)
        within(o[s], o2[s], 2 * oe, "out")
        within(l[s], l2[s], 2 * le[:, 0], "lse")

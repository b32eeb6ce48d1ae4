"""The paged cache -- writing rows, reading them back, decode attention over it --
against the plain 64-bit implementations of grouped.py, with bounds that count
the roundings (derived there)."""
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

from grouped import (F64, U8, U16, Cache, attention, quantise, rotate, rotate_bound, within)

pytestmark = pytest.mark.gpu
BASE = 10000.0


@pytest.fixture(scope="module")
def na():
    from causal_self_attention_gb300 import build, ne_attn
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ne_attn


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cu(n):
    return _i32([0] + [sum(n[:i + 1]) for i in range(len(n))])


def _randn(seed, *shape, scale=1.0):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).bfloat16().cuda()


def _append(na, c, k, v, cu, start, base, max_seqlen, **kw):
    na.ne_kv_append(k, v, cu, start, c.k, c.v, c.table, max_seqlen, c.ks, c.vs, rope_base=base,
                    **kw)


def _decode(na, c, q, lens, max_seqlen, base=BASE, **kw):
    return na.ne_attn_decode_paged(q, c.k, c.v, c.table, lens, max_seqlen, c.ks, c.vs,
                                   rope_base=base, **kw)


# ------------------------------------------------------------ append and read

def _check_append(na, c, rows, start, base, seed):
    """Appends `rows[s]` rows at start[s]; checks them, and that nothing else moved."""
    tot = sum(rows)
    behind = 3  # rows behind the last sequence
    k, v = (_randn(seed + i, tot + behind, c.Hkv, 64) for i in range(2))
    before = [t.clone() for t in (c.k, c.v, c.ks, c.vs) if t is not None]
    max_seqlen = max(s + r for s, r in zip(start, rows))
    _append(na, c, k, v, _cu(rows), _i32(start), base, max(max_seqlen, 1))
    assert na.ne_attn_get_device_status() == 0
    at = 0
    touched = torch.zeros(c.k.shape[:3], dtype=torch.bool, device="cuda")
    for s, n in enumerate(rows):
        page, slot = c.where(s, start[s] + torch.arange(n))
        touched[page.cuda(), :, slot.cuda()] = True
        got_k, got_v = c.rows(s, n, start[s])
        kk, vv = k[at:at + n].to(F64), v[at:at + n].to(F64)
        pos = start[s] + torch.arange(n, device="cuda")
        want = rotate(kk, pos, base) if base else kk
        err = rotate_bound(kk) if base else torch.zeros_like(kk)
        at += n
        if n == 0:
            continue
        if not c.e4m3:
            assert torch.equal(got_v, vv)
            if base:
                within(got_k, want, err + U16 * want.abs(), "k'")
            else:
                assert torch.equal(got_k, kk)
            continue
        x8, e = quantise(vv)
        assert torch.equal(got_v, x8 * torch.exp2(e)[..., None])
        two = torch.exp2(quantise(want)[1])[..., None]
        if not base:
            assert torch.equal(got_k, quantise(kk)[0] * two)
        # A key whose largest value sits at a border may take the next scale.
        within(got_k, want, U8 * want.abs() + (1 + U8) * err + 2.0 ** -9 * two, "k'")
    for t, b in zip((t for t in (c.k, c.v, c.ks, c.vs) if t is not None), before):
        a, b = (x.view(torch.uint8 if x.dtype != torch.bfloat16 else torch.int16) for x in (t, b))
        assert torch.equal(a[~touched], b[~touched])


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("base", [BASE, 0.0])
def test_append_prompts(na, page, e4m3, base):
    lens = [1, 0, 15, 16, 17, 300, 64, 0, 129]
    _check_append(na, Cache(lens, 3, page, e4m3, seed=1), lens, [0] * len(lens), base, 11)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("Hkv", [1, 2, 5, 12])
def test_append_one_token_each_and_parts_of_prompts(na, e4m3, Hkv):
    start = [0, 1, 15, 16, 17, 255, 256, 5000, 77]
    rows = [1] * 8 + [40]
    lens = [s + r for s, r in zip(start, rows)]
    _check_append(na, Cache(lens, Hkv, 16, e4m3, seed=2), rows, start, BASE, 12)


def test_append_many_sequences(na):
    rows = [(i * 7) % 4 for i in range(3000)]
    start = [(i * 13) % 50 for i in range(3000)]
    lens = [s + r for s, r in zip(start, rows)]
    _check_append(na, Cache(lens, 1, 16, True, seed=3), rows, start, BASE, 13)


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1.0, 1e30, 1e38])
def test_append_quantises_over_the_range_of_bf16(na, scale):
    c = Cache([64], 2, 64, True, seed=4)
    k = _randn(20, 64, 2, 64, scale=scale)
    v = _randn(21, 64, 2, 64, scale=scale)
    v[5] = 0  # an all-zero row: scale 2^-100
    v[6, :, 1:] = 0
    v[6, :, 0] = 448.0  # exactly on the border: scale 1
    v[7, :, 1:] = 0
    v[7, :, 0] = 450.0  # just past it
    _append(na, c, k, v, _cu([64]), _i32([0]), 0.0, 64)
    for got, x in zip(c.rows(0), (k, v)):
        x8, e = quantise(x.to(F64))
        # fp32 arithmetic below its smallest normal number: absolute 2^-126.
        within(got, x8 * torch.exp2(e)[..., None], torch.full_like(got, 2.0 ** -126), "values")
    page, slot = c.where(0, torch.tensor([5, 6, 7]))
    assert c.vs[page.cuda(), 0, slot.cuda()].tolist() == [27, 127, 128]


def test_append_marks_rows_with_infinities_or_nan(na):
    c = Cache([8], 2, 16, True, seed=5)
    k, v = _randn(22, 8, 2, 64), _randn(23, 8, 2, 64)
    k[1, 0, 3] = float("inf")
    k[2, 1, 63] = float("nan")
    v[4, 0, 0] = float("-inf")
    _append(na, c, k, v, _cu([8]), _i32([0]), BASE, 8)
    kk, vv = na.ne_kv_read(c.k, c.v, c.table, _cu([8]), _i32([0]), 8, c.ks, c.vs)
    bad_k = torch.zeros((8, 2), dtype=torch.bool, device="cuda")
    bad_k[1, 0] = bad_k[2, 1] = True
    bad_v = torch.zeros_like(bad_k)
    bad_v[4, 0] = True
    for got, bad in ((kk, bad_k), (vv, bad_v)):
        assert torch.equal(torch.isnan(got), bad[..., None].expand_as(got))


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("e4m3", [False, True])
def test_read_ranges(na, page, e4m3):
    lens = [1, 300, 17, 64, 500]
    c = Cache(lens, 3, page, e4m3, seed=6).fill_random(60)
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


@pytest.mark.parametrize("e4m3", [False, True])
def test_bad_positions_and_pages_are_reported_and_left_alone(na, e4m3):
    lens = [40, 40, 40]
    c = Cache(lens, 2, 16, e4m3, seed=7, fill=1.0)
    c.table[1, 1] = c.n_pages      # positions 16..31 of sequence 1
    c.table[2, 0] = -5
    k, v = _randn(30, 120, 2, 64), _randn(31, 120, 2, 64)
    clean = Cache(lens, 2, 16, e4m3, seed=7, fill=1.0)
    _append(na, c, k, v, _cu(lens), _i32([0] * 3), BASE, 40)
    assert na.ne_attn_get_device_status() == 9
    _append(na, clean, k, v, _cu(lens), _i32([0] * 3), BASE, 40)
    assert na.ne_attn_get_device_status() == 0
    want = [t.clone() for t in clean.rows(0)]
    assert all(torch.equal(a, b) for a, b in zip(c.rows(0), want))
    out_k = torch.full((120, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    out_v = out_k.clone()
    na.ne_kv_read(c.k, c.v, c.table, _cu(lens), _i32([0] * 3), 120, c.ks, c.vs, k=out_k, v=out_v)
    assert na.ne_attn_get_device_status() == 9
    for out in (out_k, out_v):
        assert bool((out[56:72] == 3).all()) and bool((out[80:96] == 3).all())
        assert not bool((out[40:56] == 3).all()) and not bool((out[96:112] == 3).all())
    # Positions below 0 and from max_seqlen on.
    c = Cache([40], 2, 16, e4m3, seed=8)
    before = c.k.view(torch.uint8).clone()
    for start in (-3, 38, 2 ** 31 - 2):
        _append(na, c, k[:3], v[:3], _cu([3]), _i32([start]), BASE, 38)
        assert na.ne_attn_get_device_status() == 7
    page, slot = c.where(0, torch.tensor([0]))  # position -3 + 3 - 1 < 0: nothing was written
    assert torch.equal(c.k.view(torch.uint8), before)


# -------------------------------------------------------------- decode

def _check_decode(na, c, H, lens, base, seed, max_seqlen=None, qscale=1.0, **kw):
    q = _randn(seed, len(lens), H, 64, scale=qscale)
    out, lse = _decode(na, c, q, _i32(lens), max_seqlen or max(max(lens), 1), base, **kw)
    assert na.ne_attn_get_device_status() == 0
    worst = 0.0
    for s, n in enumerate(lens):
        if n == 0:
            assert bool((out[s] == 0).all()) and bool((lse[s] == -float("inf")).all())
            continue
        qq = q[s:s + 1].to(F64)
        if base:
            # q' as the operator rounds it, and the effect of a value at a rounding
            # border that fp32 puts on its other side (one bf16 step, two halves).
            exact = rotate(qq, torch.tensor([n - 1], device="cuda"), base)
            qq = exact.to(torch.float32).to(torch.bfloat16).to(F64)
            off = rotate_bound(q[s:s + 1])
            near = ((exact - off).to(torch.bfloat16) != (exact + off).to(torch.bfloat16)).any()
        k, v = c.rows(s, n)
        o, l, oe, le = attention(qq, k, v, 0.125)
        if base and bool(near):
            G = H // c.Hkv
            slack = 0.125 * 2 * U16 * torch.einsum(
                "hgd,mhd->hgm", qq[0].abs().view(c.Hkv, G, 64), k.abs()).amax(-1).reshape(H)
            le = le + slack[:, None]
            oe = oe + 4 * slack[None, :, None] * v.abs().amax(0).repeat_interleave(G, 0)[None]
        worst = max(worst, within(out[s], o[0], oe[0], f"out of sequence {s}"),
                    within(lse[s], l[:, 0], le[:, 0], f"lse of sequence {s}"))
    return worst


LENS = [1, 0, 2, 15, 16, 17, 63, 64, 65, 255, 256, 257, 1000]


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H,Hkv", [(6, 2), (5, 5)])
def test_decode_lengths_and_pages(na, page, e4m3, H, Hkv):
    c = Cache(LENS, Hkv, page, e4m3, seed=40).fill_random(41)
    _check_decode(na, c, H, LENS, BASE, 42)
    _check_decode(na, c, H, LENS, 0.0, 43)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (12, 4), (8, 1), (9, 1), (16, 1), (17, 1), (32, 2),
                                   (40, 1), (32, 8), (21, 7), (12, 12)])
def test_decode_head_layouts(na, e4m3, H, Hkv):
    lens = [333, 1, 77]
    c = Cache(lens, Hkv, 32, e4m3, seed=44).fill_random(45)
    _check_decode(na, c, H, lens, BASE, 46)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B,n", [(1, 20000), (2, 9001), (3, 5000)])
def test_decode_long(na, e4m3, B, n):
    lens = [n - 777 * i for i in range(B)]
    c = Cache(lens, 2, 64, e4m3, seed=47).fill_random(48)
    _check_decode(na, c, 8, lens, BASE, 49)


@pytest.mark.parametrize("e4m3,B", [(False, 300), (True, 300), (False, 1100)])
def test_decode_many_sequences(na, e4m3, B):
    """More than a launch takes (512) among them."""
    lens = [(37 * i) % 200 for i in range(B)]
    c = Cache(lens, 1, 16, e4m3, seed=50).fill_random(51)
    _check_decode(na, c, 4, lens, BASE, 52)


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_with_a_bound_far_above_the_lengths(na, e4m3):
    """max_seqlen only bounds: lengths far below it give the same answer."""
    lens = [5, 700, 0, 64]
    c = Cache(lens, 2, 16, e4m3, seed=53, extra_columns=3000).fill_random(54)
    _check_decode(na, c, 4, lens, BASE, 55, max_seqlen=40000)


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_sharp_scores(na, e4m3):
    """Scores far apart (one key takes all the weight) and rising along the
    sequence, so that the running maximum keeps moving."""
    lens = [900, 129]
    c = Cache(lens, 2, 64, e4m3, seed=56).fill_random(57)
    _check_decode(na, c, 6, lens, 0.0, 58, qscale=30.0)
    c = Cache(lens, 2, 64, False, seed=59).fill_random(60)
    for s, n in enumerate(lens):
        page, slot = (t.cuda() for t in c.where(s, torch.arange(n)))
        ramp = torch.linspace(0, 60, n, device="cuda")[:, None, None].expand(n, 2, 64)
        c.k[page, :, slot] = ramp.bfloat16()
    q = torch.full((2, 6, 64), 0.5, dtype=torch.bfloat16, device="cuda")
    out, lse = _decode(na, c, q, _i32(lens), 900, 0.0)
    for s, n in enumerate(lens):
        o, l, oe, le = attention(q[s:s + 1], *c.rows(s, n), 0.125)
        within(out[s], o[0], oe[0], "out")
        within(lse[s], l[:, 0], le[:, 0], "lse")


def test_decode_values_of_very_different_scales(na):
    """e4m3 rows whose scales differ by 2^40: the small ones with the weight."""
    lens = [200]
    c = Cache(lens, 1, 64, True, seed=61).fill_random(62)
    page, slot = (t.cuda() for t in c.where(0, torch.arange(200)))
    c.vs[page, 0, slot] = torch.where(torch.arange(200) < 3, 150, 110).to(torch.uint8).cuda()
    _check_decode(na, c, 4, lens, BASE, 63)
    # The keys with large values get almost no weight (scores near -60).
    c.k.view(torch.uint8)[page[:3], 0, slot[:3]] = \
        torch.full((3, 64), -8.0, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    c.ks[page[:3], 0, slot[:3]] = 127
    q = torch.ones((1, 4, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = _decode(na, c, q, _i32(lens), 200, 0.0)
    o, l, oe, le = attention(q, *c.rows(0, 200), 0.125)
    within(out[0], o[0], oe[0], "out")
    within(lse[0], l[:, 0], le[:, 0], "lse")


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_bad_lengths_and_pages_give_zero_and_minus_infinity(na, e4m3):
    lens = [600, 600, 600, 30]
    c = Cache(lens, 2, 16, e4m3, seed=64).fill_random(65)
    want_out, want_lse = _decode(na, c, _randn(66, 4, 4, 64), _i32(lens), 600)
    want_out, want_lse = want_out.clone(), want_lse.clone()
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
        for s in (0, 2, 3):
            # Another batch may be split at other positions: the difference of two
            # results that are each within the bound of the exact one.
            q1 = rotate(_randn(66, 4, 4, 64)[s:s + 1], torch.tensor([lens[s] - 1], device="cuda"))
            _, _, oe, le = attention(q1.bfloat16(), *c.rows(s, lens[s]), 0.125)
            within(out[s], want_out[s], 2 * oe[0], "out")
            within(lse[s], want_lse[s], 2 * le[:, 0], "lse")


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_nan_of_an_attended_row_shows(na, e4m3):
    lens = [100, 100]
    c = Cache(lens, 1, 16, e4m3, seed=67).fill_random(68)
    page, slot = c.where(1, torch.tensor([50]))
    if e4m3:
        c.vs[page.cuda(), 0, slot.cuda()] = 255
    else:
        c.v[page.cuda(), 0, slot.cuda()] = float("nan")
    out, lse = _decode(na, c, _randn(69, 2, 3, 64), _i32(lens), 100)
    assert not bool(torch.isnan(out[0]).any()) and bool(torch.isnan(out[1]).all())
    assert bool(torch.isfinite(lse).all())


def test_decode_agrees_with_the_contiguous_cache(na):
    """The same rows in a contiguous cache: ne_attn_decode_rotated, within the
    bounds of either."""
    B, H, n = 3, 4, 500
    c = Cache([n] * B, H, 64, False, seed=70).fill_random(71)
    k, v = na.ne_kv_read(c.k, c.v, c.table, _cu([n] * B), _i32([0] * B), B * n)
    q = _randn(72, B, H, 64)
    out, lse = _decode(na, c, q, _i32([n] * B), n, 0.0)
    o2, l2 = na.ne_attn_decode_rotated(q, k.view(B, n, H, 64), v.view(B, n, H, 64),
                                       _i32([n - 1] * B))
    for b in range(B):
        _, _, oe, le = attention(q[b:b + 1], *c.rows(b, n), 0.125)
        within(out[b], o2[b], 2 * oe[0], "out")
        within(lse[b], l2[b], 2 * le[:, 0], "lse")


# ---------------------------------------------------- streams, graphs, workspaces

def test_decode_workspace_streams_and_graphs(na):
    lens, H = [700, 3, 0, 257], 6
    c = Cache(lens, 2, 32, True, seed=80).fill_random(81)
    q, n = _randn(82, 4, H, 64), _i32(lens)
    want, wl = (t.clone() for t in _decode(na, c, q, n, 700))
    need = na.ne_attn_decode_paged_workspace_bytes(4, H, 2, 700)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # dirty: NaN patterns
    out, lse = _decode(na, c, q, n, 700, workspace=ws)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = _decode(na, c, q, n, 700, workspace=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    out, lse = _decode(na, c, q, n, 700, workspace=ws, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(out, want)
    # Two graphs sharing one workspace, replayed in turn on one stream.
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            graphs.append((g, _decode(na, c, q, n, 700, workspace=ws if i else None)))
    for _ in range(2):
        for g, (out, lse) in graphs:
            out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(lse, wl)
    # Lengths are read on the device: a replay sees new ones.
    n.copy_(_i32([10, 3, 5, 0][:2] + [0, 100]))
    eager = [t.clone() for t in _decode(na, c, q, n, 700)]
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(graphs[0][1], eager))
    assert na.ne_attn_get_device_status() == 0


def test_two_calls_at_once(na):
    """Calls in flight on two streams, no workspace given: as one after the other."""
    lens = [3000, 100]
    c = Cache(lens, 2, 64, False, seed=83).fill_random(84)
    qs = [_randn(85 + i, 2, 8, 64) for i in range(8)]
    want = [[t.clone() for t in _decode(na, c, q, _i32(lens), 3000)] for q in qs]
    n = _i32(lens)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [_decode(na, c, q, n, 3000, stream=streams[i % 2]) for i, q in enumerate(qs)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_first_call_of_a_thread(na):
    """A host thread that has made no CUDA call before."""
    c = Cache([100], 2, 64, False, seed=88).fill_random(89)
    q, n = _randn(95, 1, 8, 64), _i32([100])
    want = [t.clone() for t in _decode(na, c, q, n, 100)]
    qkv = [_randn(96 + i, 1, 64, 2, 64) for i in range(3)]
    fwd = na.ne_attn_fwd(*qkv)
    outs = [torch.empty_like(t) for t in (*want, *fwd)]
    torch.cuda.synchronize()
    calls = (lambda: _decode(na, c, q, n, 100, out=outs[0], lse=outs[1]),
             lambda: na.ne_attn_fwd(*qkv, out=outs[2], lse=outs[3]))
    for call in calls:
        with ThreadPoolExecutor(1) as pool:
            pool.submit(call).result()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, (*want, *fwd)))


def test_threads_on_their_own_default_streams(na):
    """cudaStreamPerThread (the handle 2) names another stream in each thread."""
    lens = [3000, 100]
    c = Cache(lens, 2, 64, False, seed=86).fill_random(87)
    n = _i32(lens)
    qs = [_randn(90 + i, 2, 8, 64) for i in range(4)]
    want = [[t.clone() for t in _decode(na, c, q, n, 3000)] for q in qs]
    need = na.ne_attn_decode_paged_workspace_bytes(2, 8, 2, 3000)
    bufs = [(torch.empty_like(q), torch.empty((2, 8), device="cuda"),
             torch.empty(need, dtype=torch.uint8, device="cuda")) for q in qs]
    torch.cuda.synchronize()

    def run(i):
        out, lse, ws = bufs[i]
        for _ in range(50):
            _decode(na, c, qs[i], n, 3000, out=out, lse=lse, workspace=ws, stream=2)

    with ThreadPoolExecutor(len(qs)) as pool:
        list(pool.map(run, range(len(qs))))
    torch.cuda.synchronize()
    for (out, lse, _), w in zip(bufs, want):
        assert torch.equal(out, w[0]) and torch.equal(lse, w[1])


def test_append_replayed_from_a_graph(na):
    lens = [20, 40]
    c = Cache(lens, 2, 16, True, seed=86, fill=0.0)
    k, v = _randn(87, 2, 2, 64), _randn(88, 2, 2, 64)
    start = _i32([3, 17])
    cu = _cu([1, 1])
    _append(na, c, k, v, cu, start, BASE, 40)  # the RoPE table
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        _append(na, c, k, v, cu, start, BASE, 40)
    start.copy_(_i32([5, 30]))
    g.replay()
    torch.cuda.synchronize()
    other = Cache(lens, 2, 16, True, seed=86, fill=0.0)
    _append(na, other, k, v, cu, _i32([3, 17]), BASE, 40)
    _append(na, other, k, v, cu, _i32([5, 30]), BASE, 40)
    for a, b in ((c.k, other.k), (c.v, other.v)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(c.ks, other.ks) and torch.equal(c.vs, other.vs)

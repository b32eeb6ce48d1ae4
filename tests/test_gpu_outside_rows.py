"""Rows that do not belong to a sequence never reach its results, whatever they
hold: rows behind the last sequence of a packed batch (padding that nothing has
written), a neighbour's rows, and the rows of a sequence that is skipped.  A tile
of 128 rows that a sequence ends inside reaches into them, and a weight of zero
times NaN is NaN."""
import pytest
import torch

from grouped import attention, attention_grads, rotate, unrotate_bound, within

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
STALE = [NAN, INF, -3e38]
HEADS = [(4, 2), (3, 1), (4, 4), (12, 4)]
# The last sequences end 1, 44, 100 and 127 rows into a tile, and at its end.
LENS = [100, 129, 400, 60, 255, 1, 300, 128]


@pytest.fixture(scope="module")
def na():
    from causal_self_attention_gb300 import build, ne_attn
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ne_attn


def _cu(n):
    return torch.tensor([0] + [sum(n[:i + 1]) for i in range(len(n))], dtype=torch.int32,
                        device="cuda")


def _randn(seed, *shape):
    g = torch.Generator("cpu").manual_seed(seed)
    return torch.randn(shape, generator=g).bfloat16().cuda()


def _inputs(seed, n, H, Hkv):
    return [_randn(seed + i, n, h, 64) for i, h in enumerate((H, Hkv, Hkv, H))]


def _full(x, *shapes):
    return [torch.full(s, x, dtype=t, device="cuda") for s, t in shapes]


def _forward(na, q, k, v, cu, mx, fill):
    n, H, _ = q.shape
    b = torch.bfloat16
    out, lse, qr, kr = _full(fill, (q.shape, b), ((H, n), torch.float32), (q.shape, b),
                             (k.shape, b))
    return na.ne_attn_gqa_varlen_fwd(q, k, v, cu, mx, out=out, lse=lse, qr=qr, kr=kr)


def _backward(na, f, v, do, cu, mx, fill):
    out, lse, qr, kr = f
    b = torch.bfloat16
    dq, dk, dv = _full(fill, (qr.shape, b), (kr.shape, b), (kr.shape, b))
    return na.ne_attn_gqa_varlen_bwd(qr, kr, v, out, do, lse, cu, mx, dq=dq, dk=dk, dv=dv)


def _holds(t, x):
    """Every element of t is still x."""
    return bool(torch.isnan(t).all()) if x != x else bool((t == torch.tensor(x, dtype=t.dtype)).all())


def _check_forward(f, v, lens, which):
    out, lse, qr, kr = f
    at = 0
    for s, m in enumerate(lens):
        r = slice(at, at + m)
        at += m
        if s not in which:
            continue
        o, l, oe, le = attention(qr[r], kr[r], v[r], 0.125)
        within(out[r], o, oe, f"out of sequence {s}")
        within(lse[:, r], l, le, f"lse of sequence {s}")


def _check_backward(f, g, v, do, lens, which):
    (out, lse, qr, kr), (dq, dk, dv) = f, g
    at = 0
    for s, m in enumerate(lens):
        r = slice(at, at + m)
        at += m
        if s not in which:
            continue
        (gq, gk, gv), (eq, ek, ev) = attention_grads(qr[r], kr[r], v[r], out[r], do[r], lse[:, r],
                                                     0.125)
        p = torch.arange(m, device="cuda")
        for name, a, b, e in (
                ("dq", dq[r], rotate(gq, p, back=True), unrotate_bound(gq, eq, 1)),
                ("dk", dk[r], rotate(gk, p, back=True), unrotate_bound(gk, ek, 1)),
                ("dv", dv[r], gv, ev)):
            within(a, b, e, f"{name} of sequence {s}")


# ------------------------------------------------------------------- backward

@pytest.mark.parametrize("last", [1, 60, 127, 128, 300])
@pytest.mark.parametrize("H,Hkv", HEADS)
@pytest.mark.parametrize("stale", STALE)
def test_backward_with_stale_rows_behind(na, stale, H, Hkv, last):
    """A padded packed buffer: behind the last sequence every input of the backward
    holds what it may (and the outputs there stay as they were)."""
    lens = [70, last]
    tot, behind = sum(lens), 150
    q, k, v, do = _inputs(1, tot + behind, H, Hkv)
    cu = _cu(lens)
    f = _forward(na, q, k, v, cu, 300, 0.0)
    for t in (v, do, f[0], f[2], f[3]):
        t[tot:] = stale
    f[1][:, tot:] = stale
    g = _backward(na, f, v, do, cu, 300, stale)
    assert na.ne_attn_get_device_status() == 0
    _check_backward(f, g, v, do, lens, range(2))
    assert all(_holds(t[tot:], stale) for t in g)


@pytest.mark.parametrize("stale", [NAN, INF])
@pytest.mark.parametrize("name", ["qr", "kr", "v", "dout", "out", "lse"])
@pytest.mark.parametrize("H,Hkv", HEADS)
def test_backward_beside_a_bad_neighbour(na, H, Hkv, name, stale):
    """One tensor of one sequence at a time is all NaN or infinite: the gradients of
    the others are those of the clean batch."""
    q, k, v, do = _inputs(11, sum(LENS), H, Hkv)
    cu = _cu(LENS)
    f = _forward(na, q, k, v, cu, 400, 0.0)
    want = _backward(na, f, v, do, cu, 400, 0.0)
    for bad in range(len(LENS)):
        r = slice(sum(LENS[:bad]), sum(LENS[:bad + 1]))
        ff, vv, dd = [t.clone() for t in f], v.clone(), do.clone()
        spoiled = dict(qr=ff[2], kr=ff[3], v=vv, dout=dd, out=ff[0], lse=ff[1].T)[name]
        spoiled[r] = stale
        g = _backward(na, ff, vv, dd, cu, 400, 0.0)
        assert na.ne_attn_get_device_status() == 0
        others = torch.ones(sum(LENS), dtype=torch.bool, device="cuda")
        others[r] = False
        for a, w in zip(g[1:], want[1:]):
            assert torch.equal(a[others], w[others])
        _check_backward(f, g, v, do, LENS, [s for s in range(len(LENS)) if s != bad])


@pytest.mark.parametrize("H,Hkv", [(12, 4), (12, 1)])
def test_backward_of_a_larger_batch_beside_a_bad_neighbour(na, H, Hkv):
    """So many rows that a group stays whole (12 on 4), or is split in shares of
    several heads (12 on 1): a unit then walks a sequence's last tile once a head."""
    lens = [1000 - 9 * i for i in range(8)]
    q, k, v, do = _inputs(71, sum(lens), H, Hkv)
    cu = _cu(lens)
    f = _forward(na, q, k, v, cu, 1000, 0.0)
    for bad in (0, 3, 7):
        r = slice(sum(lens[:bad]), sum(lens[:bad + 1]))
        ff, vv, dd = [t.clone() for t in f], v.clone(), do.clone()
        for t in (ff[0], ff[1].T, ff[2], ff[3], vv, dd):
            t[r] = NAN
        g = _backward(na, ff, vv, dd, cu, 1000, 0.0)
        assert na.ne_attn_get_device_status() == 0
        _check_backward(f, g, v, do, lens, [s for s in range(8) if s != bad])


def test_backward_beside_a_skipped_sequence(na):
    """A sequence longer than the bound is reported and skipped by the forward, which
    leaves its rotated operands unwritten; the backward of the same call gives the
    others' gradients."""
    lens = [100, 400, 60]
    q, k, v, do = _inputs(21, sum(lens), 4, 2)
    cu = _cu(lens)
    f = _forward(na, q, k, v, cu, 399, NAN)
    assert na.ne_attn_get_device_status() == 7
    assert all(_holds(t[100:500], NAN) for t in (f[0], f[1].T, f[2], f[3]))
    g = _backward(na, f, v, do, cu, 399, NAN)
    assert na.ne_attn_get_device_status() == 7
    assert all(_holds(t[100:500], NAN) for t in g)
    _check_backward(f, g, v, do, lens, (0, 2))


def test_backward_of_a_padded_step_in_a_graph(na):
    """The forward and backward of a padded batch, captured once and replayed with
    other lengths on the device; the padding holds NaN throughout."""
    room = 1000
    q, k, v, do = _inputs(31, room, 6, 2)
    cu = _cu([300, 200, 100])
    f = _forward(na, q, k, v, cu, 400, 0.0)  # outside the capture first
    _backward(na, f, v, do, cu, 400, 0.0)
    clean = [t.clone() for t in (q, k, v, do)]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        f = _forward(na, q, k, v, cu, 400, NAN)
        g = _backward(na, f, v, do, cu, 400, NAN)
    for lens in ([300, 200, 100], [1, 0, 129], [400, 399, 77]):
        for t, c in zip((q, k, v, do), clean):
            t.copy_(c)
            t[sum(lens):] = NAN
        cu.copy_(_cu(lens))
        graph.replay()
        torch.cuda.synchronize()
        assert na.ne_attn_get_device_status() == 0
        which = [s for s in range(3) if lens[s]]
        _check_forward(f, v, lens, which)
        _check_backward(f, g, v, do, lens, which)
        assert all(_holds(t[sum(lens):], NAN) for t in (f[0], f[1].T, f[2], f[3], *g))


# -------------------------------------------------------------------- forward

@pytest.mark.parametrize("last", [1, 60, 127, 128, 300])
@pytest.mark.parametrize("H,Hkv", HEADS)
@pytest.mark.parametrize("stale", STALE)
def test_forward_with_stale_rows_behind(na, stale, H, Hkv, last):
    lens = [70, last]
    tot, behind = sum(lens), 150
    q, k, v, _ = _inputs(41, tot + behind, H, Hkv)
    for t in (q, k, v):
        t[tot:] = stale
    f = _forward(na, q, k, v, _cu(lens), 300, stale)
    assert na.ne_attn_get_device_status() == 0
    _check_forward(f, v, lens, range(2))
    assert all(_holds(t[tot:], stale) for t in (f[0], f[1].T, f[2], f[3]))


@pytest.mark.parametrize("stale", [NAN, INF])
@pytest.mark.parametrize("name", ["q", "k", "v"])
@pytest.mark.parametrize("H,Hkv", HEADS)
def test_forward_beside_a_bad_neighbour(na, H, Hkv, name, stale):
    q, k, v, _ = _inputs(51, sum(LENS), H, Hkv)
    cu = _cu(LENS)
    want = _forward(na, q, k, v, cu, 400, 0.0)
    for bad in range(len(LENS)):
        r = slice(sum(LENS[:bad]), sum(LENS[:bad + 1]))
        x = dict(q=q, k=k, v=v)
        x[name] = x[name].clone()
        x[name][r] = stale
        f = _forward(na, x["q"], x["k"], x["v"], cu, 400, 0.0)
        assert na.ne_attn_get_device_status() == 0
        others = torch.ones(sum(LENS), dtype=torch.bool, device="cuda")
        others[r] = False
        for a, w in zip((f[0], f[1].T, f[2], f[3]), (want[0], want[1].T, want[2], want[3])):
            assert torch.equal(a[others], w[others])


def test_forward_of_a_bound_without_a_work_list_beside_stale_rows(na):
    """A bound so far above the lengths that no list of the items is made."""
    lens = [(i * 7) % 23 for i in range(300)] + [700]
    tot = sum(lens)
    q, k, v, do = _inputs(61, tot + 50, 6, 2)
    for t in (q, k, v, do):
        t[tot:] = NAN
    cu = _cu(lens)
    f = _forward(na, q, k, v, cu, 40000, NAN)
    g = _backward(na, f, v, do, cu, 40000, NAN)
    assert na.ne_attn_get_device_status() == 0
    which = [s for s in range(0, 301, 20) if lens[s]]
    _check_forward(f, v, lens, which)
    _check_backward(f, g, v, do, lens, which)

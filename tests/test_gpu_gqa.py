"""Attention with shared key/value heads over packed prompts, and its gradients,
against the plain 64-bit implementations of grouped.py with bounds that count
the roundings (derived there)."""
import pytest
import torch

from grouped import (F64, U16, Cache, attention, attention_grads, positions, rotate,
                     rotate_bound, unrotate_bound, within)

pytestmark = pytest.mark.gpu
BASE = 10000.0


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


def _randn(seed, *shape, scale=1.0):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).bfloat16().cuda()


def _check(na, lens, H, Hkv, seed=0, qscale=1.0, max_seqlen=None, behind=0, grads=True):
    tot = sum(lens)
    q = _randn(seed, tot + behind, H, 64, scale=qscale)
    k, v = (_randn(seed + i, tot + behind, Hkv, 64, scale=qscale if i == 1 else 1) for i in (1, 2))
    do = _randn(seed + 3, tot + behind, H, 64)
    cu, mx = _cu(lens), max_seqlen or max(lens)
    seven = lambda *s, t=torch.bfloat16: torch.full(s, 7.0, dtype=t, device="cuda")  # noqa: E731
    n = tot + behind
    out, lse, qr, kr = na.ne_attn_gqa_varlen_fwd(
        q, k, v, cu, mx, out=seven(n, H, 64), lse=seven(H, n, t=torch.float32),
        qr=seven(n, H, 64), kr=seven(n, Hkv, 64))
    assert na.ne_attn_get_device_status() == 0
    pos = positions(cu.tolist(), "cuda")
    for got, x in ((qr, q), (kr, k)):
        want = rotate(x[:tot], pos, BASE)
        within(got[:tot], want, rotate_bound(x[:tot]) + U16 * want.abs(), "rotation")
    if grads:
        dq, dk, dv = na.ne_attn_gqa_varlen_bwd(
            qr, kr, v, out, do, lse, cu, mx, dq=seven(n, H, 64), dk=seven(n, Hkv, 64),
            dv=seven(n, Hkv, 64))
        assert na.ne_attn_get_device_status() == 0
    for t in [out, qr, kr] + ([dq, dk, dv] if grads else []):
        assert bool((t[tot:] == 7).all())
    assert bool((lse[:, tot:] == 7).all())
    worst, at = {}, 0
    for s, m in enumerate(lens):
        r = slice(at, at + m)
        at += m
        if m == 0:
            continue
        o, l, oe, le = attention(qr[r], kr[r], v[r], 0.125)
        res = [("out", out[r], o, oe), ("lse", lse[:, r], l, le)]
        if grads:
            (gq, gk, gv), (eq, ek, ev) = attention_grads(qr[r], kr[r], v[r], out[r], do[r],
                                                         lse[:, r], 0.125)
            p = torch.arange(m, device="cuda")
            res += [("dq", dq[r], rotate(gq, p, BASE, back=True), unrotate_bound(gq, eq, 1)),
                    ("dk", dk[r], rotate(gk, p, BASE, back=True), unrotate_bound(gk, ek, 1)),
                    ("dv", dv[r], gv, ev)]
        for name, a, b, e in res:
            worst[name] = max(worst.get(name, 0.0), within(a, b, e, f"{name} of sequence {s}"))
    print({k: round(x, 3) for k, x in worst.items()})


LENS = [1, 2, 0, 63, 64, 65, 127, 128, 129, 255, 256, 257, 384, 500]


@pytest.mark.parametrize("H,Hkv", [(4, 2), (6, 2), (2, 1), (3, 1)])
def test_ragged(na, H, Hkv):
    _check(na, LENS, H, Hkv, seed=100, behind=5)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 4), (12, 4), (12, 2), (16, 1), (5, 1), (14, 2),
                                   (32, 8), (17, 1)])
def test_head_layouts(na, H, Hkv):
    _check(na, [300, 5], H, Hkv, seed=110)


@pytest.mark.parametrize("n", [1, 127, 128, 129, 1000, 2049])
@pytest.mark.parametrize("H,Hkv", [(4, 1), (3, 1)])
def test_one_sequence(na, n, H, Hkv):
    _check(na, [n], H, Hkv, seed=120)


def test_long(na):
    _check(na, [5000], 4, 2, seed=130)


def test_sharp_scores(na):
    _check(na, [400, 130], 4, 2, seed=140, qscale=4.0)


def test_many_short_sequences(na):
    _check(na, [(i * 11) % 40 for i in range(200)], 4, 1, seed=150)


def test_a_bound_above_the_lengths(na):
    _check(na, [100, 300], 6, 3, seed=160, max_seqlen=4000)


def _shares(na, lens, H, Hkv):
    """Units per (key tile, key/value head): the partials that the workspace holds."""
    al = lambda x: (x + 255) // 256 * 256  # noqa: E731
    n = sum(lens)
    extra = na.ne_attn_gqa_bwd_workspace_bytes(n, max(lens), H, Hkv) - al(n * H * 256) - al(n * H * 4)
    return max(1, round(extra / (2 * n * Hkv * 256)))


def test_no_tokens(na):
    """Every sequence is empty: nothing is written."""
    _check(na, [0, 0], 3, 1, seed=166, max_seqlen=300, behind=7)


def test_two_calls_at_once(na):
    """Calls in flight on two streams: as one after the other."""
    lens = [900, 40, 300]
    cu, sets = _cu(lens), []
    for i in range(6):
        q, k, v, do = (_randn(300 + 4 * i + j, sum(lens), h, 64) for j, h in enumerate((6, 2, 2, 6)))
        sets.append((q, k, v, do))

    def step(q, k, v, do, stream=None):
        f = na.ne_attn_gqa_varlen_fwd(q, k, v, cu, 900, stream=stream)
        return f + tuple(na.ne_attn_gqa_varlen_bwd(f[2], f[3], v, f[0], do, f[1], cu, 900,
                                                   stream=stream))

    want = [step(*x) for x in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [step(*x, stream=streams[i % 2]) for i, x in enumerate(sets)]
    torch.cuda.synchronize()
    assert na.ne_attn_get_device_status() == 0
    for g, w in zip(got, want):
        for i, (a, b) in enumerate(zip(g, w)):
            if i == 4:  # dq: the order of its fp32 sums
                assert float((a.double() - b.double()).norm()) <= 1e-3 * float(b.double().norm())
            else:
                assert torch.equal(a, b), i


def test_more_items_than_a_list_holds(na):
    """A bound so far above the lengths that nearly all of the items are empty."""
    _check(na, [(i * 7) % 23 for i in range(300)] + [700], 6, 2, seed=165, max_seqlen=40000)


@pytest.mark.parametrize("shares", [1, 2, 3, 5])
def test_every_share_of_a_group(na, shares):
    """A group as one unit, in shares of several heads, even and uneven, and with a
    head each: the smallest batch (of up to 40 sequences, the last one shorter)
    that the backward splits so."""
    for H, Hkv in ((5, 1), (10, 2), (6, 1), (12, 4)):
        for n in (300, 900, 1500):
            for nseq in range(1, 40):
                lens = [n] * nseq + [n // 3]
                if _shares(na, lens, H, Hkv) == shares:
                    _check(na, lens, H, Hkv, seed=170)
                    return
    pytest.fail("no such batch")


def test_agrees_with_the_ungrouped_pair_when_heads_are_not_shared(na):
    """The same operands and the same weights: what differs is the order of the fp32
    row sums (2^-20 of them at most) and, in dk, that the ungrouped pair rounds twice."""
    lens = [1, 300, 129, 0, 700]
    tot = sum(lens)
    q, k, v, do = (_randn(180 + i, tot, 3, 64) for i in range(4))
    cu = _cu(lens)
    a = na.ne_attn_gqa_varlen_fwd(q, k, v, cu, 700)
    b = na.ne_attn_varlen_fwd_train(q, k, v, cu, 700)
    assert torch.equal(a[2], b[2]) and torch.equal(a[3], b[3])
    step = 2 * U16  # one bf16 step: a value at a rounding border may fall on either side
    within(a[0], b[0].to(F64), step * b[0].to(F64).abs() + 1e-6, "out")
    within(a[1], b[1].to(F64), torch.full_like(b[1].to(F64), 2.0 ** -19), "lse")
    out, lse, qr, kr = a
    g = na.ne_attn_gqa_varlen_bwd(qr, kr, v, out, do, lse, cu, 700)
    w = na.ne_attn_varlen_bwd_train(qr, kr, v, out, do, lse, cu, 700)
    assert torch.equal(g[2], w[2])
    # dk = R^T x: one rounding of it against a rounding of x's pair of elements (each
    # at most U16 of the pair's length r, sqrt(2) of that together) and one of dk.
    x = w[1].to(F64)
    r = torch.hypot(x[..., :32], x[..., 32:]).repeat(1, 1, 2)
    within(g[1], x, (2 + 1.5) * U16 * r + 1e-6, "dk")


def test_bad_sequence_is_reported_and_skipped(na):
    lens = [100, 400, 60]
    tot = sum(lens)
    q, k, v, do = (_randn(190 + i, tot, h, 64) for i, h in enumerate((4, 2, 2, 4)))
    cu = _cu(lens)
    want = na.ne_attn_gqa_varlen_fwd(q, k, v, cu, 400)
    wg = na.ne_attn_gqa_varlen_bwd(want[2], want[3], v, want[0], do, want[1], cu, 400)
    assert na.ne_attn_get_device_status() == 0
    mark = [torch.full_like(t, 7.0) for t in want]
    out, lse, qr, kr = na.ne_attn_gqa_varlen_fwd(q, k, v, cu, 399, out=mark[0], lse=mark[1],
                                                 qr=mark[2], kr=mark[3])
    assert na.ne_attn_get_device_status() == 7
    for t, w in ((out, want[0]), (qr, want[2]), (kr, want[3])):
        assert torch.equal(t[:100], w[:100]) and torch.equal(t[500:], w[500:])
        assert bool((t[100:500] == 7).all())
    gm = [torch.full_like(t, 7.0) for t in wg]
    g = na.ne_attn_gqa_varlen_bwd(want[2], want[3], v, want[0], do, want[1], cu, 399, dq=gm[0],
                                  dk=gm[1], dv=gm[2])
    assert na.ne_attn_get_device_status() == 7
    for t, w in zip(g[1:], wg[1:]):
        assert torch.equal(t[:100], w[:100]) and torch.equal(t[500:], w[500:])
    assert all(bool((t[100:500] == 7).all()) for t in g)


def test_gradients_are_deterministic_but_for_dq(na):
    lens = [700, 700]
    q, k, v, do = (_randn(200 + i, 1400, h, 64) for i, h in enumerate((6, 2, 2, 6)))
    cu = _cu(lens)
    out, lse, qr, kr = na.ne_attn_gqa_varlen_fwd(q, k, v, cu, 700)
    runs = [na.ne_attn_gqa_varlen_bwd(qr, kr, v, out, do, lse, cu, 700) for _ in range(4)]
    for g in runs[1:]:
        assert torch.equal(g[1], runs[0][1]) and torch.equal(g[2], runs[0][2])


def test_streams_workspaces_and_graphs(na):
    lens = [700, 3, 0, 257]
    tot = sum(lens)
    q, k, v, do = (_randn(210 + i, tot, h, 64) for i, h in enumerate((6, 2, 2, 6)))
    cu = _cu(lens)

    def step(stream=None, ws=None):
        out, lse, qr, kr = na.ne_attn_gqa_varlen_fwd(q, k, v, cu, 700, stream=stream)
        return (out, lse, qr, kr) + tuple(na.ne_attn_gqa_varlen_bwd(
            qr, kr, v, out, do, lse, cu, 700, workspace=ws, stream=stream))

    def same(a, b):
        for i, (x, y) in enumerate(zip(a, b)):
            if i == 4:  # dq: the order of its fp32 sums
                assert float((x.double() - y.double()).norm()) <= 1e-3 * float(y.double().norm())
            else:
                assert torch.equal(x, y), i

    want = step()
    torch.cuda.synchronize()
    need = na.ne_attn_gqa_bwd_workspace_bytes(tot, 700, 6, 2)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    same(step(ws=ws), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side, ws=ws)
    side.synchronize()
    same(got, want)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        outs = step()
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        same(outs, want)
    assert na.ne_attn_get_device_status() == 0


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_model_run_prompt_cache_generate(na, e4m3):
    """The operators as they are used together: prompts through the forward, its
    k' into the cache, then two generated tokens per sequence, each appended and
    attended; against attention over all rows so far in 64 bits (on the cache's
    own values)."""
    lens, H, Hkv, page = [70, 1, 300], 6, 2, 32
    B, tot = len(lens), sum(lens)
    c = Cache([n + 2 for n in lens], Hkv, page, e4m3, seed=300)
    q, k, v = (_randn(301 + i, tot, h, 64) for i, h in enumerate((H, Hkv, Hkv)))
    cu = _cu(lens)
    out, lse, qr, kr = na.ne_attn_gqa_varlen_fwd(q, k, v, cu, max(lens))
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    na.ne_kv_append(kr, v, cu, zero, c.k, c.v, c.table, 302, c.ks, c.vs, rope_base=0.0)
    now = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ones = _cu([1] * B)
    for t in range(2):
        q1, k1, v1 = (_randn(310 + 3 * t + i, B, h, 64) for i, h in enumerate((H, Hkv, Hkv)))
        na.ne_kv_append(k1, v1, ones, now, c.k, c.v, c.table, 302, c.ks, c.vs, rope_base=BASE)
        now = now + 1
        o1, l1 = na.ne_attn_decode_paged(q1, c.k, c.v, c.table, now, 302, c.ks, c.vs,
                                         rope_base=BASE)
        assert na.ne_attn_get_device_status() == 0
        for s in range(B):
            n = lens[s] + t + 1
            kk, vv = c.rows(s, n)
            qq = rotate(q1[s:s + 1], torch.tensor([n - 1], device="cuda"), BASE)
            o, l, oe, le = attention(qq, kk, vv, 0.125)
            # q' is rounded to bf16: a score moves by at most this.
            G = H // Hkv
            slack = 0.125 * U16 * torch.einsum("hgd,mhd->hgm", qq[0].abs().view(Hkv, G, 64),
                                               kk.abs()).amax(-1).reshape(H)
            le = le + slack[:, None]
            oe = oe + 2 * slack[None, :, None] * vv.abs().amax(0).repeat_interleave(G, 0)[None]
            within(o1[s], o[0], oe[0], "out")
            within(l1[s], l[:, 0], le[:, 0], "lse")
    if not e4m3:  # the prompt's rows come back as the forward wrote them
        kb, vb = na.ne_kv_read(c.k, c.v, c.table, cu, zero, tot)
        assert torch.equal(kb, kr) and torch.equal(vb, v)
    # The first generated token equals row n of a prompt one token longer.
    assert torch.isfinite(out.float()).all()

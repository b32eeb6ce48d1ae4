"""Norms of queries and keys with the rotation in the same pass, and their gradients,
against the plain 64-bit implementations of step.py (bounds derived there)."""
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import step
from grouped import F64, within

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module")
def na():
    from causal_self_attention_gb300 import build, ne_attn
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ne_attn


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _randn(seed, *shape, scale=1.0):
    g = torch.Generator("cpu").manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).bfloat16().cuda()


def _inputs(seed, N, H, Hkv, joint):
    """q, k (slices of a joint projection's output, or alone), weights, positions."""
    if joint:
        qkv = _randn(seed, N, H + 2 * Hkv, 64, scale=2)
        q, k = qkv[:, :H], qkv[:, H:H + Hkv]
    else:
        q, k = _randn(seed, N, H, 64), _randn(seed + 1, N, Hkv, 64)
    wq, wk = (_randn(seed + 2 + i, 64) for i in range(2))
    g = torch.Generator("cpu").manual_seed(seed + 4)
    pos = torch.randint(0, 5000, (N,), generator=g).to(torch.int32).cuda()
    return q, k, wq, wk, pos


def _check_forward(na, q, k, wq, wk, pos, base=1e4, eps=EPS):
    qr, kr = na.ne_qk_norm_rope_fwd(q, k, wq, wk, pos, 5000, eps=eps, rope_base=base)
    assert na.ne_attn_get_device_status() == 0
    assert qr.is_contiguous() and kr.is_contiguous()
    for got, x, w, name in ((qr, q, wq, "qr"), (kr, k, wk, "kr")):
        want, err = step.norm(x, w, eps, pos, base)
        within(got, want, err, name)


def _check_backward(na, q, k, wq, wk, pos, base=1e4, eps=EPS, seed=90, **kw):
    dqr, dkr = (_randn(seed + i, *t.shape) for i, t in enumerate((q, k)))
    dq, dk, dwq, dwk = na.ne_qk_norm_rope_bwd(dqr, dkr, q, k, wq, wk, pos, 5000, eps=eps,
                                              rope_base=base, **kw)
    assert na.ne_attn_get_device_status() == 0
    for dr, x, w, dx, dw, name in ((dqr, q, wq, dq, dwq, "dq"), (dkr, k, wk, dk, dwk, "dk")):
        gx, gw, ex, ew = step.norm_grads(dr, x, w, eps, pos, base)
        within(dx, gx, ex, name)
        within(dw, gw, ew, name + "_weight")


@pytest.mark.parametrize("N", [1, 2, 7, 64, 65, 700])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (12, 4), (3, 5), (33, 1), (32, 8)])
@pytest.mark.parametrize("joint", [False, True])
def test_sizes_and_layouts(na, N, H, Hkv, joint):
    a = _inputs(N + H, N, H, Hkv, joint)
    _check_forward(na, *a)
    _check_backward(na, *a)


@pytest.mark.parametrize("N,H,Hkv", [(9001, 12, 4), (20011, 2, 1)])
def test_many_rows(na, N, H, Hkv):
    a = _inputs(1, N, H, Hkv, True)
    _check_forward(na, *a)
    _check_backward(na, *a)


@pytest.mark.parametrize("N,H,Hkv", [(9001, 9, 3), (3001, 33, 1), (20001, 3, 2), (20003, 1, 3),
                                     (40001, 1, 1)])
def test_many_rows_of_odd_heads(na, N, H, Hkv):
    """Rows enough to fill the GPU, with heads that a quad's share divides or not."""
    a = _inputs(2, N, H, Hkv, False)
    _check_forward(na, *a)
    _check_backward(na, *a)


def test_rows_far_apart(na):
    """Rows 2^30 elements apart (2 GiB): offsets past 32 bits, of inputs and of gradients."""
    N, H, Hkv, far = 3, 5, 2, 2 ** 30
    q, k, wq, wk, pos = _inputs(8, N, H, Hkv, False)

    def spread(x, at):
        room = torch.empty((N - 1) * far + 1024, dtype=torch.bfloat16, device="cuda")
        y = room.as_strided(x.shape, (far, 64, 1), at)
        y.copy_(x)
        return y

    a = spread(q, 0), spread(k, 64), wq, wk, pos
    _check_forward(na, *a)
    _check_backward(na, *a, dq=spread(torch.zeros_like(q), 8), dk=spread(torch.zeros_like(k), 512))


def test_norm_alone(na):
    q, k, wq, wk, _ = _inputs(3, 130, 4, 2, True)
    for pos in (None, _i32([5] * 130)):
        _check_forward(na, q, k, wq, wk, pos, base=0.0)
        _check_backward(na, q, k, wq, wk, pos, base=0.0)


@pytest.mark.parametrize("scale", [1e-30, 1e-3, 1e15])
def test_magnitudes(na, scale):
    """Small rows are eps's, large ones their own norm's; a row of zeros stays zero."""
    q, k, wq, wk, pos = _inputs(5, 100, 4, 2, False)
    q, k = (q.float() * scale).bfloat16(), (k.float() * scale).bfloat16()
    q[3] = 0
    k[:, 1] = 0
    _check_forward(na, q, k, wq, wk, pos)
    qr, kr = na.ne_qk_norm_rope_fwd(q, k, wq, wk, pos, 5000)
    assert bool((qr[3] == 0).all()) and bool((kr[:, 1] == 0).all())


@pytest.mark.parametrize("scale", [1e-3, 1e3])
def test_gradients_of_magnitudes(na, scale):
    q, k, wq, wk, pos = _inputs(6, 100, 4, 2, False)
    q, k = (q.float() * scale).bfloat16(), (k.float() * scale).bfloat16()
    q[3] = 0
    _check_backward(na, q, k, wq, wk, pos)


def test_rows_of_no_sequence_and_bad_positions(na):
    """Position -1: left alone, whatever the row holds; other bad ones are reported."""
    N = 300
    q, k, wq, wk, pos = _inputs(7, N, 12, 4, True)
    dead = torch.zeros(N, dtype=torch.bool, device="cuda")
    dead[[0, 5, 150, 298, 299]] = True
    pos[dead] = -1
    live = ~dead
    q[dead], k[dead] = float("nan"), float("inf")
    qr, kr = torch.full((N, 12, 64), 7.0, dtype=torch.bfloat16, device="cuda"), \
        torch.full((N, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    na.ne_qk_norm_rope_fwd(q, k, wq, wk, pos, 5000, qr=qr, kr=kr)
    assert na.ne_attn_get_device_status() == 0
    for got, x, w in ((qr, q, wq), (kr, k, wk)):
        assert bool((got[dead] == 7).all())
        want, err = step.norm(x[live], w, EPS, pos[live])
        within(got[live], want, err, "live rows")
    dqr, dkr = _randn(70, N, 12, 64), _randn(71, N, 4, 64)
    dqr[dead], dkr[dead] = float("inf"), float("nan")
    dq, dk = torch.full_like(qr, 7.0), torch.full_like(kr, 7.0)
    _, _, dwq, dwk = na.ne_qk_norm_rope_bwd(dqr, dkr, q, k, wq, wk, pos, 5000, dq=dq, dk=dk)
    assert na.ne_attn_get_device_status() == 0
    for dr, x, w, dx, dw in ((dqr, q, wq, dq, dwq), (dkr, k, wk, dk, dwk)):
        assert bool((dx[dead] == 7).all())
        gx, gw, ex, ew = step.norm_grads(dr[live], x[live], w, EPS, pos[live])
        within(dx[live], gx, ex, "dx")
        within(dw, gw, ew, "dw")
    for bad in (5000, -2, 2 ** 31 - 1, -2 ** 31):
        pos[dead] = bad
        qr.fill_(7.0)
        na.ne_qk_norm_rope_fwd(q, k, wq, wk, pos, 5000, qr=qr, kr=kr)
        assert na.ne_attn_get_device_status() == 7
        assert bool((qr[dead] == 7).all())
        _, _, other, _ = na.ne_qk_norm_rope_bwd(dqr, dkr, q, k, wq, wk, pos, 5000)
        assert na.ne_attn_get_device_status() == 7
        assert torch.equal(other, dwq)
    pos.fill_(-1)  # no row at all
    _, _, dwq, dwk = na.ne_qk_norm_rope_bwd(dqr, dkr, q, k, wq, wk, pos, 5000)
    assert bool((dwq == 0).all()) and bool((dwk == 0).all())


def test_a_bad_row_shows_in_itself_alone(na):
    q, k, wq, wk, pos = _inputs(8, 50, 4, 2, False)
    want = na.ne_qk_norm_rope_fwd(q, k, wq, wk, pos, 5000)
    q[7, 1, 5] = float("nan")
    k[9, 0, 0] = float("inf")
    qr, kr = na.ne_qk_norm_rope_fwd(q, k, wq, wk, pos, 5000)
    for got, w, at in ((qr, want[0], (7, 1)), (kr, want[1], (9, 0))):
        same = torch.ones(got.shape[:2], dtype=torch.bool, device="cuda")
        same[at] = False
        assert torch.equal(got[same], w[same]) and not bool(torch.isfinite(got[at]).all())


def test_no_rows(na):
    q, k, wq, wk, pos = _inputs(9, 4, 4, 2, False)
    qr, kr = na.ne_qk_norm_rope_fwd(q[:0], k[:0], wq, wk, pos[:0], 5000)
    assert qr.shape == (0, 4, 64) and kr.shape == (0, 2, 64)
    got = na.ne_qk_norm_rope_bwd(q[:0], k[:0], q[:0], k[:0], wq, wk, pos[:0], 5000)
    assert bool((got[2] == 0).all()) and bool((got[3] == 0).all())


def test_gradients_into_a_joint_tensor(na):
    """dq, dk as slices: what lies between their rows stays."""
    N, H, Hkv = 90, 6, 3
    a = _inputs(10, N, H, Hkv, True)
    joint = torch.full((N, H + 2 * Hkv, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    _check_backward(na, *a, dq=joint[:, :H], dk=joint[:, H:H + Hkv])
    assert bool((joint[:, H + Hkv:] == 5).all())


def test_same_bits_streams_workspaces_and_graphs(na):
    a = _inputs(11, 800, 12, 4, True)
    d = _randn(80, 800, 12, 64), _randn(81, 800, 4, 64)
    fwd = [t.clone() for t in na.ne_qk_norm_rope_fwd(*a, 5000)]
    want = [t.clone() for t in na.ne_qk_norm_rope_bwd(*d, *a, 5000)]
    need = na.ne_qk_norm_rope_bwd_workspace_bytes()
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for kw in (dict(workspace=ws[:need]), dict(stream=side), dict(stream=side.cuda_stream)):
        got = na.ne_qk_norm_rope_bwd(*d, *a, 5000, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert bool((ws[need:] == 255).all())
    graphs = []
    for i in range(2):  # two graphs on one workspace, replayed in turn
        g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            graphs.append((g, na.ne_qk_norm_rope_fwd(*a, 5000),
                           na.ne_qk_norm_rope_bwd(*d, *a, 5000, workspace=ws[:need] if i else None)))
    for _ in range(2):
        for g, f, b in graphs:
            for t in (*f, *b):
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip((*f, *b), (*fwd, *want)))


def test_two_calls_at_once(na):
    """Calls in flight on two streams, no workspace given; and from two threads."""
    a = _inputs(12, 3000, 12, 4, True)
    ds = [(_randn(82 + i, 3000, 12, 64), _randn(92 + i, 3000, 4, 64)) for i in range(4)]
    want = [[t.clone() for t in na.ne_qk_norm_rope_bwd(*d, *a, 5000)] for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [na.ne_qk_norm_rope_bwd(*ds[i % 4], *a, 5000, stream=streams[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(g, want[i % 4]))
    with ThreadPoolExecutor(4) as pool:
        got = list(pool.map(lambda i: na.ne_qk_norm_rope_bwd(*ds[i], *a, 5000, stream=2), range(4)))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(g, w))


# ------------------------------------------------- attention on what it gives

@pytest.mark.parametrize("lens", [[300, 0, 129, 1, 700], [5]])
@pytest.mark.parametrize("H,Hkv", [(6, 2), (4, 4), (12, 1)])
def test_attention_of_rotated_operands(na, lens, H, Hkv):
    """The *_rotated prompt calls: bit for bit the calls that rotate, from their qr, kr;
    the gradients turned back are those calls' gradients."""
    from grouped import U16, positions, unrotate_bound
    n = sum(lens)
    cu = _i32([0] + [sum(lens[:i + 1]) for i in range(len(lens))])
    q, do = _randn(20, n, H, 64), _randn(21, n, H, 64)
    k, v = _randn(22, n, Hkv, 64), _randn(23, n, Hkv, 64)
    out, lse, qr, kr = na.ne_attn_gqa_varlen_fwd(q, k, v, cu, max(lens))
    o2, l2 = na.ne_attn_gqa_varlen_fwd_rotated(qr, kr, v, cu, max(lens))
    assert torch.equal(o2, out) and torch.equal(l2, lse)
    dq, dk, dv = na.ne_attn_gqa_varlen_bwd(qr, kr, v, out, do, lse, cu, max(lens))
    dqr, dkr, dv2 = na.ne_attn_gqa_varlen_bwd_rotated(qr, kr, v, out, do, lse, cu, max(lens))
    assert na.ne_attn_get_device_status() == 0
    assert torch.equal(dv2, dv)
    pos = positions(cu, q.device)
    for r, d, name in ((dqr, dq, "dq"), (dkr, dk, "dk")):
        # One rounding more (of the rotated gradient), and dq's sums in any order: n terms
        # scale dS k with sum |dS| <= 2 max |dP| <= 2 |do| |v|, the weights' sum being 1.
        turned = step.rotate(r, pos, back=True)
        most = 0.25 * float(kr.abs().max()) * float(do.float().norm(dim=-1).max()) * \
            float(v.float().norm(dim=-1).max())
        off = n * 2.0 ** -24 * most * torch.ones_like(r, dtype=F64)
        within(d, turned, unrotate_bound(r.to(F64), off, 2) + U16 * turned.abs(), name)


def test_attention_of_rotated_operands_with_many_items(na):
    """More work items than a list is made for, and a captured call."""
    nseq, H = 70, 2
    lens = [(7 * i) % 40 for i in range(nseq)]
    n = sum(lens)
    cu = _i32([0] + [sum(lens[:i + 1]) for i in range(nseq)])
    q, k, v, do = (_randn(30 + i, n, H, 64) for i in range(4))
    most = 128 * 1000  # far above the lengths: 70 * 1000 items
    out, lse, qr, kr = na.ne_attn_gqa_varlen_fwd(q, k, v, cu, most)
    got = na.ne_attn_gqa_varlen_fwd_rotated(qr, kr, v, cu, most)
    assert torch.equal(got[0], out) and torch.equal(got[1], lse)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        got = na.ne_attn_gqa_varlen_fwd_rotated(qr, kr, v, cu, 40)
        grads = na.ne_attn_gqa_varlen_bwd_rotated(qr, kr, v, out, do, lse, cu, 40)
    want = na.ne_attn_gqa_varlen_bwd_rotated(qr, kr, v, out, do, lse, cu, 40)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], out) and torch.equal(grads[1], want[1]) and torch.equal(grads[2], want[2])
    assert na.ne_attn_get_device_status() == 0


def test_training_through_norm_and_attention(na):
    """Norm, rotation and grouped attention, and back to q, k, v and the weights: the
    gradients against those of the whole in 64 bits."""
    from grouped import attention, positions
    lens, H, Hkv = [90, 130], 4, 2
    n = sum(lens)
    cu = _i32([0, 90, 220])
    q, k, wq, wk, _ = _inputs(40, n, H, Hkv, True)
    v, do = _randn(46, n, Hkv, 64), _randn(47, n, H, 64)
    pos = positions(cu, q.device).to(torch.int32)
    qr, kr = na.ne_qk_norm_rope_fwd(q, k, wq, wk, pos, 130)
    out, lse = na.ne_attn_gqa_varlen_fwd_rotated(qr, kr, v, cu, 130)
    dqr, dkr, dv = na.ne_attn_gqa_varlen_bwd_rotated(qr, kr, v, out, do, lse, cu, 130)
    got = (*na.ne_qk_norm_rope_bwd(dqr, dkr, q, k, wq, wk, pos, 130), dv)
    leaves = [t.detach().to(F64).requires_grad_() for t in (q, k, wq, wk, v)]
    a, _ = step.norm(leaves[0], leaves[2], EPS, pos)
    b, _ = step.norm(leaves[1], leaves[3], EPS, pos)
    outs = [attention(a[s:e], b[s:e], leaves[4][s:e], 0.125)[0] for s, e in ((0, 90), (90, n))]
    (torch.cat(outs) * do.to(F64)).sum().backward()
    for g, x, name in zip(got, leaves, ("dq", "dk", "dwq", "dwk", "dv")):
        # Roundings to bf16 in a row (operands, weights, dS, gradients): eight, each at most
        # 2^-8 of the value it is made of, on sums whose terms partly cancel.
        assert float((g.to(F64) - x.grad).norm()) <= 8 * 2.0 ** -8 * float(x.grad.norm()), name

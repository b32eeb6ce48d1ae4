"""Rows outside a sequence never reach its results, with a head each: a neighbour of
a packed batch or of a fixed-length one that holds NaN or infinities, and a
sequence that is skipped, whose rotated operands nothing has written."""
import pytest
import torch

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
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


def _inputs(seed, *shape):
    g = torch.Generator("cpu").manual_seed(seed)
    return [torch.randn(shape, generator=g).bfloat16().cuda() for _ in range(4)]


def _same(got, want, rows, dq=None):
    """Bit for bit in `rows`; got[dq] to the order of its fp32 sums."""
    for i, (a, b) in enumerate(zip(got, want)):
        a, b = a[rows], b[rows]
        if i == dq:
            assert bool(torch.isfinite(a).all())
            assert float((a.double() - b.double()).norm()) <= 1e-3 * float(b.double().norm())
        else:
            assert torch.equal(a, b), i


# ------------------------------------------------------------------- backward

@pytest.mark.parametrize("stale", [NAN, INF])
@pytest.mark.parametrize("name", ["q", "k", "v", "dout", "out"])
@pytest.mark.parametrize("train", [False, True])
def test_packed_backward_beside_a_bad_neighbour(na, train, name, stale):
    q, k, v, do = _inputs(1, sum(LENS), 3, 64)
    cu = _cu(LENS)
    fwd = na.ne_attn_varlen_fwd_train if train else na.ne_attn_varlen_fwd
    bwd = na.ne_attn_varlen_bwd_train if train else na.ne_attn_varlen_bwd
    f = fwd(q, k, v, cu, 400)
    x = dict(q=f[2] if train else q, k=f[3] if train else k, v=v, out=f[0], dout=do)
    want = bwd(*x.values(), f[1], cu, 400)
    for bad in range(len(LENS)):
        r = slice(sum(LENS[:bad]), sum(LENS[:bad + 1]))
        y = dict(x)
        y[name] = y[name].clone()
        y[name][r] = stale
        others = torch.ones(sum(LENS), dtype=torch.bool, device="cuda")
        others[r] = False
        _same(bwd(*y.values(), f[1], cu, 400), want, others, dq=0)
        assert na.ne_attn_get_device_status() == 0


@pytest.mark.parametrize("T", [1, 200, 256])
@pytest.mark.parametrize("name", ["q", "k", "v", "dout", "out"])
@pytest.mark.parametrize("pair", ["plain", "train", "rotated", "noalloc"])
def test_fixed_length_backward_beside_a_bad_neighbour(na, pair, name, T):
    q, k, v, do = _inputs(2, 3, T, 2, 64)
    f = {"train": na.ne_attn_fwd_train, "rotated": na.ne_attn_fwd_rotated}.get(
        pair, na.ne_attn_fwd)(q, k, v)
    bwd = dict(plain=na.ne_attn_bwd, train=na.ne_attn_bwd_train, rotated=na.ne_attn_bwd_rotated,
               noalloc=na.ne_attn_bwd_noalloc)[pair]
    x = dict(q=f[2] if pair == "train" else q, k=f[3] if pair == "train" else k, v=v, out=f[0],
             dout=do)
    want = bwd(*x.values(), f[1])
    for bad in range(3):
        y = dict(x)
        y[name] = y[name].clone()
        y[name][bad] = NAN
        _same(bwd(*y.values(), f[1]), want, [b for b in range(3) if b != bad], dq=0)
        assert na.ne_attn_get_device_status() == 0


@pytest.mark.parametrize("train", [False, True])
def test_packed_backward_beside_a_skipped_sequence(na, train):
    lens = [100, 400, 60]
    q, k, v, do = _inputs(3, sum(lens), 3, 64)
    cu = _cu(lens)
    nan = lambda *s, t=torch.bfloat16: torch.full(s, NAN, dtype=t, device="cuda")  # noqa: E731
    n = sum(lens)
    others = torch.ones(n, dtype=torch.bool, device="cuda")
    others[100:500] = False

    def step(mx):
        outs = dict(out=nan(n, 3, 64), lse=nan(3, n, t=torch.float32))
        if train:
            outs.update(qr=nan(n, 3, 64), kr=nan(n, 3, 64))
            f = na.ne_attn_varlen_fwd_train(q, k, v, cu, mx, **outs)
            return na.ne_attn_varlen_bwd_train(f[2], f[3], v, f[0], do, f[1], cu, mx)
        f = na.ne_attn_varlen_fwd(q, k, v, cu, mx, **outs)
        need = na.ne_attn_bwd_workspace_bytes(n, 3)
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN patterns
        return na.ne_attn_varlen_bwd(q, k, v, f[0], do, f[1], cu, mx, workspace=ws)

    want = step(400)
    assert na.ne_attn_get_device_status() == 0
    got = step(399)
    assert na.ne_attn_get_device_status() == 7
    _same(got, want, others, dq=0)


# -------------------------------------------------------------------- forward

@pytest.mark.parametrize("stale", [NAN, INF])
@pytest.mark.parametrize("name", ["q", "k", "v"])
@pytest.mark.parametrize("form", ["plain", "f32out", "train"])
def test_packed_forward_beside_a_bad_neighbour(na, form, name, stale):
    q, k, v, _ = _inputs(4, sum(LENS), 3, 64)
    cu = _cu(LENS)

    def fwd(q, k, v):
        if form == "train":
            f = na.ne_attn_varlen_fwd_train(q, k, v, cu, 400)
        else:
            f = na.ne_attn_varlen_fwd(q, k, v, cu, 400, out_f32=form == "f32out")
        return (f[0], f[1].T) + tuple(f[2:])

    want = fwd(q, k, v)
    for bad in range(len(LENS)):
        r = slice(sum(LENS[:bad]), sum(LENS[:bad + 1]))
        x = dict(q=q, k=k, v=v)
        x[name] = x[name].clone()
        x[name][r] = stale
        others = torch.ones(sum(LENS), dtype=torch.bool, device="cuda")
        others[r] = False
        _same(fwd(**x), want, others)
        assert na.ne_attn_get_device_status() == 0


@pytest.mark.parametrize("T", [1, 200, 256, 2100])
@pytest.mark.parametrize("name", ["q", "k", "v"])
def test_fixed_length_forward_beside_a_bad_neighbour(na, name, T):
    """Short sequences rotate their keys in the tiles, long ones (2100) in a pass."""
    q, k, v, _ = _inputs(5, 3, T, 2, 64)
    for fwd in (na.ne_attn_fwd, na.ne_attn_fwd_train, na.ne_attn_fwd_rotated):
        want = fwd(q, k, v)
        for bad in range(3):
            x = dict(q=q, k=k, v=v)
            x[name] = x[name].clone()
            x[name][bad] = NAN
            _same(fwd(*x.values()), want, [b for b in range(3) if b != bad])
            assert na.ne_attn_get_device_status() == 0

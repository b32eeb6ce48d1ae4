"""The calls of a generation step as they are marshalled in native code (the regular ones)
and in Python (the others): the same results, the same refusals."""
import gc
import threading

import numpy as np
import pytest
import torch

from grouped import Cache
from step import Cache4
from test_gpu_paged import _cu, _i32, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def na():
    from causal_self_attention_gb300 import build, ne_attn
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ne_attn.lib()
    return ne_attn


def _norm_args():
    qkv = _randn(1, 40, 10, 64)
    return [qkv[:, :6], qkv[:, 6:8], _randn(2, 64), _randn(3, 64),
            torch.arange(40, dtype=torch.int32, device="cuda"), 64]


def _pages_args():
    table = torch.full((3, 8), -1, dtype=torch.int32, device="cuda")
    table[1, 0] = 9
    return [_i32([0, 5, 0]), table, torch.arange(20, dtype=torch.int32, device="cuda"), _i32([9])]


def _caches():
    lens = [40, 0, 70]
    return [Cache(lens, 2, 16, False, seed=4).fill_random(5), Cache(lens, 2, 16, True, seed=4).fill_random(5),
            Cache4(lens, 2, 16, seed=4).fill_random(5)]


def _calls(na):
    """(name in ne_step, call(**kw) -> tensors and written state): fresh arguments each."""
    def norm(**kw):
        return na.ne_qk_norm_rope_fwd(*_norm_args(), **kw)

    def norm_bwd(**kw):
        a = _norm_args()
        return na.ne_qk_norm_rope_bwd(_randn(6, 40, 6, 64), _randn(7, 40, 2, 64), *a, **kw)

    def reserve(**kw):
        a = _pages_args()
        return (*na.ne_kv_reserve(_i32([20, 30, 1]), *a, 60, 16, 128, **kw), *a)

    def release(**kw):
        a = _pages_args()
        na.ne_kv_release(torch.tensor([0, 1, 0], device="cuda").bool(), *a, 16, 128, **kw)
        return a

    def append(**kw):
        got = []
        for c in _caches():
            na.ne_kv_append(_randn(8, 6, 2, 64), _randn(9, 6, 2, 64), _cu([3, 0, 3]), _i32([37, 0, 11]),
                            c.k, c.v, c.table, 70, c.ks, c.vs, **kw)
            got += [x.view(torch.uint8) for x in (c.k, c.v)] + [x for x in (c.ks, c.vs) if x is not None]
        return got

    def read(**kw):
        got = []
        for c in _caches():
            for top in (None, 70):
                got += na.ne_kv_read(c.k, c.v, c.table, _cu([40, 0, 70]), _i32([0, 0, 0]), 110, c.ks,
                                     c.vs, max_seqlen=top, **kw)
        return got

    def decode(**kw):
        got = []
        for c in _caches():
            for scale in (None, 0.25, 1):
                got += na.ne_attn_decode_paged(_randn(10, 3, 4, 64), c.k, c.v, c.table,
                                               _i32([40, 0, 70]), 70, c.ks, c.vs, scale=scale, **kw)
        return got

    return [("norm_fwd", norm), ("norm_bwd", norm_bwd), ("reserve", reserve), ("release", release),
            ("append", append), ("read", read), ("decode", decode)]


class Spy:
    """ne_step, with what each call returned."""

    def __init__(self, step):
        self.step, self.seen = step, []

    def __getattr__(self, name):
        def call(*a):
            got = getattr(self.step, name)(*a)
            self.seen.append((name, got))
            return got
        return call


@pytest.fixture
def spy(na, monkeypatch):
    s = Spy(na._step)
    monkeypatch.setattr(na, "_step", s)
    return s


def _same(x, y):
    return len(x) == len(y) and all(a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b)
                                    for a, b in zip(x, y))


def test_both_ways_give_the_same(na, spy):
    for name, call in _calls(na):
        want = call(stream=torch.cuda.current_stream())
        assert not spy.seen  # (a stream given: the other way)
        got = call()
        assert spy.seen and all(n == name and x is not None for n, x in spy.seen), name
        spy.seen.clear()
        assert _same(got, want), name
        assert na.ne_attn_get_device_status() == 0


def test_outputs_given_come_back(na, spy):
    a, e = _norm_args(), lambda *s, d=torch.bfloat16: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    want = na.ne_qk_norm_rope_fwd(*a)
    qr, kr = e(40, 6, 64), e(40, 2, 64)
    got = na.ne_qk_norm_rope_fwd(*a, qr=qr, kr=kr)
    assert got[0] is qr and got[1] is kr and _same(got, want)
    dr = _randn(6, 40, 6, 64), _randn(7, 40, 2, 64)
    want = na.ne_qk_norm_rope_bwd(*dr, *a)
    joint = e(40, 10, 64)
    out = joint[:, :6], joint[:, 6:8], e(64, d=torch.float32), e(64, d=torch.float32)
    got = na.ne_qk_norm_rope_bwd(*dr, *a, dq=out[0], dk=out[1], dq_weight=out[2], dk_weight=out[3])
    assert all(x is y for x, y in zip(got, out)) and _same(got, want)
    assert bool((joint[:, 8:] == 0).all())
    p = _pages_args()
    ints = [torch.full((n,), -9, dtype=torch.int32, device="cuda") for n in (4, 3, 60, 60, 3, 1)]
    got = na.ne_kv_reserve(_i32([20, 30, 1]), *p, 60, 16, 128, *ints)
    assert all(x is y for x, y in zip(got, ints[:4]))
    assert ints[0].tolist() == [0, 20, 50, 51] and ints[4].tolist() == [20, 35, 1]
    assert p[0].tolist() == [0, 5, 0] and p[3].tolist() == [9] and ints[5].tolist() == [4]
    c = _caches()[2]
    k, v = e(110, 2, 64), e(110, 2, 64)
    got = na.ne_kv_read(c.k, c.v, c.table, _cu([40, 0, 70]), _i32([0, 0, 0]), 110, c.ks, c.vs, k=k, v=v)
    assert got[0] is k and got[1] is v and bool((k != 0).any())
    out, lse = e(3, 4, 64), e(3, 4, d=torch.float32)
    got = na.ne_attn_decode_paged(_randn(10, 3, 4, 64), c.k, c.v, c.table, _i32([40, 0, 70]), 70, c.ks,
                                  c.vs, out=out, lse=lse)
    assert got[0] is out and got[1] is lse and bool((out[0] != 0).any())
    assert [x is not None for _, x in spy.seen] == [True] * 7


def test_refusals(na, spy):
    """What is not regular is handed back, and refused as before; nothing is written."""
    bf, i32 = torch.bfloat16, torch.int32
    a, p = _norm_args(), _pages_args()
    c4, c8 = _caches()[2], _caches()[1]
    new = _i32([1, 1, 1])
    q = _randn(11, 3, 4, 64)
    lens = _i32([40, 0, 70])
    k1 = _randn(12, 6, 2, 64)
    cu, at = _cu([3, 0, 3]), _i32([0, 0, 0])

    def swap(args, i, x):
        return [*args[:i], x, *args[i + 1:]]

    def decode(q=q, c=c4, lens=lens, ks=None, **kw):
        return na.ne_attn_decode_paged(q, c.k, c.v, c.table, lens, 70, c.ks if ks is None else ks, c.vs, **kw)

    bad = [
        lambda: na.ne_qk_norm_rope_fwd(*swap(a, 0, a[0].half())),
        lambda: na.ne_qk_norm_rope_fwd(*swap(a, 0, a[0].cpu())),
        lambda: na.ne_qk_norm_rope_fwd(*swap(a, 0, a[0][:, ::2])),
        lambda: na.ne_qk_norm_rope_fwd(*swap(a, 1, a[1][:39])),
        lambda: na.ne_qk_norm_rope_fwd(*swap(a, 2, a[2][:32])),
        lambda: na.ne_qk_norm_rope_fwd(*swap(a, 3, a[3].float())),
        lambda: na.ne_qk_norm_rope_fwd(*swap(a, 4, a[4].long())),
        lambda: na.ne_qk_norm_rope_fwd(*swap(a, 4, None)),
        lambda: na.ne_qk_norm_rope_fwd(*a, qr=a[0]),
        lambda: na.ne_qk_norm_rope_bwd(a[0], a[1], *a),
        lambda: na.ne_qk_norm_rope_bwd(a[0].contiguous(), a[1].contiguous(), *a, dq=a[0].float()),
        lambda: na.ne_kv_reserve(new.long(), *p, 3, 16, 128),
        lambda: na.ne_kv_reserve(new[:2], *p, 3, 16, 128),
        lambda: na.ne_kv_reserve(new, *p, 3, 16, 128, positions=new[:2]),
        lambda: na.ne_kv_reserve(new, *swap(p, 1, p[1][:2]), 3, 16, 128),
        lambda: na.ne_kv_release(new, *p, 16, 128),
        lambda: na.ne_kv_append(k1, k1[:5], cu, at, c4.k, c4.v, c4.table, 70, c4.ks, c4.vs),
        lambda: na.ne_kv_append(k1, k1, cu[:3], at, c4.k, c4.v, c4.table, 70, c4.ks, c4.vs),
        lambda: na.ne_kv_append(k1, k1, cu, at, c4.k, c4.v, c4.table, 70),
        lambda: na.ne_kv_append(k1, k1, cu, at, c8.k, c8.v, c8.table, 70, c4.ks, c4.vs),
        lambda: na.ne_kv_append(k1, k1, cu, at, c4.k, c4.v[:1], c4.table, 70, c4.ks, c4.vs),
        lambda: na.ne_kv_read(c4.k, c4.v, c4.table, cu, at, 6, c4.ks, c4.vs, k=k1[:5]),
        lambda: decode(q=_randn(13, 3, 3, 64)),
        lambda: decode(lens=lens[:2]),
        lambda: decode(ks=c8.ks),
        lambda: decode(out=q[:2]),
        lambda: decode(lse=torch.zeros((3, 4), dtype=bf, device="cuda")),
        lambda: decode(c=_caches()[0], ks=c4.ks),
    ]
    state = [x.clone() for x in (*p, c4.k, c4.ks)]
    for n, call in enumerate(bad):
        spy.seen.clear()
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"refusal {n} did not happen")
        assert [x for _, x in spy.seen] == [None], n
    refused = [  # by the library: its status
        (lambda: na.ne_qk_norm_rope_fwd(*a, eps=-1.0), 1),
        (lambda: na.ne_qk_norm_rope_fwd(*swap(a, 0, _randn(1, 40 * 640 + 4)[4:].view(40, 10, 64)[:, :6])), 3),
        (lambda: na.ne_kv_reserve(new, *p, 3, 24, 128), 2),
        (lambda: na.ne_kv_release(new.bool(), *p, 16, 1 << 20), 1),
        (lambda: na.ne_kv_append(k1, k1, cu, at, c4.k, c4.v, c4.table, 1 << 20, c4.ks, c4.vs), 1),
        (lambda: na.ne_kv_read(c4.k, c4.v, c4.table, cu, at, 6, c4.ks, c4.vs, max_seqlen=0), 1),
        (lambda: decode(scale=-1.0), 1),
    ]
    for n, (call, code) in enumerate(refused):
        spy.seen.clear()
        with pytest.raises(na.NeAttnError) as e:
            call()
        assert e.value.status == code and [x for _, x in spy.seen] == [code], n
    assert all(torch.equal(x, y) for x, y in zip((*p, c4.k, c4.ks), state))
    assert na.ne_attn_get_device_status() == 0 and i32 is torch.int32


def test_the_other_way_takes_what_it_took(na, spy):
    """Integers of other types, lengths of another shape, subclasses, no rows."""
    a, c = _norm_args(), _caches()[2]
    want = na.ne_qk_norm_rope_fwd(*a)
    spy.seen.clear()
    assert _same(na.ne_qk_norm_rope_fwd(*a[:5], np.int64(64)), want)

    class Sub(torch.Tensor):
        pass

    assert all(torch.equal(x, y) for x, y in
               zip(na.ne_qk_norm_rope_fwd(a[0].as_subclass(Sub), *a[1:]), want))
    q, lens = _randn(10, 3, 4, 64), _i32([40, 0, 70])
    way = lambda n: na.ne_attn_decode_paged(q, c.k, c.v, c.table, n, 70, c.ks, c.vs)  # noqa: E731
    got = way(lens.view(3, 1))
    assert [x for _, x in spy.seen] == [None] * 3
    assert _same(got, way(lens)) and spy.seen[-1][1] is not None
    assert na.ne_qk_norm_rope_fwd(a[0][:0], a[1][:0], *a[2:4], a[4][:0], 64)[0].shape == (0, 6, 64)
    param = torch.nn.Parameter(a[2])  # (a parameter is regular, and stays out of the graph)
    got = na.ne_qk_norm_rope_fwd(*a[:2], param, *a[3:])
    assert spy.seen[-1][1] is not None and not got[0].requires_grad and _same(got, want)


def test_tensors_that_stand_for_others(na, spy):
    """In a transform a tensor has no memory of its own: an error, as it was."""
    a = _norm_args()
    many = torch.stack([a[0], a[0]])
    with pytest.raises(RuntimeError):
        torch.vmap(lambda q: na.ne_qk_norm_rope_fwd(q, *a[1:]))(many)
    assert spy.seen == [("norm_fwd", None)]
    assert na.ne_qk_norm_rope_fwd(*a)[0].shape == a[0].shape


def test_current_stream_and_threads(na):
    """The stream that is current where the call is made, in any thread."""
    a = _norm_args()
    want = na.ne_qk_norm_rope_fwd(*a)
    torch.cuda.synchronize()
    side, got = torch.cuda.Stream(), []

    def work():
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)  # (about a millisecond, on the side stream)
            late = a[0] * 1
            got.append(na.ne_qk_norm_rope_fwd(late, *a[1:]))

    t = threading.Thread(target=work)
    t.start()
    t.join()
    side.synchronize()
    assert _same(got[0], want)


def test_nothing_is_kept(na):
    a = _norm_args()
    na.ne_qk_norm_rope_fwd(*a)
    torch.cuda.synchronize()
    gc.collect()  # (what other tests left)
    before = torch.cuda.memory_allocated()
    for _ in range(200):
        na.ne_qk_norm_rope_fwd(*a)
        with pytest.raises(na.NeAttnError):
            na.ne_qk_norm_rope_fwd(*a, eps=-1.0)
    assert torch.cuda.memory_allocated() == before

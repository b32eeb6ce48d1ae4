"""What the paged decode keeps between calls: the arrival counters of streams and of
captured calls."""
import ctypes

import pytest
import torch

from grouped import Cache

pytestmark = pytest.mark.gpu


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


def _decode(na, c, q, lens, **kw):
    return na.ne_attn_decode_paged(q, c.k, c.v, c.table, lens, max(c.lens), c.ks, c.vs, **kw)


def _driver(name, *args):
    assert getattr(ctypes.CDLL("libcuda.so.1"), name)(*args) == 0, name


@pytest.mark.parametrize("drop", [7, 20, 100])
def test_a_call_after_one_whose_wait_ran_out(na, drop):
    """A tile never arrives at one CTA.  That is reported, the heads that it concerns
    have no result, the others do, and later calls on the stream are as before."""
    # About eight tiles a CTA, so that the parts of a sequence arrive at different times
    # (a CTA's share may end in one sequence and begin in the next).
    c = Cache([19000 - 10 * i for i in range(12)], 1, 64, False, seed=4).fill_random(5)
    q, lens = _randn(6, 12, 4, 64), _i32(c.lens)
    later = [_randn(7 + i, 12, 4, 64) for i in range(3)]
    want, wl = (t.clone() for t in _decode(na, c, q, lens, rope_base=0.0))
    others = [[t.clone() for t in _decode(na, c, x, lens, rope_base=0.0)] for x in later]
    assert na.ne_attn_get_device_status() == 0
    for _ in range(2):
        out, lse = na.ne_debug_decode_drop(q, c.k, c.v, c.table, lens, 19000, drop)
        assert na.ne_attn_get_device_status() == 5
        none = (out == 0).all(-1) & (lse == -float("inf"))
        same = (out == want).all(-1) & (lse == wl)
        assert bool((none | same).all()) and bool(none.any()) and bool(same.any())
        for x, w in zip(later, others):
            got = _decode(na, c, x, lens, rope_base=0.0)
            assert na.ne_attn_get_device_status() == 0
            assert all(torch.equal(a, b) for a, b in zip(got, w))


KERNEL_NODE = 0  # CU_GRAPH_NODE_TYPE_KERNEL


def test_any_number_of_captured_calls_are_a_kernel_each(na):
    """As many as a model's layers times its batch sizes make, with a workspace: each is
    its kernel and nothing in front of it, and each has counters of its own."""
    P, n = ctypes.c_void_p, 400
    c = Cache([900, 300], 2, 64, False, seed=1).fill_random(2)
    q, lens = _randn(3, 2, 6, 64), _i32(c.lens)
    want = [t.clone() for t in _decode(na, c, q, lens)]
    ws = torch.empty(na.ne_attn_decode_paged_workspace_bytes(2, 6, 2, 900), dtype=torch.uint8,
                     device="cuda")
    outs = torch.zeros((n, 2, 6, 64), dtype=torch.bfloat16, device="cuda")
    lses = torch.zeros((n, 2, 6), device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    raw, graph, executable = P(stream.cuda_stream), P(), P()
    with torch.cuda.stream(stream):
        _driver("cuStreamBeginCapture_v2", raw, 0)  # of the global mode, the strictest
        for i in range(n):
            _decode(na, c, q, lens, out=outs[i], lse=lses[i], workspace=ws)
        _driver("cuStreamEndCapture", raw, ctypes.byref(graph))
    count = ctypes.c_size_t()
    _driver("cuGraphGetNodes", graph, None, ctypes.byref(count))
    nodes = (P * count.value)()
    _driver("cuGraphGetNodes", graph, nodes, ctypes.byref(count))
    kinds = []
    for node in nodes:
        kind = ctypes.c_int()
        _driver("cuGraphNodeGetType", P(node), ctypes.byref(kind))
        kinds.append(kind.value)
    assert kinds == [KERNEL_NODE] * n
    _driver("cuGraphInstantiateWithFlags", ctypes.byref(executable), graph, ctypes.c_ulonglong(0))
    for _ in range(2):
        outs.zero_()
        lses.zero_()
        torch.cuda.synchronize()
        _driver("cuGraphLaunch", executable, raw)
        torch.cuda.synchronize()
        assert bool((outs == want[0]).all()) and bool((lses == want[1]).all())
    _driver("cuGraphExecDestroy", executable)
    _driver("cuGraphDestroy", graph)
    assert all(torch.equal(a, b) for a, b in zip(_decode(na, c, q, lens), want))
    assert na.ne_attn_get_device_status() == 0

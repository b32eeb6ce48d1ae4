"""A native call's tensors given other memory by another thread meanwhile: the library gets an
address and a size that belong together."""
import ctypes
import itertools
import sys
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
P, I = ctypes.c_void_p, ctypes.c_int


@pytest.fixture(scope="module")
def na():
    from causal_self_attention_gb300 import build, ne_attn
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ne_attn.lib()
    return ne_attn


def test_addresses_and_sizes_belong_together(na):
    """(In place of the library stands a function that writes down what it is given: no
    kernel runs.)"""
    if na._step is None:
        pytest.skip("the module is not built")
    L, seen = na.lib(), set()

    @ctypes.CFUNCTYPE(I, P, P, I, P, I, P, P, I, I, I, P)
    def release(finished, lens, nseq, table, width, free, n_free, n_pages, page, longest, stream):
        seen.add((free, n_pages))
        return 0

    def address(fn):
        return ctypes.cast(fn, P).value

    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    few, many, free = i32(8), i32(4096), i32(8)
    free.data = few
    finished, lens, table, n_free = i32(2).bool(), i32(2), i32(2, 3), i32(1)
    pairs = {(t.data_ptr(), t.numel()) for t in (few, many)}
    done = threading.Event()

    def swap():
        for t in itertools.cycle((many, few)):
            free.data = t
            if done.is_set():
                return

    threads, interval = [threading.Thread(target=swap) for _ in range(2)], sys.getswitchinterval()
    real = [address(fn) for fn in (L.ne_qk_norm_rope_fwd, L.ne_qk_norm_rope_bwd, L.ne_kv_reserve,
                                   L.ne_kv_release, L.ne_kv_append, L.ne_kv_read,
                                   L.ne_attn_decode_paged)]
    na._step.bind(*real[:3], address(release), *real[4:])
    sys.setswitchinterval(1e-6)
    try:
        for t in threads:
            t.start()
        for _ in range(20000):
            assert na._step.release(finished, lens, table, free, n_free, 16, 48) == 0
    finally:
        done.set()
        sys.setswitchinterval(interval)
        for t in threads:
            t.join()
        na._step.bind(*real)
    assert seen <= pairs

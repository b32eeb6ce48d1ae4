"""The caller's current context is left as it is."""
import ctypes
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

pytestmark = pytest.mark.gpu
UNSUPPORTED = 2


@pytest.fixture(scope="module")
def na():
    from causal_self_attention_gb300 import build, ne_attn
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ne_attn


def _with_a_context_of_its_own(call):
    """call() in a thread whose current context it has made itself: (what it returns,
    whether that context is current afterwards)."""
    P, cuda = ctypes.c_void_p, ctypes.CDLL("libcuda.so.1")

    def run():
        mine, now = P(), P()
        assert cuda.cuCtxCreate_v2(ctypes.byref(mine), 0, 0) == 0
        try:
            got = call()
            assert cuda.cuCtxGetCurrent(ctypes.byref(now)) == 0
            return got, now.value == mine.value
        finally:
            assert cuda.cuCtxDestroy_v2(mine) == 0

    with ThreadPoolExecutor(1) as pool:
        return pool.submit(run).result()


def test_a_thread_with_a_context_of_its_own(na):
    """The tables and counters live in one context of a device: a call from another one
    is refused, and the thread's context stays current."""
    torch.zeros(1, device="cuda")
    assert na.ne_attn_get_device_status() == 0
    assert _with_a_context_of_its_own(
        lambda: na.lib().ne_attn_get_device_status(None)) == (UNSUPPORTED, True)
    assert na.ne_attn_get_device_status() == 0


def test_release_from_a_thread_with_a_context_of_its_own(na):
    """What is kept is freed where it lives; the next call makes it anew."""
    qkv = [torch.randn(1, 200, 2, 64, device="cuda").bfloat16() for _ in range(3)]
    want = na.ne_attn_fwd(*qkv)
    torch.cuda.synchronize()
    assert _with_a_context_of_its_own(lambda: na.lib().ne_attn_release())[1]
    got = na.ne_attn_fwd(*qkv)
    assert na.ne_attn_get_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))

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


def test_a_thread_with_a_context_of_its_own(na):
    """The tables and counters live in one context of a device: a call from another one
    is refused, and the thread's context stays current."""
    P = ctypes.c_void_p
    torch.zeros(1, device="cuda")
    assert na.ne_attn_get_device_status() == 0
    cuda = ctypes.CDLL("libcuda.so.1")

    def run():
        mine, now = P(), P()
        assert cuda.cuCtxCreate_v2(ctypes.byref(mine), 0, 0) == 0
        try:
            status = na.lib().ne_attn_get_device_status(None)
            assert cuda.cuCtxGetCurrent(ctypes.byref(now)) == 0
            return status, now.value == mine.value
        finally:
            assert cuda.cuCtxDestroy_v2(mine) == 0

    with ThreadPoolExecutor(1) as pool:
        assert pool.submit(run).result() == (UNSUPPORTED, True)
    assert na.ne_attn_get_device_status() == 0

"""A RoPE table is complete when the call that makes it launches, on any stream."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def na():
    from causal_self_attention_gb300 import build, ne_attn
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ne_attn


@pytest.mark.parametrize("n", [100, 9000])
def test_first_call_for_a_base_on_a_non_blocking_stream(na, n):
    """torch's side streams do not wait for the legacy stream; the second call reads a
    table that has long been there."""
    x = torch.randn(n, 2, 64, device="cuda").bfloat16()
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for i in range(5):
        base = 20000.0 + n + i
        first = na.ne_attn_gqa_varlen_fwd(x, x, x, cu, n, rope_base=base, stream=side)
        side.synchronize()
        again = na.ne_attn_gqa_varlen_fwd(x, x, x, cu, n, rope_base=base, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    assert na.ne_attn_get_device_status() == 0

"""Prompt attention on rotated operands where the work has no list (more items than one is
made for): eager, and captured behind whatever kernel comes before it."""
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


@pytest.mark.parametrize("H,Hkv", [(4, 2), (3, 3)])
def test_more_items_than_a_list_holds(na, H, Hkv):
    nseq, longest = 9000, 4096
    lens = torch.tensor([(i * 7) % 5 for i in range(nseq)])
    lens[4321] = 700
    cu = torch.cat((torch.zeros(1, dtype=torch.int64), lens.cumsum(0))).to(torch.int32).cuda()
    n = int(lens.sum())
    g = torch.Generator("cpu").manual_seed(3)
    q, k, v = (torch.randn((n, h, 64), generator=g).bfloat16().cuda() for h in (H, Hkv, Hkv))
    out, lse, qr, kr = na.ne_attn_gqa_varlen_fwd(q, k, v, cu, longest)
    want = (out, lse)
    got = na.ne_attn_gqa_varlen_fwd_rotated(qr, kr, v, cu, longest)
    assert na.ne_attn_get_device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph, x = torch.cuda.CUDAGraph(), qr.clone()
    with torch.cuda.graph(graph, stream=s):
        y = x * 1  # a kernel right before
        captured = na.ne_attn_gqa_varlen_fwd_rotated(y, kr, v, cu, longest)
    for _ in range(3):
        for t in captured:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, want))

"""The backward with shared heads asks for what it keeps, no more: also with a head
each, where the size that its query gives serves the ungrouped backward, too."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p
FAKE = P(0x10000)  # never dereferenced: every call below fails its host check first
INVALID, MISALIGNED = 1, 3


def _need(n, H):
    """dQ' and D in fp32, each in whole 256 bytes (a head each: no partials)."""
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    return up(n * H * 64 * 4) + up(n * H * 4)


@pytest.fixture(scope="module")
def na():
    from causal_self_attention_gb300 import build, ne_attn
    build.build()
    ne_attn.lib()
    return ne_attn


@pytest.mark.parametrize("n,H", [(100, 4), (1, 1), (8192, 12)])
def test_what_a_head_each_needs(na, n, H):
    def call(ws, ws_bytes):
        return na.lib().ne_attn_gqa_varlen_bwd(
            FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2, n, n, H, H, 64, 1e4, 0.125, FAKE, FAKE,
            FAKE, ws, ws_bytes, None)

    assert call(FAKE, _need(n, H) - 1) == INVALID
    assert call(P(0x10010), _need(n, H)) == MISALIGNED  # the size was enough
    assert na.ne_attn_gqa_bwd_workspace_bytes(n, n, H, H) >= _need(n, H)


@pytest.mark.gpu
def test_a_head_each_in_the_smallest_workspace(na):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lens, H = [300, 129], 3
    n, need = sum(lens), _need(sum(lens), H)
    g = torch.Generator("cpu").manual_seed(1)
    q, k, v, do = (torch.randn((n, H, 64), generator=g).bfloat16().cuda() for _ in range(4))
    cu = torch.tensor([0, 300, 429], dtype=torch.int32, device="cuda")
    out, lse, qr, kr = na.ne_attn_gqa_varlen_fwd(q, k, v, cu, 300)
    want = na.ne_attn_gqa_varlen_bwd(qr, kr, v, out, do, lse, cu, 300)
    room = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    got = na.ne_attn_gqa_varlen_bwd(qr, kr, v, out, do, lse, cu, 300, workspace=room[:need])
    assert na.ne_attn_get_device_status() == 0
    assert bool((room[need:] == 77).all())
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    assert float((got[0].double() - want[0].double()).norm()) <= 1e-3 * float(want[0].double().norm())

"""A generated token is the last row of a prompt one token longer: the prompt through
the forward, its k', v and the token's into the cache, the token through the decode,
against the forward over all of it."""
import pytest
import torch

from grouped import Cache, attention, within

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


def _cu(n):
    return _i32([0] + [sum(n[:i + 1]) for i in range(len(n))])


@pytest.mark.parametrize("H,Hkv", [(6, 2), (12, 4), (16, 1), (3, 3)])
@pytest.mark.parametrize("lens", [[1, 127, 128, 129], [5, 1000, 0, 300]])
def test_the_next_token_is_the_last_row_of_a_longer_prompt(na, H, Hkv, lens):
    whole, B = [n + 1 for n in lens], len(lens)
    g = torch.Generator("cpu").manual_seed(1)
    q, k, v = (torch.randn((sum(whole), h, 64), generator=g).bfloat16().cuda()
               for h in (H, Hkv, Hkv))
    out, lse, qr, kr = na.ne_attn_gqa_varlen_fwd(q, k, v, _cu(whole), max(whole))
    last = _cu(whole)[1:].long() - 1
    prompt = torch.ones(sum(whole), dtype=torch.bool, device="cuda")
    prompt[last] = False
    # The prompts alone, and their rows and the tokens' into the cache.
    _, _, _, kp = na.ne_attn_gqa_varlen_fwd(q[prompt], k[prompt], v[prompt], _cu(lens), max(lens))
    c = Cache(whole, Hkv, 32, False, seed=2)
    na.ne_kv_append(kp, v[prompt], _cu(lens), _i32([0] * B), c.k, c.v, c.table, max(whole),
                    rope_base=0.0)
    na.ne_kv_append(k[last], v[last], _cu([1] * B), _i32(lens), c.k, c.v, c.table, max(whole))
    one, one_lse = na.ne_attn_decode_paged(q[last], c.k, c.v, c.table, _i32(whole), max(whole))
    assert na.ne_attn_get_device_status() == 0
    kb, vb = na.ne_kv_read(c.k, c.v, c.table, _cu(whole), _i32([0] * B), sum(whole))
    assert torch.equal(kb, kr) and torch.equal(vb, v)  # the same keys, bit for bit
    for s, n in enumerate(whole):
        r = slice(int(last[s]) + 1 - n, int(last[s]) + 1)
        _, _, oe, le = attention(qr[last[s]:last[s] + 1], kr[r], v[r], 0.125)
        # Either is within its bound of the exact value.
        within(one[s], out[last[s]], 2 * oe[0], f"out of sequence {s}")
        within(one_lse[s], lse[:, last[s]], 2 * le[:, 0], f"lse of sequence {s}")

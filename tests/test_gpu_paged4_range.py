"""Decode attention over the 4-bit cache at the ends of the range: sums that are zero when
the references move, against the plain 64-bit implementation of grouped.py."""
import pytest
import torch

from step import Cache4
from test_gpu_paged import _decode, _i32
from test_gpu_paged4 import _check_sequence

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def na():
    from causal_self_attention_gb300 import build, ne_attn
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ne_attn


class Rows:
    """One sequence of n keys; what() sets some of them."""

    def __init__(self, n, Hkv=1, page=64, seed=1):
        self.c, self.n = Cache4([n], Hkv, page, seed=seed).fill_random(seed + 1), n

    def what(self, pool, rows, code, byte, half=None):
        """The rows' value bytes (two e2m1 codes each; None: as they are) and scale bytes, in
        one half of the dims or both."""
        rows = torch.as_tensor(rows)
        page, slot = (t.cuda() for t in self.c.where(0, rows))
        values, scales = (self.c.k, self.c.ks) if pool == "k" else (self.c.v, self.c.vs)
        for h in (0, 1) if half is None else (half,):
            if code is not None:  # (a half's bytes: two of every four)
                at = torch.tensor([b for b in range(32) if b % 4 // 2 == h], device="cuda")
                values[page[:, None], :, slot[:, None], at] = code
            byte = torch.as_tensor(byte, dtype=torch.uint8, device="cuda")
            scales[page, :, slot, h] = byte.reshape(-1, 1)
        return self

    def decode(self, na, q, **kw):
        out, lse = _decode(na, self.c, q, _i32([self.n]), self.n, 0.0, **kw)
        assert na.ne_attn_get_device_status() == 0
        return out[0], lse[0]

    def check(self, na, q):
        _check_sequence(self.c, 0, self.n, q, *self.decode(na, q))


def _ones(H, x=1.0):
    return torch.full((1, H, 64), x, dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("H", [4, 13])
@pytest.mark.parametrize("halves", [(0,), (1,), (0, 1)])
@pytest.mark.parametrize("n,zeros", [(512, 27), (512, 127), (20000, 127)])
def test_zero_rows_before_scales_far_apart(na, H, halves, n, zeros):
    """The keys with all the weight hold zeros; rows whose scales are far apart come after
    them, with scores 1100 (in powers of two) below."""
    r = Rows(n).what("k", range(n), 0xff, 130)  # -6 * 2^3: scores of -384 ...
    i = torch.arange(n)
    first, late = (i[(i // 256 % 2 == x) & (i % 256 < 64)] for x in (0, 1))
    r.what("k", first, 0x77, 130)               # ... and 384
    for h in halves:
        r.what("v", first, 0x00, zeros, h)
        r.what("v", late, None, 110 + 40 * (late % 2), h)
    q = _ones(H)
    out, _ = r.decode(na, q)
    for h in halves:
        assert bool((out[:, 32 * h:32 * h + 32] == 0).all())
    r.check(na, q)

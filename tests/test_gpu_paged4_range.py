"""Decode attention over the 4-bit cache at the ends of the range: sums that are zero when
the references move, large keys beside small queries, scores of any size, values up to bf16's largest, against
the plain 64-bit implementation of grouped.py."""
import pytest
import torch

from grouped import F64, U16, U32, within
from step import Cache4
from test_gpu_paged import _decode, _i32, _randn
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


@pytest.mark.parametrize("H", [4, 13])
@pytest.mark.parametrize("q_exp,lo,hi", [
    (-118, 245, 252), (-126, 250, 252),  # large keys: the sums before the query's factor pass 2^128
    (-133, 250, 252),                    # a query below the smallest normal number
    (100, 27, 33), (118, 1, 8), (125, 0, 4), (126, 0, 2)])  # and the other way round
def test_keys_and_queries_of_far_apart_sizes(na, H, q_exp, lo, hi):
    n = 700
    r, i = Rows(n, Hkv=1), torch.arange(n)
    for h in (0, 1):
        r.what("k", i, None, lo + (i + h) % (hi - lo + 1), h)
    q = (_randn(3, 1, H, 64).double().clamp(-1.9, 1.9) * 2.0 ** q_exp).bfloat16()
    assert bool((q != 0).any()) and bool(torch.isfinite(q).all())
    r.check(na, q)


def _winner(na, n, H, k, sign, v_byte, at, spread=0):
    """Scores of 15 * 2^k: sign times that for the key `at`, which has all the weight, and
    -2 (sign > 0: -1) times that for the others.  What comes out is its value row."""
    r = Rows(n)
    half = k // 2
    q = _ones(H, 1.25 * 2.0 ** half)           # 64 * 1.25 * 1.5 / 8 = 15
    r.what("k", range(n), 0xbb, 127 + k - half + (sign < 0))
    r.what("k", [at], 0x33 if sign > 0 else 0xbb, 127 + k - half)
    i = torch.arange(n)
    r.what("v", i, None, v_byte + spread * (i % 2))
    out, lse = r.decode(na, q)
    v = r.c.rows(0)[1][at].expand(H, 64)
    # The weight in a half, its sum in fp32 (and the powers of two, 2^-22 each); bf16.
    within(out, v, v.abs() * (U16 + 2.0 ** -11 + 16 * U32), "out")
    score = torch.full((H,), sign * 15 * 2.0 ** k, dtype=F64, device="cuda")
    within(lse, score, score.abs() * 72 * U32 + 16 * U32, "lse")


@pytest.mark.parametrize("n,at", [(1, 0), (100, 77), (700, 3), (700, 699)])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("H", [4, 13])
def test_scores_of_any_size(na, n, at, sign, H):
    for k in (*range(4, 40), 60, 90, 97, 100, 110, 118):
        _winner(na, n, H, k, sign, 127, at)


@pytest.mark.parametrize("n,at", [(1, 0), (100, 76), (100, 77), (700, 3), (700, 698)])
@pytest.mark.parametrize("v_byte,spread", [(122, 0), (130, 0), (110, 40), (116, 9)])
@pytest.mark.parametrize("H", [4, 13])
def test_exponents_of_values_beside_scores_of_any_size(na, n, at, v_byte, spread, H):
    """The value rows' scales, alike or far apart (both modes)."""
    for k in (4, 10, *range(18, 34), 60, 110):
        for sign in (1, -1):
            _winner(na, n, H, k, sign, v_byte, at, spread)


@pytest.mark.parametrize("H", [4, 13])
@pytest.mark.parametrize("n", [1, 5, 300, 1500, 20000])
@pytest.mark.parametrize("lo,hi", [(245, 252), (252, 252), (200, 252), (27, 252), (27, 28)])
def test_values_of_any_size(na, H, n, lo, hi):
    """Scale bytes up to the largest that the cache writes (2^125): one key, several, parts
    that are joined; alike and far apart."""
    r, i = Rows(n), torch.arange(n)
    for h in (0, 1):
        r.what("v", i, None, lo + (i * 7 + h) % (hi - lo + 1), h)
    r.check(na, _randn(5, 1, H, 64))
    # All of the largest size and one sign: nothing is larger on the way.
    r.what("v", i, 0x77, hi)
    out, _ = r.decode(na, _randn(5, 1, H, 64))
    want = 6 * 2.0 ** (hi - 127)
    # Weights in halves (2^-11) and their sum of n terms, bf16.
    err = want * (U16 + 2.0 ** -11 + (n + 32) * U32)
    within(out, torch.full_like(out, want), torch.full_like(out, err, dtype=F64), "out")


def test_values_whose_scales_are_beyond_bf16(na):
    """Scale bytes that the cache itself never writes, of values that bf16 holds."""
    for byte, code in ((253, 0x22), (254, 0x11), (0, 0x77), (20, 0x22)):
        r = Rows(300).what("v", range(300), code, byte)
        out, _ = r.decode(na, _randn(6, 1, 4, 64))
        want = r.c.rows(0)[1][0, 0, 0]
        within(out, want.expand(4, 64), (want * (U16 + 2.0 ** -11 + 332 * U32)).expand(4, 64), "out")


@pytest.mark.parametrize("H", [4, 13])
@pytest.mark.parametrize("halves", [(0,), (1,), (0, 1)])
@pytest.mark.parametrize("n,at", [(1, 0), (64, 5), (500, 3), (500, 301), (5000, 4000)])
@pytest.mark.parametrize("gap", [10, 24, 30, 60])
def test_zeros_with_the_largest_score(na, n, at, halves, H, gap):
    """A row of zeros, as the cache holds them (scale byte 27), has nearly all the weight: what
    comes out is the others', 2^-gap of it, as exact as their weights among themselves."""
    r = Rows(n).what("k", range(n), 0x00, 127)  # scores of 0
    r.what("k", [at], 0x22, 127)                # (1) a score of 8 |q|: 8 q / ln 2 in powers of two
    for h in halves:
        r.what("v", [at], 0x00, 27, h)
    r.check(na, _ones(H, gap * 0.6931 / 8))


@pytest.mark.parametrize("H", [4, 13])
@pytest.mark.parametrize("above", [1, 7, 8, 9, 20, 31, 32, 33, 50])
def test_rows_of_the_smallest_scale_beside_others(na, H, above):
    """Rows of scale 2^-100 that hold values, beside a few a little larger."""
    for n in (64, 700):
        r, i = Rows(n), torch.arange(n)
        r.what("v", i, 0x77, 27)
        r.what("v", i[::50], 0x11, 27 + above)
        # (What is left out is 12 2^-32 of the largest rows' values a key, n keys.)
        out, _ = r.decode(na, _ones(H, 0.0))
        v = r.c.rows(0)[1].mean(0)[0].expand(H, 64)
        left = 12 * 2.0 ** -32 * 2.0 ** (above - 101) if above >= 32 else 0.0
        within(out * 2.0 ** 90, v * 2.0 ** 90,
               (v.abs() * (U16 + 2.0 ** -10 + (n + 32) * U32) + left) * 2.0 ** 90, "out")

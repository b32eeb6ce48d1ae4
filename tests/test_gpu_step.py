"""Steps of generation as a server runs them: pages and positions on the GPU, norms and
rotation, rows into the paged cache, attention over it -- eager and as a replayed graph,
with requests that end and others in their place."""
import pytest
import torch

import step
from grouped import F64, Cache, attention, quantise, within
from step import Cache4, quantise4

pytestmark = pytest.mark.gpu
B, H, HKV, PAGE, WIDTH, ROOM = 5, 6, 2, 16, 12, 96
LONGEST = PAGE * WIDTH


@pytest.fixture(scope="module")
def na():
    from causal_self_attention_gb300 import build, ne_attn
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return ne_attn


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cache(kind):
    lens = [LONGEST] * B
    c = Cache4(lens, HKV, PAGE, seed=1, spare=0, extra_columns=0) if kind == "e2m1" else \
        Cache(lens, HKV, PAGE, kind == "e4m3", seed=1, spare=0, extra_columns=0)
    c.table.fill_(-1)
    return c


class Server:
    """The state that a server keeps, and one step on it."""

    def __init__(self, na, kind):
        self.na, self.c = na, _cache(kind)
        n_pages = self.c.n_pages
        self.free, self.n_free = _i32([(7 * i) % n_pages for i in range(n_pages)]), _i32([n_pages])
        self.lens = _i32([0] * B)
        self.new, self.done = _i32([0] * B), torch.zeros(B, dtype=torch.bool, device="cuda")
        self.qkv = torch.zeros((ROOM, H + 2 * HKV, 64), dtype=torch.bfloat16, device="cuda")
        self.qr, self.kr = (torch.zeros((ROOM, h, 64), dtype=torch.bfloat16, device="cuda")
                            for h in (H, HKV))
        self.wq, self.wk = ((torch.arange(64, device="cuda") / 64 + x).bfloat16() for x in (0.5, 0.8))

    def step(self):
        na, c = self.na, self.c
        na.ne_kv_release(self.done, self.lens, c.table, self.free, self.n_free, PAGE, LONGEST)
        cu, start, pos, slots = na.ne_kv_reserve(self.new, self.lens, c.table, self.free,
                                                 self.n_free, ROOM, PAGE, LONGEST)
        q, k, v = self.qkv[:, :H], self.qkv[:, H:H + HKV], self.qkv[:, H + HKV:].contiguous()
        qr, kr = na.ne_qk_norm_rope_fwd(q, k, self.wq, self.wk, pos, LONGEST, qr=self.qr, kr=self.kr)
        na.ne_kv_append(kr, v, cu, start, c.k, c.v, c.table, LONGEST, c.ks, c.vs, rope_base=0.0)
        prompt = na.ne_attn_gqa_varlen_fwd_rotated(qr, kr, v, cu, ROOM)
        last = qr[(cu[1:].long() - 1).clamp(min=0)]  # each sequence's last new row
        got = na.ne_attn_decode_paged(last, c.k, c.v, c.table, self.lens, LONGEST, c.ks, c.vs,
                                      rope_base=0.0)
        return dict(cu=cu, start=start, pos=pos, slots=slots, qr=qr, kr=kr, v=v, last=last,
                    prompt=prompt[0], prompt_lse=prompt[1], out=got[0], lse=got[1])


# (new rows, finished before): prompts, tokens, an idle sequence, a request that ends and
# another in its place, a step without any row.
STEPS = [([17, 1, 40, 0, 30], [0] * 5), ([1, 1, 1, 1, 1], [0] * 5), ([1, 0, 1, 1, 1], [0] * 5),
         ([0] * 5, [0] * 5), ([1, 1, 60, 1, 1], [0, 0, 1, 0, 0]), ([1] * 5, [0] * 5),
         ([2, 0, 1, 33, 5], [1, 1, 0, 1, 0]), ([1] * 5, [0] * 5)]


def _set(s, i):
    g = torch.Generator("cpu").manual_seed(100 + i)
    s.qkv.copy_(torch.randn(s.qkv.shape, generator=g).bfloat16())
    s.new.copy_(_i32(STEPS[i][0]))
    s.done.copy_(torch.tensor(STEPS[i][1], device="cuda").bool())


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
def test_steps(na, kind):
    s, c = Server(na, kind), None
    n_pages = s.c.n_pages
    plain = step.Pages(B, WIDTH, n_pages, PAGE, [(7 * i) % n_pages for i in range(n_pages)])
    held = [[torch.zeros((0, HKV, 64), dtype=F64, device="cuda")] * 2 for _ in range(B)]
    for i, (new, done) in enumerate(STEPS):
        _set(s, i)
        got = s.step()
        assert na.ne_attn_get_device_status() == 0
        plain.release(done)
        want = plain.reserve(new, ROOM)
        for name, w in zip(("cu", "start", "pos", "slots"), want):
            assert got[name].tolist() == w
        assert s.lens.tolist() == plain.lens and s.c.table.tolist() == plain.table
        cu, n, pos = want[0], sum(new), torch.tensor(want[2][:sum(new)], device="cuda")
        for name, x, w in (("qr", s.qkv[:n, :H], s.wq), ("kr", s.qkv[:n, H:H + HKV], s.wk)):
            y, err = step.norm(x, w, 1e-5, pos)
            within(got[name][:n], y, err, name)
        c = s.c
        for b in range(B):
            if done[b]:
                held[b] = [t[:0] for t in held[b]]
            for j, x in enumerate((got["kr"], got["v"])):
                x = x[cu[b]:cu[b + 1]].to(F64)
                if kind == "e4m3":
                    x8, e = quantise(x)
                    x = x8 * torch.exp2(e)[..., None]
                elif kind == "e2m1":
                    x = quantise4(x)[0]
                held[b] = [torch.cat((t, x)) if k == j else t for k, t in enumerate(held[b])]
            if not plain.lens[b]:
                assert bool((got["out"][b] == 0).all())
                continue
            rows = c.rows(b, plain.lens[b])
            assert torch.equal(rows[0], held[b][0]) and torch.equal(rows[1], held[b][1])
            o, l, oe, le = attention(got["last"][b:b + 1], *rows, 0.125)
            oe = oe[0]
            if kind == "e2m1":
                oe = oe + step.half_weights(got["last"][b], rows[0],
                                            c.value_scales(b, plain.lens[b]), 0.125)
            within(got["out"][b], o[0], oe, f"out of {b} in step {i}")
            within(got["lse"][b], l[:, 0], le[:, 0], f"lse of {b} in step {i}")
            if new[b] and new[b] == plain.lens[b]:  # a whole prompt: its own attention
                r = slice(cu[b], cu[b + 1])
                o, l, oe, le = attention(got["qr"][r], got["kr"][r], got["v"][r], 0.125)
                within(got["prompt"][r], o, oe, f"prompt {b}")
                within(got["prompt_lse"][:, r], l, le, f"prompt lse {b}")


@pytest.mark.parametrize("kind", ["bf16", "e2m1"])
def test_steps_replayed_from_a_graph(na, kind):
    eager, s = Server(na, kind), Server(na, kind)
    _set(eager, 0)
    _set(s, 0)
    first = eager.step(), s.step()
    torch.cuda.synchronize()
    assert all(torch.equal(first[0][x], first[1][x]) for x in ("cu", "out", "lse"))
    g, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        got = s.step()
    for i in range(1, len(STEPS)):
        _set(eager, i)
        _set(s, i)
        want = eager.step()
        g.replay()
        torch.cuda.synchronize()
        n = sum(STEPS[i][0])
        for name, w in want.items():
            x = got[name]
            if name in ("qr", "kr", "v", "prompt"):
                x, w = x[:n], w[:n]
            elif name == "prompt_lse":
                x, w = x[:, :n], w[:, :n]
            elif name == "last":
                continue  # (of a sequence without rows: whatever lay there)
            elif name in ("out", "lse"):
                has = torch.tensor([m > 0 for m in STEPS[i][0]], device="cuda")
                x, w = x[has], w[has]
            assert torch.equal(x, w), (i, name)
        assert torch.equal(s.lens, eager.lens) and torch.equal(s.c.table, eager.c.table)
    assert na.ne_attn_get_device_status() == 0

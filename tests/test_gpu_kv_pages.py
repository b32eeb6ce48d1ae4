"""Pages handed out and taken back on the GPU, with the positions and slots of a step's
rows, against the plain implementation of step.py: every number equal."""
import random

import pytest
import torch

import step

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


class Gpu:
    """The same state on the GPU; unused stack entries hold garbage."""

    def __init__(self, plain):
        self.p = plain
        free = plain.free + [-7] * (plain.n_pages - len(plain.free))
        self.table, self.lens = _i32(plain.table), _i32(plain.lens)
        self.free, self.n_free = _i32(free), _i32([len(plain.free)])
        self.max_seqlen = len(plain.table[0]) * plain.page

    def reserve(self, na, new, room, **kw):
        return na.ne_kv_reserve(_i32(new), self.lens, self.table, self.free, self.n_free, room,
                                self.p.page, self.max_seqlen, **kw)

    def release(self, na, finished):
        na.ne_kv_release(torch.tensor(finished, device="cuda").bool(), self.lens, self.table,
                         self.free, self.n_free, self.p.page, self.max_seqlen)

    def state(self):
        n = int(self.n_free)
        return self.table.tolist(), self.lens.tolist(), self.free[:n].tolist()

    def check(self):
        assert self.state() == (self.p.table, self.p.lens, self.p.free)


def _steps(na, nseq, page, max_pages, steps, most, seed, bounds=None):
    """Random steps, in place, with sequences finishing; all state compared each time."""
    rng = random.Random(seed)
    n_pages = nseq * max_pages
    order = list(range(n_pages))
    rng.shuffle(order)
    plain = step.Pages(nseq, max_pages, n_pages, page, order)
    gpu = Gpu(plain)
    for i in range(steps):
        new = [min(rng.choice((0, 1, 1, rng.randint(0, most))), max_pages * page - n)
               for n in plain.lens]
        room = sum(new) + rng.choice((0, 1, 5, 4096))
        got = gpu.reserve(na, new, room)
        assert na.ne_attn_get_device_status() == 0
        for g, w, name in zip(got, plain.reserve(new, room),
                              ("cu_seqlens", "start_pos", "positions", "slots")):
            assert g.tolist() == w, (i, name)
        gpu.check()
        finished = [rng.random() < 0.3 for _ in range(nseq)]
        gpu.release(na, finished)
        assert na.ne_attn_get_device_status() == 0
        plain.release(finished)
        gpu.check()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("nseq", [1, 3, 64])
def test_steps(na, page, nseq):
    _steps(na, nseq, page, 5, 12, 2 * page, seed=page + nseq)


@pytest.mark.parametrize("nseq,most", [(1023, 40), (1024, 200), (1025, 3), (5000, 60), (16384, 2)])
def test_many_sequences(na, nseq, most):
    """Several CTAs, and more sequences than one of them has threads."""
    _steps(na, nseq, 16, 8, 3, most, seed=nseq)


def test_one_long_sequence(na):
    _steps(na, 1, 16, 20000, 3, 300000, seed=9)


def test_new_values_beside_the_old(na):
    """seq_lens_out, n_free_out given: the inputs stay, and the call can be repeated."""
    plain = step.Pages(4, 6, 30, 16, range(30))
    gpu = Gpu(plain)
    gpu.reserve(na, [20, 0, 33, 1], 54)
    plain.reserve([20, 0, 33, 1], 54)
    before = gpu.state()
    lens, n_free = _i32([0] * 4), _i32([0])
    want = plain.reserve([1, 40, 15, 0], 60)
    for _ in range(2):
        got = gpu.reserve(na, [1, 40, 15, 0], 60, seq_lens_out=lens, n_free_out=n_free)
        assert [t.tolist() for t in got] == list(want)
        assert (lens.tolist(), n_free.tolist()) == (plain.lens, [len(plain.free)])
        assert gpu.state()[1:] == before[1:] and gpu.table.tolist() == plain.table


def test_nothing_wanted_but_the_table(na):
    """No positions, no slots: the number of rows has no bound."""
    plain = step.Pages(2, 6, 12, 16, range(12))
    gpu = Gpu(plain)
    got = gpu.reserve(na, [50, 20], 0)
    want = plain.reserve([50, 20], 70)
    assert na.ne_attn_get_device_status() == 0
    assert got[0].tolist() == want[0] and got[2].numel() == 0
    gpu.check()


@pytest.mark.parametrize("nseq", [2, 3000])
@pytest.mark.parametrize("new,code", [
    ([65, 0], 7), ([-1, 5], 7), ([0, 60], 7), ([40, 30], 7),   # past the table, negative, rows
    ([2 ** 31 - 1, 2 ** 31 - 1], 7), ([33, 40], 10),           # sums past 32 bits; pages
])
def test_all_or_nothing(na, nseq, new, code):
    """What does not fit leaves everything as it was, and there are no rows."""
    plain = step.Pages(nseq, 4, 6, 16, range(6))
    gpu = Gpu(plain)
    fill = [0] * (nseq - 2)
    gpu.reserve(na, [1, 20, *fill], 32)
    plain.reserve([1, 20, *fill], 32)
    before = gpu.state()
    room = 4096 * 5 if code == 10 else 69  # several CTAs
    got = gpu.reserve(na, [*new, *fill], room)
    assert na.ne_attn_get_device_status() == code
    assert got[0].tolist() == [0] * (nseq + 1) and got[1].tolist() == plain.lens
    assert got[2].tolist() == [-1] * room and got[3].tolist() == [-1] * room
    assert gpu.state() == before
    got = gpu.reserve(na, [0, 1, *fill], 4)  # and the next step is sound
    assert na.ne_attn_get_device_status() == 0
    assert [t.tolist() for t in got] == list(plain.reserve([0, 1, *fill], 4))


def test_bad_lengths_and_counts(na):
    for lens, n_free, code in (([-1, 0], 4, 7), ([65, 0], 4, 7), ([0, 2 ** 31 - 1], 4, 7),
                               ([0, 0], -3, 10), ([0, 0], 9, 10), ([0, 0], 2 ** 31 - 1, 10)):
        plain = step.Pages(2, 4, 8, 16, range(8))
        gpu = Gpu(plain)
        gpu.lens, gpu.n_free = _i32(lens), _i32([n_free])
        for call in (lambda: gpu.reserve(na, [1, 1], 5), lambda: gpu.release(na, [1, 1])):
            call()
            assert na.ne_attn_get_device_status() == code
            assert gpu.lens.tolist() == lens and gpu.n_free.tolist() == [n_free]
            assert gpu.table.tolist() == plain.table and gpu.free.tolist() == list(range(8))


def test_a_page_outside_the_pool(na):
    """Entries are handed out as they are; the rows there have no slot, and it is told."""
    plain = step.Pages(2, 4, 8, 16, [0, 1, 2, 99, 4])
    gpu = Gpu(plain)
    _, _, pos, slots = gpu.reserve(na, [20, 16], 36)
    assert na.ne_attn_get_device_status() == 9
    assert pos.tolist() == list(range(20)) + list(range(16))
    assert slots.tolist() == [4 * 16 + i for i in range(16)] + [-1] * 4 + \
        [2 * 16 + i for i in range(16)]
    assert gpu.table.tolist()[0][:2] == [4, 99]
    _, _, _, slots = gpu.reserve(na, [5, 0], 5)  # the rest of that page
    assert na.ne_attn_get_device_status() == 9 and slots.tolist() == [-1] * 5


@pytest.mark.parametrize("left", ["cu_seqlens", "start_pos", "positions", "slots", "both", "all"])
@pytest.mark.parametrize("shift", [0, 1])
def test_outputs_that_are_not_wanted(na, left, shift):
    """The C entry with NULL for some of the outputs, and outputs that are 4-byte aligned."""
    lens, new = [0, 30, 5], [40, 3, 0]
    plain = step.Pages(3, 6, 18, 16, range(18))
    gpu = Gpu(plain)
    gpu.reserve(na, lens, 35)
    plain.reserve(lens, 35)
    want = plain.reserve(new, 50)
    room = [torch.full((n + shift,), -9, dtype=torch.int32, device="cuda")[shift:] for n in (4, 3, 50, 50)]
    names = ("cu_seqlens", "start_pos", "positions", "slots")
    none = {"both": names[2:], "all": names}.get(left, (left,))
    out = [None if n in none else t.data_ptr() for n, t in zip(names, room)]
    more = _i32(new)
    rc = na.lib().ne_kv_reserve(
        more.data_ptr(), gpu.lens.data_ptr(), 3, gpu.table.data_ptr(), 6, gpu.free.data_ptr(),
        gpu.n_free.data_ptr(), 18, 16, 96, 50, *out, gpu.lens.data_ptr(), gpu.n_free.data_ptr(),
        torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and na.ne_attn_get_device_status() == 0
    for n, t, w in zip(names, room, want):
        assert t.tolist() == ([-9] * t.numel() if n in none else w), n
    gpu.check()


def test_slots_up_to_31_bits(na):
    """The largest pool: its last pages' slots, and rows of a long sequence of them."""
    n_pages = (2 ** 31 - 1) // 256
    free = torch.arange(n_pages, dtype=torch.int32, device="cuda")
    lens, n_free = _i32([0, 3]), _i32([n_pages])
    table = torch.full((2, 5000), -1, dtype=torch.int32, device="cuda")
    table[1, 0] = 7
    m = 1000 * 256 + 5
    cu, start, pos, slots = na.ne_kv_reserve(_i32([m, 2]), lens, table, free, n_free, m + 2, 256,
                                             5000 * 256)
    assert na.ne_attn_get_device_status() == 0
    assert cu.tolist() == [0, m, m + 2] and start.tolist() == [0, 3] and lens.tolist() == [m, 5]
    assert n_free.tolist() == [n_pages - 1001]
    i = torch.arange(m, device="cuda")
    assert torch.equal(pos[:m].long(), i)
    assert torch.equal(slots[:m].long(), (n_pages - 1 - i // 256) * 256 + i % 256)
    assert slots[m:].tolist() == [7 * 256 + 3, 7 * 256 + 4]
    na.ne_kv_release(torch.tensor([1, 0], dtype=torch.uint8, device="cuda"), lens, table, free,
                     n_free, 256, 5000 * 256)
    assert na.ne_attn_get_device_status() == 0
    assert n_free.tolist() == [n_pages] and lens.tolist() == [0, 5]
    assert torch.equal(free[-1001:].flip(0), torch.arange(n_pages - 1001, n_pages, device="cuda"))


def test_giving_back_too_much(na):
    """A stack that would hold more than there is stays as it was."""
    plain = step.Pages(2, 4, 4, 16, range(4))
    gpu = Gpu(plain)
    gpu.reserve(na, [40, 0], 40)
    gpu.n_free.fill_(2)
    before = gpu.state()
    gpu.release(na, [1, 0])
    assert na.ne_attn_get_device_status() == 10
    assert gpu.state() == before


def test_streams_and_replays(na):
    """A captured step, replayed: the state moves on by itself, step after step."""
    plain = step.Pages(5, 8, 40, 16, range(40))
    gpu = Gpu(plain)
    new = _i32([1, 3, 0, 7, 20])
    done = torch.zeros(5, dtype=torch.uint8, device="cuda")
    room = 8192  # two CTAs

    def one(**kw):
        got = na.ne_kv_reserve(new, gpu.lens, gpu.table, gpu.free, gpu.n_free, room, 16, 128, **kw)
        na.ne_kv_release(done, gpu.lens, gpu.table, gpu.free, gpu.n_free, 16, 128, **kw)
        return got

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = one(stream=side)
    torch.cuda.synchronize()
    assert [t.tolist() for t in got] == list(plain.reserve([1, 3, 0, 7, 20], room))
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        got = one()
    rng = random.Random(4)
    for _ in range(12):
        n, f = [rng.randint(0, 15) for _ in range(5)], [int(rng.random() < 0.3) for _ in range(5)]
        n = [min(x, 128 - y) for x, y in zip(n, plain.lens)]
        new.copy_(_i32(n))
        done.copy_(torch.tensor(f, dtype=torch.uint8))
        g.replay()
        torch.cuda.synchronize()
        assert na.ne_attn_get_device_status() == 0
        assert [t.tolist() for t in got] == list(plain.reserve(n, room))
        plain.release(f)
        gpu.check()


def test_two_streams_at_once(na):
    """Calls of several CTAs in flight on two streams, each on its own state."""
    plains = [step.Pages(2000, 8, 16000, 16, range(16000)) for _ in range(2)]
    gpus = [Gpu(p) for p in plains]
    new = [(i * 5) % 9 for i in range(2000)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    n = _i32(new)
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        for g, s in zip(gpus, streams):
            got.append(na.ne_kv_reserve(n, g.lens, g.table, g.free, g.n_free, 9000, 16, 128, stream=s))
    torch.cuda.synchronize()
    assert na.ne_attn_get_device_status() == 0
    for i in range(6):
        for j, p in enumerate(plains):
            assert [t.tolist() for t in got[2 * i + j]] == list(p.reserve(new, 9000))
    for g in gpus:
        g.check()

"""Pages handed out and taken back: bounds on rows whose places nobody wants, and entries
that are no page of the pool."""
import pytest
import torch

import step
from test_gpu_kv_pages import Gpu, _i32, na  # noqa: F401

pytestmark = pytest.mark.gpu


def _c_reserve(na, gpu, new, n_tot, outs):
    """The C entry, with the outputs named in outs."""
    nseq, width = gpu.table.shape
    room = {n: torch.full((m,), -9, dtype=torch.int32, device="cuda") for n, m in
            (("cu_seqlens", nseq + 1), ("start_pos", nseq), ("positions", n_tot), ("slots", n_tot))}
    more = _i32(new)
    rc = na.lib().ne_kv_reserve(
        more.data_ptr(), gpu.lens.data_ptr(), nseq, gpu.table.data_ptr(), width, gpu.free.data_ptr(),
        gpu.n_free.data_ptr(), gpu.p.n_pages, gpu.p.page, gpu.max_seqlen, n_tot,
        *(t.data_ptr() if n in outs else None for n, t in room.items()), gpu.lens.data_ptr(),
        gpu.n_free.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    return na.ne_attn_get_device_status(), room


@pytest.mark.parametrize("nseq", [3, 3000])
@pytest.mark.parametrize("outs", [(), ("cu_seqlens", "start_pos"), ("positions",), ("slots",)])
def test_more_rows_than_there_is_room_for(na, outs, nseq):  # noqa: F811
    """n_tot bounds the rows whichever outputs are wanted: one too many, and nothing is
    handed out; as many as that, and all is."""
    fill = [0] * (nseq - 3)
    plain = step.Pages(nseq, 6, 18, 16, range(18))
    gpu = Gpu(plain)
    gpu.reserve(na, [0, 30, 5, *fill], 35)
    plain.reserve([0, 30, 5, *fill], 35)
    before = gpu.state()
    new = [40, 3, 0, *fill]
    for n_tot in (42, 1):
        code, room = _c_reserve(na, gpu, new, n_tot, outs)
        assert code == 7 and gpu.state() == before
        if "cu_seqlens" in outs:
            assert room["cu_seqlens"].tolist() == [0] * (nseq + 1)
    code, room = _c_reserve(na, gpu, new, 43, outs)
    want = dict(zip(("cu_seqlens", "start_pos", "positions", "slots"), plain.reserve(new, 43)))
    assert code == 0 and all(room[n].tolist() == want[n] for n in outs)
    gpu.check()


@pytest.mark.parametrize("outs", [(), ("cu_seqlens", "start_pos")])
def test_no_bound_without_rows_wanted(na, outs):  # noqa: F811
    plain = step.Pages(3, 6, 18, 16, range(18))
    gpu = Gpu(plain)
    code, room = _c_reserve(na, gpu, [40, 3, 0], 0, outs)
    want = dict(zip(("cu_seqlens", "start_pos"), plain.reserve([40, 3, 0], 43)))
    assert code == 0 and all(room[n].tolist() == want[n] for n in outs)
    gpu.check()


@pytest.mark.parametrize("nseq", [2, 1024, 3000, 16384])
@pytest.mark.parametrize("bad", [-1, -2 ** 31, 2 ** 31 - 1, "n_pages"])
def test_release_of_what_is_no_page(na, nseq, bad):  # noqa: F811
    """All or nothing: an entry outside the pool is told, and none of the others is given
    back; entries of sequences that go on, and behind a sequence's pages, do not matter."""
    width, page = 4, 16
    plain = step.Pages(nseq, width, nseq * width, page, range(nseq * width))
    gpu = Gpu(plain)
    new = [(7 * s) % (width * page) + 1 for s in range(nseq)]
    gpu.reserve(na, new, sum(new))
    plain.reserve(new, sum(new))
    bad = plain.n_pages if bad == "n_pages" else bad
    on = nseq // 2  # the sequence that goes on
    finished = [s != on for s in range(nseq)]
    for s in {0, nseq // 3, nseq - 1} - {on}:
        for col in {0, (new[s] - 1) // page}:
            good = int(gpu.table[s, col])
            gpu.table[s, col] = bad
            before = gpu.state()
            gpu.release(na, finished)
            assert na.ne_attn_get_device_status() == 9
            assert gpu.state() == before
            gpu.table[s, col] = good
    gpu.table[on] = bad
    gpu.table[0, 3] = bad  # (its one row is on page 0)
    gpu.release(na, finished)
    plain.release(finished)
    assert na.ne_attn_get_device_status() == 0
    gpu.table[on] = _i32(plain.table[on])
    gpu.table[0, 3] = -1
    gpu.check()


def test_release_of_many_pages(na):  # noqa: F811
    """Several CTAs' shares of one sequence's pages beside many short ones."""
    nseq, width = 5000, 3000
    plain = step.Pages(nseq, width, 8000, 16, range(8000))
    gpu = Gpu(plain)
    new = [1] * nseq
    new[1234] = width * 16
    gpu.reserve(na, new, sum(new))
    plain.reserve(new, sum(new))
    good = gpu.table[1234, 2999].clone()
    gpu.table[1234, 2999] = 8000
    before = gpu.state()
    gpu.release(na, [True] * nseq)
    assert na.ne_attn_get_device_status() == 9 and gpu.state() == before
    gpu.table[1234, 2999] = good
    gpu.release(na, [True] * nseq)
    plain.release([True] * nseq)
    assert na.ne_attn_get_device_status() == 0
    gpu.check()

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

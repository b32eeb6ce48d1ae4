"""A step in which no sequence has a row: nothing is written, nothing is refused."""
import pytest
import torch

from grouped import Cache


def _empty(dev):
    return torch.empty((0, 2, 64), dtype=torch.bfloat16, device=dev)


def _zeros(n, dev):
    return torch.zeros(n, dtype=torch.int32, device=dev)


def _step(na, c, dev):
    before = [t.clone() for t in (c.k, c.v, c.ks, c.vs) if t is not None]
    pools = na.ne_kv_append(_empty(dev), _empty(dev), _zeros(4, dev), _zeros(3, dev), c.k, c.v,
                            c.table, 40, c.ks, c.vs)
    assert pools[0] is c.k and pools[1] is c.v
    for a, b in zip((t for t in (c.k, c.v, c.ks, c.vs) if t is not None), before):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    k, v = na.ne_kv_read(c.k, c.v, c.table, _zeros(4, dev), _zeros(3, dev), 0, c.ks, c.vs)
    assert k.shape == v.shape == (0, 2, 64) and k.dtype == v.dtype == torch.bfloat16
    given = _empty(dev), _empty(dev)
    k, v = na.ne_kv_read(c.k, c.v, c.table, _zeros(4, dev), _zeros(3, dev), 0, c.ks, c.vs,
                         k=given[0], v=given[1])
    assert k is given[0] and v is given[1]
    with pytest.raises(ValueError):  # the checks of the arguments are made all the same
        na.ne_kv_append(_empty(dev)[:, :1], _empty(dev), _zeros(4, dev), _zeros(3, dev), c.k, c.v,
                        c.table, 40, c.ks, c.vs)


@pytest.mark.parametrize("e4m3", [False, True])
def test_no_rows_without_a_gpu(monkeypatch, e4m3):
    from causal_self_attention_gb300 import ne_attn as na
    monkeypatch.setattr(na, "lib", lambda: pytest.fail("the library was called"))
    monkeypatch.setattr(na, "_device", lambda t, name: -1)
    monkeypatch.setattr(na, "_need_on", lambda t, dtype, dev, name: None)
    monkeypatch.setattr(na, "_on", lambda stream, dev: (0, None))
    _step(na, Cache([40] * 3, 2, 16, e4m3, seed=1, device="cpu"), "cpu")


@pytest.mark.gpu
@pytest.mark.parametrize("e4m3", [False, True])
def test_no_rows(e4m3):
    from causal_self_attention_gb300 import build, ne_attn as na
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _step(na, Cache([40] * 3, 2, 16, e4m3, seed=1), "cuda")
    assert na.ne_attn_get_device_status() == 0

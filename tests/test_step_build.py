"""The native module beside the library: what it takes to have it, and what works without."""
import pytest
import torch


@pytest.fixture
def fresh(monkeypatch):
    """The binding as before its first call (the library is built)."""
    from causal_self_attention_gb300 import build, ne_attn
    build.build()
    monkeypatch.setattr(ne_attn, "_lib", None)
    monkeypatch.setattr(ne_attn, "_step", None)
    return ne_attn


def test_calls_without_the_module(fresh, monkeypatch, tmp_path):
    """The binding is complete without it: the library loads and its calls are made."""
    monkeypatch.setattr(fresh._build, "step_path", lambda: str(tmp_path / "none.so"))
    L = fresh.lib()
    assert fresh._step is None and fresh.lib() is L
    assert L.ne_status_string(7) == b"NE_ERR_BAD_SEQLEN"
    assert fresh.ne_attn_decode_paged_workspace_bytes(4, 8, 2, 500) > 0
    bf, i = torch.zeros((4, 2, 64), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):  # (CPU tensors: said in Python)
        fresh.ne_qk_norm_rope_fwd(bf, bf, bf[0, 0], bf[0, 0], i, 4)


@pytest.mark.gpu
def test_the_same_results_without_the_module(monkeypatch):
    from causal_self_attention_gb300 import build, ne_attn as na
    from test_gpu_step_calls import _calls, _same
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    na.lib()
    calls = _calls(na)
    want = [call() for _, call in calls]
    monkeypatch.setattr(na, "_step", None)
    for (name, call), w in zip(calls, want):
        assert _same(call(), w), name
    assert na.ne_attn_get_device_status() == 0


def test_the_module_belongs_to_this_python_and_torch():
    """Its name says for which interpreter and torch it was built: another one's is not
    loaded."""
    import importlib.machinery
    import sysconfig

    from causal_self_attention_gb300 import build
    name = build.step_path()
    assert torch.__version__ in name and name.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert sysconfig.get_config_var("EXT_SUFFIX") in importlib.machinery.EXTENSION_SUFFIXES

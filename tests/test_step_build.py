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


class Compiler:
    """In subprocess.run's place: notes the commands, and makes (or not) what they name."""

    def __init__(self, fail=()):
        self.commands, self.fail = [], fail

    def __call__(self, cmd, **kw):
        import subprocess
        self.commands.append(cmd)
        bad = any(cmd[0].endswith(f) for f in self.fail)
        if not bad:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, int(bad), "", "no such header" if bad else "")


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """build() into an empty folder, by a compiler that makes empty files."""
    from causal_self_attention_gb300 import build
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libne_attn.so"))
    monkeypatch.delenv("CXX", raising=False)
    monkeypatch.setattr(build.subprocess, "run", Compiler())
    return build


def test_the_module_alone_needs_no_nvcc(elsewhere, monkeypatch, tmp_path):
    elsewhere.build()
    run = elsewhere.subprocess.run
    assert (tmp_path / "libne_attn.so").exists() and run.commands
    import os
    os.remove(elsewhere.step_path())
    run.commands.clear()
    monkeypatch.setattr(elsewhere, "nvcc_path", lambda: pytest.fail("nvcc is asked for"))
    assert elsewhere.build() == str(tmp_path / "libne_attn.so")
    assert [c[0] for c in run.commands] == ["g++"] and os.path.exists(elsewhere.step_path())
    run.commands.clear()
    elsewhere.build()
    assert not run.commands  # both are fresh


def test_the_library_is_built_where_the_module_cannot_be(elsewhere, monkeypatch, tmp_path):
    """(Without Python's or torch's headers, say.)  It is told, and the next build tries again."""
    import os
    monkeypatch.setattr(elsewhere.subprocess, "run", Compiler(fail=("g++",)))
    open(elsewhere.step_path(), "w").close()  # one of older sources
    os.utime(elsewhere.step_path(), (0, 0))
    for _ in range(2):
        with pytest.warns(RuntimeWarning, match="no such header"):
            assert elsewhere.build() == str(tmp_path / "libne_attn.so")
        assert os.path.exists(elsewhere.LIB_PATH) and not os.path.exists(elsewhere.step_path())
    monkeypatch.setattr(elsewhere.subprocess, "run", Compiler(fail=("nvcc",)))
    with pytest.raises(RuntimeError, match="nvcc failed"):
        elsewhere.build(force=True)

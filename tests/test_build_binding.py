"""When the compiled Python module is linked again (CPU only, no compiler runs:
the module, its object and the library are empty files of chosen ages)."""
import os

import pytest

from sparse_attention_kv_qsa_gb300 import build, qsa


@pytest.fixture
def files(tmp_path, monkeypatch):
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    for name in ("LIB", "OPS", "OPS_KEY"):
        monkeypatch.setattr(build, name, str(tmp_path / name.lower()))
    monkeypatch.setattr(build, "build_calls", [], raising=False)

    def run(cmd, **kw):                                   # stands for g++: makes the file named after -o
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        build.build_calls.append(os.path.basename(out))
        return type("R", (), {"returncode": 0})

    monkeypatch.setattr(build.subprocess, "run", run)
    open(build.LIB, "w").close()
    os.utime(build.LIB, (1, 1))
    return build


def steps(b):
    """What build() does for the module; the number of compilations and links it took."""
    before = len(b.build_calls)
    obj = b._compile_binding(False)
    if not b._binding_is_current(obj):
        b._link_binding(obj)
    return len(b.build_calls) - before


def test_another_torch_and_back_links_the_right_object(files, monkeypatch):
    own = files.binding_key()
    assert steps(files) == 2 and steps(files) == 0 and files.linked_for() == own
    monkeypatch.setattr(files, "binding_key", lambda: "torch other")
    assert steps(files) == 2 and files.linked_for() == "torch other"
    monkeypatch.setattr(files, "binding_key", lambda: own)
    assert steps(files) == 1                              # its object is there, and older than the module
    assert files.linked_for() == own and steps(files) == 0


def test_the_key_names_torch_and_python(files):
    import sysconfig

    import torch
    key = files.binding_key()
    assert torch.__version__ in key and os.path.dirname(torch.__file__) in key
    assert sysconfig.get_config_var("SOABI") in key


def test_a_module_without_a_key_or_of_an_older_library_is_linked_again(files):
    steps(files)
    os.remove(files.OPS_KEY)
    assert steps(files) == 1
    os.utime(files.LIB, None)
    os.utime(files.OPS, (2, 2))
    assert steps(files) == 1 and steps(files) == 0


def test_a_module_of_another_torch_is_not_loaded(files, monkeypatch):
    steps(files)
    monkeypatch.setattr(qsa, "_ops_module", None)
    monkeypatch.setattr(qsa, "lib", lambda: None)
    monkeypatch.setattr(files, "binding_key", lambda: "torch other")
    with pytest.raises(RuntimeError, match="torch other"):
        qsa._ops()

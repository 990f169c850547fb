"""Without the native binding every call still works through the checks in
Python: the products do not need it, nor does a machine without a host compiler
or headers for it."""

import os
import sys
import warnings

import pytest

import bit_quantized_gemm_qgemm_amd as qg
from bit_quantized_gemm_qgemm_amd import build


@pytest.fixture
def fresh(monkeypatch):
    """The module as before its first call, the binding not importable."""
    if not os.path.exists(qg.LIB_PATH):
        build.build()
    monkeypatch.setattr(qg, "_lib", None)
    monkeypatch.setattr(qg, "_native", None)
    monkeypatch.delattr(qg, "_binding", raising=False)
    monkeypatch.setitem(sys.modules, qg.__name__ + "._binding", None)


def test_the_library_loads_without_the_binding(fresh):
    with pytest.warns(RuntimeWarning, match="binding"):
        lib = qg.lib()
    assert qg._native is None
    with warnings.catch_warnings():
        warnings.simplefilter("error")          # said once
        assert qg.lib() is lib
        assert lib.qgemm_prepack_bytes(1, 1024, 1024) == 1024 * 1024 // 2
        assert qg.qgemm_paged_attention_workspace_bytes(1, 8, 2, 64, 100) >= 0


def test_the_binding_belongs_to_one_interpreter():
    import sysconfig

    assert build.BINDING_PATH.endswith("_binding" + sysconfig.get_config_var("EXT_SUFFIX"))


@pytest.mark.parametrize("missing", ["compiler", "headers"])
def test_the_library_builds_without_a_host_toolchain(monkeypatch, tmp_path, missing):
    calls = []

    def run(cmd, what, verbose):
        calls.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("x")

    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libqgemm.so"))
    monkeypatch.setattr(build, "BINDING_PATH", str(tmp_path / "_binding.so"))
    (tmp_path / "_binding.so").write_text("of another build")
    if missing == "compiler":
        which = build.shutil.which
        monkeypatch.setattr(build.shutil, "which", lambda name: None if name == "g++" else which(name))
    else:
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    with pytest.warns(RuntimeWarning, match="binding"):
        assert build.build() == str(tmp_path / "libqgemm.so")
    assert (tmp_path / "libqgemm.so").exists()
    assert not (tmp_path / "_binding.so").exists()
    assert not any(cmd[0] == "g++" for cmd in calls)

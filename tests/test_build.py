"""What build() makes and when: the library needs no Python, the module of the
cache calls belongs to one interpreter."""
import os
import sysconfig

import pytest

from bf16_gemm_skinny_gb300 import _native as bsk
from bf16_gemm_skinny_gb300 import build as b


@pytest.fixture(scope="module", autouse=True)
def built():
    b.build()


@pytest.fixture
def no_compiler(monkeypatch):
    def run(*args, **kwargs):
        raise AssertionError("nothing is to be compiled")

    monkeypatch.setattr(b.subprocess, "run", run)


def test_the_module_carries_the_interpreters_tag():
    assert os.path.basename(b.CALLS_PATH) == "_calls" + sysconfig.get_config_var("EXT_SUFFIX")
    assert os.path.exists(b.CALLS_PATH) and bsk._load_calls().__file__ == b.CALLS_PATH


def test_nothing_is_built_twice(no_compiler):
    assert not b.is_stale() and b.build() == b.LIB_PATH


def test_another_interpreter_builds_its_own_module_and_not_the_library(monkeypatch):
    monkeypatch.setattr(b, "CALLS_PATH", os.path.join(b.BUILD_DIR, "_calls.cpython-399-none.so"))
    assert b.is_stale() and not b._lib_stale()


def test_without_python_headers_the_library_is_enough(monkeypatch, no_compiler, tmp_path):
    monkeypatch.setattr(b.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    monkeypatch.setattr(b, "CALLS_PATH", str(tmp_path / "_calls.so"))
    assert not b.is_stale() and b.build() == b.LIB_PATH
    monkeypatch.setattr(bsk, "_calls", None)
    with pytest.raises(RuntimeError, match="Python.h"):
        bsk._load_calls()


@pytest.mark.slow
def test_a_module_that_does_not_compile_leaves_the_library(monkeypatch, tmp_path):
    (tmp_path / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    (tmp_path / "py_calls.cpp").write_text("#error not today\n")
    for name, value in (("CSRC", str(tmp_path)), ("BUILD_DIR", str(tmp_path / "out")), ("LIB_PATH", str(tmp_path / "out" / "libbsk.so")),
                        ("CALLS_PATH", str(tmp_path / "out" / "_calls.so")), ("CALLS_SOURCE", str(tmp_path / "py_calls.cpp"))):
        monkeypatch.setattr(b, name, value)
    with pytest.raises(RuntimeError, match="py_calls"):
        b.build()
    assert os.path.exists(b.LIB_PATH) and not os.path.exists(b.CALLS_PATH)
    assert b.is_stale() and not b._lib_stale()

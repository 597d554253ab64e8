"""The build: the C library stands on its own, and the Python module follows the PyTorch it is for."""
import ctypes
import os

import pytest

from gathered_rank_gemm_gb300 import build


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """A build of one small source in a folder of its own."""
    src = tmp_path / "one.cu"
    src.write_text('extern "C" __attribute__((visibility("default"))) int one() { return 1; }\n')
    for name, value in dict(LIB_PATH="lib.so", NATIVE_PATH="_native.so", BUILD_DIR="_build",
                            NATIVE_FOR="_build/native_for").items():
        monkeypatch.setattr(build, name, str(tmp_path / value), raising=False)
    monkeypatch.setattr(build, "_sources", lambda: [str(src)])
    return tmp_path


def test_the_library_is_there_where_the_module_does_not_compile(elsewhere, monkeypatch):
    def fails():
        raise RuntimeError("no PyTorch headers")
    monkeypatch.setattr(build, "_compile_native", fails)
    with pytest.raises(RuntimeError, match="no PyTorch headers"):
        build.build()
    assert ctypes.CDLL(build.LIB_PATH).one() == 1
    assert not os.path.exists(build.NATIVE_PATH) and build.is_stale()


def test_the_module_is_stale_under_another_pytorch(elsewhere, monkeypatch):
    def compiles():
        return "object"

    def links(obj):
        open(build.NATIVE_PATH, "w").close()
        with open(build.NATIVE_FOR, "w") as f:
            f.write(build._pytorch())
    monkeypatch.setattr(build, "_compile_native", compiles)
    monkeypatch.setattr(build, "_link_native", links)
    build.build()
    assert not build.is_stale()
    monkeypatch.setattr(build, "_pytorch", lambda: "another one")
    assert build.is_stale()
    when = os.path.getmtime(build.LIB_PATH)
    build.build()
    assert not build.is_stale() and os.path.getmtime(build.LIB_PATH) == when  # the library is none the older

"""What the build makes anew, and when: compilers that only note their calls stand in for nvcc and g++."""
import os
import stat

import pytest

SCRIPT = """#!/bin/bash
echo "$@" >> {log}
if [ -n "{fail}" ]; then echo "{fail}" >&2; exit 1; fi
while [ $# -gt 0 ]; do if [ "$1" = -o ]; then echo made > "$2"; fi; shift; done
"""


@pytest.fixture
def box(tmp_path, monkeypatch):
    """The build in a folder of its own: box.nvcc() and box.cxx() are the calls since the last look."""
    from verify_gemm_gb300 import build

    class Box:
        module, out = build, tmp_path / "out"

        def tool(self, name, fail=""):
            path = tmp_path / name
            path.write_text(SCRIPT.format(log=tmp_path / (name + ".log"), fail=fail))
            path.chmod(path.stat().st_mode | stat.S_IXUSR)
            return str(path)

        def calls(self, name):
            log = tmp_path / (name + ".log")
            lines = log.read_text().splitlines() if log.exists() else []
            log.unlink(missing_ok=True)
            return lines

        def again(self):
            """As a new process finds the folder."""
            if hasattr(build, "_binding_failed"):
                monkeypatch.setattr(build, "_binding_failed", None)

    b = Box()
    monkeypatch.setattr(build, "OUT_DIR", str(b.out))
    monkeypatch.setattr(build, "LIB", str(b.out / "libvgemm.so"))
    monkeypatch.setattr(build, "TORCH_LIB", str(b.out / "_vgtorch.so"))
    (tmp_path / "torch").mkdir()
    (tmp_path / "torch" / "version.py").write_text("__version__ = '2.9.1'\n")
    monkeypatch.setattr(build, "_torch_dir", lambda: str(tmp_path / "torch"))
    monkeypatch.setattr(build, "nvcc", lambda: b.tool("nvcc"))
    monkeypatch.setattr(build, "_cxx", lambda: b.tool("g++"))
    b.again()
    return b


def test_the_library_is_built_where_the_torch_binding_cannot_be(box, monkeypatch):
    """Users of the C ABI need neither torch's nor Python's headers."""
    os.makedirs(box.out)
    (box.out / "_vgtorch.so").write_text("of another build")
    os.utime(box.out / "_vgtorch.so", (1, 1))
    monkeypatch.setattr(box.module, "_cxx", lambda: box.tool("g++", fail="Python.h: No such file or directory"))
    with pytest.warns(RuntimeWarning, match="Python.h"):
        assert box.module.build() == box.module.LIB
    assert (box.out / "libvgemm.so").exists() and not (box.out / "_vgtorch.so").exists()
    assert len(box.calls("nvcc")) == len(box.module.SOURCES) + 1
    box.module.build()                                    # nothing to do: tried once a process
    assert not box.calls("nvcc") and len(box.calls("g++")) == 1
    # headers that came later are found, and the library stays as it is
    box.again()
    monkeypatch.setattr(box.module, "_cxx", lambda: box.tool("g++"))
    box.module.build()
    assert (box.out / "_vgtorch.so").exists() and not box.calls("nvcc")


def test_calls_that_need_the_binding_say_that_it_is_missing(tmp_path, monkeypatch):
    from verify_gemm_gb300 import _lib, build

    build.build()
    monkeypatch.setattr(_lib, "_torch_module", None)
    monkeypatch.setattr(_lib, "TORCH_PATH", str(tmp_path / "_vgtorch.so"))
    with pytest.raises(RuntimeError, match="no fallback"):
        _lib.load_torch()


def test_a_finished_build_is_left_alone(box):
    box.module.build()
    assert len(box.calls("nvcc")) == len(box.module.SOURCES) + 1 and len(box.calls("g++")) == 2
    box.again()
    box.module.build()
    assert not box.calls("nvcc") and not box.calls("g++")


def test_another_torch_makes_the_binding_anew(box):
    """The binding is compiled against one torch's headers; the library is not."""
    box.module.build()
    box.calls("nvcc"), box.calls("g++")
    version = os.path.join(box.module._torch_dir(), "version.py")
    with open(version, "w") as f:
        f.write("__version__ = '2.11.0'\n")
    os.utime(version, (1, 1))                             # (an older file than the build, as wheels hold)
    box.again()
    box.module.build()
    assert len(box.calls("g++")) == 2 and not box.calls("nvcc")
    box.again()
    box.module.build()
    assert not box.calls("g++")


def test_builds_at_the_same_time_make_everything_once(box, tmp_path, monkeypatch):
    """Processes that build at once (parallel tests, several ranks) do not write one another's objects."""
    from concurrent.futures import ThreadPoolExecutor

    slow = SCRIPT.replace("while [", "sleep 0.3\nwhile [")
    for name in ("nvcc", "g++"):
        path = tmp_path / name
        path.write_text(slow.format(log=tmp_path / (name + ".log"), fail=""))
        path.chmod(0o755)
    monkeypatch.setattr(box.module, "nvcc", lambda: str(tmp_path / "nvcc"))
    monkeypatch.setattr(box.module, "_cxx", lambda: str(tmp_path / "g++"))
    with ThreadPoolExecutor(3) as ex:                     # (the lock is a file's: threads and processes wait alike)
        assert [f.result() for f in [ex.submit(box.module.build) for _ in range(3)]] == [box.module.LIB] * 3
    assert len(box.calls("nvcc")) == len(box.module.SOURCES) + 1 and len(box.calls("g++")) == 2

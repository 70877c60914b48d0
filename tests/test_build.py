"""What the build makes where torch is missing or another one than the extension was compiled for. The compilers are
stand-ins that write their output file."""

import os
import stat

import pytest

from expert_major_chunked_gb300 import build

COMPILER = """#!/bin/sh
while [ $# -gt 0 ]; do
  if [ "$1" = -o ]; then echo made > "$2"; echo "$2" >> "{log}"; fi
  shift
done
"""


@pytest.fixture
def made(tmp_path, monkeypatch):
    """A build into an empty folder; returns the names of what has been made since the last call."""
    log, bin_dir, lib = tmp_path / "log", tmp_path / "bin", tmp_path / "lib"
    bin_dir.mkdir()
    for name in ("nvcc", "g++"):
        exe = bin_dir / name
        exe.write_text(COMPILER.format(log=log))
        exe.chmod(exe.stat().st_mode | stat.S_IEXEC)
    monkeypatch.setenv("NVCC", str(bin_dir / "nvcc"))
    monkeypatch.setenv("PATH", f"{bin_dir}:{os.environ['PATH']}")
    for name in ("LIB_PATH", "EXT_PATH", "EXT_KEY_PATH"):
        monkeypatch.setattr(build, name, str(lib / os.path.basename(getattr(build, name))))
    monkeypatch.setattr(build, "LIB_DIR", str(lib))

    def since():
        lines = log.read_text().split() if log.exists() else []
        log.unlink(missing_ok=True)
        return sorted({os.path.basename(x).split(".tmp")[0] for x in lines if not x.endswith(".o")})
    return since


def test_the_library_needs_no_torch(made, monkeypatch):
    find = build.importlib.util.find_spec
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert build.build() == build.LIB_PATH and made() == ["libmoe_prefill.so"]
    assert build.up_to_date() and build.build() == build.LIB_PATH and made() == []
    with pytest.raises(RuntimeError, match="torch is not installed"):
        build.build_extension()


def test_the_library_alone(made):
    build.build(extension=False)
    assert made() == ["libmoe_prefill.so"]
    build.build()
    assert made() == ["attention_py.so"]
    build.build(force=True)
    assert made() == ["attention_py.so", "libmoe_prefill.so"]


def test_an_extension_of_another_torch_or_python_is_made_anew(made, monkeypatch):
    build.build()
    assert made() == ["attention_py.so", "libmoe_prefill.so"]
    build.build()
    build.build_extension()
    assert made() == []
    original, key = build._extension_key, build._extension_key()
    monkeypatch.setattr(build, "_extension_key", lambda: key.replace("__version__ = '", "__version__ = '9"))
    assert build._extension_key() != key
    assert not build.extension_up_to_date() and build.up_to_date()
    build.build_extension()
    assert made() == ["attention_py.so"] and build.extension_up_to_date()
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: "another-abi")
    monkeypatch.setattr(build, "_extension_key", original)
    build.build()
    assert made() == ["attention_py.so"]

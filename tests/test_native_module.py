"""The binding's native module: only the calls that go through it need it, and the library is built without it (CPU)."""
import os
import stat
import subprocess
import sys

import pytest
import torch

from tp_reduce_moe_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = """
import torch
from tp_reduce_moe_gb300 import build
build.marshal_path = lambda: "/nowhere/_marshal.so"
import tp_reduce_moe_gb300 as arf
arf.load_library({path!r})
assert arf.ar_status_string(0)
new = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)
ws = arf.ar_workspace_create(2, 0, 1024, 8, 1e-6, flags=arf.AR_WS_DRY_RUN)
parts = [new(3, 1024) for _ in range(2)]
out, h = arf.ar_rmsnorm(ws, parts, new(3, 1024), new(1024), 0.0, 1e-6)
assert out.shape == h.shape == (3, 1024)
attn = arf.ar_attn_create(4, 2, 64, 16, 4, flags=arf.AR_WS_DRY_RUN)
arf.ar_attn_set_rope(attn, [0.5] * 32)
cache = arf.ar_kv_cache(new(3, 16, 2, 64), new(3, 16, 2, 64))
ints = new(2, dtype=torch.int32)
for call in (lambda: arf.ar_rmsnorm_q8(ws, parts, new(3, 1024), new(1024), 0.0, 1e-6),
             lambda: arf.ar_attn_append(attn, cache, new(2, 512), ints, ints),
             lambda: arf.ar_attn_decode(attn, cache, new(2, 4, 64), new(2, 1, dtype=torch.int32), ints)):
    try:
        call()
    except RuntimeError as e:
        assert "_marshal.so" in str(e) and "build" in str(e), e
    else:
        raise AssertionError("answered without the module")
print("done")
"""


@pytest.mark.parametrize("elsewhere", [False, True])
def test_other_calls_do_without_it(elsewhere, tmp_path):
    path = None
    build.build()
    if elsewhere:  # a library that lies somewhere else
        path = str(tmp_path / "libarfuse.so")
        os.symlink(build.LIB, path)
    r = subprocess.run([sys.executable, "-c", WITHOUT.format(path=path)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, r.stderr[-2000:]


def test_its_name_is_that_of_one_torch_and_one_interpreter(monkeypatch):
    import sysconfig
    name = os.path.basename(build.marshal_path())
    assert name.startswith(f"_marshal.{torch.__version__}.") and sysconfig.get_config_var("SOABI") in name
    monkeypatch.setattr(sysconfig, "get_config_var", lambda n: "cpython-399-other")
    assert os.path.basename(build.marshal_path()) != name


@pytest.fixture()
def stubs(tmp_path, monkeypatch):
    """A build into a folder of its own with a compiler that only makes its output."""
    cc = tmp_path / "nvcc"
    cc.write_text('#!/bin/sh\nwhile [ $# -gt 0 ]; do if [ "$1" = -o ]; then echo made > "$2"; fi; shift; done\n')
    cc.chmod(cc.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setattr(build, "nvcc", lambda: str(cc))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "build"))
    monkeypatch.setattr(build, "LIBDIR", str(tmp_path / "lib"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib" / "libarfuse.so"))
    return tmp_path


@pytest.mark.parametrize("why", ["no torch", "no headers"])
def test_the_library_is_built_where_the_module_cannot_be(stubs, monkeypatch, capsys, why):
    monkeypatch.setattr(build, "torch_paths", lambda: None if why == "no torch" else (str(stubs / "torch"), "9.9"))
    for _ in range(2):
        assert os.path.exists(build.build())
        assert "left out" in capsys.readouterr().err
    assert not [f for f in os.listdir(stubs / "lib") if f.startswith("_marshal")]


def test_a_module_that_does_not_compile_is_an_error_behind_the_library(stubs, monkeypatch):
    monkeypatch.setattr(build, "_marshal_command", lambda target: [sys.executable, "-c", "raise SystemExit(3)"])
    with pytest.raises(RuntimeError, match="marshal.cpp"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.marshal_path())

"""The compiled module of the paged-cache calls is theirs alone: without it the
library builds and the package's other calls work."""
import importlib.util
import shutil
import subprocess
import sys
from pathlib import Path

import segmented_gather_gemm_sgmv_amd as sg

PACKAGE = Path(sg.__file__).resolve().parent


def test_package_without_the_compiled_module(tmp_path):
    there = tmp_path / PACKAGE.name
    there.mkdir()
    for name in ("__init__.py", "libsgmv.so"):
        shutil.copy(PACKAGE / name, there / name)
    script = f"""
import torch
import {PACKAGE.name} as sg
assert sg.__file__.startswith({str(tmp_path)!r})
assert sg.sgmv_version() > 0 and sg.sgmv_workspace_bytes(1, 1, 64, 64, 8, torch.float32) > 0
x = torch.zeros(2, dtype=torch.int32)
try:
    sg.sgmv_kv_tables(*[x] * 3, 16, *[x] * 7, stream=0)
except ImportError as e:
    assert "_kv_binding" in str(e) and e.__cause__ is not None
else:
    raise AssertionError("no error")
"""
    run = subprocess.run([sys.executable, "-c", script], cwd=tmp_path, capture_output=True, text=True)
    assert run.returncode == 0, run.stderr


def test_build_without_gxx_leaves_the_module_out(tmp_path, monkeypatch, capsys):
    spec = importlib.util.spec_from_file_location("_sgmv_build_under_test", PACKAGE / "build.py")
    build = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build)
    stale = tmp_path / "_kv_binding.so"
    stale.write_bytes(b"of an earlier build")
    monkeypatch.setattr(build, "BINDING", stale)
    monkeypatch.setattr(build, "_run", lambda *a: (_ for _ in ()).throw(AssertionError("nothing to run")))
    which = shutil.which
    monkeypatch.setattr(build.shutil, "which", lambda name: None if name == "g++" else which(name))
    assert build.build_binding() is None
    assert not stale.exists() and "g++" in capsys.readouterr().err


def test_alignment_error_names_no_operand_that_a_call_does_not_have():
    for call in ("sgmv_rope_table", "sgmv_rope_append", "sgmv_paged_attention"):
        error = sg.SGMVError(call, -5)
        assert error.status == -5 and "aligned" in str(error) and call in str(error)
        assert "X, Y" not in str(error)
    assert sg.lib.sgmv_status_string(-5).decode() in str(sg.SGMVError("sgmv_shrink", -5))

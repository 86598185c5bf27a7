"""The package without _torch_calls.so, or with one that does not fit: the calls go through Python."""
import os
import shutil
import subprocess
import sys

import pytest

from swiglu_gated_mlp_gb300 import build

TRY = """
import sys, warnings
{before}
with warnings.catch_warnings(record=True) as said:
    warnings.simplefilter("always")
    import swiglu_gated_mlp_gb300 as sg
    assert sg.swiglu_packed_weight_bytes(896, 4864) == 2 * 4864 * 896 * 2
said = [str(w.message) for w in said if "swiglu_gated_mlp_gb300.build" in str(w.message)]
import torch
from swiglu_gated_mlp_gb300 import _native
assert __import__("os").path.dirname(_native.__file__) == {package!r}
t = torch.zeros(4, 64, dtype=torch.bfloat16)
if {fits}:
    assert not said and _native._calls.__name__.endswith("_torch_calls")
else:
    assert len(said) == 1, said
    for name in ("quantize_int8", "forward_int8", "down_forward_int8", "forward_checkpoint", "checkpoint_output",
                 "backward_checkpoint"):
        assert getattr(_native._calls, name)(t) is None
try:
    sg.swiglu_quantize_int8(t)
except ValueError:
    print("ok")
"""


def run(tmp_path, calls, before="", fits=False):
    package = tmp_path / "swiglu_gated_mlp_gb300"
    package.mkdir()
    for name in os.listdir(build.PKG_DIR):
        if name.endswith(".py") or name == "libswiglu.so":
            shutil.copy2(os.path.join(build.PKG_DIR, name), package / name)
    if calls is not None:
        calls(package / "_torch_calls.so")
    r = subprocess.run([sys.executable, "-c", TRY.format(before=before, package=str(package), fits=fits)], cwd=tmp_path,
                       capture_output=True, text=True, env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr


def built(to):
    shutil.copy2(build.CALLS_PATH, to)


def test_as_built(native_lib, tmp_path):
    run(tmp_path, built, fits=True)


def test_missing(native_lib, tmp_path):
    run(tmp_path, None)


def test_cannot_be_loaded(native_lib, tmp_path):
    run(tmp_path, lambda to: to.write_bytes(b"not a library"))


def test_built_for_another_pytorch(native_lib, tmp_path):
    run(tmp_path, built, before="import torch; torch.__version__ = '0.1.0'")


def test_the_library_itself_is_not_optional(tmp_path):
    package = tmp_path / "swiglu_gated_mlp_gb300"
    package.mkdir()
    for name in os.listdir(build.PKG_DIR):
        if name.endswith(".py"):
            shutil.copy2(os.path.join(build.PKG_DIR, name), package / name)
    r = subprocess.run([sys.executable, "-c", "from swiglu_gated_mlp_gb300 import _native"], cwd=tmp_path, text=True,
                       capture_output=True, env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode != 0 and "ImportError" in r.stderr and "is not built" in r.stderr


@pytest.mark.parametrize("lacks", ["torch", "compiler", "python headers"])
def test_the_library_is_built_without(lacks, monkeypatch, tmp_path):
    if lacks == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)  # importing it raises
    elif lacks == "compiler":
        monkeypatch.setattr(build.shutil, "which", lambda name: None)
    else:
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert build._calls_flags() is None
    assert build._stamp(build._nvcc())

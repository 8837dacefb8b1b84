"""Linear attention and rotary positions from plain C: tests/c_client/linear_client.c is compiled with gcc as C11 against
include/*.h alone, linked to libgdn_decode.so, and run without a GPU. The structs must have the layout that the library and the
Python binding use, and the host-side checks must answer with the documented codes."""
import ctypes
import os
import shutil
import subprocess

import pytest

import ssm_recurrent_decode_gb300 as gdn
from ssm_recurrent_decode_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def out(tmp_path_factory):
    if not shutil.which("gcc"):
        pytest.skip("gcc is needed to build the C client")
    lib = _build.build()
    exe = tmp_path_factory.mktemp("c_client") / "linear_client"
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "c_client", "linear_client.c"), "-o", str(exe),
                    "-L", os.path.dirname(lib), "-lgdn_decode", f"-Wl,-rpath,{os.path.dirname(lib)}"], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, check=True)
    return dict(line.split(" ", 1) for line in run.stdout.strip().splitlines())


def test_layouts_agree(out):
    structs = (gdn.LinearArgs, gdn.LinearGradArgs, gdn.LinearStepArgs, gdn.RotaryArgs)
    sizes = [ctypes.sizeof(s) for s in structs]
    assert [int(v) for v in out["c_sizes"].split()] == sizes == [int(v) for v in out["lib_sizes"].split()]
    assert [int(v) for v in out["offsets"].split()] == [
        gdn.LinearArgs.workspace.offset, gdn.LinearGradArgs.d_o.offset, gdn.LinearStepArgs.state.offset, gdn.RotaryArgs.magnitude.offset]
    assert int(out["version"]) == gdn.ABI_VERSION


def test_host_checks(out):
    assert int(out["attention_null"]) == -1 and int(out["attention_no_workspace"]) == -1
    assert int(out["attention_bad_K"]) == -2 and int(out["attention_bad_heads"]) == -2
    assert int(out["gradient_no_d_o"]) == -1 and int(out["workspace_grows"]) == 1
    assert int(out["step_null"]) == -1 and int(out["step_empty"]) == -2
    assert int(out["rotary_odd"]) == -2 and int(out["rotary_null"]) == -1

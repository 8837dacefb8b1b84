"""The sequence and search operators from plain C: tests/c_client/sequence_client.c is compiled with gcc as C11 against
include/*.h alone, linked to libgdn_decode.so, and run without a GPU. The structs must have the layout that the library
and the Python binding use, and the host-side checks must answer with the documented codes."""
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
    exe = tmp_path_factory.mktemp("c_client") / "sequence_client"
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "c_client", "sequence_client.c"), "-o", str(exe),
                    "-L", os.path.dirname(lib), "-lgdn_decode", f"-Wl,-rpath,{os.path.dirname(lib)}"], check=True)
    run = subprocess.run([str(exe)], capture_output=True, text=True, check=True)
    return dict(line.split(" ", 1) for line in run.stdout.strip().splitlines())


def test_layouts_agree(out):
    structs = (gdn.MambaScanArgs, gdn.MambaScanGradArgs, gdn.BeamSelectArgs, gdn.BeamReorderArgs, gdn.BeamPool)
    sizes = [ctypes.sizeof(s) for s in structs]
    assert [int(v) for v in out["c_sizes"].split()] == sizes == [int(v) for v in out["lib_sizes"].split()]
    assert [int(v) for v in out["offsets"].split()] == [
        gdn.MambaScanArgs.num_states.offset, gdn.MambaScanArgs.err_flags.offset, gdn.MambaScanGradArgs.dh0.offset,
        gdn.BeamSelectArgs.eos_token.offset, gdn.BeamReorderArgs.slots.offset, gdn.BeamPool.slot_bytes.offset]
    assert int(out["version"]) == gdn.ABI_VERSION


def test_the_header_states_the_version():
    text = open(os.path.join(ROOT, "include", "gdn_decode.h")).read()
    assert f"currently {gdn.ABI_VERSION})" in text


def test_host_checks(out):
    assert int(out["scan_null"]) == -1 and int(out["scan_bad_N"]) == -2 and int(out["scan_no_workspace"]) == -1
    assert int(out["dz_without_z"]) == -6 and int(out["workspace_grows"]) == 1
    assert int(out["select_no_workspace"]) == -1 and int(out["select_bad_K"]) == -2
    assert int(out["reorder_over_parents"]) == -6

"""The KV-block allocator where host memory runs out: kv_memory_check.cpp lets every allocation within a call fail in turn."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CALLS = ("release", "trim", "grow", "fork", "unshare", "compact", "announce")


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    exe = tmp_path_factory.mktemp("kv") / "kv_memory_check"
    subprocess.run([gxx, "-O1", "-std=c++17", os.path.join(HERE, "kv_memory_check.cpp"), "-o", str(exe)], check=True)
    return str(exe)


@pytest.mark.parametrize("call", ["release", "trim", "grow", "fork", "compact", "announce"])
def test_a_call_out_of_memory_changes_nothing(program, call):
    out = subprocess.run([program, "".join("1" if c == call else "0" for c in CALLS)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr

"""State that belongs to a device is kept per device: a kernel's shared-memory
allowance, set on the host against a fake runtime of several devices."""
import glob
import os
import re
import shutil
import subprocess

from skinny_gemv_gb300 import _build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_shared_memory_is_allowed_on_every_device(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    assert cxx, "a C++ compiler is needed"
    cuda = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc())), "include")
    exe = tmp_path / "device_smem_check"
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", _build.CSRC, "-I", cuda,
                    os.path.join(HERE, "native", "device_smem_check.cc"), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0 and out.stdout == "ok\n", out.stdout + out.stderr


def test_no_launch_remembers_the_allowance_for_the_process():
    """A kernel's attribute is set through allow_dynamic_smem, or before each launch."""
    for path in glob.glob(os.path.join(_build.CSRC, "*.cu")):
        text = open(path, encoding="utf-8").read()
        assert not re.search(r"static\s+bool\s+\w+\s*=\s*false", text), path

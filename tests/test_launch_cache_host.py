"""The launch cache over a fake runtime, on the CPU (tests/host_checks/launch_cache.cpp)."""
import os
import subprocess

from block_quantized_wire_gb300 import build

SRC = os.path.join(build.ROOT, "tests", "host_checks", "launch_cache.cpp")


def test_shared_memory_limits_never_fall(tmp_path):
    exe = str(tmp_path / "launch_cache")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-pthread", "-I", build.CSRC, SRC, "-o",
                        exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout

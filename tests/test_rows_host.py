"""How the expert-layer kernels cut rows into 16-byte pieces, evaluated on the CPU
(tests/host_checks/rows_cut.cu): no piece leaves its buffer, rows without columns have none."""
import os
import subprocess

from block_quantized_wire_gb300 import build

SRC = os.path.join(build.ROOT, "tests", "host_checks", "rows_cut.cu")


def test_pieces_and_windows_stay_in_their_rows(tmp_path):
    exe = str(tmp_path / "rows_cut")
    r = subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-O1", "-I", build.INCLUDE, "-I", build.CSRC, SRC, "-o",
                        exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout

"""How the expert-layer kernels cut rows into 16-byte pieces and into passes, evaluated on the
CPU (tests/host_checks): no piece leaves its buffer, rows without columns have none, and
passes end at the largest number of rows."""
import os
import subprocess

from block_quantized_wire_gb300 import build


def run_check(name, tmp_path):
    src, exe = os.path.join(build.ROOT, "tests", "host_checks", name + ".cu"), str(tmp_path / name)
    r = subprocess.run([build.nvcc(), *build.ARCH, "-std=c++17", "-O1", "-I", build.INCLUDE, "-I", build.CSRC, src, "-o",
                        exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_pieces_and_windows_stay_in_their_rows(tmp_path):
    run_check("rows_cut", tmp_path)


def test_passes_end_at_the_largest_number_of_rows(tmp_path):
    run_check("row_passes", tmp_path)

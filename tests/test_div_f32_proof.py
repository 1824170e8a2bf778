"""CPU proof that the kernels' reciprocal-based division equals IEEE binary32 division for every binary32
dividend too (rows that the norm and the gate quantize): every pair whose quotient lies close enough to a
border between two numbers for the last rounding to go wrong is tried.  Builds tests/cpu/div_f32_proof.cpp
against the library's own fp8q_math.h with the host compiler."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)


@pytest.mark.slow
def test_division_of_binary32_rows_is_correctly_rounded(tmp_path):
    exe = tmp_path / "div_f32_proof"
    subprocess.run(["g++", "-std=c++17", "-O2", "-ffp-contract=off", "-fopenmp",
                    "-I", os.path.join(ROOT, "fp8_e4m3_quantization_amd", "csrc"),
                    os.path.join(HERE, "cpu", "div_f32_proof.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600)
    print(r.stdout, r.stderr)
    assert r.returncode == 0, r.stdout
    lines = r.stdout.splitlines()
    assert len(lines) == 3 and all(line.endswith(" 0") for line in lines), r.stdout

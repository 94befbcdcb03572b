"""The shared-prefix decode's line of work on the host (tests/prefix_line.cpp, built from
the kernels' own header): which plans serve, and that every tile of keys is computed once,
every partial row has a place of its own, and the merge reads exactly what was written."""
import os
import re
import shutil
import subprocess

import pytest

from mla_decode_attention_folded_gb300 import build

HERE = os.path.dirname(os.path.abspath(__file__))


def test_pieces_slots_and_plans(tmp_path):
    cxx = shutil.which("g++")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    if cxx is None or not os.path.exists(os.path.join(cuda, "cuda_runtime.h")):
        pytest.skip("no host compiler or CUDA headers")
    exe = str(tmp_path / "prefix_line")
    r = subprocess.run([cxx, "-std=c++17", "-O2", "-w", "-I", cuda, "-o", exe,
                        os.path.join(HERE, "prefix_line.cpp")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe, "40000"], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    counts = [int(v) for v in re.findall(r"\d+", r.stdout)]
    assert len(counts) == 4 and min(counts) > 1000, r.stdout

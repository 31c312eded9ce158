"""The forward schedule of up to 128 tokens, whose column ranges outnumber those of larger batches (no GPU needed)."""

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_single_cta_schedules_stay_in_their_slots(tmp_path):
    exe = tmp_path / "logp_single_check"
    subprocess.run(["g++", "-std=c++17", "-O2", "-o", str(exe), os.path.join(HERE, "native", "logp_single_check.cpp")],
                   check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=600)
    assert out.returncode == 0 and out.stdout.startswith("OK"), out.stdout + out.stderr

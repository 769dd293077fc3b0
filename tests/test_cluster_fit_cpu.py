"""A cluster of 16 blocks that the device has no place for becomes one of 8: the rule by itself,
compiled for the host (the occupancy of a real device is the library's question to the driver)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_clusters_fall_back_to_what_fits(tmp_path):
    cxx = os.environ.get("CXX") or shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    exe = str(tmp_path / "cluster_fit_check")
    r = subprocess.run([cxx, "-std=c++17", "-I", os.path.join(ROOT, "selective_ssm_sequence_b200", "csrc"),
                        os.path.join(ROOT, "tests", "cluster_fit_check.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and "0 failures" in r.stdout, r.stdout

"""csrc/per_device.h: a device's value is asked for once, and no thread sees it half made (no GPU needed)."""

import os
import subprocess

from token_permute_grouped_gb300 import build


def test_threads_see_whole_values(tmp_path):
    exe = str(tmp_path / "probe")
    src = os.path.join(os.path.dirname(__file__), "per_device_probe.cc")
    subprocess.run(["g++", "-std=c++17", "-O2", "-pthread", "-I", build.CSRC, src, "-o", exe], check=True)
    for _ in range(5):
        # asked twice (one failure, which one call reports), nothing half made, no device out of range
        assert subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split() == ["2", "1", "0", "0"]

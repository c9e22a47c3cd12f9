"""The group norm's thread map covers every group width it takes (CPU).

`norm_width_check.hip` is built for the host only, from the function that the launches choose a
variant by, and goes through all widths to 8192 for aligned rows and others.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def test_every_channel_has_a_place(tmp_path):
    if not os.path.exists(HIPCC) and shutil.which("hipcc") is None:
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "norm_width_check")
    subprocess.run([HIPCC if os.path.exists(HIPCC) else "hipcc", "--cuda-host-only", "-O1", "-std=c++17",
                    "-I" + os.path.join(ROOT, "gated_delta_rule_85_amd", "csrc"), "-I" + os.path.join(ROOT, "include"),
                    "-o", exe, os.path.join(ROOT, "tests", "norm_width_check.hip")],
                   check=True, capture_output=True, text=True)
    out = subprocess.run([exe], check=True, capture_output=True, text=True).stdout
    assert out.splitlines() == ["widths checked 16384"], out

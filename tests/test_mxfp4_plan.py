"""CPU tests of how the 4-bit product cuts its work, compiled from the kernel's own header."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = tmp_path_factory.mktemp("plan") / "check"
    subprocess.run(["g++", "-O2", "-std=c++17", "-fwrapv", os.path.join(HERE, "mxfp4_plan_check.cpp"), "-o", str(exe)],
                   check=True)
    return str(exe)


def test_tiles_cover_an_experts_rows(check):
    """Up to 2^24 - 1 rows of one expert."""
    p = subprocess.run([check], capture_output=True, text=True, timeout=120)
    assert p.returncode == 0 and p.stdout == "ok\n", p.stdout

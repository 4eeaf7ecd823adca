"""CPU tests of how the 4-bit product cuts its work, compiled from the kernel's own header."""
import os
import shutil
import subprocess

import pytest

from tests import test_gpu_mxfp4 as GPU

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


def tile_rows(check, T, G, M, K, N):
    return int(subprocess.run([check, *map(str, (T, G, M, K, N))], capture_output=True, text=True, check=True).stdout)


def test_row_offsets_of_the_large_tiles_fit_32_bits(check):
    """(T + 1) rows of K / 2 bytes below 4 GiB: where nothing else speaks against the large tiles, that decides."""
    for K in (1024, 1152, 16384):
        T = 2 ** 32 // (K // 2) - 2                  # the last row of zeros included, the most below 4 GiB
        T += ((T + 2) * (K // 2) < 2 ** 32)
        assert (T + 1) * (K // 2) < 2 ** 32 <= (T + 2) * (K // 2)
        assert tile_rows(check, T, 1, 64, K, 30976) == 256 and tile_rows(check, T + 1, 1, 64, K, 30976) == 128
    assert tile_rows(check, 2 ** 24 - 1, 1, 2 ** 24 - 1, 1024, 65536) == 128


@pytest.mark.parametrize("T,k,G,K,N", GPU.MANY_TILES + GPU.LARGE_TILES)
def test_shapes_that_test_the_large_tiles_take_them(check, T, k, G, K, N):
    M = T * k
    assert tile_rows(check, T, G, M, K, N) == 256


def test_every_kernel_is_tested(check):
    """The shapes of the GPU tests reach each of the four."""
    assert {tile_rows(check, T, G, T * k, K, N) for T, k, G, K, N in GPU.GEMM + GPU.LARGE + GPU.MANY_TILES} >= {32, 64, 256}
    assert {tile_rows(check, M, G, M, K, N) for M, G, K, N in GPU.BETWEEN} == {32, 64, 128}

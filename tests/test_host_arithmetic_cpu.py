"""Arithmetic of the library that no call on the CPU reaches, compiled from its headers."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("clang++")
    if cxx is None:
        pytest.skip("no host compiler")
    out = str(tmp_path_factory.mktemp("host") / "libhost.so")
    subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-Wno-unknown-pragmas", "-fPIC", "-shared",
                    "-D__HIP_PLATFORM_AMD__", "-isystem", "/opt/rocm/include", "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "kda_recurrent_state_amd", "csrc"),
                    os.path.join(ROOT, "tests", "host_arithmetic.cpp"), "-o", out], check=True)
    return ctypes.CDLL(out)


@pytest.mark.parametrize("lanes", [16, 32, 64])
@pytest.mark.parametrize("each", [1, 2])
def test_cache_calls_go_in_launches_of_fewer_than_2_to_32_threads(host, lanes, each):
    """Workgroups of 256 threads take 256 / lanes rows (L <= 128, <= 256, above), twice as many in large calls."""
    host.cache_slice_rows.restype = ctypes.c_int64
    rows = 256 // lanes * each
    most = host.cache_slice_rows(rows)
    assert most % rows == 0 and most // rows * 256 < 2 ** 32 <= (most // rows + 1) * 256
    # calls of up to 2^28 - 1 rows are taken: one launch holds them where a workgroup takes more than 16
    assert (most >= 2 ** 28 - 1) == (rows > 16)

"""Arithmetic of the library that no call on the CPU reaches, compiled from its headers."""
import ctypes
import os
import random
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
    lib = ctypes.CDLL(out)
    for name in ("cache_slice_rows", "plan_quotient", "plan_share_begin"):
        getattr(lib, name).restype = ctypes.c_int64
    return lib


def _i64(*x):
    return [ctypes.c_int64(v) for v in x]


def _call(f, n, *args, kind=ctypes.c_int64):
    out = (kind * n)()
    f(*args, out)
    return list(out)


@pytest.mark.parametrize("lanes", [16, 32, 64])
@pytest.mark.parametrize("each", [1, 2])
def test_cache_calls_go_in_launches_of_fewer_than_2_to_32_threads(host, lanes, each):
    """Workgroups of 256 threads take 256 / lanes rows (L <= 128, <= 256, above), twice as many in large calls."""
    rows = 256 // lanes * each
    most = host.cache_slice_rows(rows)
    assert most % rows == 0 and most // rows * 256 < 2 ** 32 <= (most // rows + 1) * 256
    # calls of up to 2^28 - 1 rows are taken: one launch holds them where a workgroup takes more than 16
    assert (most >= 2 ** 28 - 1) == (rows > 16)


def test_quotients_of_the_plan(host):
    """Exact up to 2^52, at multiples of the divisor and next to them; in 32 bits below 2^31."""
    rng = random.Random(1)
    for bits in range(1, 53):
        for _ in range(200):
            a = rng.getrandbits(bits)
            b = rng.getrandbits(rng.randint(1, bits)) + 1
            for x in {a, a // b * b, a // b * b + b - 1, max(0, a // b * b - 1), (1 << bits) - 1}:
                if x >= 1 << 52:
                    continue
                assert host.plan_quotient(*_i64(x, b), 0) == x // b, (x, b)
                if x < 2 ** 31 and b < 2 ** 31:
                    assert host.plan_quotient(*_i64(x, b), 1) == x // b, (x, b)


@pytest.mark.parametrize("team", [1, 2, 3, 5, 11, 16])
def test_shares_of_the_line(host, team):
    """They cover the line one behind the other, differ by one place at most, and each place is found in its share: short
    lines, those around 2^31 places and the longest, beyond 2^42."""
    rng = random.Random(team)
    most = 256 // team
    for total in [1, 2, most - 1, most, most + 1, 3 * most - 1, 12345, 2 ** 31 - 1, 2 ** 31, 2 ** 31 + 1, 2 ** 32 + 5,
                  2 ** 42 + 7, 2 ** 51 + 12345]:
        quot, rem, count, narrow = _call(host.plan_shares, 4, team, *_i64(total))
        assert narrow == (total < 2 ** 31) and count == min(total, most)
        begins = [host.plan_share_begin(team, *_i64(total), w) for w in range(count + 1)]
        assert begins[0] == 0 and begins[-1] == total
        sizes = [b - a for a, b in zip(begins, begins[1:])]
        assert min(sizes) >= 1 and max(sizes) - min(sizes) <= 1
        for w in range(count):
            for x in {begins[w], begins[w + 1] - 1, rng.randrange(begins[w], begins[w + 1])}:
                assert host.plan_share_at(team, *_i64(total, x)) == w, (total, w, x)


@pytest.mark.parametrize("tiles,row_blocks,share", [
    (1, 1, 1), (1, 7, 1), (100, 1, 3), (512, 2, 4), (512, 3, 6), (513, 5, 9), (100, 9, 100), (100, 9, 101), (1000, 12, 7),
    (1 << 24, 1, 1000), (1 << 24, 4096, 1 << 20), (1 << 24, 4096, (1 << 28) + 77), (16777213, 4095, 12345), (1 << 24, 127, 1 << 23),
    (1 << 24, 1 << 18, (1 << 30))])
def test_places_of_an_entitys_units(host, tiles, row_blocks, share):
    """Units lie one behind the other, and each place is of the unit and tile whose place it is (the room before a unit: of
    its first tile), with lines of up to 2^42 places."""
    chunks, chunk, longer, room, line = _call(host.plan_cut, 5, tiles, row_blocks, share)
    assert 1 <= chunks <= tiles and chunks * chunk + longer == tiles and 0 <= longer < max(chunks, 1)
    assert (chunks == 1 and chunk == tiles) or chunk >= share
    assert room == (4 if chunks == 1 else 0) and line == row_blocks * (tiles + room)
    rng = random.Random(tiles + row_blocks)
    units = {(k, rb) for k in {0, 1, longer - 1, longer, chunks - 1} for rb in {0, 1, row_blocks - 1}}
    units |= {(rng.randrange(chunks), rng.randrange(row_blocks)) for _ in range(50)}
    for k, rb in units:
        if not (0 <= k < chunks and 0 <= rb < row_blocks):
            continue
        begin, n = _call(host.plan_unit, 2, tiles, row_blocks, share, k, rb)
        assert n == chunk + (k < longer)
        assert begin == (k * chunk + min(k, longer)) * row_blocks + rb * (n + room)
        for t in {0, n - 1, rng.randrange(n)}:
            for narrow in {0, int(line < 2 ** 31)}:
                assert _call(host.plan_at, 3, tiles, row_blocks, share, *_i64(begin + room + t), narrow,
                             kind=ctypes.c_int) == [k, rb, t]
        for before in range(room):
            assert _call(host.plan_at, 3, tiles, row_blocks, share, *_i64(begin + before), 0, kind=ctypes.c_int) == [k, rb, 0]

"""Index arithmetic that kernels share with the host, compiled for the host: at
sizes that no test allocates."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "decode_attention_preallocated_gb300", "csrc")


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    at = tmp_path_factory.mktemp("host")
    src, lib = at / "host.cpp", at / "host.so"
    src.write_text("""
#include "fd_internal.h"
extern "C" void run_of(int32_t total, int32_t threads, int32_t thread, int32_t *to) {
    const fd::Run r = fd::run_of(total, threads, thread);
    to[0] = r.lo;
    to[1] = r.hi;
}
extern "C" int32_t steps_from(uint32_t start, uint32_t len, uint32_t tiles, uint32_t tile) {
    return fd::steps_from(start, len, tiles, tile);
}
""")
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O1", "-fPIC", "-shared", "-I", CSRC, str(src), "-o",
                    str(lib)], check=True)
    return ctypes.CDLL(str(lib))


@pytest.mark.parametrize("total", [0, 1, 7, 1023, 1024, 1025, 8191, 8193, 2 ** 31 - 8193, 2 ** 31 - 8191, 2 ** 31 - 1])
@pytest.mark.parametrize("threads", [1024, 8192])
def test_runs_cover_every_item_once(host, total, threads):
    # up to 2^31 - 1 table entries may be written in one reservation
    to, at = (ctypes.c_int32 * 2)(), 0
    for thread in range(threads):
        host.run_of(total, threads, thread, to)
        assert to[0] == at and to[0] <= to[1] <= total
        at = to[1]
    assert at == total


@pytest.mark.parametrize("length", [1, 31, 32, 33, 255, 256, 257, 5000, 2 ** 31 - 257, 2 ** 31 - 256, 2 ** 31 - 33, 2 ** 31 - 2,
                                    2 ** 31 - 1])
@pytest.mark.parametrize("streams", [3, 4, 6, 8])
def test_steps_of_the_last_tile_stay_within_the_length(host, length, streams):
    # the last tile of a prefix near 2^31 positions: some of its streams start
    # past the prefix, and past what 31 bits hold
    tile = 32 * streams
    tiles = -(-length // tile)
    for first in {0, tiles // 2, tiles - 1}:
        for stream in range(streams):
            start = first * tile + 32 * stream
            want = max(0, min(tiles - first, -(-(length - start) // tile)))
            assert host.steps_from(start, length, tiles - first, tile) == want
            assert host.steps_from(start, length, 1, tile) == min(want, 1)

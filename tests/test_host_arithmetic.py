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

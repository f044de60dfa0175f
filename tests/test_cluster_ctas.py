"""CPU tests of how many CTAs a cluster of the decodes over a bounded cache gets: the rule, compiled by itself, with
devices that run clusters of some sizes only."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_kvcache_gb300", "csrc")

SOURCE = """
#include "cta_count.h"
extern "C" int ctas(int64_t units, int64_t keys, int whole, const int *at_once, int fails)
{
    int n = -1;
    const int rc = pa::count_cluster_ctas(units, keys, whole != 0,
                                          [&](int c, int *got) { return *got = at_once[c], c == fails ? 7 : 0; }, &n);
    return rc ? -rc : n;
}
"""


@pytest.fixture(scope="module")
def ctas(tmp_path_factory):
    at = tmp_path_factory.mktemp("ctas")
    (at / "ctas.cpp").write_text(SOURCE)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, "ctas.cpp", "-o", "ctas.so"], cwd=at)
    f = ctypes.CDLL(str(at / "ctas.so")).ctas
    f.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_int]

    def call(units, keys, whole, at_once, fails=-1):
        return f(units, keys, int(whole), (ctypes.c_int * 17)(0, *at_once), fails)

    return call


def device(places, largest=16):
    """A device of so many places that runs no cluster of more than `largest` CTAs."""
    return [places // c if c <= largest else 0 for c in range(1, 17)]


@pytest.mark.parametrize("largest", [1, 2, 5, 8, 15, 16])
def test_a_size_that_does_not_run_is_not_taken(ctas, largest):
    for units in (1, 2, 7, 38, 64, 256, 800, 5000):
        for keys in (1, 63, 128, 500, 1024, 3584, 4160, 8192, 65536, 2 ** 31 - 17):
            for whole in (False, True):
                n = ctas(units, keys, whole, device(456, largest))
                assert 1 <= n <= largest, (units, keys, whole)
                if not whole and n > 1:
                    assert 456 // n >= units


def test_sizes(ctas):
    whole_device = device(456)
    assert ctas(1, 3584, False, whole_device) == 16
    assert ctas(1, 3584, False, device(456, 8)) == 8
    assert ctas(1, 40, False, whole_device) == 1
    assert ctas(64, 512, False, whole_device) == 4
    assert ctas(256, 4160, False, whole_device) == 1
    assert ctas(256, 8192, True, whole_device) == 4   # up to 1024 CTAs
    assert ctas(480, 516, True, whole_device) == 1
    assert ctas(5000, 2 ** 31 - 17, True, whole_device) == 1
    assert ctas(1, 8192, True, [0] * 16) == 1         # nothing runs: the launch says so


def test_an_error_is_handed_on(ctas):
    assert ctas(1, 3584, False, device(456), fails=16) == -7
    assert ctas(1, 3584, False, device(456), fails=1) == -7
    assert ctas(256, 8192, True, device(456), fails=4) == -7

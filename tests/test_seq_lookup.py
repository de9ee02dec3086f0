"""The look-up of a token's sequence, compiled for the host: right, and inside the starts, up to as
many sequences as the calls take."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "kimi_delta_attention_12_gb300", "csrc")
MOST = 0x7fff0000

# start of sequence i: i / per * step, so that `per` of them share one (all but the last are empty)
SOURCE = """
#define __device__
#define __forceinline__ inline
#include "kda_seqlens.cuh"
struct Starts {
    int n, per;
    int64_t step;
    mutable int outside;
    int64_t operator[](int i) const {
        if (i < 0 || i > n) { outside = 1; return 0; }
        return i / per * step;
    }
};
extern "C" int look_up(int n, int per, int64_t step, int64_t t, int* outside) {
    Starts s = {n, per, step, 0};
    const int found = kda::last_start(s, n, t);
    *outside = s.outside;
    return found;
}
"""


@pytest.fixture(scope="module")
def look_up(tmp_path_factory):
    at = tmp_path_factory.mktemp("look_up")
    (at / "l.cpp").write_text(SOURCE)
    # (an overflow wraps, as it does on the device, instead of being undefined)
    subprocess.run(["g++", "-O1", "-fwrapv", "-shared", "-fPIC", "-I", CSRC, str(at / "l.cpp"),
                    "-o", str(at / "l.so")], check=True)
    L = ctypes.CDLL(str(at / "l.so"))
    L.look_up.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int64, ctypes.c_int64,
                          ctypes.c_void_p]

    def call(n, per, step, t):
        outside = ctypes.c_int()
        found = L.look_up(n, per, step, t, ctypes.addressof(outside))
        assert not outside.value
        return found
    return call


@pytest.mark.parametrize("n", [1, 2, 3, 5, 64, 1000, (1 << 30) - 1, 1431655767, 0x60000000, MOST])
@pytest.mark.parametrize("per,step", [(1, 1), (1, 3), (4, 1)])
def test_the_sequence_of_a_token(look_up, n, per, step):
    last = (n - 1) // per                 # group of the last sequence
    groups = {0, 1, 2, n // 3, n // 2, 2 * (n // 3), last - 1, last}
    for k in sorted(g for g in groups if 0 <= g <= last):
        for t in {k * step, k * step + step - 1}:
            assert look_up(n, per, step, t) == min((k + 1) * per, n) - 1
    assert look_up(n, per, step, 1 << 40) == n - 1

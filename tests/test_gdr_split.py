"""The choice of the fp32 prefill's split (csrc/gdr_split.h, host code), compiled alone: the rule as its
comment states it, turn by turn, and the same cost whatever the head count."""
import ctypes
import pathlib
import random
import subprocess
import time

import pytest

import rwkv_linear_attention_gb300 as wkv7

SHIM = """#include "gdr_split.h"
extern "C" int choose(int s, int t, int hv, int n, const int32_t *cu) { return wkv7::gdr_choose_split(s, t, hv, n, cu); }
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    d = tmp_path_factory.mktemp("split")
    (d / "shim.cpp").write_text(SHIM)
    csrc = pathlib.Path(wkv7.__file__).parent / "csrc"
    subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", str(csrc), str(d / "shim.cpp"), "-o", str(d / "shim.so")], check=True)
    f = ctypes.CDLL(str(d / "shim.so")).choose
    f.argtypes = [ctypes.c_int] * 4 + [ctypes.c_void_p]

    def call(lens, Hv, N, host=True, T=None):
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        arr = (ctypes.c_int32 * len(cu))(*cu)
        return f(len(lens), cu[-1], Hv, N, ctypes.cast(arr, ctypes.c_void_p) if host else None)

    return call


def _by_turns(lens, Hv, N):
    if len(lens) * Hv * (N // 32) > 1 << 24:
        return 2
    total, sms = float(sum(lens)), 152
    order = sorted(map(float, lens), reverse=True) if len(lens) <= 32 else []
    longest = max(max(lens), total / len(lens))

    def busiest(ctas):
        most, turn = max(longest, total * ctas / sms), 1
        while turn * sms // ctas < len(order):
            most = max(most, (turn + 1) * order[turn * sms // ctas])
            turn += 1
        return most

    wide, narrow = busiest(Hv * (N // 64)), 0.72 * busiest(Hv * (N // 32))
    shared = 0.3 * longest + 0.75 * wide
    return 0 if narrow <= min(wide, shared) else 1 if wide <= shared else 2


def test_the_rule_turn_by_turn(choose):
    rng = random.Random(1)
    seen = set()
    for _ in range(3000):
        lens = [rng.choice((0, 1, rng.randint(2, 50), rng.randint(50, 4000))) for _ in range(rng.choice((1, 2, 3, 8, 31, 32, 33, 60)))]
        Hv, N = rng.choice((1, 3, 8, 40, 64, 151, 152, 153, 400, 1000)), rng.choice((64, 128))
        want = _by_turns(lens, Hv, N)
        seen.add(want)
        assert choose(lens, Hv, N) == want, (lens, Hv, N)
    assert seen == {0, 1, 2}


def test_without_a_host_copy_the_mean_length_counts(choose):
    for S, n, Hv, N in ((1, 1000, 40, 64), (2, 1000, 40, 64), (4, 1000, 32, 128), (16, 1000, 40, 64), (40, 30, 8, 64)):
        assert choose([n] * S, Hv, N, host=False) == choose([n] * S, Hv, N)


def test_the_cost_does_not_grow_with_the_heads(choose):
    """As many heads as a call may have (2^30 with 32 sequences): a few comparisons, not one for each SM's turn."""
    lens = [1] * 32
    choose(lens, 1, 64)
    began = time.perf_counter()
    for _ in range(10):
        for Hv in (1 << 18, 1 << 25):
            assert choose(lens, Hv, 64) == 2
    assert time.perf_counter() - began < 0.01

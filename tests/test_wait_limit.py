"""When a bounded device wait runs out (csrc/wait_limit.h), compiled for the host: neither a timer that is
stepped back nor one that is stepped forward ends a wait at once."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "diffusion_transformer_ultra_b200", "csrc")
LIMIT = 2_000_000_000
SECOND = 1_000_000_000


@pytest.fixture(scope="module")
def over(tmp_path_factory):
    d = tmp_path_factory.mktemp("wait")
    src, so = d / "w.cpp", d / "w.so"
    src.write_text('#include "wait_limit.h"\nextern "C" int over(uint64_t now, uint64_t t0, uint64_t limit, uint32_t looks)'
                   ' { return ug::wait_over(now, t0, limit, looks); }\n')
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(so)], check=True)
    f = ctypes.CDLL(str(so)).over
    f.argtypes = [ctypes.c_uint64] * 3 + [ctypes.c_uint32]
    return lambda now, t0, looks, limit=LIMIT: bool(f(now, t0, limit, looks))


@pytest.mark.parametrize("t0", [5, 1_700_000_000 * SECOND, 2 ** 63 - 7, 2 ** 64 - 3])
def test_time_and_looks(over, t0):
    def at(ns):
        return (t0 + ns) % 2 ** 64
    assert not over(at(0), t0, 10 ** 6) and not over(at(LIMIT), t0, 10 ** 6)
    assert over(at(LIMIT + 1), t0, 10 ** 6) and over(at(LIMIT + 1), t0, 2048)
    for back in (1, 32, 1000, SECOND, 3600 * SECOND):          # stepped back
        assert not over(at(-back), t0, 10 ** 6)
    for ahead in (LIMIT + 1, 3600 * SECOND):                   # stepped forward: the first looks do not end it
        assert not over(at(ahead), t0, 1) and not over(at(ahead), t0, 2047)


def test_a_timer_stepped_far_back_does_not_hold_a_wait(over):
    t0 = 1_700_000_000 * SECOND
    back = t0 - 24 * 3600 * SECOND
    assert not over(back, t0, 2 ** 26 - 1) and over(back, t0, 2 ** 26) and over(t0, t0, 2 ** 26)

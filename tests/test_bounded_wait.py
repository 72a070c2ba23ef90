"""The kernels' bounded wait (csrc/bounded.h), compiled for the host and run against a clock and a barrier that are scripted."""
import os
import subprocess

import pytest

from bitlinear_w1_a8_02_b200 import build

PROGRAM = r"""
#include <stdio.h>
#include <stdlib.h>
#include "bounded.h"

// now() advances by `tick`; before its `stop_at`-th look the thread is stopped for `stopped` and what it waits for comes.
int main(int argc, char** argv) {
    const uint64_t limit = strtoull(argv[1], 0, 10), tick = strtoull(argv[2], 0, 10), stopped = strtoull(argv[4], 0, 10);
    const int stop_at = atoi(argv[3]), there = atoi(argv[5]);  // there: polls that fail before it is there anyway, -1 never
    uint64_t t = 1000;
    int polls = 0, looks = 0;
    bool come = false;
    auto poll = [&] { ++polls; return come || (there >= 0 && polls > there); };
    auto now = [&] {
        if (++looks == stop_at) t += stopped, come = true;
        t += tick;
        return t;
    };
    const bool ok = bl::bounded_wait<ROUND>(poll, now, limit);
    printf("%d %d %llu\n", ok, polls, (unsigned long long)(t - 1000));
}
"""


@pytest.fixture(scope="module", params=[1, 32])
def wait(request, tmp_path_factory):
    polls = request.param
    d = tmp_path_factory.mktemp("wait")
    (d / "wait.cpp").write_text(PROGRAM)
    subprocess.check_call(["g++", "-std=c++17", "-O1", f"-DROUND={polls}", "-I", build.CSRC, str(d / "wait.cpp"), "-o", str(d / "wait")])

    def run(limit, tick, stop_at=0, stopped=0, there=-1):
        out = subprocess.check_output([str(d / "wait"), *map(str, (limit, tick, stop_at, stopped, there))], text=True)
        ok, n, t = map(int, out.split())
        return bool(ok), n, t, polls

    return run


def test_what_is_there_needs_no_clock(wait):
    assert wait(100, 10, there=0)[:3] == (True, 1, 0)


def test_what_comes_in_time_is_seen(wait):
    for there in (1, 5, 40):
        ok, n, _, _ = wait(10 ** 6, 10, there=there)
        assert ok and n == there + 1


def test_it_gives_up_and_not_before_the_limit(wait):
    ok, n, t, polls = wait(1000, 10)
    assert not ok and 1000 < t <= 1040 and n <= 1 + polls * (t // 10 + 1)
    assert wait(0, 10)[0] is False


@pytest.mark.parametrize("stop_at", [1, 2, 3, 50])
def test_a_thread_stopped_beyond_the_limit_still_sees_what_came_meanwhile(wait, stop_at):
    """It was stopped between a poll that failed and the look at the clock; the clock alone says that it is too late."""
    ok, _, t, _ = wait(1000, 10, stop_at=stop_at, stopped=2000)
    assert ok and t > 1000

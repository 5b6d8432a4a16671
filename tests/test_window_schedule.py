"""The sliding-window work decomposition, brute-forced on the host
(tests/window_schedule_check.cpp compiled with g++): each visible pair is
computed exactly once by the forward's, the dQ's and the dK/dV's units, inside
the tensors' rows."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("sched") / "window_schedule_check")
    subprocess.run(["g++", "-std=c++17", "-O2", "-x", "c++", os.path.join(HERE, "window_schedule_check.cpp"), "-o", exe],
                   check=True)

    def run(*args):
        r = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, (args, r.stdout[-500:])
        return int(r.stdout.split()[1])

    return run


def _pairs(sq, skv, window, sinks):
    return sum(sum(1 for j in range(p + 1) if p - j < window or j < sinks) for p in range(skv - sq, skv))


UNIFORM = [
    # b, sq, skv, hq, hkv, window, sinks
    (1, 1, 1, 1, 1, 1, 0),
    (1, 128, 128, 2, 1, 128, 0),
    (2, 129, 129, 4, 2, 64, 4),
    (1, 700, 700, 2, 2, 100, 4),        # tile pairs, an even tile count
    (1, 641, 641, 3, 1, 129, 1),        # tile pairs, one head group of three
    (2, 1, 500, 4, 2, 200, 4),          # a single query at the end
    (1, 77, 900, 4, 1, 300, 130),       # first tokens over two tiles
    (1, 300, 1000, 2, 2, 50, 0),        # keys that no query sees
    (1, 1000, 1000, 2, 1, 1, 0),        # a window of one key
    (1, 1000, 1000, 2, 1, 1, 7),
    (1, 900, 900, 2, 1, 5000, 3),       # wider than the sequence: causal
    (1, 900, 900, 2, 1, 16, 5000),      # every key is a first token
    (1, 3500, 3500, 2, 2, 130, 4),      # walks of the first tile cut into parts
    (1, 2500, 3700, 2, 1, 64, 200),     # two cut tiles, queries from position 1200 on
    (3, 1300, 1500, 1, 1, 128, 128),
    (8, 2300, 2300, 4, 4, 16, 4),       # as long walks, but enough of them to stay whole
]


@pytest.mark.parametrize("case", UNIFORM)
def test_uniform(check, case):
    b, sq, skv, hq, hkv, window, sinks = case
    assert check(*case) == b * hq * _pairs(sq, skv, window, sinks)


PACKED = [
    # hq, hkv, window, sinks, lengths
    (4, 2, 64, 4, [300, 0, 1, 129, 512]),
    (3, 3, 200, 1, [1, 127, 128, 640, 0, 257]),
    (2, 1, 30, 140, [2500, 10, 1500]),   # cut walks, samples shorter than a cut part
    (1, 1, 7, 0, [0, 0, 5]),
]


@pytest.mark.parametrize("hq,hkv,window,sinks,lengths", PACKED)
def test_packed(check, hq, hkv, window, sinks, lengths):
    want = hq * sum(_pairs(n, n, window, sinks) for n in lengths)
    assert check("packed", hq, hkv, window, sinks, *lengths) == want

"""Cut walks in the dK/dV schedule of the window form, on the host: where the
parts' fp32 results lie (tests/window_parts_check.cpp compiled with g++), how
many there are, and the workspace that the calls ask for."""
import ctypes
import os
import subprocess
from collections import namedtuple

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
Cost = namedtuple("Cost", "units parts longest blocks busiest")


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("parts") / "window_parts_check")
    subprocess.run(["g++", "-std=c++17", "-O2", "-x", "c++", os.path.join(HERE, "window_parts_check.cpp"), "-o", exe],
                   check=True)

    def run(*args):
        r = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0, (args, r.stdout[-500:])
        return Cost(*map(int, r.stdout.split()[1:]))

    return run


@pytest.fixture(scope="module")
def lib():
    import context_blockwise_causal_gb300 as pkg
    from context_blockwise_causal_gb300._build import is_stale

    if is_stale():
        pkg.build()
    return pkg.library()


def _packed_bytes(lib, lengths, hq, hkv, d, window, sinks):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return lib.cpattn_bwd_window_varlen_workspace_bytes((ctypes.c_int * len(cu))(*cu), len(lengths), hq, hkv, d, window, sinks)


@pytest.mark.parametrize("args,cuts", [
    ((1, 3500, 3500, 2, 2, 130, 4), True),
    ((1, 2500, 3700, 2, 1, 64, 200), True),      # two cut tiles, queries from the middle on
    ((3, 5000, 5000, 4, 2, 64, 300), True),      # three of each sequence
    ((1, 9300, 9300, 1, 1, 64, 140), True),      # ten parts
    ((1, 1700, 2300, 2, 1, 64, 200), False),
    (("packed", 2, 1, 30, 140, 2500, 10, 1500), True),
    (("packed", 4, 2, 30, 140, 0, 2500, 10, 0, 1025, 1024, 3000, 0), True),
    (("packed", 3, 3, 64, 1, 9000, *[3] * 60), True),
    (("packed", 2, 1, 30, 140, 1500, 10, 700), False),
])
def test_every_part_is_where_the_join_looks(check, args, cuts):
    assert (check(*args).parts > 0) == cuts


def test_short_samples_beside_a_long_one_take_no_results(check, lib):
    """A sample no longer than a part keeps its walk whole: the fp32 results
    are the long sample's, whatever is packed beside it."""
    alone = check("packed", 32, 8, 1024, 4, 32768)
    assert alone.parts == 8 * 29
    mixed = check("packed", 32, 8, 1024, 4, 32768, *[64] * 32)
    assert mixed.parts == alone.parts
    # two row vectors, padded to the longest sample, and dK and dV of each part
    need = _packed_bytes(lib, [32768] + [64] * 32, 32, 8, 128, 1024, 4)
    assert need == 2 * 33 * 32 * 32768 * 4 + 2 * alone.parts * 128 * 128 * 4


def test_shorter_samples_take_the_parts_they_have(check):
    """Seven samples of 8191 tokens: each has the parts of its own length."""
    lengths = (1709, 333, 2048, 85, 1500, 1409, 1107)
    c = check("packed", 8, 8, 300, 1, *lengths)
    tiles = [-(-n // 128) for n in lengths]
    assert c.parts in (0, 8 * sum(-(-t // 8) for t in tiles if t > 8))

"""How calls over a cache in pages are cut, on the host (tests/paged_shape_check.cpp
compiled with g++): the workspace that is asked for holds what the call that takes
it leaves there, also next to the largest counts."""
import os
import random
import subprocess
from collections import namedtuple

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
Shape = namedtuple("Shape", "bytes form ctas part_rows own_runs")


@pytest.fixture(scope="module")
def exe(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("shapes") / "paged_shape_check")
    subprocess.run(["g++", "-std=c++17", "-O2", os.path.join(HERE, "paged_shape_check.cpp"), "-o", exe], check=True)
    return exe


@pytest.fixture(scope="module")
def shapes(exe):
    def run(cases):
        text = "\n".join(" ".join(map(str, c)) for c in cases)
        r = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=300, check=True)
        got = [Shape(*map(int, line.split())) for line in r.stdout.splitlines()]
        assert len(got) == len(cases)
        return got

    return run


def _agrees(case, s):
    """The workspace holds a place for each group, and values and a log-sum-exp for each row's results."""
    sms, b, hq, hkv, d, groups, max_group, cap = case
    if s.form < 0:
        assert s.bytes == 0
        return
    if s.form == 2:  # as cpattn_decode_paged, in so few runs that they need none
        assert s.own_runs == 0 and groups > 1024
        return
    rows = s.ctas * s.part_rows + b * hq * s.own_runs
    assert s.bytes >= groups * 8 + rows * (d + 1) * 4, case
    assert 0 < s.ctas < 1 << 26 and s.ctas + b * hq * s.own_runs < 1 << 31


@pytest.mark.parametrize("sms", [152, 148, 1])
def test_workspace_next_to_the_largest_count_of_groups(shapes, sms):
    """Groups of one, as many KV heads as query heads, b hq next to 2^25: the form
    for few rows can still be numbered where the prefix kernel's whole SMs cannot."""
    cases = [(sms, b, 8, 8, 64, b, 1, cap) for b in range((1 << 22) - 400, 1 << 22) for cap in (16, 1 << 30)]
    got = shapes(cases)
    for c, s in zip(cases, got):
        _agrees(c, s)
    if sms == 152:
        assert got[cases.index((152, 4194298, 8, 8, 64, 4194298, 1, 16))].bytes > 78 * 10 ** 9
    assert all(s.form >= 0 for c, s in zip(cases, got) if 2 * 8 * c[1] + sms < 1 << 26)


def test_workspace_of_all_sorts_of_shapes(shapes):
    rng = random.Random(1)
    cases = []
    while len(cases) < 20000:
        hkv, d = rng.choice([1, 2, 8, 40]), rng.choice([64, 128])
        hq = hkv * rng.choice([1, 2, 4, 8, 9, 17, 64, 300])
        b = int(2 ** rng.uniform(0, 25))
        if b * hq * 64 >= 1 << 31:  # refused before
            continue
        groups, most = max(1, int(b * 2 ** -rng.uniform(0, 12))), max(1, int(b * 2 ** -rng.uniform(0, 25)))
        cases.append((rng.choice([152, 148]), b, hq, hkv, d, groups, most, 16 << rng.randrange(27)))
    got = shapes(cases)
    for c, s in zip(cases, got):
        _agrees(c, s)
    assert {s.form for s in got} == {-1, 0, 1, 2}


def test_no_kernel_looks_through_more_groups_than_pays(shapes):
    """Every CTA of the prefix kernel looks through all groups, of which there
    may be as many as CTAs: 128 of few rows, 1024 of others at most."""
    cases = [(152, g * most, 4 * hkv, hkv, d, g, most, cap) for g in (1, 100, 128, 129, 1000, 1024, 1025, 5000, 60000) for hkv in (1, 8)
             for d in (64, 128) for most in (5, 16, 17, 40) for cap in (256, 131072) if g * most * 4 * hkv < 1 << 24]
    for c, s in zip(cases, shapes(cases)):
        _agrees(c, s)
        groups, most = c[5], c[6]
        assert s.form in ((1,) if most <= 16 and groups > 128 else (0, 1) if groups <= 1024 else (2,)), (c, s)


def test_the_tables_room_does_not_change_the_workspace(shapes):
    for b, hq, hkv, groups, most in ((4, 32, 8, 1, 4), (46, 24, 8, 5, 20), (16, 32, 8, 1, 16), (64, 32, 8, 1, 64)):
        got = shapes([(152, b, hq, hkv, 128, groups, most, cap) for cap in (16, 1024, 1 << 20, 1 << 30)])
        assert len({s.bytes for s in got}) == 1


def test_runs_fill_the_places_that_there_are(exe):
    """A quarter of an SM's registers holds 16384 / 32 threads' worth: units of 16
    heads take 129 registers or more, so three of a CTA's five warps fit it
    and two CTAs an SM; units of 8 heads of 64 stay within 102, four CTAs. Runs below
    2048 keys never take a second turn for the sake of their number."""
    cases = [(152, d, G, units, keys) for d in (64, 128) for G in (1, 8, 9, 16, 40) for units in (1, 2, 7, 19, 24, 40, 57, 100, 152, 300)
             for keys in (100, 1000, 1500, 4000, 8000)]
    r = subprocess.run([exe, "runs"], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True, text=True,
                       timeout=60, check=True)
    for (sms, d, G, units, keys), runs in zip(cases, map(int, r.stdout.split())):
        places = sms * (4 if d == 64 and G <= 8 else 2)
        assert runs == 1 or keys / runs >= 2048 or units * runs <= places, (d, G, units, keys, runs)

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


@pytest.mark.parametrize("case", [
    # b, sq, skv, hq, hkv, d, window, sinks
    (1, 65536, 65536, 1, 1, 128, 128, 65536),    # every key a first token
    (1, 65536, 65536, 4, 4, 128, 128, 16384),
    (1, 12800, 12800, 1, 1, 64, 16, 6400),
    (2, 9000, 30000, 2, 1, 64, 100, 20000),
    (1, 32768, 32768, 32, 8, 128, 1024, 4),
    (1, 1 << 20, 1 << 20, 4, 2, 64, 10, 100),
])
def test_the_results_of_parts_are_bounded(check, lib, case):
    """At most four times the bytes of dk and dv, in whole tiles; walks are
    still cut where whole ones do not balance."""
    b, sq, skv, hq, hkv, d, window, sinks = case
    need = lib.cpattn_bwd_window_workspace_bytes(*case) - 2 * b * hq * (-(-sq // 128) * 128) * 4
    grads = 2 * b * hkv * (-(-skv // 128) * 128) * d * 2
    assert 0 <= need <= 4 * grads
    if skv <= 65536:
        c = check(b, sq, skv, hq, hkv, window, sinks)
        assert need == c.parts * 2 * 128 * d * 4
        assert c.longest <= max(c.blocks / 152, 9 * hq // hkv)


def test_the_results_of_packed_parts_are_bounded(check, lib):
    for lengths, hkv, sinks in (([20000, 5000, 4000, 100], 1, 3000), ([9000] * 7 + [3] * 100, 2, 5000), ([30000, 2000], 1, 1)):
        need = _packed_bytes(lib, lengths, hkv, hkv, 64, 64, sinks) - 2 * len(lengths) * hkv * (-(-max(lengths) // 128) * 128) * 4
        assert 0 <= need <= 4 * 2 * hkv * sum(-(-n // 128) * 128 for n in lengths) * 64 * 2
        assert need == check("packed", hkv, hkv, 64, sinks, *lengths).parts * 2 * 128 * 64 * 4


@pytest.mark.parametrize("extra", [0, 32, 64, 200, 480])
def test_short_samples_leave_the_long_walk_cut(check, extra):
    """Work balances by the samples' own lengths: the longest unit stays under
    a quarter of a CTA's even share, and the busiest CTA near it."""
    c = check("packed", 32, 8, 1024, 4, 32768, *[64] * extra)
    assert 4 * c.longest <= c.blocks / 152
    assert c.busiest <= 1.1 * c.blocks / 152


@pytest.mark.parametrize("b,sq,skv,hkv,sinks", [(1, 2000, 2000, 1, 4), (2, 700, 3000, 2, 1500), (1, 3000, 3000, 1, 3000),
                                                (1, 1000, 5000, 1, 4500), (3, 129, 500, 1, 400), (1, 1, 1, 1, 1)])
def test_walks_of_the_first_tokens_are_counted(tmp_path, b, sq, skv, hkv, sinks):
    """win_first_walks against the units' own walks."""
    src = tmp_path / "walks.cpp"
    src.write_text('#include <cstdio>\n#include "%s"\n' % os.path.join(
        os.path.dirname(HERE), "context_blockwise_causal_gb300", "csrc", "win_schedule.cuh") + """
int main() {
  using namespace cpattn;
  CpGeom g{};
  g.b = %d; g.s = %d; g.kv_s = %d; g.hq = g.hkv = %d; g.sinks = %d; g.cp = g.causal = g.window = 1;
  win_finish(g, false);
  const WinSeq s = win_seq(g, 0);
  long n = 0;
  for (int kt = 0; kt * kTile < g.sinks; ++kt) { int qa, nq; win_query_tiles(g, s, kt, qa, nq); n += nq; }
  std::printf("%%ld %%ld", n, long(win_first_walks(g, g.tpc, s.off)));
}
""" % (b, sq, skv, hkv, sinks))
    exe = str(tmp_path / "walks")
    subprocess.run(["g++", "-std=c++17", "-O1", str(src), "-o", exe], check=True)
    want, got = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert want == got

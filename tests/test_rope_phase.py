"""Phases of the rotation at the furthest positions and the largest
frequencies that the calls admit, against exact rational arithmetic: the
64-bit fraction of a turn that the host forms (csrc/rope_turns.h), and rotated
rows on the GPU."""
import math
import os
import random
import subprocess
from fractions import Fraction

import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "context_blockwise_causal_gb300", "csrc")
# 1 / (2 pi) to 80 digits
INV_TWO_PI = Fraction("0.15915494309189533576888376337251436203445964574045644874766734405889679763422654")


def _turns(radians):
    """Exact turns of a double of radians, modulo 1."""
    return Fraction(float(radians)) * INV_TWO_PI % 1


def test_fraction_of_a_turn_is_within_one_unit(tmp_path):
    src = tmp_path / "turns.cpp"
    src.write_text('#include <cstdio>\n#include <cstdlib>\n#include "%s"\n' % os.path.join(CSRC, "rope_turns.h") +
                   'int main(int, char** v) { while (*++v) std::printf("%llu\\n", (unsigned long long)'
                   'cpattn::turn_fraction(std::strtod(*v, nullptr))); }\n')
    exe = str(tmp_path / "turns")
    subprocess.run(["g++", "-std=c++17", "-O2", str(src), "-o", exe], check=True)
    rng = random.Random(1)
    f = [0.0, 1.0, 0.5, 2 * math.pi, 4 * math.pi, math.pi, 1e6, 1000.0, 1e-3, 1e-9, 1e-30, 5e-324]
    f += [math.exp(rng.uniform(math.log(1e-7), math.log(1e6))) for _ in range(2000)]
    f += [math.nextafter(2 * math.pi * k, 0) for k in (1, 3, 100, 159154)]
    out = subprocess.run([exe, *map(repr, f)], capture_output=True, text=True, check=True).stdout.split()
    for x, got in zip(f, map(int, out), strict=True):
        off = (got - _turns(x) * 2 ** 64) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 1, (x, float(off))


@pytest.mark.gpu
def test_far_positions_and_fast_pairs():
    """y_a, y_b of pairs that turn by up to 1e6 radians per position, out to
    both ends of int32. Tolerance as for every rotation: the output's rounding,
    2^-8 |y|, and 2^-21 (|x_a| + |x_b|) for cosine, sine, products and phase."""
    from context_blockwise_causal_gb300 import cpattn_rope

    freq = torch.tensor([1e6, 1e5 / 3, 1000.0, 37.7, 1.0, 0.3, 1e-3, 999999.9], dtype=torch.float64)
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, 1234567890, -77, 1 << 20, 3, 0]
    gen = torch.Generator().manual_seed(7)
    x = torch.randn(1, len(pos), 3, 64, generator=gen).bfloat16()
    y = cpattn_rope(x.cuda(), positions=torch.tensor(pos, dtype=torch.int32, device="cuda"), inv_freq=freq,
                    out=torch.empty_like(x, device="cuda")).cpu()
    assert torch.equal(y[..., 16:], x[..., 16:])
    for t, p in enumerate(pos):
        for i in range(8):
            theta = 2 * math.pi * float((p * Fraction(float(freq[i])) * INV_TWO_PI) % 1)
            a, b = x[0, t, :, i].double(), x[0, t, :, 8 + i].double()
            for got, ref in ((y[0, t, :, i], a * math.cos(theta) - b * math.sin(theta)),
                             (y[0, t, :, 8 + i], a * math.sin(theta) + b * math.cos(theta))):
                off = (got.double() - ref).abs()
                assert (off <= 2.0 ** -8 * ref.abs() + 2.0 ** -21 * (a.abs() + b.abs())).all(), (p, float(freq[i]))

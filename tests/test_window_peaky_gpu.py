"""The window forward where the running maximum moves from tile to tile.

A row's largest probability enters P V as exactly 1, whichever tile it comes
from, so a row that one key dominates is that key's value times p, rounded
once. (A maximum that lags would round its P, to 2^-8 of the value, before
the output's own rounding.)
"""
import math

import pytest
import torch

import oracle
from context_blockwise_causal_gb300 import cpattn_device_status, cpattn_fwd_window

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


def _randn(*shape, seed, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(torch.bfloat16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(2, 1), (1, 1)])  # pairs of heads, pairs of tiles
@pytest.mark.parametrize("window,sinks", [(5000, 0), (300, 0), (140, 4)])  # the last: first tokens' own product
def test_a_new_maximum_is_exact(d, hq, hkv, window, sinks):
    """Keys score 0 but for one in the second tile and one in the third, which
    score x and 1.5 x in log2 units, x from 1 to 7.97 by row; only they have a
    value. Besides the output's rounding there are fp32 exponentials and sums
    of up to 440 terms of one sign, under 2^-17 together, 2^-8 of half a step
    of bf16."""
    s, first, second = 440, 150, 300
    x = (1 + 0.03125 * torch.randint(0, 224, (s, hq), generator=torch.Generator().manual_seed(d + hq))).to(torch.bfloat16)
    q, k, v = torch.zeros(1, s, hq, d), torch.zeros(1, s, hkv, d), torch.zeros(1, s, hkv, d)
    q[0, :, :, 5] = x.float()
    k[0, first, :, 5], k[0, second, :, 5] = 1.0, 1.5
    v[0, first] = _randn(hkv, d, seed=1).float()
    # rows that see both: the first key's part is of the same sign and at most 2^-0.5 of the second's
    v[0, second] = v[0, first] * 3
    q, k, v = (t.to(torch.bfloat16) for t in (q, k, v))
    o, lse = cpattn_fwd_window(q.cuda(), k.cuda(), v.cuda(), window, sinks, scale=math.log(2.0))
    torch.cuda.synchronize()
    assert cpattn_device_status() == 0
    got = o[0].double().cpu()
    see = oracle.window_mask(s, s, window, sinks)
    alone = see[:, first] & ~see[:, second]
    assert alone.sum() >= 60
    # rows without either key are zero
    assert (got[~see[:, first] & ~see[:, second]] == 0).all()
    for h in range(hq):
        r = oracle.window_attention(q[0, :, h:h + 1], k[0], v[0], window, sinks, scale=math.log(2.0))
        assert (lse[0, h].double().cpu() - r["lse"][0]).abs().max().item() <= 1e-5
        for rows in (alone, see[:, second] & ~see[:, first]):  # one key: its P is 1
            ref = r["o"][rows, 0]
            half = 2.0 ** (torch.floor(torch.log2(ref.abs())) - 8)  # half a step of bf16 at ref
            worst = ((got[rows, h] - ref).abs() / half).nan_to_num().max().item() if rows.any() else 0.0
            print(f"one key: {worst:.3f} half steps")
            assert worst <= 1 + 2.0 ** -8, worst
        both = see[:, first] & see[:, second]
        if both.any():
            # the second key's P is 1 and the first's, which was 1 when it came, was rescaled in fp32
            ref = r["o"][both, 0]
            half = 2.0 ** (torch.floor(torch.log2(ref.abs())) - 8)
            worst = ((got[both, h] - ref).abs() / half).max().item()
            print(f"both keys: {worst:.3f} half steps")
            assert worst <= 1 + 2.0 ** -8, worst


@pytest.mark.parametrize("case", [
    # b, sq, skv, hq, hkv, d, window, sinks, std of q and k
    (1, 700, 700, 4, 2, 128, 5000, 0, 3.0),   # pairs of heads, every tile
    (1, 700, 700, 2, 1, 128, 260, 4, 2.0),
    (1, 641, 641, 3, 1, 128, 300, 1, 3.0),    # pairs of tiles
    (1, 500, 900, 4, 2, 64, 300, 130, 3.0),   # a chunk
    (1, 641, 641, 1, 1, 64, 5000, 0, 2.0),
])
def test_peaky_scores_all_elements(case):
    """Scores of spread 4 to 9 units a row: the maximum moves in most tiles.
    Scores are off by up to e = 2^-17 sum |q k| scale (128 fp32 terms), which
    moves O by 2 e sum P |v| and the LSE by e; else as for unit normals: P
    rounded once, the output once."""
    b, sq, skv, hq, hkv, d, window, sinks, std = case
    q, k = _randn(b, sq, hq, d, seed=1, std=std), _randn(b, skv, hkv, d, seed=2, std=std)
    v = _randn(b, skv, hkv, d, seed=3)
    o, lse = cpattn_fwd_window(q.cuda(), k.cuda(), v.cuda(), window, sinks)
    torch.cuda.synchronize()
    assert cpattn_device_status() == 0
    for bi in range(b):
        r = oracle.window_attention(q[bi], k[bi], v[bi], window, sinks)
        for h in range(hq):
            e = 2.0 ** -17 * (q[bi, :, h].double().abs() @ k[bi, :, h // (hq // hkv)].double().abs().T).amax(1) / d ** 0.5
            off = (o[bi, :, h].double().cpu() - r["o"][:, h]).abs()
            allowed = r["o_err"][:, h] * (1 + 1 / 16 + 2 * e[:, None] / U) + U * r["o"][:, h].abs() + 1e-6
            assert (off <= allowed).all(), (off / allowed).max().item()
            assert ((lse[bi, h].double().cpu() - r["lse"][h]).abs() <= e + 1e-5).all()

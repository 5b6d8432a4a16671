"""The window backward where the walks of the first tokens' key tiles are cut
into parts and their fp32 results joined: against the CPU fp64 oracle, every
element.

Tolerances as in test_window_gpu.py. The sums are longer here, up to 9300
queries for a first token, but a part adds at most 8 tiles of 8 K-steps and
the join up to 10 parts: 80 fp32 additions, 2^-16 of the sum of the terms'
sizes, where the rounding of dS allows 2^-7 of it and P's 2^-8.
"""
import pytest
import torch

import context_blockwise_causal_gb300 as pkg
import oracle
from context_blockwise_causal_gb300 import (cpattn_bwd_window, cpattn_bwd_window_varlen, cpattn_device_status,
                                            cpattn_fwd_window, cpattn_fwd_window_varlen)
from test_window_gpu import _check, _randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", [
    # b, sq, skv, hq, hkv, d, window, sinks, parts in all
    (1, 2500, 3700, 2, 1, 128, 64, 200, 6),      # two cut tiles, queries from the middle on
    (2, 2400, 2400, 2, 2, 64, 130, 4, 12),       # two sequences, two KV heads
    (1, 9300, 9300, 1, 1, 64, 64, 140, 20),      # two tiles of ten parts: more than the join's warps
    (1, 9300, 9300, 2, 1, 128, 64, 4, 10),
])
def test_uniform(case):
    b, sq, skv, hq, hkv, d, window, sinks, parts = case
    vectors = 2 * b * hq * (-(-sq // 128) * 128) * 4
    need = pkg.cpattn_bwd_window_workspace_bytes(b, sq, skv, hq, hkv, d, window, sinks)
    assert need == vectors + 2 * parts * 128 * d * 4  # the walks are cut
    q, do = _randn(b, sq, hq, d, seed=1), _randn(b, sq, hq, d, seed=2)
    k, v = _randn(b, skv, hkv, d, seed=3), _randn(b, skv, hkv, d, seed=4)
    x = [t.cuda() for t in (q, k, v, do)]
    ws = torch.full((need + 256,), 0xff, dtype=torch.uint8, device="cuda")  # NaN where nothing was written
    o, lse = cpattn_fwd_window(x[0], x[1], x[2], window, sinks)
    grads = cpattn_bwd_window(x[0], x[1], x[2], o, lse, x[3], window, sinks, workspace=ws[:need])
    torch.cuda.synchronize()
    assert cpattn_device_status() == 0
    assert (ws[need:] == 0xff).all()
    for bi in range(b):
        r = oracle.window_attention(q[bi], k[bi], v[bi], window, sinks, do=do[bi])
        _check(r, o[bi], lse[bi], [g[bi] for g in grads])


@pytest.mark.parametrize("lengths,hq,hkv,d,window,sinks", [
    ([2500, 10, 1500], 2, 1, 128, 30, 140),
    ([0, 2500, 1025, 0, 1024, 1300], 4, 2, 64, 64, 4),  # samples of a part, of one row more, of none
    ([2600] + [5] * 40, 3, 3, 64, 100, 1),
])
def test_packed(lengths, hq, hkv, d, window, sinks):
    import ctypes

    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    total = cu[-1]
    need = pkg.library().cpattn_bwd_window_varlen_workspace_bytes((ctypes.c_int * len(cu))(*cu), len(lengths), hq, hkv, d,
                                                                  window, sinks)
    assert need > 2 * len(lengths) * hq * (-(-max(lengths) // 128) * 128) * 4  # some walk is cut
    q, do = _randn(total, hq, d, seed=11), _randn(total, hq, d, seed=12)
    k, v = _randn(total, hkv, d, seed=13), _randn(total, hkv, d, seed=14)
    x = [t.cuda() for t in (q, k, v, do)]
    ws = torch.full((need + 256,), 0xff, dtype=torch.uint8, device="cuda")
    o, lse = cpattn_fwd_window_varlen(x[0], x[1], x[2], cu, window, sinks)
    grads = cpattn_bwd_window_varlen(x[0], x[1], x[2], o, lse, x[3], cu, window, sinks, workspace=ws[:need])
    torch.cuda.synchronize()
    assert cpattn_device_status() == 0
    assert (ws[need:] == 0xff).all()
    parts = [oracle.window_attention(q[a:e], k[a:e], v[a:e], window, sinks, do=do[a:e])
             for a, e in zip(cu, cu[1:]) if e > a]
    r = {n: torch.cat([p[n] for p in parts], dim=1 if n == "lse" else 0) for n in parts[0]}
    _check(r, o, lse, grads)


def test_checked_build_is_silent_and_identical():
    """The bounds tests of the checked build over cut walks, a packed call."""
    import ctypes

    lib = pkg.checked_library()
    cu, hq, hkv, d, window, sinks = [0, 2500, 2510, 4010, 5035], 2, 1, 128, 30, 140
    q, do = (_randn(cu[-1], hq, d, seed=20 + i).cuda() for i in range(2))
    k, v = (_randn(cu[-1], hkv, d, seed=22 + i).cuda() for i in range(2))
    o, lse = cpattn_fwd_window_varlen(q, k, v, cu, window, sinks)
    grads = cpattn_bwd_window_varlen(q, k, v, o, lse, do, cu, window, sinks)
    torch.cuda.synchronize()
    c = (ctypes.c_int * len(cu))(*cu)
    n = lib.cpattn_bwd_window_varlen_workspace_bytes(c, len(cu) - 1, hq, hkv, d, window, sinks)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    got = [torch.full_like(t, 7.0) for t in grads]
    p = [t.data_ptr() for t in (q, k, v, o, lse, do, *got, ws)]
    assert lib.cpattn_bwd_window_varlen(*p, n, c, len(cu) - 1, hq, hkv, d, window, sinks, 0.0, None) == 0
    torch.cuda.synchronize()
    st = ctypes.c_int(0)
    lib.cpattn_device_status(None, ctypes.byref(st))
    assert st.value == 0, hex(st.value)
    for a, e in zip(grads, got):
        assert torch.equal(a, e)

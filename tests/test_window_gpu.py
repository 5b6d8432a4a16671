"""Sliding-window attention with visible first tokens through the C ABI
against the CPU fp64 oracle, every element.

Tolerances, from the roundings that the kernels make (u = 2^-8, a bf16
rounding relative to the value; everything else is fp32):
  O:   P is rounded before P V:             u sum_j P_ij |v_j|
  dV:  the same P:                          u sum_i P_ij |dO_i|
  dS = P (dP - D): P and dS are rounded, D comes from the rounded O, whose P
       was rounded too:                     2 u |dS| + P sum_d |dO| u (|O| + sum_j P |v_j|)
  dQ, dK: that, through |K| or |Q| and the scale.
The oracle computes these bounds (``*_err``); the output's own rounding adds
u |value|. fp32 sums, exponentials and second-order terms are under 1/16 of
them: a product of 128 fp32 terms is off by at most 2^-17 of its absolute sum,
u / 2^-17 = 512. LSE: scores off by up to 2^-17 sum |q k| scale, which is
below 5e-5 for the inputs here (sum |q k| scale < 7): 1e-4.
"""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import context_blockwise_causal_gb300 as pkg
import oracle
from context_blockwise_causal_gb300 import (cpattn_bwd_window, cpattn_bwd_window_varlen, cpattn_device_status,
                                            cpattn_fwd_window, cpattn_fwd_window_varlen)

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
LSE_TOL = 1e-4


def _randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def _within(name, got, ref, err):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), name
    off = (got - ref).abs()
    allowed = err * (1 + 1 / 16) + U * ref.abs() + 1e-6
    worst = (off / allowed).max().item()
    print(f"{name}: {worst:.2f} of the allowance")
    assert worst <= 1.0, (name, worst)


def _check(r, o, lse, grads=None):
    _within("o", o, r["o"], r["o_err"])
    assert (lse.double().cpu() - r["lse"]).abs().max().item() <= LSE_TOL
    for name, g in zip(("dq", "dk", "dv"), grads or ()):
        _within(name, g, r[name], r[name + "_err"])


UNIFORM = [
    # b, sq, skv, hq, hkv, d, window, sinks, scale
    (1, 1, 1, 1, 1, 128, 1, 0, None),        # one token
    (1, 2, 2, 2, 1, 64, 1, 1, None),
    (1, 128, 128, 2, 1, 128, 128, 0, None),
    (2, 129, 129, 4, 2, 64, 64, 4, None),    # one row in the second tile, batch
    (1, 300, 300, 2, 2, 128, 100, 4, None),  # one head per group: pairs of tiles, an odd number of them
    (1, 641, 641, 3, 1, 64, 129, 1, 0.2),    # groups of three heads, a scale
    (2, 1, 500, 4, 2, 128, 200, 4, None),    # a single query after 499 tokens
    (1, 77, 700, 8, 2, 64, 300, 130, None),  # first tokens over two tiles
    (1, 200, 700, 2, 1, 128, 50, 0, None),   # keys that no query sees
    (1, 400, 400, 2, 1, 128, 1, 0, None),    # a window of one key: every row its own value
    (1, 400, 400, 2, 1, 64, 1, 9, None),
    (1, 330, 330, 2, 1, 128, 5000, 3, None),  # wider than the sequence
    (1, 330, 330, 2, 2, 64, 16, 5000, None),  # every key a first token
    (1, 2100, 2100, 2, 2, 64, 130, 4, None),  # the first tile's walk cut into parts, pairs of tiles
    (1, 1700, 2300, 2, 1, 128, 64, 200, None),  # two cut tiles, queries from the middle on
]


@pytest.mark.parametrize("case", UNIFORM)
def test_uniform_all_elements(case):
    b, sq, skv, hq, hkv, d, window, sinks, scale = case
    q, do = _randn(b, sq, hq, d, seed=1 + sq), _randn(b, sq, hq, d, seed=2 + sq)
    k, v = _randn(b, skv, hkv, d, seed=3 + skv), _randn(b, skv, hkv, d, seed=4 + skv)
    x = [t.cuda() for t in (q, k, v, do)]
    # outputs inside larger buffers: what lies around them stays
    def room(like, dtype=torch.bfloat16, n=64):
        buf = torch.full((like.numel() + 2 * n,), 7.0, dtype=dtype, device="cuda")
        return buf, buf[n:n + like.numel()].view(like.shape)

    lse_like = torch.empty(b, hq, sq)
    bufs = [room(q), room(lse_like, torch.float32), room(q), room(k), room(v)]
    for _, t in bufs:
        t.fill_(float("nan"))
    o, lse = cpattn_fwd_window(x[0], x[1], x[2], window, sinks, scale=scale, o=bufs[0][1], lse=bufs[1][1])
    grads = cpattn_bwd_window(x[0], x[1], x[2], o, lse, x[3], window, sinks, scale=scale, dq=bufs[2][1],
                              dk=bufs[3][1], dv=bufs[4][1])
    torch.cuda.synchronize()
    assert cpattn_device_status() == 0
    for buf, _ in bufs:
        assert (buf[:64] == 7).all() and (buf[-64:] == 7).all()
    for bi in range(b):
        r = oracle.window_attention(q[bi], k[bi], v[bi], window, sinks, scale, do=do[bi])
        _check(r, o[bi], lse[bi], [g[bi] for g in grads])


PACKED = [
    # lengths, hq, hkv, d, window, sinks
    ([300, 0, 1, 129, 512], 4, 2, 128, 64, 4),
    ([1, 127, 128, 640, 0, 257], 3, 3, 64, 200, 1),   # pairs of tiles
    ([1500, 10, 700], 2, 1, 128, 30, 140),            # cut walks
    ([3] * 600, 2, 1, 64, 2, 1),                      # more samples than one launch takes
]


@pytest.mark.parametrize("lengths,hq,hkv,d,window,sinks", PACKED)
def test_packed_all_elements(lengths, hq, hkv, d, window, sinks):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    total = cu[-1]
    q, do = _randn(total, hq, d, seed=11), _randn(total, hq, d, seed=12)
    k, v = _randn(total, hkv, d, seed=13), _randn(total, hkv, d, seed=14)
    x = [t.cuda() for t in (q, k, v, do)]
    o, lse = cpattn_fwd_window_varlen(x[0], x[1], x[2], cu, window, sinks)
    grads = cpattn_bwd_window_varlen(x[0], x[1], x[2], o, lse, x[3], cu, window, sinks)
    torch.cuda.synchronize()
    assert cpattn_device_status() == 0
    parts = [oracle.window_attention(q[a:e], k[a:e], v[a:e], window, sinks, do=do[a:e])
             for a, e in zip(cu, cu[1:]) if e > a]
    r = {n: torch.cat([p[n] for p in parts], dim=1 if n == "lse" else 0) for n in parts[0]}
    _check(r, o, lse, grads)


def test_no_rows_and_windows_beyond_int32():
    q, k = (torch.empty(0, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    o, lse = cpattn_fwd_window_varlen(q, k, k, [0, 0, 0], 16)
    grads = cpattn_bwd_window_varlen(q, k, k, o, lse, q, [0, 0, 0], 16)
    assert o.shape == q.shape and lse.shape == (4, 0) and grads[1].shape == k.shape
    x = [_randn(1, 200, h, 64, seed=15 + i).cuda() for i, h in enumerate((2, 1, 1))]
    want = cpattn_fwd_window(*x, 200)
    for window, sinks in ((2 ** 32 + 1, 0), (2 ** 40, 2 ** 33)):  # all keys, not what 32 bits leave of the number
        got = cpattn_fwd_window(*x, window, sinks)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        got = cpattn_fwd_window_varlen(*(t[0] for t in x), [0, 200], window, sinks)
        assert torch.equal(got[0], want[0][0]) and torch.equal(got[1], want[1][0])


def test_first_call_may_be_captured():
    """The library's first call on a device inside a capture, in a fresh process."""
    code = """
import sys, torch
sys.path.insert(0, sys.argv[1])
import context_blockwise_causal_gb300 as pkg
g = torch.Generator(device="cuda").manual_seed(1)
q, k, v = (torch.randn(1, 300, h, 64, generator=g, device="cuda").bfloat16() for h in (2, 1, 1))
n = torch.tensor([300], dtype=torch.int32, device="cuda")
w = torch.ones(64, device="cuda")
def step():
    qn, kn = pkg.cpattn_qk_norm_rope(q, k, w, w)
    o, lse = pkg.cpattn_fwd_window(qn, kn, v, 40, 2)
    grads = pkg.cpattn_bwd_window(qn, kn, v, o, lse, q, 40, 2)
    dx = pkg.cpattn_qk_norm_rope_bwd(q, k, w, w, grads[0], grads[1])
    return (o, *grads, *dx, pkg.cpattn_decode(qn[:, -1], kn, v, n, 40, 2)[0])
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, step()))
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code, root], capture_output=True, text=True, timeout=200)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-1500:]


def test_packed_equals_the_samples_alone():
    cu, hq, hkv, d = [0, 700, 701, 1300], 4, 2, 128
    x = [_randn(1300, h, d, seed=20 + i).cuda() for i, h in enumerate((hq, hkv, hkv, hq))]
    o, lse = cpattn_fwd_window_varlen(*x[:3], cu, 100, 3)
    grads = cpattn_bwd_window_varlen(*x[:3], o, lse, x[3], cu, 100, 3)
    for a, e in zip(cu, cu[1:]):
        y = [t[None, a:e].contiguous() for t in x]
        o1, l1 = cpattn_fwd_window(*y[:3], 100, 3)
        assert torch.equal(o1[0], o[a:e]) and torch.equal(l1[0], lse[:, a:e])
        g1 = cpattn_bwd_window(*y[:3], o1, l1, y[3], 100, 3)
        assert torch.equal(g1[0][0], grads[0][a:e])  # dQ: the same tiles in the same order


def test_repeatable_and_grid_independent():
    b, s, hq, hkv, d = 1, 2100, 4, 2, 128
    x = [_randn(b, s, h, d, seed=30 + i).cuda() for i, h in enumerate((hq, hkv, hkv, hq))]

    def once():
        o, lse = cpattn_fwd_window(*x[:3], 130, 4)
        return (o, lse, *cpattn_bwd_window(*x[:3], o, lse, x[3], 130, 4))

    first = once()
    try:
        for cap in (0, 1, 37):
            pkg.cpattn_set_max_ctas(cap)
            assert all(torch.equal(a, c) for a, c in zip(first, once())), cap
    finally:
        pkg.cpattn_set_max_ctas(0)
    assert cpattn_device_status() == 0


def test_long_sequence_sampled_rows():
    """32K tokens, the rows of a few tiles against 64-bit attention on the GPU."""
    s, hq, hkv, d, window, sinks = 32768, 8, 2, 128, 1024, 4
    gen = torch.Generator(device="cuda").manual_seed(40)
    q, k, v = (torch.randn(1, s, h, d, generator=gen, device="cuda").bfloat16() for h in (hq, hkv, hkv))
    o, lse = cpattn_fwd_window(q, k, v, window, sinks)
    for p0 in (0, 1000, 1020, 16380, 32704):
        rows = torch.arange(p0, min(p0 + 64, s), device="cuda")
        j = torch.arange(s, device="cuda")
        see = (j[None] <= rows[:, None]) & ((rows[:, None] - j[None] < window) | (j[None] < sinks))
        for h in range(hq):
            sc = (q[0, rows, h].double() @ k[0, :, h // 4].double().T / d ** 0.5).masked_fill(~see, float("-inf"))
            p = torch.softmax(sc, -1)
            vd = v[0, :, h // 4].double()
            ref, mass = p @ vd, p @ vd.abs()
            off = (o[0, rows, h].double() - ref).abs()
            assert (off <= U * mass * (1 + 1 / 16) + U * ref.abs() + 1e-6).all()
            assert (lse[0, h, rows].double() - torch.logsumexp(sc, -1)).abs().max().item() <= LSE_TOL


def test_captured_graphs_share_a_workspace():
    """Two captured training steps replayed in turn with one workspace, on a
    stream of their own, give what the plain calls give."""
    s, hq, hkv, d = 700, 4, 2, 64
    sets = [[_randn(1, s, h, d, seed=50 + 10 * j + i).cuda() for i, h in enumerate((hq, hkv, hkv, hq))]
            for j in range(2)]
    need = pkg.cpattn_bwd_window_workspace_bytes(1, s, s, hq, hkv, d, 100, 4)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def step(x):
        o, lse = cpattn_fwd_window(*x[:3], 100, 4)
        return (o, lse, *cpattn_bwd_window(*x[:3], o, lse, x[3], 100, 4, workspace=ws))

    want = [step(x) for x in sets]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(x))
        graphs.append(g)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for g in (*graphs, *graphs):
            g.replay()
    side.synchronize()
    for w, got in zip(want, outs):
        assert all(torch.equal(a, c) for a, c in zip(w, got))


def test_given_stream():
    s, d = 300, 128
    x = [_randn(1, s, h, d, seed=70 + i).cuda() for i, h in enumerate((2, 1, 1, 2))]
    o, lse = cpattn_fwd_window(*x[:3], 40, 2)
    grads = cpattn_bwd_window(*x[:3], o, lse, x[3], 40, 2)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o2, l2 = cpattn_fwd_window(*x[:3], 40, 2, stream=side)
    g2 = cpattn_bwd_window(*x[:3], o2, l2, x[3], 40, 2, stream=side)
    side.synchronize()
    for a, c in zip((o, lse, *grads), (o2, l2, *g2)):
        assert torch.equal(a, c)


def test_checked_build_is_silent_and_identical():
    lib = pkg.checked_library()
    for b, sq, skv, hq, hkv, d, window, sinks in ((2, 641, 641, 3, 1, 128, 100, 4), (1, 77, 700, 4, 2, 64, 300, 130),
                                                  (1, 2100, 2100, 2, 1, 128, 130, 4)):
        q, do = (_randn(b, sq, hq, d, seed=80 + i).cuda() for i in range(2))
        k, v = (_randn(b, skv, hkv, d, seed=82 + i).cuda() for i in range(2))
        o, lse = cpattn_fwd_window(q, k, v, window, sinks)
        grads = cpattn_bwd_window(q, k, v, o, lse, do, window, sinks)
        torch.cuda.synchronize()
        got = [torch.full_like(t, 7.0) for t in (o, lse, *grads)]
        n = pkg.cpattn_bwd_window_workspace_bytes(b, sq, skv, hq, hkv, d, window, sinks)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        p = [t.data_ptr() for t in (q, k, v, *got, do, ws)]
        assert lib.cpattn_fwd_window(p[0], p[1], p[2], p[3], p[4], b, sq, skv, hq, hkv, d, window, sinks, 0.0,
                                     None) == 0
        assert lib.cpattn_bwd_window(p[0], p[1], p[2], p[3], p[4], p[8], p[5], p[6], p[7], p[9], n, b, sq, skv, hq,
                                     hkv, d, window, sinks, 0.0, None) == 0
        torch.cuda.synchronize()
        st = ctypes.c_int(0)
        lib.cpattn_device_status(None, ctypes.byref(st))
        assert st.value == 0, hex(st.value)
        for a, c in zip((o, lse, *grads), got):
            assert torch.equal(a, c)


def test_refusals():
    q, k = torch.zeros(1, 8, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 8, 2, 64, dtype=torch.bfloat16,
                                                                                      device="cuda")
    with pytest.raises(pkg.CpattnError):
        cpattn_fwd_window(q, k, k, 0)
    with pytest.raises(pkg.CpattnError):
        cpattn_fwd_window(q, k, k, 4, -1)
    with pytest.raises(pkg.CpattnError):
        cpattn_fwd_window(q, k[:, :4].contiguous(), k[:, :4].contiguous(), 4)  # fewer keys than queries
    with pytest.raises(pkg.CpattnError):
        cpattn_fwd_window(q, k, k, 4, scale=-1.0)
    with pytest.raises(TypeError):
        cpattn_fwd_window(q.half(), k.half(), k.half(), 4)
    with pytest.raises(ValueError):
        cpattn_fwd_window(q.transpose(1, 2), k, k, 4)
    o, lse = cpattn_fwd_window(q, k, k, 4)
    with pytest.raises(pkg.CpattnError):
        cpattn_bwd_window(q, k, k, o, lse, q, 4, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        cpattn_fwd_window_varlen(q[0], k[0], k[0], [0, 4], 4)


@pytest.mark.parametrize("s,window,d", [(85, 228, 64), (116, 246, 128), (128, 128, 64)])
def test_gradients_of_short_sequences_carry_two_roundings(s, window, d):
    """dQ and dK are off by the rounding of dS and by their own, no more: a
    bf16 rounding of values spread over a binade is off by 2^-7 sqrt(0.541 / 12)
    = 1.66e-3 in the mean square, two of them by 2.35e-3, and 8 % are left for
    the spread over few elements. (O's rounding in D, which single-tile rows do
    not take, would add up to 20 %.)"""
    q, do, k, v = (_randn(4, s, h, d, seed=30 + i) for i, h in enumerate((4, 4, 2, 2)))
    o, lse = cpattn_fwd_window(q.cuda(), k.cuda(), v.cuda(), window)
    grads = cpattn_bwd_window(q.cuda(), k.cuda(), v.cuda(), o, lse, do.cuda(), window)
    want = [oracle.window_attention(q[i], k[i], v[i], window, do=do[i]) for i in range(4)]
    for name, g in zip(("dq", "dk"), grads):
        ref = torch.stack([w[name] for w in want])
        err = ((g.double().cpu() - ref).norm() / ref.norm()).item()
        print(name, err)
        assert err <= 2.0 ** -7 * (0.541 / 12) ** 0.5 * 2 ** 0.5 * 1.08

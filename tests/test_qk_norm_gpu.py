"""Rotary positions in their general form and the q/k norms with the rotation
through the C ABI against the CPU fp64 oracle, every element; and the whole
path of a windowed layer.

Tolerances (u = 2^-8: the output's rounding, relative to the value):
  rotation: u |y| + 2^-21 m (|x_a| + |x_b|): cosine, sine, two products and a
    sum, each good to a few 2^-24, and the phase (a 32-bit fraction of a turn
    rounded to fp32: 2^-24 of half a turn, 2^-22.3 rad).
  norm: u |y| + 2^-18 (pair sum of |x r w|): besides, a sum of squares of
    17 + 3 fp32 additions (2^-19.6, halved by the root) and the root.
  dx: u |dx| + 2^-17 r (pair sums of |dy| m |w| and |xh| mean |t w xh|).
  dw: 2^-17 sum |t xh|: fp32 sums of at most 2^6 terms a thread in these
    tests, a few more across threads, and the rotation's own error.
"""
import ctypes

import pytest
import torch

import context_blockwise_causal_gb300 as pkg
import oracle
from context_blockwise_causal_gb300 import (cpattn_bwd_window, cpattn_decode, cpattn_device_status, cpattn_fwd_window,
                                            cpattn_qk_norm_rope, cpattn_qk_norm_rope_bwd, cpattn_rope,
                                            cpattn_rope_frequencies)

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


def _randn(*shape, seed, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(torch.bfloat16)


def _pair_sum(a, rot, layout):
    """|a| summed over each rotated pair, at both of its features."""
    a = a.double().abs().clone()
    r = a[..., :rot]
    if layout == "half":
        s = r[..., :rot // 2] + r[..., rot // 2:]
        a[..., :rot] = torch.cat([s, s], -1)
    else:
        s = r[..., 0::2] + r[..., 1::2]
        a[..., :rot] = s.repeat_interleave(2, -1)
    return a


def _within(name, got, ref, err):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), name
    worst = ((got - ref).abs() / (err + U * ref.abs() + 1e-12)).max().item()
    print(f"{name}: {worst:.2f} of the allowance")
    assert worst <= 1.0, (name, worst)


ROPE = [
    # b, n, h, d, rot, layout, scaling arguments, magnitude
    (1, 1, 1, 64, 64, "half", {}, 1.0),
    (2, 37, 5, 128, 128, "half", {"scaling": "linear", "factor": 4.0}, 1.0),
    (2, 37, 5, 128, 128, "interleaved", {"scaling": "base", "factor": 8.0}, 1.0),
    (3, 19, 3, 128, 64, "half", {"scaling": "turns", "factor": 8.0, "original_len": 8192, "low": 1.0, "high": 4.0}, 1.2),
    (3, 19, 3, 128, 96, "interleaved",
     {"scaling": "index", "factor": 16.0, "original_len": 4096, "low": 1.0, "high": 32.0}, 1.3),
    (1, 300, 40, 64, 16, "half", {}, 1.0),
    (1, 300, 9, 64, 48, "interleaved", {}, 1.0),
    (1, 5, 33, 128, 112, "half", {}, 1.0),
]


@pytest.mark.parametrize("case", ROPE)
def test_rope_general_form(case):
    b, n, h, d, rot, layout, scaling, mag = case
    freq = cpattn_rope_frequencies(rot, 500000.0, **scaling)
    assert torch.allclose(freq, oracle.scaled_frequencies(rot, 500000.0, **scaling), rtol=1e-12)
    # the heads of interest inside wider rows, in and out
    wide = _randn(b, n, h + 3, d, seed=1, std=2.0)
    x = wide[:, :, 1:h + 1]
    buf = torch.full((b, n, h + 2, d), 7.0, dtype=torch.bfloat16, device="cuda")
    y = buf[:, :, 1:h + 1]
    xd = wide.cuda()[:, :, 1:h + 1]
    given = torch.randint(0, 1 << 20, (b, n), generator=torch.Generator().manual_seed(2))
    for pos, arg in ((torch.arange(n), None), (given, given.int().cuda())):
        got = cpattn_rope(xd, inv_freq=freq, layout=layout, magnitude=mag, positions=arg, out=y)
        assert got is y
        err = 2.0 ** -21 * mag * _pair_sum(x, rot, layout)
        _within("y", y, oracle.rotate(x, pos, freq, layout, mag), err)
        assert torch.equal(y[..., rot:], xd[..., rot:])
        assert (buf[:, :, 0] == 7).all() and (buf[:, :, -1] == 7).all()
        back = cpattn_rope(xd, inv_freq=freq, layout=layout, magnitude=mag, positions=arg, inverse=True,
                           out=torch.empty(b, n, h, d, dtype=torch.bfloat16, device="cuda"))
        _within("inverse", back, oracle.rotate(x, pos, freq, layout, mag, inverse=True), err)
        inplace = wide.cuda()
        cpattn_rope(inplace[:, :, 1:h + 1], inv_freq=freq, layout=layout, magnitude=mag, positions=arg)
        assert torch.equal(inplace[:, :, 1:h + 1], y) and torch.equal(inplace[:, :, 0], wide.cuda()[:, :, 0])


def test_rope_position_sources():
    d = 128
    freq = cpattn_rope_frequencies(d)
    # zigzag shards and packed samples, as the plain call
    s, cp = 96 * 3, 3
    cu = [0, 100, 101, s]
    cu_dev = torch.tensor(cu, dtype=torch.int32, device="cuda")
    x = _randn(1, s, 2, d, seed=3)
    for r in range(cp):
        idx = oracle.zigzag_global_index(s, cp)[r]
        shard = x[:, idx].contiguous()
        for c, cdev in ((None, None), (cu, cu_dev)):
            got = cpattn_rope(shard.cuda(), cp=cp, rank=r, s=s, cu_seqlens=cdev, layout="interleaved", inv_freq=freq)
            pos = oracle.rank_local_positions(s, cp, r, c)
            _within("shard", got, oracle.rotate(shard, pos, freq, "interleaved"),
                    2.0 ** -21 * _pair_sum(shard, d, "interleaved"))
    # shared positions, extremes and negative ones (2^31 positions: the phase is still exact)
    pos = torch.tensor([0, -1, 1, -100000, 2 ** 31 - 1, -2 ** 31])
    x = _randn(2, 6, 2, d, seed=4)
    got = cpattn_rope(x.cuda(), positions=pos.int().cuda(), inv_freq=freq)
    # the 64-bit fractions are rounded from fp64 frequencies: 2^31 * 2^-54 turns at the first pairs
    _within("extremes", got, oracle.rotate(x, pos, freq), (2.0 ** -21 + 2.0 ** -19) * _pair_sum(x, d, "half"))


def test_rope_default_agrees_with_the_plain_call():
    x = _randn(2, 500, 3, 128, seed=5).cuda()
    a = cpattn_rope(x.clone())
    c = cpattn_rope(x, out=torch.empty_like(x))
    # two roundings of values 2^-20 apart differ by at most one step
    assert ((a.double() - c.double()).abs() <= 2 * U * a.double().abs() + 1e-5).all()


NORM = [
    # b, n, hq, hkv, d, rot, layout, weights, eps, explicit positions
    (1, 1, 1, 1, 128, 128, "half", torch.float32, 1e-6, False),
    (2, 33, 6, 2, 128, 128, "half", torch.bfloat16, 1e-6, False),
    (2, 33, 6, 2, 64, 32, "interleaved", torch.float32, 1e-5, True),
    (3, 17, 5, 5, 128, 96, "interleaved", torch.bfloat16, 1e-6, True),
    (1, 700, 3, 1, 64, 64, "half", torch.float32, 0.1, False),
    (5, 1, 32, 8, 128, 64, "half", torch.bfloat16, 1e-6, True),
    (1, 9, 70, 1, 64, 16, "half", torch.float32, 1e-6, True),
]


@pytest.mark.parametrize("case", NORM)
def test_norm_rope_forward_backward(case):
    b, n, hq, hkv, d, rot, layout, wt, eps, explicit = case
    qkv = _randn(b, n, hq + 2 * hkv, d, seed=6, std=3.0)
    qkv[0, 0, 0] = 0  # a head of zeros: r = eps^-1/2, output zero
    gq, gk = _randn(b, n, hq, d, seed=7), _randn(b, n, hkv, d, seed=8)
    wq, wk = ((1 + 0.3 * _randn(d, seed=s).float()).to(wt) for s in (9, 10))
    freq = cpattn_rope_frequencies(rot, 10000.0)
    pos = torch.randint(0, 1 << 17, (b, n), generator=torch.Generator().manual_seed(11)) if explicit else torch.arange(n)
    kw = {"eps": eps, "inv_freq": freq, "layout": layout, "magnitude": 1.1,
          "positions": pos.int().cuda() if explicit else None}
    dev = qkv.cuda()
    q, k = dev[:, :, :hq], dev[:, :, hq:hq + hkv]
    qo, ko = cpattn_qk_norm_rope(q, k, wq.cuda(), wk.cuda(), **kw)
    dq, dk, dwq, dwk = cpattn_qk_norm_rope_bwd(q, k, wq.cuda(), wk.cuda(), gq.cuda(), gk.cuda(), **kw)
    torch.cuda.synchronize()
    assert cpattn_device_status() == 0
    for x, w, g, y, dx, dw in ((qkv[:, :, :hq], wq, gq, qo, dq, dwq), (qkv[:, :, hq:hq + hkv], wk, gk, ko, dk, dwk)):
        xd, wd = x.double(), w.double()
        r = 1 / torch.sqrt((xd * xd).mean(-1, keepdim=True) + eps)
        _within("y", y, oracle.norm_rotate(x, w, pos, freq, eps, layout, 1.1),
                2.0 ** -18 * 1.1 * _pair_sum(xd * r * wd, rot, layout))
        ref, dw_ref = oracle.norm_rotate_backward(x, w, g, pos, freq, eps, layout, 1.1)
        t = 1.1 * _pair_sum(g, rot, layout)
        xh = (xd * r).abs()
        _within("dx", dx, ref, 2.0 ** -17 * r * (t * wd.abs() + xh * (t * wd.abs() * xh).mean(-1, keepdim=True)))
        off = (dw.double().cpu() - dw_ref).abs()
        assert (off <= 2.0 ** -17 * (t * xh).sum(dim=(0, 1, 2)) + 1e-9).all()
    # in place, into the fused rows; the values beside them stay
    cpattn_qk_norm_rope(q, k, wq.cuda(), wk.cuda(), q_out=q, k_out=k, **kw)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(dev[:, :, hq + hkv:], qkv.cuda()[:, :, hq + hkv:])
    # the gradients over their own inputs
    dq2, dk2 = gq.cuda(), gk.cuda()
    dev = qkv.cuda()
    r2 = cpattn_qk_norm_rope_bwd(dev[:, :, :hq], dev[:, :, hq:hq + hkv], wq.cuda(), wk.cuda(), dq2, dk2, dq=dq2, dk=dk2,
                                 **kw)
    assert all(torch.equal(a, c) for a, c in zip(r2, (dq, dk, dwq, dwk)))


def test_norm_weight_gradient_over_many_rows():
    """Enough rows that every CTA takes several tokens: dw within fp32 sums
    (2^6 terms a thread at most: 2^13 tokens x 2 rows a pass / 8 warps a CTA)."""
    b, n, hq, hkv, d = 1, 8192, 8, 2, 128
    q, k = _randn(b, n, hq, d, seed=20).cuda(), _randn(b, n, hkv, d, seed=21).cuda()
    gq, gk = _randn(b, n, hq, d, seed=22).cuda(), _randn(b, n, hkv, d, seed=23).cuda()
    w = torch.ones(d, device="cuda")
    _, _, dwq, dwk = cpattn_qk_norm_rope_bwd(q, k, w, w, gq, gk, inv_freq=cpattn_rope_frequencies(d))
    again = cpattn_qk_norm_rope_bwd(q, k, w, w, gq, gk, inv_freq=cpattn_rope_frequencies(d))
    assert torch.equal(dwq, again[2]) and torch.equal(dwk, again[3])
    for x, g, dw in ((q, gq, dwq), (k, gk, dwk)):
        xd = x.double().cpu()
        r = 1 / torch.sqrt((xd * xd).mean(-1, keepdim=True) + 1e-6)
        t = oracle.rotate(g.cpu(), torch.arange(n), cpattn_rope_frequencies(d), inverse=True)
        ref, mag = (t * xd * r).sum(dim=(0, 1, 2)), (_pair_sum(g.cpu(), d, "half") * (xd * r).abs()).sum(dim=(0, 1, 2))
        assert ((dw.double().cpu() - ref).abs() <= 2.0 ** -17 * mag).all()


def test_layer_of_them_together():
    """A windowed layer's path: norms and rotation of a fused projection,
    attention, its backward and the norms', against the oracle's chain; then
    one more token through the single-token forms with a cache."""
    s, hq, hkv, d, window, sinks = 301, 4, 2, 64, 50, 3
    qkv = _randn(1, s, hq + 2 * hkv, d, seed=30)
    wq, wk = (1 + 0.2 * _randn(d, seed=31).float()), (1 + 0.2 * _randn(d, seed=32).float())
    do = _randn(1, s - 1, hq, d, seed=33)
    freq = cpattn_rope_frequencies(32, 10000.0, "linear", 2.0)
    kw = {"inv_freq": freq, "layout": "interleaved"}
    dev = qkv.cuda()
    q, k, v = dev[:, :s - 1, :hq], dev[:, :s - 1, hq:hq + hkv], dev[:, :s - 1, hq + hkv:].contiguous()
    qn, kn = cpattn_qk_norm_rope(q, k, wq.cuda(), wk.cuda(), **kw)
    o, lse = cpattn_fwd_window(qn, kn, v, window, sinks)
    dqn, dkn, dv = cpattn_bwd_window(qn, kn, v, o, lse, do.cuda(), window, sinks)
    dq, dk, dwq, dwk = cpattn_qk_norm_rope_bwd(q, k, wq.cuda(), wk.cuda(), dqn, dkn, **kw)
    torch.cuda.synchronize()
    # stage by stage: each stage's oracle on the stage's own inputs
    r = oracle.window_attention(qn[0].cpu(), kn[0].cpu(), v[0].cpu(), window, sinks, do=do[0])
    for name, got in (("o", o), ("dq", dqn), ("dk", dkn), ("dv", dv)):
        _within(name, got[0], r[name], r[name + "_err"] * (1 + 1 / 16) + 1e-6)
    # the chain as a whole by automatic differentiation in 64 bits: the
    # relative error of each stage's roundings, a handful of u in the norm
    leaves = [qkv[:, :s - 1].double().requires_grad_(), wq.double().requires_grad_(), wk.double().requires_grad_()]
    qa = oracle_norm(leaves[0][:, :, :hq], leaves[1], freq)
    ka = oracle_norm(leaves[0][:, :, hq:hq + hkv], leaves[2], freq)
    see = oracle.window_mask(s - 1, s - 1, window, sinks)
    sc = torch.einsum("bqhd,bkhd->bhqk", qa, ka.repeat_interleave(hq // hkv, 2)) * d ** -0.5
    p = torch.softmax(sc.masked_fill(~see, float("-inf")), -1)
    oa = torch.einsum("bhqk,bkhd->bqhd", p, leaves[0][:, :, hq + hkv:].repeat_interleave(hq // hkv, 2))
    gx, gwq, gwk = torch.autograd.grad(oa, leaves, do.double())

    def rel(a, c):
        return ((a.double().cpu() - c).norm() / c.norm()).item()

    assert rel(o, oa.detach()) <= 4 * U
    # q, k, P, dS, D and the gradients themselves are rounded: eight roundings at most on any way
    assert rel(dq, gx[:, :, :hq]) <= 8 * U and rel(dk, gx[:, :, hq:hq + hkv]) <= 8 * U
    assert rel(dv, gx[:, :, hq + hkv:]) <= 8 * U
    assert rel(dwq, gwq) <= 8 * U and rel(dwk, gwk) <= 8 * U
    # one more token: its q and k at position s - 1, appended to the cache
    cache_k, cache_v = (torch.full((1, s + 5, hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache_k[:, :s - 1], cache_v[:, :s - 1] = kn, v
    at = torch.tensor([[s - 1]], dtype=torch.int32, device="cuda")
    q1, _ = cpattn_qk_norm_rope(dev[:, s - 1:, :hq], dev[:, s - 1:, hq:hq + hkv], wq.cuda(), wk.cuda(), positions=at,
                                k_out=cache_k[:, s - 1:s], **kw)
    cache_v[:, s - 1] = dev[:, s - 1, hq + hkv:]
    o1, l1 = cpattn_decode(q1[:, 0], cache_k, cache_v, torch.tensor([s], dtype=torch.int32, device="cuda"), window, sinks)
    qf, kf = cpattn_qk_norm_rope(dev[:, :, :hq], dev[:, :, hq:hq + hkv], wq.cuda(), wk.cuda(), **kw)
    assert torch.equal(kf, cache_k[:, :s]) and torch.equal(qf[:, -1:], q1)
    of, lf = cpattn_fwd_window(qf, kf, dev[:, :, hq + hkv:].contiguous(), window, sinks)
    r = oracle.window_attention(qf[0].cpu(), kf[0].cpu(), qkv[0, :, hq + hkv:], window, sinks)
    _within("token", o1[0], r["o"][-1], r["o_err"][-1] * (1 + 1 / 16) + 1e-6)
    _within("row", of[0, -1], r["o"][-1], r["o_err"][-1] * (1 + 1 / 16) + 1e-6)
    assert (l1 - lf[:, :, -1]).abs().max().item() <= 2e-4


def oracle_norm(x, w, freq):
    """norm and interleaved rotation of half of the head, differentiable."""
    n, rot = x.shape[1], 2 * freq.numel()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
    ang = (torch.arange(n).double()[:, None] * freq)[None, :, None]
    a, b = y[..., 0:rot:2], y[..., 1:rot:2]
    r = torch.stack([a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()], -1).flatten(-2)
    return torch.cat([r, y[..., rot:]], -1)


def test_captured_and_on_a_given_stream():
    b, n, hq, hkv, d = 2, 50, 4, 2, 64
    q, k = _randn(b, n, hq, d, seed=40).cuda(), _randn(b, n, hkv, d, seed=41).cuda()
    gq, gk = _randn(b, n, hq, d, seed=42).cuda(), _randn(b, n, hkv, d, seed=43).cuda()
    w = torch.ones(d, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    freq = cpattn_rope_frequencies(d)

    def step(stream=None):
        return (*cpattn_qk_norm_rope(q, k, w, w, inv_freq=freq, positions=pos, stream=stream),
                *cpattn_qk_norm_rope_bwd(q, k, w, w, gq, gk, inv_freq=freq, positions=pos, stream=stream))

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    pos += 7  # the positions are read at replay
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(step(), got)) and not torch.equal(want[0], got[0])


def test_checked_build_is_silent_and_identical():
    lib = pkg.checked_library()
    b, n, hq, hkv, d = 2, 33, 5, 2, 128
    q, k = _randn(b, n, hq, d, seed=50).cuda(), _randn(b, n, hkv, d, seed=51).cuda()
    w = torch.ones(d, device="cuda")
    freq = cpattn_rope_frequencies(d)
    want = (*cpattn_qk_norm_rope(q, k, w, w, inv_freq=freq), *cpattn_qk_norm_rope_bwd(q, k, w, w, q, k, inv_freq=freq))
    normal, pkg._LIB = pkg._LIB, lib
    try:
        got = (*cpattn_qk_norm_rope(q, k, w, w, inv_freq=freq), *cpattn_qk_norm_rope_bwd(q, k, w, w, q, k, inv_freq=freq))
    finally:
        pkg._LIB = normal
    torch.cuda.synchronize()
    st = ctypes.c_int(0)
    lib.cpattn_device_status(None, ctypes.byref(st))
    assert st.value == 0, hex(st.value)
    assert all(torch.equal(a, c) for a, c in zip(want, got))


def test_refusals():
    x = torch.zeros(2, 8, 3, 64, dtype=torch.bfloat16, device="cuda")
    freq = cpattn_rope_frequencies(64)
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        cpattn_rope(x, layout="quarter")
    with pytest.raises(ValueError):
        cpattn_rope(x, rot_dim=32, inv_freq=freq)
    with pytest.raises(pkg.CpattnError):
        cpattn_rope(x, rot_dim=24)  # not a multiple of 16
    with pytest.raises(pkg.CpattnError):
        cpattn_rope(x, rot_dim=128)  # more than the head
    with pytest.raises(pkg.CpattnError):
        cpattn_rope(x, inv_freq=freq, magnitude=0.0)
    with pytest.raises(pkg.CpattnError):
        cpattn_rope(x, inv_freq=-freq)
    with pytest.raises(TypeError):
        cpattn_rope(x, inv_freq=freq.float())
    with pytest.raises(ValueError):
        cpattn_rope(x, positions=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        cpattn_rope(x, positions=torch.zeros(8, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        cpattn_rope(x.transpose(1, 2), inv_freq=freq)  # heads apart
    with pytest.raises(ValueError):
        cpattn_rope(x, out=x[:, :4])
    with pytest.raises(pkg.CpattnError):
        cpattn_rope(x, out=x[:, :1].expand(2, 8, 3, 64))  # an output whose tokens overlap
    with pytest.raises(pkg.CpattnError):
        cpattn_rope(x, out=x[:1].expand(2, 8, 3, 64))     # or whose batch elements do
    with pytest.raises(TypeError):
        cpattn_qk_norm_rope(x, x, w, w.half())
    with pytest.raises(TypeError):
        cpattn_qk_norm_rope(x, x, w, w.bfloat16())
    with pytest.raises(ValueError):
        cpattn_qk_norm_rope(x, x[:, :4], w, w)
    with pytest.raises(pkg.CpattnError):
        cpattn_qk_norm_rope(x, x, w, w, eps=-1.0)
    with pytest.raises(pkg.CpattnError):
        cpattn_qk_norm_rope_bwd(x, x, w, w, x, x, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    for kw in ({"scaling": "linear", "factor": 0.5}, {"scaling": "turns", "factor": 2.0}, {"base": 1.0}):
        with pytest.raises(pkg.CpattnError):
            cpattn_rope_frequencies(64, **kw)
    with pytest.raises(ValueError):
        cpattn_rope_frequencies(64, scaling="other")


def test_refusals_of_offsets_and_of_sizes_beyond_int32():
    x = torch.zeros(1, 8, 3, 64, dtype=torch.bfloat16, device="cuda")
    for n in (0, 1):
        with pytest.raises(ValueError):  # offsets without a sample, not taken for none
            cpattn_rope(x, rot_dim=32, cu_seqlens=torch.zeros(n, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        cpattn_rope(x, rot_dim=32, rank=0, cp=1 << 20, s=1 << 40)
    with pytest.raises(ValueError):
        cpattn_rope(x, rot_dim=32, rank=0, cp=1 << 30)  # s = n cp
    with pytest.raises(pkg.CpattnError):
        cpattn_rope(x[:, :1].expand(1, (1 << 32) + 1, 3, 64), rot_dim=32)
    with pytest.raises(TypeError):
        cpattn_rope(x, rot_dim=32, positions=[0] * 8)
    with pytest.raises(TypeError):
        cpattn_rope(x, rot_dim=32.5)
    with pytest.raises(AttributeError):
        cpattn_rope(x, rot_dim=32, stream=7)
    assert torch.equal(x, torch.zeros_like(x))


def test_given_outputs_are_returned_and_new_ones_are_kept_apart():
    x = torch.randn(2, 5, 3, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    out = torch.empty_like(x)
    q, k = cpattn_qk_norm_rope(x, x, w, w, q_out=out)
    assert q is out and k is not out and torch.equal(q, k)
    assert k.is_contiguous() and not k.requires_grad and k.data_ptr() != q.data_ptr()
    assert cpattn_rope(x, rot_dim=32) is x
    grads = cpattn_qk_norm_rope_bwd(x, x, w, w, x, x)
    assert len({t.data_ptr() for t in grads}) == 4 and torch.equal(grads[0], grads[1])
    with torch.cuda.stream(torch.cuda.Stream()):
        s = torch.cuda.Stream()
        before = torch.cuda.current_stream()
        cpattn_qk_norm_rope(x, x, w, w, stream=s)
        assert torch.cuda.current_stream() == before
        with pytest.raises(pkg.CpattnError):
            cpattn_qk_norm_rope(x, x, w, w, eps=-1.0, stream=s)
        assert torch.cuda.current_stream() == before
        s.synchronize()

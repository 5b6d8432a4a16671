"""CPU pins of the oracle's windowed attention and q/k norms: hand values,
identities with the plain oracle, automatic differentiation and differences."""
import math

import torch

import oracle

F64 = torch.float64


def _x(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F64)


def test_mask_by_hand():
    m = oracle.window_mask(6, 6, 2, 1)
    want = ["100000", "110000", "111000", "101100", "100110", "100011"]
    assert ["".join(str(int(x)) for x in row) for row in m] == want
    assert torch.equal(oracle.window_mask(2, 6, 2, 1), m[4:])
    assert torch.equal(oracle.window_mask(6, 6, 1, 0), torch.eye(6, dtype=torch.bool))


def test_wide_window_is_causal_attention():
    q, k, v, do = _x(40, 4, 64, seed=1), _x(40, 2, 64, seed=2), _x(40, 2, 64, seed=3), _x(40, 4, 64, seed=4)
    o, lse = oracle.attention_forward(q[None], k[None], v[None])
    grads = oracle.attention_backward(q[None], k[None], v[None], do[None])
    for window, sinks in ((40, 0), (1000, 3), (1, 40)):
        r = oracle.window_attention(q, k, v, window, sinks, do=do)
        assert torch.allclose(r["o"], o[0], atol=1e-12) and torch.allclose(r["lse"], lse[0], atol=1e-12)
        for n, g in zip(("dq", "dk", "dv"), grads):
            assert torch.allclose(r[n], g[0], atol=1e-12), n


def test_window_of_one_returns_its_own_value():
    q, k, v = _x(9, 2, 64, seed=5), _x(9, 1, 64, seed=6), _x(9, 1, 64, seed=7)
    r = oracle.window_attention(q, k, v, 1)
    assert torch.allclose(r["o"], v.expand(9, 2, 64), atol=1e-14)
    assert torch.allclose(r["lse"], ((q * k).sum(-1) / 8.0).T, atol=1e-12)


def test_gradients_against_autograd_and_differences():
    q, k, v, do = _x(11, 4, 64, seed=8), _x(17, 2, 64, seed=9), _x(17, 2, 64, seed=10), _x(11, 4, 64, seed=11)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    see = oracle.window_mask(11, 17, 5, 2)
    kk, vv = (x.repeat_interleave(2, dim=1) for x in leaves[1:])
    s = torch.einsum("qhd,khd->hqk", leaves[0], kk) / 8.0
    p = torch.softmax(s.masked_fill(~see, -math.inf), -1)
    o = torch.einsum("hqk,khd->qhd", p, vv)
    grads = torch.autograd.grad(o, leaves, do)
    r = oracle.window_attention(q, k, v, 5, 2, do=do)
    assert torch.allclose(r["o"], o.detach(), atol=1e-12)
    for n, g in zip(("dq", "dk", "dv"), grads):
        assert torch.allclose(r[n], g, atol=1e-12), n
    h = 1e-6
    for n, x, at in (("dq", q, (3, 1, 5)), ("dk", k, (0, 1, 7)), ("dv", v, (9, 0, 2))):
        vals = []
        for sign in (1, -1):
            args = {"dq": q, "dk": k, "dv": v}
            y = x.clone()
            y[at] += sign * h
            args[n] = y
            vals.append((oracle.window_attention(args["dq"], args["dk"], args["dv"], 5, 2)["o"] * do).sum().item())
        assert abs((vals[0] - vals[1]) / (2 * h) - r[n][at].item()) < 1e-7, n


def test_decode_is_the_last_row():
    q, k, v = _x(30, 4, 64, seed=12), _x(30, 2, 64, seed=13), _x(30, 2, 64, seed=14)
    for window, sinks in ((0, 0), (7, 0), (7, 3), (100, 5)):
        o, lse, _ = oracle.decode_attention(q[29], k, v, 30, window, sinks)
        r = oracle.window_attention(q, k, v, window or 30, sinks)
        assert torch.allclose(o, r["o"][29], atol=1e-13) and torch.allclose(lse, r["lse"][:, 29], atol=1e-13)
    o, lse, _ = oracle.decode_attention(q[0], k, v, 0)
    assert (o == 0).all() and (lse == -math.inf).all()


def test_rotation_layouts_and_parts():
    x = _x(2, 5, 3, 64, seed=15)
    pos = torch.tensor([0, 1, 7, 100, 131071])
    f = oracle.scaled_frequencies(64, 10000.0)
    assert torch.allclose(oracle.rotate(x, pos, f), oracle.rope_apply(x, pos), atol=1e-9)
    # interleaved = half on the features sorted into evens and odds
    perm = torch.cat([torch.arange(0, 64, 2), torch.arange(1, 64, 2)])
    y = oracle.rotate(x, pos, f, "interleaved")
    assert torch.allclose(y[..., perm], oracle.rotate(x[..., perm], pos, f), atol=1e-12)
    # part of the head: the rest passes; turning back undoes it up to the magnitude squared
    g = f[:16]
    for layout in ("half", "interleaved"):
        y = oracle.rotate(x, pos, g, layout, magnitude=1.5)
        assert torch.equal(y[..., 32:], x[..., 32:])
        z = oracle.rotate(y, pos, g, layout, magnitude=1.5, inverse=True)
        assert torch.allclose(z[..., :32], 2.25 * x[..., :32], atol=1e-12)


def test_scaled_frequencies_by_hand():
    f = oracle.scaled_frequencies(8, 10000.0)
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=F64))
    assert torch.allclose(oracle.scaled_frequencies(8, 10000.0, "linear", 4.0), f / 4)
    # base 10^4 * 10^(8/6): the slowest pair is slowed down by exactly the factor
    assert abs(oracle.scaled_frequencies(8, 10000.0, "base", 10.0)[3].item() / (0.001 / 10.0) - 1) < 1e-12
    # turns over 1000 positions: 159, 15.9, 1.59, 0.159
    t = oracle.scaled_frequencies(8, 10000.0, "turns", 8.0, 1000.0, low=1.0, high=4.0)
    share = (1000 * 0.01 / (2 * math.pi) - 1) / 3
    want = torch.tensor([1.0, 0.1, 0.01 * (share + (1 - share) / 8), 0.001 / 8], dtype=F64)
    assert torch.allclose(t, want, rtol=1e-12)
    # pairs with 4 turns and 1 turn: indexes 1.6 and 2.2 -> 1 and 3
    t = oracle.scaled_frequencies(8, 10000.0, "index", 8.0, 1000.0, low=1.0, high=4.0)
    want = torch.tensor([1.0, 0.1, 0.01 * (0.5 + 0.5 / 8), 0.001 / 8], dtype=F64)
    assert torch.allclose(t, want, rtol=1e-12)


def test_norm_gradients_against_autograd_and_differences():
    x, w, dy = _x(2, 3, 4, 64, seed=16), 1 + 0.1 * _x(64, seed=17), _x(2, 3, 4, 64, seed=18)
    pos, f = torch.tensor([5, 0, 999]), oracle.scaled_frequencies(32, 500000.0)
    for layout in ("half", "interleaved"):
        xl, wl = x.clone().requires_grad_(), w.clone().requires_grad_()
        y = oracle.norm_rotate(xl, wl, pos, f, 1e-5, layout, 1.2)
        gx, gw = torch.autograd.grad(y, (xl, wl), dy)
        dx, dw = oracle.norm_rotate_backward(x, w, dy, pos, f, 1e-5, layout, 1.2)
        assert torch.allclose(dx, gx, atol=1e-12) and torch.allclose(dw, gw, atol=1e-11)
    h, at = 1e-6, (1, 2, 3, 9)
    vals = []
    for sign in (1, -1):
        z = x.clone()
        z[at] += sign * h
        vals.append((oracle.norm_rotate(z, w, pos, f, 1e-5, "interleaved", 1.2) * dy).sum().item())
    assert abs((vals[0] - vals[1]) / (2 * h) - dx[at].item()) < 1e-7

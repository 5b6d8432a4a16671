"""Rotary positions in their general form and the RMS norm of heads in front
of them, with gradients, fp64 on the CPU. TEST INFRASTRUCTURE (see the package
docstring).

Pair i of the first rot features turns by pos * inv_freq[i]: features i and
i + rot/2 (half) or 2i and 2i + 1 (interleaved), cosines and sines times a
magnitude; the other features pass.
"""
import math

import torch

_F64 = torch.float64


def scaled_frequencies(rot, base, scaling=None, factor=1.0, original_len=0.0, low=1.0, high=32.0):
    """Pair by pair, in Python floats."""
    out = []
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    for i in range(rot // 2):
        f = 1.0 / base ** (2 * i / rot)
        if scaling == "linear":
            f = f / factor
        elif scaling == "turns":
            turns = original_len * f / (2 * math.pi)
            share = min(1.0, max(0.0, (turns - low) / (high - low)))
            f = share * f + (1 - share) * f / factor
        elif scaling == "index":
            def index(turns):
                return rot * math.log(original_len / (2 * math.pi * turns)) / (2 * math.log(base))

            first, last = max(math.floor(index(high)), 0), min(math.ceil(index(low)), rot - 1)
            divided = min(1.0, max(0.0, (i - first) / max(last - first, 1e-3)))
            f = (1 - divided) * f + divided * f / factor
        out.append(f)
    return torch.tensor(out, dtype=_F64)


def rotate(x, pos, inv_freq, layout="half", magnitude=1.0, inverse=False):
    """x [b, n, h, d], pos [n] or [b, n] -> fp64."""
    b, n, h, d = x.shape
    half = inv_freq.numel()
    ang = (pos if pos.dim() == 2 else pos[None].expand(b, n)).to(_F64)[..., None, None] * inv_freq
    c, s = magnitude * torch.cos(ang), magnitude * torch.sin(ang)
    if inverse:
        s = -s
    out = x.to(_F64).clone()
    if layout == "half":
        ia, ib = torch.arange(half), torch.arange(half) + half
    else:
        ia, ib = 2 * torch.arange(half), 2 * torch.arange(half) + 1
    xa, xb = x[..., ia].to(_F64), x[..., ib].to(_F64)
    out[..., ia] = xa * c - xb * s
    out[..., ib] = xa * s + xb * c
    return out


def norm_rotate(x, w, pos, inv_freq, eps, layout="half", magnitude=1.0):
    x = x.to(_F64)
    r = 1.0 / torch.sqrt((x * x).mean(dim=-1, keepdim=True) + eps)
    return rotate(x * r * w.to(_F64), pos, inv_freq, layout, magnitude)


def norm_rotate_backward(x, w, dy, pos, inv_freq, eps, layout="half", magnitude=1.0):
    """(dx, dw) by the formulas: t = R^T dy, dw = sum t xh,
    dx = r (t w - xh mean(t w xh))."""
    x, w = x.to(_F64), w.to(_F64)
    r = 1.0 / torch.sqrt((x * x).mean(dim=-1, keepdim=True) + eps)
    xh = x * r
    t = rotate(dy, pos, inv_freq, layout, magnitude, inverse=True)
    dw = (t * xh).sum(dim=(0, 1, 2))
    t = t * w
    return r * (t - xh * (t * xh).mean(dim=-1, keepdim=True)), dw

"""Attention with a sliding window and visible first tokens, and its gradients,
fp64 on the CPU. TEST INFRASTRUCTURE (see the package docstring).

The query at position p of its sequence sees key j when
    j <= p  and  (p - j < window  or  j < sinks).
A sequence has klen keys and qlen <= klen queries, its last positions. Each
function takes one sequence (no batch), the mask is written out as a matrix and
the formulas are applied to whole matrices: small sizes only.
"""
import math

import torch

_F64 = torch.float64


def window_mask(qlen, klen, window, sinks):
    """[qlen, klen], true where the query sees the key."""
    p = torch.arange(klen - qlen, klen)[:, None]
    j = torch.arange(klen)[None, :]
    return (j <= p) & ((p - j < window) | (j < sinks))


def _probabilities(q, k, see, scale):
    s = (q @ k.T) * scale
    s = s.masked_fill(~see, float("-inf"))
    m = s.amax(dim=1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(s - m)
    total = e.sum(dim=1, keepdim=True)
    lse = (m + torch.log(total)).squeeze(1)
    return torch.where(total > 0, e / total, torch.zeros_like(e)), lse


def window_attention(q, k, v, window, sinks=0, scale=None, do=None):
    """q [qlen, hq, d], k/v [klen, hkv, d]. Returns a dict of fp64 tensors: o,
    lse [hq, qlen], and with ``do`` the gradients dq, dk, dv; beside each of
    them ``*_err``, what rounding to bf16 where the kernels round may move it
    by (element-wise; see the derivation in the tests)."""
    qlen, hq, d = q.shape
    klen, hkv, _ = k.shape
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    see = window_mask(qlen, klen, window, sinks)
    u = 2.0 ** -8  # a bf16 rounding, relative to the value
    out = {"o": torch.zeros(qlen, hq, d, dtype=_F64), "lse": torch.zeros(hq, qlen, dtype=_F64)}
    out["o_err"] = torch.zeros_like(out["o"])
    if do is not None:
        for n, x in (("dq", q), ("dk", k), ("dv", v)):
            out[n] = torch.zeros(x.shape, dtype=_F64)
            out[n + "_err"] = torch.zeros(x.shape, dtype=_F64)
    for h in range(hq):
        g = h // (hq // hkv)
        qh, kh, vh = q[:, h].to(_F64), k[:, g].to(_F64), v[:, g].to(_F64)
        p, lse = _probabilities(qh, kh, see, scale)
        o = p @ vh
        out["o"][:, h], out["lse"][h] = o, lse
        # P enters the product rounded: sum_j P_ij |v_j| u
        mass = p @ vh.abs()
        out["o_err"][:, h] = u * mass
        if do is None:
            continue
        dh = do[:, h].to(_F64)
        dp = dh @ vh.T
        dd = (dh * o).sum(dim=1, keepdim=True)
        ds = p * (dp - dd)
        out["dv"][:, g] += p.T @ dh
        out["dq"][:, h] = scale * (ds @ kh)
        out["dk"][:, g] += scale * (ds.T @ qh)
        # dS: P and dS rounded (2 u of it), and D formed from the rounded O
        # whose own P was rounded: P * sum_d |dO| (u |O| + u mass)
        dd_err = (dh.abs() * (u * o.abs() + u * mass)).sum(dim=1, keepdim=True)
        ds_err = 2 * u * ds.abs() + p * dd_err
        out["dv_err"][:, g] += u * (p.T @ dh.abs())
        out["dq_err"][:, h] = scale * (ds_err @ kh.abs())
        out["dk_err"][:, g] += scale * (ds_err.T @ qh.abs())
    return out


def decode_attention(q, k, v, length, window=0, sinks=0, scale=None):
    """One query [hq, d] against the first ``length`` of k/v [cap, hkv, d].
    Returns (o, lse, o_err)."""
    hq, d = q.shape
    if length == 0:
        z = torch.zeros(hq, d, dtype=_F64)
        return z, torch.full((hq,), float("-inf"), dtype=_F64), z
    w = window if window > 0 else length
    r = window_attention(q[None], k[:length], v[:length], w, sinks if window > 0 else 0, scale)
    return r["o"][0], r["lse"][:, 0], r["o_err"][0]

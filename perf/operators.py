"""Operators around windowed attention: what is measured, and their plain forms.

  rope    rotary positions: half or interleaved pairs, part of the head,
          frequencies scaled for long contexts, explicit positions
  norm    RMS norm of each query and key head and the position rotation in one
          pass; with its backward in training
  window  attention with a sliding window and a few first tokens that stay
          visible: forward, and forward with backward
  decode  the same attention for one new token per sequence over a cache

Tensors are bf16 ([batch, tokens, heads, head_dim] unless said otherwise), as
everywhere in the package. With `own` false the operators are computed by
elementary torch operations in 32 bits, angles of positions in 64.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
BASE = 500000.0


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one new token of one sequence far into a long context, as a server decodes it
        {"name": "rope_token", "op": "rope", "b": 1, "n": 1, "h": 40, "d": 128, "rot": 128, "layout": "half",
         "scaled": True, "explicit": True},
        # queries and keys of the 32K training sequence, rotated in the fused projection's own rows
        {"name": "rope_sequence", "op": "rope", "b": 1, "n": 32768, "h": 40, "d": 128, "rot": 64,
         "layout": "interleaved", "scaled": True, "explicit": False},
        # a serving step: one new token for each of 128 sequences
        {"name": "norm_tokens", "op": "norm", "b": 128, "n": 1, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "layout": "half", "train": False, "explicit": True, "w32": False},
        # the 32K training workload's queries and keys, forward and backward
        {"name": "norm_train", "op": "norm", "b": 1, "n": 32768, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "layout": "half", "train": True, "explicit": False, "w32": True},
        # small heads, an odd length, half of the head rotated in interleaved pairs
        {"name": "norm_train_odd", "op": "norm", "b": 3, "n": 1777, "hq": 6, "hkv": 2, "d": 64, "rot": 32,
         "layout": "interleaved", "train": True, "explicit": False, "w32": False},
        # prefill of a 16K prompt with 64 query heads, a wide window
        {"name": "window_prefill", "op": "window", "b": 1, "sq": 16384, "skv": 16384, "hq": 64, "hkv": 8, "d": 128,
         "window": 4096, "sinks": 4, "train": False, "samples": 0},
        # the 32K training workload as a windowed layer
        {"name": "window_train", "op": "window", "b": 1, "sq": 32768, "skv": 32768, "hq": 32, "hkv": 8, "d": 128,
         "window": 1024, "sinks": 4, "train": True, "samples": 0},
        # packed samples of odd lengths, one KV head per query head, small heads
        {"name": "window_train_packed", "op": "window", "b": 1, "sq": 8191, "skv": 8191, "hq": 8, "hkv": 8, "d": 64,
         "window": 300, "sinks": 1, "train": True, "samples": 7},
        # a chunk of each of four prompts against what was read of them so far
        {"name": "window_chunk", "op": "window", "b": 4, "sq": 333, "skv": 8192, "hq": 32, "hkv": 8, "d": 128,
         "window": 1024, "sinks": 4, "train": False, "samples": 0},
        # one new token of one long sequence: the shortest call
        {"name": "decode_one", "op": "decode", "b": 1, "hq": 32, "hkv": 8, "d": 128, "cap": 131072, "window": 1024,
         "sinks": 4},
        # a serving step of 64 sequences of different lengths with a wide window
        {"name": "decode_batch", "op": "decode", "b": 64, "hq": 32, "hkv": 8, "d": 128, "cap": 16384, "window": 4096,
         "sinks": 4},
        # long contexts read whole (the layers of such a model that have no window)
        {"name": "decode_whole", "op": "decode", "b": 16, "hq": 64, "hkv": 8, "d": 128, "cap": 65537, "window": 0,
         "sinks": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rope", "norm", "window", "window", "decode"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 8])
    layout = rng.choice(["half", "interleaved"])
    rot = rng.choice([d, d, d // 2, d // 4, 3 * d // 4])
    if op in ("rope", "norm"):
        if rng.random() < 0.4:  # single tokens
            b, n, explicit = _log(rng, 1, 256), 1, True
        else:
            b, explicit = rng.choice([1, 1, 2, 3]), False
            n = _log(rng, 3, 32768 // b)
        if op == "rope":
            return {"op": op, "b": b, "n": n, "h": min(hq + hkv, 40), "d": d, "rot": rot, "layout": layout,
                    "scaled": rng.random() < 0.5, "explicit": explicit}
        return {"op": op, "b": b, "n": n, "hq": min(hq, 32), "hkv": hkv if hq <= 32 else 4, "d": d, "rot": rot,
                "layout": layout, "train": not explicit and rng.random() < 0.7, "explicit": explicit,
                "w32": rng.random() < 0.5}
    if op == "window":
        if hq > 32:
            hq, hkv = 32, 8
        sinks = rng.choice([0, 1, 4, 16])
        window = _log(rng, 16, 2048)
        kind = rng.choice(["train", "train", "packed", "prefill", "chunk"])
        if kind == "chunk":
            skv = _log(rng, 256, 16384)
            return {"op": op, "b": rng.choice([1, 2, 4]), "sq": _log(rng, 2, min(1024, skv)), "skv": skv, "hq": hq,
                    "hkv": hkv, "d": d, "window": window, "sinks": sinks, "train": False, "samples": 0}
        b = 1 if kind == "packed" else rng.choice([1, 1, 2])
        s = _log(rng, 64, 16384 // b)
        return {"op": op, "b": b, "sq": s, "skv": s, "hq": hq, "hkv": hkv, "d": d, "window": window, "sinks": sinks,
                "train": kind != "prefill", "samples": rng.choice([3, 5, 12]) if kind == "packed" else 0}
    b = _log(rng, 1, 64)
    cap = _log(rng, 64, min(65536, (1 << 20) // b))
    window = 0 if rng.random() < 0.4 else _log(rng, 16, 8192)
    return {"op": op, "b": b, "hq": hq, "hkv": hkv, "d": d, "cap": cap, "window": window,
            "sinks": rng.choice([0, 4, 16]) if window else 0}


# ---------------------------------------------------------------- inputs
def _frequencies(rot, scaled):
    """Angle per position of each pair; scaled: pairs that turn less than once over 8192 positions get
    an eighth of their frequency, those that turn more than four times keep it, linear in between."""
    f = BASE ** (-2.0 * torch.arange(rot // 2, dtype=F64) / rot)
    if scaled:
        keep = ((8192.0 * f / (2 * math.pi) - 1.0) / 3.0).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / 8.0)
    return f


def _randn(gen, *shape, std=1.0):
    x = torch.randn(*shape, generator=gen, device="cuda", dtype=BF16)
    return x if std == 1.0 else x.mul_(std)


def _positions(c, gen):
    return torch.randint(0, 131072, (c["b"], c["n"]), generator=gen, device="cuda", dtype=torch.int32)


def _sample_offsets(total, samples, seed):
    """Packed samples of different lengths, one of them a single token."""
    g = torch.Generator().manual_seed(seed)
    cut = torch.randperm(total - 2, generator=g)[: max(0, samples - 2)] + 1
    return [0] + sorted(cut.tolist()) + [total - 1, total]


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"c": c}
    if c["op"] == "rope":
        # the head rows of a fused projection: queries and keys, followed by the values that stay as they are
        st["x"] = _randn(gen, c["b"], c["n"], c["h"] + 8, c["d"])[:, :, : c["h"]]
        st["pos"] = _positions(c, gen) if c["explicit"] else None
        st["freq"] = _frequencies(c["rot"], c["scaled"])
        st["mag"] = 1.0 + 0.1 * math.log(8.0) if c["scaled"] else 1.0
    elif c["op"] == "norm":
        hq, hkv = c["hq"], c["hkv"]
        qkv = _randn(gen, c["b"], c["n"], hq + 2 * hkv, c["d"], std=3.0)
        st["q"], st["k"] = qkv[:, :, :hq], qkv[:, :, hq : hq + hkv]
        wt = F32 if c["w32"] else BF16
        for name in ("wq", "wk"):
            st[name] = (1.0 + 0.2 * torch.randn(c["d"], generator=gen, device="cuda")).to(wt)
        st["pos"] = _positions(c, gen) if c["explicit"] else None
        st["freq"] = _frequencies(c["rot"], False)
        if c["train"]:
            st["gq"] = _randn(gen, c["b"], c["n"], hq, c["d"])
            st["gk"] = _randn(gen, c["b"], c["n"], hkv, c["d"])
    elif c["op"] == "window":
        lead = (c["sq"],) if c["samples"] else (c["b"], c["sq"])
        leadk = (c["skv"],) if c["samples"] else (c["b"], c["skv"])
        st["q"] = _randn(gen, *lead, c["hq"], c["d"])
        st["k"] = _randn(gen, *leadk, c["hkv"], c["d"])
        st["v"] = _randn(gen, *leadk, c["hkv"], c["d"])
        if c["train"]:
            st["do"] = _randn(gen, *lead, c["hq"], c["d"])
        st["cu"] = _sample_offsets(c["sq"], c["samples"], 77) if c["samples"] else None
    else:
        st["q"] = _randn(gen, c["b"], c["hq"], c["d"])
        st["k"] = _randn(gen, c["b"], c["cap"], c["hkv"], c["d"])
        st["v"] = _randn(gen, c["b"], c["cap"], c["hkv"], c["d"])
        order = torch.randperm(c["b"], generator=gen, device="cuda")
        st["len"] = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")[order].contiguous()
    return st


def _lengths(c):
    """Tokens held of each sequence: from half of the cache to all of it."""
    return [c["cap"] - (i * (c["cap"] // 2)) // max(1, c["b"] - 1) for i in range(c["b"])]


# ---------------------------------------------------------------- the calls
def run(st):
    if own:
        return _own(st)
    return {"rope": _plain_rope, "norm": _plain_norm, "window": _plain_window, "decode": _plain_decode}[st["c"]["op"]](st)


def _own(st):
    import context_blockwise_causal_gb300 as cp

    c = st["c"]
    if c["op"] == "rope":
        y = torch.empty(c["b"], c["n"], c["h"], c["d"], dtype=BF16, device="cuda")
        return cp.cpattn_rope(st["x"], inv_freq=st["freq"], layout=c["layout"], positions=st["pos"],
                              magnitude=st["mag"], out=y)
    if c["op"] == "norm":
        kw = {"inv_freq": st["freq"], "layout": c["layout"], "positions": st["pos"], "eps": 1e-6}
        q, k = cp.cpattn_qk_norm_rope(st["q"], st["k"], st["wq"], st["wk"], **kw)
        if not c["train"]:
            return {"q": q, "k": k}
        dq, dk, dwq, dwk = cp.cpattn_qk_norm_rope_bwd(st["q"], st["k"], st["wq"], st["wk"], st["gq"], st["gk"], **kw)
        return {"q": q, "k": k, "dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    if c["op"] == "window":
        args = (c["window"], c["sinks"])
        if c["samples"]:
            o, lse = cp.cpattn_fwd_window_varlen(st["q"], st["k"], st["v"], st["cu"], *args)
        else:
            o, lse = cp.cpattn_fwd_window(st["q"], st["k"], st["v"], *args)
        if not c["train"]:
            return {"o": o, "lse": lse}
        if c["samples"]:
            dq, dk, dv = cp.cpattn_bwd_window_varlen(st["q"], st["k"], st["v"], o, lse, st["do"], st["cu"], *args)
        else:
            dq, dk, dv = cp.cpattn_bwd_window(st["q"], st["k"], st["v"], o, lse, st["do"], *args)
        return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    o, lse = cp.cpattn_decode(st["q"], st["k"], st["v"], st["len"], window=c["window"], sinks=c["sinks"])
    return {"o": o, "lse": lse}


# ---------------------------------------------------------------- plain forms
def _cos_sin(st, mag=1.0):
    """Cosine and sine [b or 1, n, 1, rot/2], the angle formed in 64 bits."""
    c = st["c"]
    pos = torch.arange(c["n"], device="cuda")[None] if st["pos"] is None else st["pos"]
    a = (pos.to(F64)[..., None] * st["freq"].cuda())[:, :, None]
    return (a.cos() * mag).to(F32), (a.sin() * mag).to(F32)


def _turn(x, cos, sin, rot, layout):
    """Rotates the first `rot` features of each head; the others pass."""
    r, rest = x[..., :rot], x[..., rot:]
    if layout == "half":
        a, b = r[..., : rot // 2], r[..., rot // 2 :]
        r = torch.cat([a * cos - b * sin, a * sin + b * cos], dim=-1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, a * sin + b * cos], dim=-1).flatten(-2)
    return torch.cat([r, rest], dim=-1)


def _plain_rope(st):
    c = st["c"]
    cos, sin = _cos_sin(st, st["mag"])
    return _turn(st["x"].to(F32), cos, sin, c["rot"], c["layout"]).to(BF16)


def _plain_norm(st):
    c = st["c"]
    cos, sin = _cos_sin(st)
    out = {}
    for name, x, w, g in (("q", st["q"], st["wq"], st.get("gq")), ("k", st["k"], st["wk"], st.get("gk"))):
        x, w = x.to(F32), w.to(F32)
        r = (x.square().mean(dim=-1, keepdim=True) + 1e-6).rsqrt()
        xh = x * r
        out[name] = _turn(xh * w, cos, sin, c["rot"], c["layout"]).to(BF16)
        if c["train"]:
            t = _turn(g.to(F32), cos, -sin, c["rot"], c["layout"])  # the gradient of the rotation turns back
            out["dw" + name] = (t * xh).sum(dim=(0, 1, 2), dtype=F64).to(F32)
            t = t * w
            out["d" + name] = (r * (t - xh * (t * xh).mean(dim=-1, keepdim=True))).to(BF16)
    return out


def _plain_window(st):
    """Blocks of queries against the stretch of keys that their windows cover, and against the first
    keys of their own sample. Query t is token skv - sq + t."""
    c = st["c"]
    packed = bool(c["samples"])
    q, k, v = (x[None] if packed else x for x in (st["q"], st["k"], st["v"]))
    b, sq, hq, d = q.shape
    skv, hkv = k.shape[1], k.shape[2]
    w, ns, grp, size = min(c["window"], skv), c["sinks"], hq // hkv, 256
    first = torch.zeros(skv, dtype=torch.long, device="cuda")
    if packed:
        cu = torch.tensor(st["cu"], device="cuda")
        first = cu[torch.searchsorted(cu, torch.arange(skv, device="cuda"), right=True) - 1]
    nb = -(-sq // size)
    rows = torch.arange(nb * size, device="cuda").view(nb, size)
    live = rows < sq
    rows = rows.clamp(max=sq - 1)
    pos = rows + (skv - sq)  # [block, query]
    keys = (skv - sq) - (w - 1) + size * torch.arange(nb, device="cuda")[:, None] + torch.arange(w - 1 + size, device="cuda")
    p3, k3 = pos[:, :, None], keys[:, None, :]
    see = (k3 <= p3) & (k3 > p3 - c["window"]) & (k3 >= first[pos][:, :, None])
    keys = keys.clamp(0, skv - 1)
    early = first[pos][:, :, None] + torch.arange(ns, device="cuda")  # the sample's first tokens
    see_early = early <= p3 - c["window"]
    early = early.clamp(max=skv - 1)
    qb = q[:, rows].to(F32).view(b, nb, size, hkv, grp, d)
    kb, vb, ke, ve = (x[:, i].to(F32) for i in (keys, early) for x in (k, v))
    scale = d ** -0.5
    s = torch.cat([torch.einsum("bnqhgd,bnlhd->bnhgql", qb, kb).mul_(scale).masked_fill_(~see[:, None, None], -math.inf),
                   torch.einsum("bnqhgd,bnqchd->bnhgqc", qb, ke).mul_(scale).masked_fill_(~see_early[:, None, None], -math.inf)], dim=-1)
    m = s.amax(dim=-1, keepdim=True)
    p = s.sub_(m).exp_()
    total = p.sum(dim=-1, keepdim=True)
    p = p.div_(total)
    n = kb.shape[2]
    o = torch.einsum("bnhgql,bnlhd->bnqhgd", p[..., :n], vb) + torch.einsum("bnhgqc,bnqchd->bnqhgd", p[..., n:], ve)
    lse = (m + total.log()).squeeze(-1).permute(0, 2, 3, 1, 4).reshape(b, hq, nb * size)[:, :, :sq]
    out = {"o": o.reshape(b, nb * size, hq, d)[:, :sq].to(BF16), "lse": lse.contiguous()}
    if c["train"]:
        do = st["do"][None] if packed else st["do"]
        g = (do[:, rows].to(F32) * live[:, :, None, None]).view(b, nb, size, hkv, grp, d)
        dd = (g * o).sum(dim=-1).permute(0, 1, 3, 4, 2)[..., None]
        dp = torch.cat([torch.einsum("bnqhgd,bnlhd->bnhgql", g, vb), torch.einsum("bnqhgd,bnqchd->bnhgqc", g, ve)], dim=-1)
        ds = dp.sub_(dd).mul_(p).mul_(scale)
        dq = torch.einsum("bnhgql,bnlhd->bnqhgd", ds[..., :n], kb) + torch.einsum("bnhgqc,bnqchd->bnqhgd", ds[..., n:], ke)
        out["dq"] = dq.reshape(b, nb * size, hq, d)[:, :sq].to(BF16)
        for name, t, x in (("dk", ds, qb), ("dv", p, g)):
            acc = torch.zeros(b, skv, hkv, d, device="cuda")
            acc.index_add_(1, keys.flatten(), torch.einsum("bnhgql,bnqhgd->bnlhd", t[..., :n], x).flatten(1, 2))
            acc.index_add_(1, early.flatten(), torch.einsum("bnhgqc,bnqhgd->bnqchd", t[..., n:], x).flatten(1, 3))
            out[name] = acc.to(BF16)
    return {name: t[0] if packed else t for name, t in out.items()}


def _plain_decode(st):
    c = st["c"]
    b, hq, d = st["q"].shape
    hkv, held = c["hkv"], st["len"].long()[:, None]
    if c["window"]:  # the window's keys and the first ones, each once
        at = held - c["window"] + torch.arange(c["window"], device="cuda")
        see = at >= 0
        early = torch.arange(c["sinks"], device="cuda").expand(b, -1)
        see = torch.cat([see, early < held - c["window"]], dim=1)
        at = torch.cat([at, early], dim=1).clamp(0, c["cap"] - 1)
        i = torch.arange(b, device="cuda")[:, None]
        k, v = st["k"][i, at].to(F32), st["v"][i, at].to(F32)
    else:
        see = torch.arange(c["cap"], device="cuda") < held
        k, v = st["k"].to(F32), st["v"].to(F32)
    s = torch.einsum("bhgd,blhd->bhgl", st["q"].to(F32).view(b, hkv, hq // hkv, d), k) * d ** -0.5
    s = s.masked_fill(~see[:, None, None], -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    p = (s - m).exp()
    total = p.sum(dim=-1, keepdim=True)
    o = torch.einsum("bhgl,blhd->bhgd", p / total, v)
    return {"o": o.reshape(b, hq, d).to(BF16), "lse": (m + total.log()).view(b, hq)}


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    c = st["c"]
    if c["op"] in ("rope", "norm"):
        pos = torch.arange(c["n"], device="cuda").expand(c["b"], -1) if st["pos"] is None else st["pos"]
        turn = torch.polar(torch.ones((), dtype=F64, device="cuda"), pos.to(F64)[:, :, None, None] * st["freq"].cuda())
        if c["op"] == "rope":
            return _exact_turn(st["x"].to(F64), turn * st["mag"], c)
        return _exact_norm(st, turn)
    if c["op"] == "window":
        matmuls = 9 if c["train"] else 2
        if matmuls * 2.0 * c["b"] * c["hq"] * c["sq"] * c["skv"] * c["d"] > 1.4e13:
            return None  # over 20 seconds at this card's 64-bit rate
        return _exact_window(st)
    return _exact_decode(st)


def _exact_turn(x, turn, c):
    """The rotated pairs as complex numbers times e^(i angle)."""
    r = x[..., : c["rot"]]
    z = torch.complex(*r.unflatten(-1, (2, -1)).unbind(-2)) if c["layout"] == "half" else torch.view_as_complex(r.unflatten(-1, (-1, 2)).contiguous())
    z = z * turn
    r = torch.cat([z.real, z.imag], -1) if c["layout"] == "half" else torch.view_as_real(z).flatten(-2)
    return torch.cat([r, x[..., c["rot"] :]], -1)


def _exact_norm(st, turn):
    out = {}
    for name, g in (("q", st.get("gq")), ("k", st.get("gk"))):
        x, w = st[name].to(F64).requires_grad_(), st["w" + name].to(F64).requires_grad_()
        y = _exact_turn(x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w, turn, st["c"])
        out[name] = y.detach()
        if g is not None:
            out["d" + name], out["dw" + name] = torch.autograd.grad(y, (x, w), g.to(F64))
    return out


def _exact_window(st):
    c = st["c"]
    packed = bool(c["samples"])
    q, k, v = (x[None] if packed else x for x in (st["q"], st["k"], st["v"]))
    b, sq, hq, d = q.shape
    skv, hkv = k.shape[1:3]
    i = torch.arange(skv - sq, skv, device="cuda")[:, None]
    j = torch.arange(skv, device="cuda")[None]
    first = torch.zeros_like(i)
    if packed:
        for a, e in zip(st["cu"], st["cu"][1:]):
            first[a:e] = a
    hidden = ~((j <= i) & (j >= first) & ((i - j < c["window"]) | (j - first < c["sinks"])))
    out = {"o": torch.empty(q.shape, dtype=F64, device="cuda"), "lse": torch.empty(b, hq, sq, dtype=F64, device="cuda")}
    if c["train"]:
        out |= {n: torch.zeros(x.shape, dtype=F64, device="cuda") for n, x in (("dq", q), ("dk", k), ("dv", v))}
        do = st["do"][None] if packed else st["do"]
    for bi in range(b):
        for h in range(hq):
            e = h * hkv // hq
            leaves = [x.to(F64).requires_grad_(c["train"]) for x in (q[bi, :, h], k[bi, :, e], v[bi, :, e])]
            s = (leaves[0] @ leaves[1].T / math.sqrt(d)).masked_fill(hidden, -math.inf)
            o = torch.softmax(s, -1) @ leaves[2]
            out["o"][bi, :, h] = o.detach()
            out["lse"][bi, h] = torch.logsumexp(s.detach(), -1)
            if c["train"]:
                grads = torch.autograd.grad(o, leaves, do[bi, :, h].to(F64))
                out["dq"][bi, :, h] = grads[0]
                out["dk"][bi, :, e] += grads[1]
                out["dv"][bi, :, e] += grads[2]
    return {n: t[0] if packed else t for n, t in out.items()}


def _exact_decode(st):
    c = st["c"]
    b, hq, d = st["q"].shape
    o, lse = torch.zeros(b, hq, d, dtype=F64, device="cuda"), torch.full((b, hq), -math.inf, dtype=F64, device="cuda")
    for i, n in enumerate(st["len"].tolist()):
        at = torch.arange(n, device="cuda")
        if c["window"]:
            at = at[(at >= n - c["window"]) | (at < c["sinks"])]
        k, v = (x[i].index_select(0, at).to(F64).repeat_interleave(hq // c["hkv"], 1) for x in (st["k"], st["v"]))
        s = (st["q"][i].to(F64)[None] * k).sum(-1) / math.sqrt(d)  # [key, head]
        lse[i] = torch.logsumexp(s, 0)
        o[i] = (torch.softmax(s, 0)[..., None] * v).sum(0)
    return {"o": o, "lse": lse}


# ---------------------------------------------------------------- work
def _pairs(sq, skv, window, sinks):
    """(query, key) pairs of one head: query at position i sees min(i + 1, window) keys and the first ones before them."""
    total = 0
    for i in range(skv - sq, skv):
        near = min(i + 1, window)
        total += near + min(sinks, i + 1 - near)
    return total


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["b"] * c["n"] * c["h"]
        return {"bytes": 4.0 * n * c["d"], "flops": 3.0 * n * c["rot"]}
    if c["op"] == "norm":
        n = c["b"] * c["n"] * (c["hq"] + c["hkv"])
        # forward: read x, write y; backward: read x and the gradient, write dx
        return {"bytes": (10.0 if c["train"] else 4.0) * n * c["d"], "flops": (24.0 if c["train"] else 8.0) * n * c["d"]}
    if c["op"] == "window":
        if c["samples"]:
            cu = _sample_offsets(c["sq"], c["samples"], 77)
            pairs = sum(_pairs(e - a, e - a, c["window"], c["sinks"]) for a, e in zip(cu, cu[1:]))
        else:
            pairs = c["b"] * _pairs(c["sq"], c["skv"], c["window"], c["sinks"])
        seen = c["b"] * min(c["skv"], c["sq"] + c["window"] - 1 + c["sinks"])
        nq, nkv = c["b"] * c["sq"] * c["hq"] * c["d"], seen * c["hkv"] * c["d"]
        if c["train"]:  # forward: q, k, v, o; backward: q, k, v, o, do and the three gradients
            return {"bytes": 2.0 * (6 * nq + 6 * nkv), "flops": 14.0 * pairs * c["hq"] * c["d"]}
        return {"bytes": 2.0 * (2 * nq + 2 * nkv), "flops": 4.0 * pairs * c["hq"] * c["d"]}
    keys = sum(n if not c["window"] else min(n, c["window"]) + min(c["sinks"], max(0, n - c["window"])) for n in _lengths(c))
    return {"bytes": 4.0 * keys * c["hkv"] * c["d"] + 4.0 * c["b"] * c["hq"] * c["d"], "flops": 4.0 * keys * c["hq"] * c["d"]}

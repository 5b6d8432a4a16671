"""Operators of a paged cache: what is measured, and their plain forms.

  append  new tokens' keys and values into the pages of their sequences, keys
          (and the queries beside them) rotated to their positions on the way
  paged   attention of one new token per sequence over the pages, whole or
          with a sliding window and a few first tokens that stay visible
  shared  the same over every key for groups of sequences that begin with the
          same tokens, whose pages are read once for the group

A page holds the keys or the values of `page` tokens of every KV head; a
sequence's table names its pages in order. Tensors are bf16, as everywhere in
the package. With `own` false the operators are computed by elementary torch
operations in 32 bits, angles of positions in 64.
"""
import math

import torch

own = False

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
BASE = 500000.0


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one new token of one sequence: the shortest call
        {"name": "append_token", "op": "append", "b": 1, "n": 1, "ragged": False, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "layout": "half", "cap": 8192, "page": 64, "heads_first": False},
        # a serving step: one new token for each of 128 sequences, small pages
        {"name": "append_step", "op": "append", "b": 128, "n": 1, "ragged": False, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "layout": "half", "cap": 1024, "page": 16, "heads_first": False},
        # chunks of different lengths of seven prompts in one call, half of a small head rotated in interleaved pairs
        {"name": "append_chunks", "op": "append", "b": 7, "n": 5331, "ragged": True, "hq": 6, "hkv": 2, "d": 64,
         "rot": 32, "layout": "interleaved", "cap": 6000, "page": 48, "heads_first": True},
        # the whole of a 32K prompt
        {"name": "append_prompt", "op": "append", "b": 1, "n": 32768, "ragged": False, "hq": 32, "hkv": 8, "d": 128,
         "rot": 128, "layout": "half", "cap": 32768, "page": 128, "heads_first": False},
        # one new token of one sequence of middling length
        {"name": "paged_one", "op": "paged", "b": 1, "hq": 32, "hkv": 8, "d": 128, "cap": 8192, "page": 64,
         "window": 0, "sinks": 0, "heads_first": False},
        # small heads, an odd number of short sequences, pages whose heads come first
        {"name": "paged_small", "op": "paged", "b": 37, "hq": 6, "hkv": 2, "d": 64, "cap": 2928, "page": 48,
         "window": 0, "sinks": 0, "heads_first": True},
        # a serving step of 64 sequences of different lengths with a wide window, small pages
        {"name": "paged_window", "op": "paged", "b": 64, "hq": 32, "hkv": 8, "d": 128, "cap": 16384, "page": 16,
         "window": 4096, "sinks": 4, "heads_first": False},
        # long contexts read whole
        {"name": "paged_whole", "op": "paged", "b": 16, "hq": 64, "hkv": 8, "d": 128, "cap": 65536, "page": 128,
         "window": 0, "sinks": 0, "heads_first": False},
        # four answers to one prompt
        {"name": "shared_few", "op": "shared", "groups": "4", "prefix": "8192", "own": 256, "hq": 32, "hkv": 8,
         "d": 128, "page": 64, "heads_first": False},
        # several prompts of odd lengths with different numbers of answers, three query heads to a KV head
        {"name": "shared_groups", "op": "shared", "groups": "3 20 1 9 13", "prefix": "9001 2049 777 4099 5000",
         "own": 300, "hq": 24, "hkv": 8, "d": 64, "page": 32, "heads_first": True},
        # a serving step of 64 sequences behind one long document
        {"name": "shared_step", "op": "shared", "groups": "64", "prefix": "32768", "own": 1024, "hq": 32, "hkv": 8,
         "d": 128, "page": 64, "heads_first": False},
        # many sequences behind a long system prompt, 64 query heads
        {"name": "shared_many", "op": "shared", "groups": "256", "prefix": "16384", "own": 2048, "hq": 64, "hkv": 8,
         "d": 128, "page": 128, "heads_first": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["append", "append", "paged", "paged", "shared", "shared"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 8])
    page = rng.choice([16, 32, 48, 64, 80, 128, 256])
    c = {"op": op, "hq": hq, "hkv": hkv, "d": d, "page": page, "heads_first": rng.random() < 0.3}
    if op == "append":
        if hq > 32:
            c["hq"], c["hkv"] = 32, 4
        kind = rng.choice(["step", "chunks", "prompt"])
        if kind == "step":
            b, n, cap = _log(rng, 1, 256), 1, _log(rng, 16, 1024)
        elif kind == "chunks":
            b, n = _log(rng, 2, 32), _log(rng, 40, 16384)
            cap = _log(rng, n, 32768)
            cap = max(n, min(cap, 131072 // b))
        else:
            b = rng.choice([1, 1, 2, 3])
            n = _log(rng, 3, 32768 // b)
            cap = _log(rng, n, 32768)
        return c | {"b": b, "n": n, "ragged": kind == "chunks", "cap": cap, "rot": rng.choice([d, d, d // 2, d // 4]),
                    "layout": rng.choice(["half", "interleaved"])}
    if op == "paged":
        b = _log(rng, 1, 64)
        window = 0 if rng.random() < 0.5 else _log(rng, 16, 8192)
        return c | {"b": b, "cap": _log(rng, 64, min(65536, (1 << 20) // b)), "window": window,
                    "sinks": rng.choice([0, 4, 16]) if window else 0}
    count = rng.choice([1, 1, 2, 3, 6])
    groups = [_log(rng, 1, 128 // count) for _ in range(count)]
    prefix = [_log(rng, 16, 32768 // count) for _ in range(count)]
    return c | {"groups": " ".join(map(str, groups)), "prefix": " ".join(map(str, prefix)), "own": _log(rng, 1, 2048)}


def _groups(c):
    """Sequences of each group, and the tokens that they begin with."""
    return [int(x) for x in c["groups"].split()], [int(x) for x in c["prefix"].split()]


# ---------------------------------------------------------------- inputs
def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=BF16)


def _frequencies(rot):
    return BASE ** (-2.0 * torch.arange(rot // 2, dtype=F64) / rot)


def _pools(gen, c, pages):
    """Keys and values of the pages, [pages, page, hkv, d]; heads_first: a view of [pages, hkv, page, d]."""
    if c["heads_first"]:
        return [_randn(gen, pages, c["hkv"], c["page"], c["d"]).transpose(1, 2) for _ in range(2)]
    return [_randn(gen, pages, c["page"], c["hkv"], c["d"]) for _ in range(2)]


def _spread(last, first, count):
    """`count` whole numbers from `last` down to `first`."""
    return [last - (i * (last - first)) // max(1, count - 1) for i in range(count)]


def _counts(c):
    """New tokens of each sequence; ragged ones differ, and one sequence has a single token."""
    if not c["ragged"]:
        return [c["n"]] * c["b"]
    weight = [2 + (i * 7) % 5 for i in range(c["b"] - 1)]
    left = c["n"] - 1
    counts = [left * w // sum(weight) for w in weight]
    counts[0] += left - sum(counts)
    return counts[: c["b"] // 2] + [1] + counts[c["b"] // 2 :]


def _appended_lengths(c):
    """Tokens held after the call: from just the new ones to a full table."""
    return [m + (i + 1) * (c["cap"] - m) // c["b"] for i, m in enumerate(_counts(c))]


def _paged_lengths(c):
    return _spread(c["cap"], (c["cap"] + 1) // 2, c["b"])


def _shared_lengths(c):
    """Of each group's sequences: the tokens they begin with and from one to `own` of their own."""
    return [p + m for size, p in zip(*_groups(c)) for m in _spread(c["own"], (c["own"] + 3) // 4, size)]


def _on_gpu(values):
    return torch.tensor(values, dtype=I32, device="cuda")


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"c": c}
    if c["op"] == "shared":
        return _prepare_shared(c, gen, st)
    cols = -(-c["cap"] // c["page"])
    pages = c["b"] * cols + 3
    st["kp"], st["vp"] = _pools(gen, c, pages)
    # the pages lie in no order, as a server hands them out
    st["tables"] = torch.randperm(pages, generator=gen, device="cuda")[: c["b"] * cols].view(c["b"], cols).to(I32)
    if c["op"] == "append":
        lead = (1, c["n"]) if c["ragged"] else (c["b"], c["n"])
        # the rows of a fused projection: queries, keys, values
        qkv = _randn(gen, *lead, c["hq"] + 2 * c["hkv"], c["d"])
        st["q"], st["k"], st["v"] = qkv.split([c["hq"], c["hkv"], c["hkv"]], dim=2)
        st["len"] = _on_gpu(_appended_lengths(c))
        ends = [0]
        for m in _counts(c):
            ends.append(ends[-1] + m)
        st["cu"] = _on_gpu(ends) if c["ragged"] else None
        st["freq"] = _frequencies(c["rot"])
        return st
    st["q"] = _randn(gen, c["b"], c["hq"], c["d"])
    order = torch.randperm(c["b"], generator=gen, device="cuda")
    st["len"] = _on_gpu(_paged_lengths(c))[order].contiguous()
    return st


def _prepare_shared(c, gen, st):
    (groups, prefix), page = _groups(c), c["page"]
    b = sum(groups)
    lengths = _shared_lengths(c)
    cols = max(-(-n // page) for n in lengths)
    whole = [p // page for p in prefix]  # pages that hold common tokens alone
    own_cols = max(-(-n // page) - w for w, n in zip([w for w, g in zip(whole, groups) for _ in range(g)], lengths))
    pages = sum(whole) + b * own_cols + 3
    st["kp"], st["vp"] = _pools(gen, c, pages)
    name = torch.randperm(pages, generator=gen, device="cuda").to(I32)
    tables = torch.full((b, cols), -1, dtype=I32, device="cuda")
    at = row = 0
    for size, p, w in zip(groups, prefix, whole):
        tables[row : row + size, :w] = name[at : at + w]
        at += w
        n = min(own_cols, cols - w)
        tables[row : row + size, w : w + n] = name[at : at + size * n].view(size, n)
        at += size * n
        rest = p - w * page  # the common tokens in the next page: each sequence writes on in its own copy
        if rest and size > 1:
            copies = tables[row + 1 : row + size, w].long()
            for pool in (st["kp"], st["vp"]):
                pool[copies, :rest] = pool[tables[row, w].long(), :rest]
        row += size
    st["tables"] = tables
    st["q"] = _randn(gen, b, c["hq"], c["d"])
    st["len"] = _on_gpu(lengths)
    st["shared"] = _on_gpu(prefix)
    ends = [0]
    for size in groups:
        ends.append(ends[-1] + size)
    st["ends"] = _on_gpu(ends) if len(groups) > 1 else None
    return st


# ---------------------------------------------------------------- the calls
def run(st):
    if own:
        return _own(st)
    return {"append": _plain_append, "paged": _plain_paged, "shared": _plain_shared}[st["c"]["op"]](st)


def _own(st):
    import context_blockwise_causal_gb300 as cp

    c = st["c"]
    if c["op"] == "append":
        q = cp.cpattn_append_paged(st["k"], st["v"], st["kp"], st["vp"], st["tables"], st["len"], cu_tokens=st["cu"],
                                   q=st["q"], inv_freq=st["freq"], layout=c["layout"])
        return {"q": q, "k_pages": st["kp"], "v_pages": st["vp"]}
    if c["op"] == "paged":
        o, lse = cp.cpattn_decode_paged(st["q"], st["kp"], st["vp"], st["tables"], st["len"], window=c["window"],
                                        sinks=c["sinks"])
    else:
        o, lse = cp.cpattn_decode_shared(st["q"], st["kp"], st["vp"], st["tables"], st["len"], st["shared"],
                                         group_offsets=st["ends"], max_group=max(_groups(c)[0]))
    return {"o": o, "lse": lse}


# ---------------------------------------------------------------- plain forms
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


def _plain_append(st):
    c = st["c"]
    held = st["len"].long()
    if st["cu"] is None:
        seq = torch.arange(c["b"], device="cuda")[:, None]
        place = held[:, None] - c["n"] + torch.arange(c["n"], device="cuda")
    else:
        cu = st["cu"].long()
        at = torch.arange(c["n"], device="cuda")
        seq = (torch.searchsorted(cu, at, right=True) - 1)[None]
        place = held[seq] - (cu[seq + 1] - at)
    angle = (place.to(F64)[..., None] * st["freq"].cuda())[:, :, None]
    cos, sin = angle.cos().to(F32), angle.sin().to(F32)
    page, slot = st["tables"].long()[seq, place // c["page"]], place % c["page"]
    st["kp"][page, slot] = _turn(st["k"].to(F32), cos, sin, c["rot"], c["layout"]).to(BF16)
    st["vp"][page, slot] = st["v"]
    return {"q": _turn(st["q"].to(F32), cos, sin, c["rot"], c["layout"]).to(BF16), "k_pages": st["kp"], "v_pages": st["vp"]}


def _attend(q, k, v, see):
    """q [b, hq, d], k and v [b, keys, hkv, d] in 32 bits, see [b, keys]: scores, then their softmax's sums
    without the division: (maximum, sum, weighted values)."""
    b, hq, d = q.shape
    hkv = k.shape[2]
    s = torch.einsum("bhgd,blhd->bhgl", q.view(b, hkv, hq // hkv, d), k).mul_(d ** -0.5)
    s.masked_fill_(~see[:, None, None], -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    p = s.sub_(m).exp_()
    return m, p.sum(dim=-1, keepdim=True), torch.einsum("bhgl,blhd->bhgd", p, v)


def _out(m, total, o):
    b, hkv, grp, d = o.shape
    return {"o": (o / total).reshape(b, hkv * grp, d).to(BF16), "lse": (m + total.log()).view(b, hkv * grp)}


def _keys(st, at):
    """Keys and values at the places [b, n] of their sequences, in 32 bits."""
    page = st["c"]["page"]
    rows = torch.arange(at.shape[0], device="cuda")[:, None]
    names = st["tables"].long()[rows, at // page]
    return st["kp"][names, at % page].to(F32), st["vp"][names, at % page].to(F32)


def _plain_paged(st):
    c = st["c"]
    held = st["len"].long()[:, None]
    if c["window"]:  # the window's keys and the first ones, each once
        w = min(c["window"], c["cap"])
        at = held - w + torch.arange(w, device="cuda")
        see = at >= 0
        early = torch.arange(min(c["sinks"], c["cap"]), device="cuda").expand(c["b"], -1)
        see = torch.cat([see, early < held - w], dim=1)
        at = torch.cat([at, early], dim=1).clamp(0, c["cap"] - 1)
    else:
        at = torch.arange(c["cap"], device="cuda").expand(c["b"], -1)
        see = at < held
    return _out(*_attend(st["q"].to(F32), *_keys(st, at), see))


def _plain_shared(st):
    """Each group's common keys against all its queries, each sequence's own keys against its query, joined."""
    c = st["c"]
    q = st["q"].to(F32)
    hkv, d = c["hkv"], c["d"]
    parts, row = [], 0
    for size, p in zip(*_groups(c)):
        cols = -(-p // c["page"])
        names = st["tables"][row, :cols].long()
        k, v = (pool[names].reshape(cols * c["page"], hkv, d)[:p].to(F32) for pool in (st["kp"], st["vp"]))
        s = torch.einsum("bhgd,lhd->bhgl", q[row : row + size].view(size, hkv, -1, d), k).mul_(d ** -0.5)
        m = s.amax(dim=-1, keepdim=True)
        e = s.sub_(m).exp_()
        parts.append((m, e.sum(dim=-1, keepdim=True), torch.einsum("bhgl,lhd->bhgd", e, v)))
        row += size
    m0, t0, o0 = (torch.cat(x) for x in zip(*parts))
    first = torch.repeat_interleave(st["shared"].long(), torch.tensor(_groups(c)[0], device="cuda"), output_size=row)[:, None]
    at = first + torch.arange(c["own"], device="cuda")
    see = at < st["len"].long()[:, None]
    at = torch.minimum(at, st["len"].long()[:, None] - 1)
    m1, t1, o1 = _attend(q, *_keys(st, at), see)
    m = torch.maximum(m0, m1)
    w0, w1 = (m0 - m).exp(), (m1 - m).exp()
    return _out(m, t0 * w0 + t1 * w1, o0 * w0 + o1 * w1)


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    c = st["c"]
    if c["op"] == "append":
        return _exact_append(st)
    lengths = st["len"].tolist()
    b, hq, d = st["q"].shape
    o, lse = torch.zeros(b, hq, d, dtype=F64, device="cuda"), torch.full((b, hq), -math.inf, dtype=F64, device="cuda")
    window = c.get("window", 0)
    for i, n in enumerate(lengths):  # every sequence by itself, whatever it shares
        names = st["tables"][i, : -(-n // c["page"])].long()
        k, v = (x.index_select(0, names).flatten(0, 1)[:n].to(F64).permute(1, 0, 2) for x in (st["kp"], st["vp"]))
        j = torch.arange(n, device="cuda")
        s = st["q"][i].to(F64).view(c["hkv"], -1, d) @ k.transpose(1, 2) / math.sqrt(d)  # [KV head, query head, key]
        if window:
            s = s.masked_fill((j < n - window) & (j >= c["sinks"]), -math.inf)
        lse[i] = torch.logsumexp(s, -1).flatten()
        o[i] = (torch.softmax(s, -1) @ v).view(hq, d)
    return {"o": o, "lse": lse}


def _exact_append(st):
    c = st["c"]
    out = {"q": st["q"].to(F64), "k_pages": st["kp"].to(F64), "v_pages": st["vp"].to(F64)}
    q, k, v = (st[x].reshape(-1, st[x].shape[2], c["d"]).to(F64) for x in ("q", "k", "v"))
    tables = st["tables"].tolist()
    row = 0
    for names, n, m in zip(tables, st["len"].tolist(), _counts(c)):
        place = torch.arange(n - m, n, device="cuda")
        turn = torch.polar(torch.ones((), dtype=F64, device="cuda"), place[:, None, None].to(F64) * st["freq"].cuda())
        at = (torch.tensor(names, device="cuda")[torch.div(place, c["page"], rounding_mode="floor")], place % c["page"])
        out["k_pages"][at] = _exact_turn(k[row : row + m], turn, c)
        out["v_pages"][at] = v[row : row + m]
        out["q"].view(-1, c["hq"], c["d"])[row : row + m] = _exact_turn(q[row : row + m], turn, c)
        row += m
    return out


def _exact_turn(x, turn, c):
    """The rotated pairs as complex numbers times e^(i angle)."""
    r = x[..., : c["rot"]]
    half = c["layout"] == "half"
    z = torch.complex(*r.unflatten(-1, (2, -1)).unbind(-2)) if half else torch.view_as_complex(r.unflatten(-1, (-1, 2)).contiguous())
    z = z * turn
    r = torch.cat([z.real, z.imag], -1) if half else torch.view_as_real(z).flatten(-2)
    return torch.cat([r, x[..., c["rot"] :]], -1)


# ---------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "append":
        tokens = c["n"] if c["ragged"] else c["b"] * c["n"]
        # every row is read once and written once
        return {"bytes": 4.0 * tokens * (c["hq"] + 2 * c["hkv"]) * c["d"],
                "flops": 3.0 * tokens * (c["hq"] + c["hkv"]) * c["rot"]}
    if c["op"] == "paged":
        b, lengths = c["b"], _paged_lengths(c)
        if c["window"]:
            lengths = [min(n, c["window"]) + min(c["sinks"], max(0, n - c["window"])) for n in lengths]
        read = seen = sum(lengths)
    else:
        b, lengths = sum(_groups(c)[0]), _shared_lengths(c)
        seen = sum(lengths)
        read = seen - sum((size - 1) * p for size, p in zip(*_groups(c)))
    return {"bytes": 4.0 * read * c["hkv"] * c["d"] + 4.0 * b * c["hq"] * c["d"] + 4.0 * b * c["hq"],
            "flops": 4.0 * seen * c["hq"] * c["d"]}

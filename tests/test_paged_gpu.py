"""The paged cache (cpattn_append_paged, cpattn_decode_paged,
cpattn_decode_shared) against the CPU fp64 oracle, every element.

Tolerances. Rotated rows: one rounding to bf16 (u |y|, u = 2^-8), and before it
fp32: products and their sum (3 roundings of 2^-24 of |a| + |b|), a phase that
is within 2^-25 turn (2 pi 2^-25 < 2^-22 of |a| + |b|) and cosines of a few ulp:
under 2^-20 (|a| + |b|) together, times the magnitude. Attention: as for
cpattn_decode (P rounded before P V, u sum_j P_j |v_j|; parts, the group's and
the sequence's own among them, are joined in fp32; the output rounded once more,
u |o|; fp32 sums and exponentials under 1/16 of the first). LSE: 1e-4 (scores are
off by at most 2^-17 sum |q k| scale, below 5e-5 here).
"""
import ctypes

import pytest
import torch

import context_blockwise_causal_gb300 as pkg
import oracle
from context_blockwise_causal_gb300 import cpattn_append_paged, cpattn_decode_paged, cpattn_decode_shared

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
NAN = float("nan")
PAGE_BIT = 1 << 17


def _randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32)


def _pools(pages, size, hkv, d, heads_first, seed):
    """Host pools, and device ones of the layout."""
    k, v = _randn(pages, size, hkv, d, seed=seed), _randn(pages, size, hkv, d, seed=seed + 1)
    return k, v, _device(k, heads_first), _device(v, heads_first)


def _device(x, heads_first):
    x = x.cuda()
    return x.transpose(1, 2).contiguous().transpose(1, 2) if heads_first else x


def _tables(b, cols, pages, seed):
    return torch.randperm(pages, generator=torch.Generator().manual_seed(seed))[: b * cols].view(b, cols).to(torch.int32)


def _status():
    st = ctypes.c_int(0)
    pkg.library().cpattn_device_status(None, ctypes.byref(st))
    return st.value


def _close(got, ref, bound):
    off = (got.double().cpu() - ref).abs()
    assert (off <= bound).all(), (off - bound).max().item()


def _pair_mass(x, rot, layout):
    """|a| + |b| of each feature's pair (0 where it passes)."""
    a = x.double().abs()
    out = torch.zeros_like(a)
    h = rot // 2
    if layout == "half":
        s = a[..., :h] + a[..., h:rot]
        out[..., :h], out[..., h:rot] = s, s
    else:
        s = a[..., 0:rot:2] + a[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = s, s
    return out


def _rotated(got, ref, x, rot, layout, magnitude):
    mass = _pair_mass(x, rot, layout)
    _close(got, ref, U * ref.abs() * (mass > 0) + magnitude * 2.0 ** -20 * mass)


# ---------------------------------------------------------------- append
APPEND = [
    # counts, lengths, dense, hq, hkv, d, rot, layout, size, cols, heads_first
    ([1], [1], True, 1, 1, 64, 64, "half", 16, 1, False),
    ([1] * 5, [1, 16, 17, 95, 96], True, 4, 2, 128, 128, "half", 16, 6, False),
    ([7] * 3, [7, 33, 100], True, 6, 2, 64, 32, "interleaved", 48, 3, True),
    ([200], [333], True, 8, 8, 128, 96, "interleaved", 80, 5, False),      # one head to a group, pages of 80
    ([3, 0, 50, 1, 17], [3, 40, 90, 64, 17], False, 10, 2, 64, 48, "half", 32, 3, False),
    ([1] * 70, [i % 60 + 1 for i in range(70)], False, 3, 1, 128, 128, "half", 64, 1, True),  # more than 32 offsets
    ([5, 2], [5, 2000], False, 0, 4, 128, 128, "half", 128, 16, False),    # no queries
    ([400], [1 << 20], True, 2, 1, 64, 64, "half", 256, 4096, False),      # far positions
]


@pytest.mark.parametrize("counts,lengths,dense,hq,hkv,d,rot,layout,size,cols,heads_first", APPEND)
def test_append_all_elements(counts, lengths, dense, hq, hkv, d, rot, layout, size, cols, heads_first):
    b, rows = len(counts), sum(counts)
    far = cols > 1000  # a table of many pages over a small pool: the pages used are the last ones
    pages = 12 if far else b * cols + 2
    tables = torch.full((b, cols), -1, dtype=torch.int32)
    if far:
        tables[0, -5:] = _i32([3, 7, 1, 0, 9])
    else:
        tables = _tables(b, cols, pages, 5)
    kp, vp, kd, vd = _pools(pages, size, hkv, d, heads_first, 1)
    qkv = _randn(rows, hq + 2 * hkv, d, seed=3)
    q, k, v = qkv.split([hq, hkv, hkv], dim=1)
    freq = pkg.cpattn_rope_frequencies(rot, 500000.0)
    mag = 1.25
    dev = qkv.cuda().view(*((b, counts[0]) if dense else (1, rows)), hq + 2 * hkv, d)
    qd, kn, vn = dev.split([hq, hkv, hkv], dim=2)
    cu = None if dense else _i32([0] + list(torch.tensor(counts).cumsum(0))).cuda()
    out = cpattn_append_paged(kn, vn, kd, vd, tables.cuda(), _i32(lengths).cuda(), cu_tokens=cu, q=qd if hq else None,
                              inv_freq=freq, layout=layout, magnitude=mag)
    torch.cuda.synchronize()
    assert _status() == 0
    rq, rk, rv, written, kept = oracle.append_tokens(k, v, q if hq else None, kp, vp, tables.tolist(), lengths, counts, freq,
                                                     layout, magnitude=mag)
    assert kept.all() and written.sum() == rows
    # what was not written keeps its bits, values are copied, keys are rotated
    got_k, got_v = kd.cpu(), vd.cpu()
    assert torch.equal(got_k[~written], kp[~written]) and torch.equal(got_v[~written], vp[~written])
    assert torch.equal(got_v[written].double(), rv[written])
    src = torch.zeros(pages, size, hkv, d, dtype=torch.float64)
    src = oracle.append_tokens(k, v, None, src, src, tables.tolist(), lengths, counts)[1]  # the keys before they turn
    _rotated(got_k[written], rk[written], src[written], rot, layout, mag)
    if hq:
        _rotated(out.view(rows, hq, d), rq, q, rot, layout, mag)
        assert torch.equal(dev.cpu().view(rows, -1, d), qkv)  # the projection itself is left alone
    else:
        assert out is None


def test_append_what_has_no_place_is_left_out():
    """Padded rows (length 0), more new tokens than a sequence holds, places past
    the table, rows around the offsets: keys are dropped, queries of no sequence
    stay as they were."""
    size, cols, hq, hkv, d = 16, 2, 2, 1, 64
    kp, vp, kd, vd = _pools(9, size, hkv, d, False, 11)
    counts, lengths = [1, 4, 3, 2], [0, 2, 34, -7]
    tables = _tables(4, cols, 9, 12)
    rows = 3 + sum(counts) + 5  # three before the first sequence, five behind the last
    k, v, q = _randn(rows, hkv, d, seed=13), _randn(rows, hkv, d, seed=14), _randn(rows, hq, d, seed=15)
    cu = _i32([3, 4, 8, 11, 13])
    mark = torch.full((1, rows, hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
    out = cpattn_append_paged(k.cuda()[None], v.cuda()[None], kd, vd, tables.cuda(), _i32(lengths).cuda(), cu_tokens=cu.cuda(),
                              q=q.cuda()[None], q_out=mark)
    assert out is mark
    torch.cuda.synchronize()
    assert _status() == 0
    freq = pkg.cpattn_rope_frequencies(d)
    rq, rk, rv, written, kept = oracle.append_tokens(k[3:13], v[3:13], q[3:13], kp, vp, tables.tolist(), lengths, counts, freq)
    assert kept.sum() == 2 + 1  # two of the four, one of the three (places 31, 32, 33 of 32)
    got_k, got_v = kd.cpu(), vd.cpu()
    assert torch.equal(got_k[~written], kp[~written]) and torch.equal(got_v.double(), rv)
    _close(got_k[written], rk[written], U * rk[written].abs() + 2.0 ** -20 * 16)
    assert (mark[0, :3] == 3.0).all() and (mark[0, 13:] == 3.0).all()
    _rotated(mark[0, 3:13], rq, q[3:13], d, "half", 1.0)


def test_append_copies_bits_and_takes_positions_and_queries_in_place():
    size, hq, hkv, d, b, n = 32, 4, 2, 128, 3, 9
    kp, vp, kd, vd = _pools(8, size, hkv, d, False, 21)
    tables, lengths = _tables(b, 2, 8, 22), [9, 33, 64]
    k, v, q = _randn(b, n, hkv, d, seed=23), _randn(b, n, hkv, d, seed=24), _randn(b, n, hq, d, seed=25)
    k.view(torch.int16)[0, 0, 0, :4] = torch.tensor([0x7fc1, -1, 0x7f80, -0x8000], dtype=torch.int16)  # NaNs, inf, -0
    args = (k.cuda(), v.cuda(), kd, vd, tables.cuda(), _i32(lengths).cuda())
    qd = q.cuda()
    assert cpattn_append_paged(*args, q=qd, rotate=False, q_out=qd) is qd
    torch.cuda.synchronize()
    assert torch.equal(qd.cpu(), q)
    for i in range(b):
        got = oracle.held_tokens(kd.cpu(), tables[i], lengths[i])[lengths[i] - n:]
        assert torch.equal(got.view(torch.int16), k[i].view(torch.int16))
        assert torch.equal(oracle.held_tokens(vd.cpu(), tables[i], lengths[i])[lengths[i] - n:], v[i])
    # explicit positions, shared by all sequences and one row each; the queries in place
    k = _randn(b, n, hkv, d, seed=26)
    for pos in (torch.arange(n) * 1000 + 5, torch.randint(-2 ** 31, 2 ** 31 - 1, (b, n), generator=torch.Generator().manual_seed(1))):
        qd = q.cuda()
        cpattn_append_paged(k.cuda(), *args[1:], q=qd, q_out=qd, positions=pos.to(torch.int32).cuda(), base=500000.0)
        freq = pkg.cpattn_rope_frequencies(d, 500000.0)
        full = pos if pos.dim() == 2 else pos[None].expand(b, n)
        # the oracle's own angles in fp64 lose 2^-53 of |pos|: 2^-22 at the ends of int32
        ref = oracle.rotate(q, full, freq)
        _rotated(qd, ref, q, d, "half", 1.0)
        ref = oracle.rotate(k, full, freq)
        for i in range(b):
            got = oracle.held_tokens(kd.cpu(), tables[i], lengths[i])[lengths[i] - n:]
            _rotated(got, ref[i], k[i], d, "half", 1.0)


def test_append_bad_pages_are_not_followed():
    size, hkv, d = 16, 2, 64
    kp, vp, kd, vd = _pools(4, size, hkv, d, False, 31)
    tables = _i32([[0, -1], [1 << 30, 2], [3, 4]])
    k = _randn(3, 20, hkv, d, seed=32)
    assert _status() == 0
    cpattn_append_paged(k.cuda(), k.cuda(), kd, vd, tables.cuda(), _i32([20, 20, 20]).cuda())
    torch.cuda.synchronize()
    assert _status() == PAGE_BIT
    written = oracle.append_tokens(k.flatten(0, 1), k.flatten(0, 1), None, kp, vp, tables.tolist(), [20] * 3, [20] * 3)[3]
    assert written.sum() == 16 + 4 + 16
    assert torch.equal(kd.cpu()[~written], kp[~written]) and not torch.equal(kd.cpu()[written], kp[written])


# ---------------------------------------------------------------- decode
def _check(q, k, v, tables, lengths, window, sinks, scale, o, lse, k_close=None):
    cap = tables.shape[1] * k.shape[1]
    for i, n in enumerate(lengths):
        n = min(max(n, 0), cap)
        kk, vv = oracle.held_tokens(k, tables[i], n), oracle.held_tokens(v, tables[i], n)
        ref, l_ref, err = oracle.decode_attention(q[i], kk, vv, n, window, sinks, scale)
        got = o[i].double().cpu()
        off = (got - ref).abs()
        assert (off <= err * (1 + 1 / 16) + U * ref.abs() + 1e-6).all(), (i, n, off.max().item())
        if n == 0:
            assert (got == 0).all() and (lse[i] == float("-inf")).all()
        else:
            assert (lse[i].double().cpu() - l_ref).abs().max().item() <= 1e-4, (i, n)


def _hide(kd, vd, tables, lengths, window, sinks):
    """Device copies of the pools in which everything that no sequence sees is NaN or infinite."""
    seen = torch.zeros(kd.shape[:2], dtype=torch.bool)
    size = kd.shape[1]
    for table, n in zip(tables.tolist(), lengths):
        n = min(max(n, 0), len(table) * size)
        for t in range(n):
            if not window or t >= n - window or t < sinks:
                if 0 <= table[t // size] < kd.shape[0]:
                    seen[table[t // size], t % size] = True
    m = ~seen.cuda()[:, :, None, None]
    return kd.masked_fill(m, NAN), vd.masked_fill(m, float("inf"))


PAGED = [
    # lengths, size, cols, hq, hkv, d, window, sinks, scale, heads_first
    ([1], 16, 1, 1, 1, 128, 0, 0, None, False),
    ([0, 1, 2, 15, 16, 17, 63, 64, 65, 200], 16, 13, 4, 2, 128, 0, 0, None, False),
    ([0, 1, 2, 15, 16, 17, 63, 64, 65, 200], 48, 5, 8, 1, 64, 16, 0, None, True),
    ([200, 199, 150, 20, 19, 18, 17, 3], 32, 7, 8, 8, 64, 16, 4, None, False),     # one head per group
    ([1000, 900, 17], 80, 13, 24, 2, 128, 100, 30, 0.3, False),                     # 12 heads per group, 30 first tokens
    ([700, 33], 64, 11, 40, 1, 64, 0, 0, None, True),                              # 40 heads per group: three row tiles
    ([5000], 128, 40, 4, 2, 128, 0, 0, None, False),                               # one sequence over many runs
    ([5000, 1], 256, 20, 4, 2, 64, 4001, 5, None, False),                          # an odd window, a sequence shorter than the runs
    ([40000], 1024, 40, 4, 1, 128, 0, 0, None, False),                             # more runs than a cluster has CTAs
    ([36000, 0, 3], 512, 79, 4, 1, 64, 35000, 4, None, False),
    ([300, 300], 16, 19, 2, 1, 128, 1, 0, None, False),                            # a window of the new token alone
    ([300, 2], 16, 19, 2, 1, 128, 1, 500, None, True),                             # every key a first token
    ([20, 37, 30], 16, 3, 2, 1, 64, 12, 9, None, False),                           # first tokens and window in one block
    ([777] * 90, 64, 13, 16, 8, 64, 500, 1, None, False),                          # more sequences than places
]


@pytest.mark.parametrize("lengths,size,cols,hq,hkv,d,window,sinks,scale,heads_first", PAGED)
def test_decode_all_elements_and_what_is_not_seen(lengths, size, cols, hq, hkv, d, window, sinks, scale, heads_first):
    b = len(lengths)
    pages = b * cols + 1
    k, v, kd, vd = _pools(pages, size, hkv, d, heads_first, 41)
    tables = _tables(b, cols, pages, 43)
    q = _randn(b, hq, d, seed=44)
    kd, vd = _hide(kd, vd, tables, lengths, window, sinks)
    # entries past a sequence's length, or wholly behind its window, are never followed
    free = tables.clone()
    for i, n in enumerate(lengths):
        free[i, -(-n // size):] = -1
        if window:
            free[i, -(-sinks // size):max(0, n - window) // size] = 1 << 30
    ln = _i32(lengths).cuda()
    o = torch.full((b, hq, d), NAN, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b, hq), NAN, device="cuda")
    cpattn_decode_paged(q.cuda(), kd, vd, free.cuda(), ln, window, sinks, scale, o=o, lse=lse)
    torch.cuda.synchronize()
    assert _status() == 0
    _check(q, k, v, tables, lengths, window, sinks, scale, o, lse)
    # queries inside wider rows, tables inside wider ones, another page order: the same bits
    wide = torch.zeros(b, hq + 3, d, dtype=torch.bfloat16, device="cuda")
    wide[:, :hq] = q.cuda()
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(9))
    back = torch.empty_like(order)
    back[order] = torch.arange(pages)
    moved = torch.full((b, cols + 2), -5, dtype=torch.int32)
    moved[:, :cols] = torch.where((free >= 0) & (free < pages), back[free.clamp(0, pages - 1).long()].to(torch.int32), free)
    o2, l2 = cpattn_decode_paged(wide[:, :hq], kd[order.cuda()], vd[order.cuda()], moved.cuda()[:, :cols], ln, window, sinks, scale)
    assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_decode_lengths_are_clamped_and_bad_pages_count_as_zeros():
    k, v, kd, vd = _pools(9, 16, 1, 64, False, 51)
    tables = _i32([[0, 1, 2], [3, 4, 5], [6, 99, -1]])
    q = _randn(3, 2, 64, seed=53)
    assert _status() == 0
    lengths = [-5, 1 << 30, 40]
    o, lse = cpattn_decode_paged(q.cuda(), kd, vd, tables.cuda(), _i32(lengths).cuda())
    torch.cuda.synchronize()
    assert _status() == PAGE_BIT
    _check(q, k, v, tables, lengths, 0, 0, None, o, lse)


# ---------------------------------------------------------------- shared
def _group_state(groups, prefix, own, size, hq, hkv, d, heads_first, seed, copies=True):
    """Pools, tables and lengths of groups that begin alike; own[i]: further
    tokens of sequence i. Whole pages of common tokens are shared, the page
    that they end in is copied."""
    b = sum(groups)
    lengths = [p + own[i] for i, p in enumerate(x for g, p in zip(groups, prefix) for x in [p] * g)]
    cols = max(1, max(-(-n // size) for n in lengths))
    whole = [p // size for p in prefix]
    pages = sum(whole) + b * cols + 2
    k, v = _randn(pages, size, hkv, d, seed=seed), _randn(pages, size, hkv, d, seed=seed + 1)
    name = torch.randperm(pages, generator=torch.Generator().manual_seed(seed + 2)).to(torch.int32).tolist()
    tables = torch.full((b, cols), -1, dtype=torch.int32)
    row = 0
    for g, p, w in zip(groups, prefix, whole):
        common = [name.pop() for _ in range(w)]
        for j in range(g):
            mine = [name.pop() for _ in range(-(-lengths[row + j] // size) - w)]
            tables[row + j, :w + len(mine)] = _i32(common + mine)
            rest = p - w * size
            if j and rest:
                first = tables[row, w]
                k[mine[0], :rest], v[mine[0], :rest] = k[first, :rest], v[first, :rest]
        row += g
    offsets = _i32([0] + list(torch.tensor(groups).cumsum(0)))
    return k, v, tables, lengths, offsets


SHARED = [
    # groups, prefix, own, size, hq, hkv, d, scale, heads_first
    ([1], [1], [0], 16, 1, 1, 64, None, False),
    ([2], [5], [1, 3], 16, 4, 2, 128, None, False),
    ([3], [127], [0, 1, 40], 32, 4, 2, 128, None, True),
    ([3], [128], [17, 0, 129], 64, 4, 2, 64, None, False),
    ([3], [129], [1, 2, 3], 48, 6, 2, 128, 0.2, False),
    ([5], [1000], [33, 100, 1, 0, 260], 80, 8, 8, 64, None, False),          # one head per group: 5 rows
    ([32], [700], list(range(32)), 16, 4, 1, 128, None, False),              # exactly 128 rows
    ([33], [700], list(range(33)), 128, 4, 1, 64, None, False),              # two row tiles, 4 rows in the second
    ([43], [515], [i % 7 for i in range(43)], 256, 6, 1, 128, None, True),    # 258 rows: two units
    ([2], [300], [50, 60], 16, 300, 1, 64, None, False),                     # 300 heads to a KV head: 600 rows
    ([3, 1, 2], [400, 0, 77], [1, 9, 30, 300, 1, 2], 32, 6, 2, 64, None, False),
    ([9, 30, 1, 2], [2049, 130, 1, 4000], [i % 40 for i in range(42)], 64, 16, 2, 128, None, False),
    ([2] * 40, [(i * 37) % 300 for i in range(40)], [i % 3 for i in range(80)], 16, 4, 4, 64, None, False),  # more groups than a warp has lanes
    ([2], [30000], [10, 3], 512, 4, 1, 128, None, False),                    # one unit over the whole chip
    # the same edges with more than 32 rows to a group
    ([9], [1], [0, 1, 15, 16, 17, 2, 3, 4, 5], 16, 8, 1, 64, None, False),
    ([9], [127], [0, 1, 15, 16, 17, 2, 3, 4, 5], 32, 16, 2, 128, None, True),
    ([9], [128], [0, 1, 15, 16, 17, 2, 3, 4, 5], 64, 16, 2, 64, None, False),
    ([9], [129], [0, 1, 15, 16, 17, 2, 3, 4, 5], 48, 12, 2, 128, 0.2, False),
    ([9], [257], [0, 1, 15, 16, 17, 2, 3, 4, 5], 144, 8, 1, 128, None, False),  # three tiles, pages of 144
    ([20, 1, 0, 12], [400, 0, 50, 77], [i % 33 for i in range(33)], 32, 6, 2, 64, None, False),  # an empty group
    ([2], [30000], [10, 3], 512, 17, 1, 64, None, False),
    ([9] * 33, [(i * 37) % 300 for i in range(33)], [i % 3 for i in range(297)], 16, 4, 1, 64, None, False),
    ([8], [2000], [i * 90 for i in range(8)], 128, 4, 1, 128, None, False),      # exactly 32 rows
    ([9] * 20, [(i * 97) % 500 for i in range(20)], [i % 5 for i in range(180)], 32, 16, 4, 64, None, False),  # more units than half of the SMs
    ([120], [600], [i % 70 for i in range(120)], 64, 16, 2, 128, None, False),   # 960 rows: three units and three quarters
    # and with more than 64
    ([9], [129], [0, 1, 15, 16, 17, 2, 3, 4, 5], 48, 32, 2, 128, 0.2, False),
    ([40, 1, 0, 33], [400, 0, 50, 77], [i % 33 for i in range(74)], 32, 6, 2, 64, None, False),
    ([2], [30000], [10, 3], 512, 33, 1, 64, None, False),
    ([9] * 33, [(i * 37) % 300 for i in range(33)], [i % 3 for i in range(297)], 16, 8, 1, 64, None, False),
    ([9] * 20, [(i * 97) % 500 for i in range(20)], [i % 5 for i in range(180)], 32, 32, 4, 64, None, False),
    ([13], [9000], [i * 7 for i in range(13)], 64, 40, 8, 128, None, False),     # 65 rows
    ([16], [9000], [i * 7 for i in range(16)], 64, 32, 8, 128, None, True),      # 64 rows, many keys
]


@pytest.mark.parametrize("groups,prefix,own,size,hq,hkv,d,scale,heads_first", SHARED)
def test_shared_all_elements_and_what_is_not_seen(groups, prefix, own, size, hq, hkv, d, scale, heads_first):
    k, v, tables, lengths, offsets = _group_state(groups, prefix, own, size, hq, hkv, d, heads_first, 61)
    b = len(lengths)
    q = _randn(b, hq, d, seed=64)
    kd, vd = _hide(_device(k, heads_first), _device(v, heads_first), tables, lengths, 0, 0)
    ln, sh = _i32(lengths).cuda(), _i32(prefix).cuda()
    off = offsets.cuda() if len(groups) > 1 else None
    o = torch.full((b, hq, d), NAN, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b, hq), NAN, device="cuda")
    cpattn_decode_shared(q.cuda(), kd, vd, tables.cuda(), ln, sh, group_offsets=off, max_group=max(groups), scale=scale, o=o, lse=lse)
    torch.cuda.synchronize()
    assert _status() == 0
    _check(q, k, v, tables, lengths, 0, 0, scale, o, lse)
    # again, with a workspace full of NaN and the queries in wider rows: the same bits
    need = pkg.cpattn_decode_shared_workspace_bytes(b, hq, hkv, d, len(groups), max(groups))
    ws = torch.full((need // 4 + 4,), NAN, device="cuda")[4:]  # 16-byte aligned, no more
    wide = torch.zeros(b, hq + 3, d, dtype=torch.bfloat16, device="cuda")
    wide[:, :hq] = q.cuda()
    o2, l2 = cpattn_decode_shared(wide[:, :hq], kd, vd, tables.cuda(), ln, sh, group_offsets=off, max_group=max(groups),
                                  scale=scale, workspace=ws)
    assert torch.equal(o, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("hq,hkv", [(4, 2), (20, 2), (40, 2)])
def test_shared_members_that_do_not_share(hq, hkv):
    """Finished sequences (length 0, a cleared table), sequences with fewer tokens
    than the group, behind max_group others, outside of every group."""
    groups, prefix, size, d = [4, 5], [300, 200], 32, 128
    k, v, tables, lengths, _ = _group_state(groups + [2], prefix + [40], [20, 5, 0, 60, 1, 2, 3, 4, 5, 7, 9], size, hq, hkv, d, False, 71)
    lengths[0], lengths[1], lengths[6] = 0, 100, 199
    tables[0] = -1  # the first member's table is gone
    q = _randn(11, hq, d, seed=74)
    # group 0 begins at sequence 0; sequences 9 and 10 are in no group; max_group leaves out sequence 8
    kd, vd = _hide(k.cuda(), v.cuda(), tables, lengths, 0, 0)
    o, lse = cpattn_decode_shared(q.cuda(), kd, vd, tables.cuda(), _i32(lengths).cuda(), _i32(prefix).cuda(),
                                  group_offsets=_i32([0, 4, 9]).cuda(), max_group=4)
    torch.cuda.synchronize()
    assert _status() == 0
    _check(q, k, v, tables, lengths, 0, 0, None, o, lse)
    # counts out of range are clamped; nobody holds as many tokens as the table has room for, so nobody shares
    for counts in ([-3, 1 << 30], [0, 0]):
        o, lse = cpattn_decode_shared(q.cuda(), kd, vd, tables.cuda(), _i32(lengths).cuda(), _i32(counts).cuda(),
                                      group_offsets=_i32([0, 4, 9]).cuda(), max_group=5)
        torch.cuda.synchronize()
        _check(q, k, v, tables, lengths, 0, 0, None, o, lse)
    # offsets outside of the batch
    o, lse = cpattn_decode_shared(q.cuda(), kd, vd, tables.cuda(), _i32(lengths).cuda(), _i32(prefix).cuda(),
                                  group_offsets=_i32([-2, 0, 500]).cuda(), max_group=11)
    torch.cuda.synchronize()
    assert o.isfinite().all()


@pytest.mark.parametrize("hq", [4, 24, 60])
def test_shared_bad_pages_count_as_zeros(hq):
    k, v, tables, lengths, _ = _group_state([3], [200], [5, 6, 7], 32, hq, 2, 64, False, 81)
    tables[:, 2] = 1 << 30
    tables[:, 4] = -2
    q = _randn(3, hq, 64, seed=84)
    assert _status() == 0
    o, lse = cpattn_decode_shared(q.cuda(), k.cuda(), v.cuda(), tables.cuda(), _i32(lengths).cuda(), _i32([200]).cuda())
    torch.cuda.synchronize()
    assert _status() == PAGE_BIT
    _check(q, k, v, tables, lengths, 0, 0, None, o, lse)


def test_shared_peaky_rows():
    """Rows that one key dominates, in the common part and in the own one."""
    k, v, tables, lengths, _ = _group_state([40], [900], [30] * 40, 64, 8, 1, 128, False, 91)
    q = (_randn(40, 8, 128, seed=94).float() * 12).to(torch.bfloat16)
    o, lse = cpattn_decode_shared(q.cuda(), k.cuda(), v.cuda(), tables.cuda(), _i32(lengths).cuda(), _i32([900]).cuda())
    for i, n in enumerate(lengths):
        ref, l_ref, err = oracle.decode_attention(q[i], oracle.held_tokens(k, tables[i], n), oracle.held_tokens(v, tables[i], n), n)
        assert ((o[i].double().cpu() - ref).abs() <= err * (1 + 1 / 16) + U * ref.abs() + 1e-6).all(), i
        # scores up to about 12 * 4 * sqrt(128) / sqrt(128): fp32 products and sums, 2^-17 sum |q k| scale
        bound = 2.0 ** -17 * (q[i].double().abs() @ oracle.held_tokens(k, tables[i], n)[:, 0].double().abs().T).amax() / 128 ** 0.5
        assert (lse[i].double().cpu() - l_ref).abs().max() <= 1e-4 + bound


# ---------------------------------------------------------------- together
def test_a_server_appends_and_decodes():
    """Prompts of two lengths go into the pages, three answers each go on from
    them for some tokens: a captured step (append with the rotation, shared and
    plain attention) is replayed while lengths grow, and every step is what the
    oracle makes of the tokens so far."""
    size, cols, hq, hkv, d, steps = 16, 6, 4, 2, 64, 20
    prompts, answers = [41, 50], 3
    b = len(prompts) * answers
    gen = torch.Generator().manual_seed(101)
    freq = pkg.cpattn_rope_frequencies(d, 500000.0)
    kd, vd = (torch.full((b * cols, size, hkv, d), NAN, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tables = torch.arange(b * cols, dtype=torch.int32).view(b, cols)
    heads = torch.randn(sum(prompts), hq + 2 * hkv, d, generator=gen).to(torch.bfloat16)
    firsts = [0, answers]
    prow = heads.cuda()[None].split([hq, hkv, hkv], dim=2)
    cpattn_append_paged(prow[1], prow[2], kd, vd, tables[firsts].cuda(), _i32(prompts).cuda(),
                        cu_tokens=_i32([0, prompts[0], sum(prompts)]).cuda(), inv_freq=freq)
    for g, p in enumerate(prompts):  # the others share its whole pages and copy the last one
        w = p // size
        for j in range(1, answers):
            tables[g * answers + j, :w] = tables[g * answers, :w]
            for pool in (kd, vd):
                pool[int(tables[g * answers + j, w])] = pool[int(tables[g * answers, w])]
    td = tables.cuda()
    ln = _i32([p for p in prompts for _ in range(answers)]).cuda()
    new = torch.empty(b, 1, hq + 2 * hkv, d, dtype=torch.bfloat16, device="cuda")
    shared, off = _i32(prompts).cuda(), _i32([0, 3, 6]).cuda()

    def step():
        q, k, v = new.split([hq, hkv, hkv], dim=2)
        ln.add_(1)
        q = cpattn_append_paged(k, v, kd, vd, td, ln, q=q, inv_freq=freq)[:, 0]
        return q, cpattn_decode_shared(q, kd, vd, td, ln, shared, group_offsets=off, max_group=answers), cpattn_decode_paged(q, kd, vd, td, ln, 20, 3)

    rows = [torch.randn(b, 1, hq + 2 * hkv, d, generator=gen).to(torch.bfloat16) for _ in range(steps)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        new.copy_(rows[0])
        step()
        ln.sub_(1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, (o, lse), (ow, lw) = step()
    for t in range(steps):
        new.copy_(rows[t])
        graph.replay()
        torch.cuda.synchronize()
        lengths = [p + t + 1 for p in prompts for _ in range(answers)]
        assert ln.tolist() == lengths and _status() == 0
        kh, vh, qh = kd.cpu(), vd.cpu(), q.cpu()
        if t in (0, 6, steps - 1):
            _check(qh, kh, vh, tables, lengths, 0, 0, None, o, lse)
            _check(qh, kh, vh, tables, lengths, 20, 3, None, ow, lw)
    # every token is where it belongs
    for i in range(b):
        g, p = i // answers, prompts[i // answers]
        src = torch.cat([heads[sum(prompts[:g]):sum(prompts[:g]) + p]] + [r[i] for r in rows])
        n = p + steps
        assert torch.equal(oracle.held_tokens(vh, tables[i], n), src[:, hq + hkv:])
        ref = oracle.rotate(src[None, :, hq:hq + hkv], torch.arange(n), freq)[0]
        _rotated(oracle.held_tokens(kh, tables[i], n), ref, src[:, hq:hq + hkv], d, "half", 1.0)


@pytest.mark.parametrize("hq", [8, 24, 48])
def test_given_streams_and_calls_at_once(hq):
    k, v, tables, lengths, off = _group_state([3, 4], [900, 1300], [5, 50, 500, 1, 2, 3, 4], 32, hq, 2, 64, False, 111)
    q, kd, vd, td, ln = _randn(7, hq, 64, seed=114).cuda(), k.cuda(), v.cuda(), tables.cuda(), _i32(lengths).cuda()
    kw = {"group_offsets": off.cuda(), "max_group": 4}
    counts = [_i32([900, 1300]).cuda(), _i32([33, 1024]).cuda()]
    want = [cpattn_decode_shared(q, kd, vd, td, ln, c, **kw) for c in counts]
    want += [cpattn_decode_paged(q, kd, vd, td, ln, w, 4) for w in (100, 0)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(5):
        got = [cpattn_decode_shared(q, kd, vd, td, ln, c, stream=s, **kw) for c, s in zip(counts, streams)]
        got += [cpattn_decode_paged(q, kd, vd, td, ln, w, 4, stream=s) for w, s in zip((100, 0), streams[2:])]
        torch.cuda.synchronize()
        for w, g in zip(want, got):
            assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


@pytest.mark.parametrize("b", [7, 40])
def test_shared_calls_one_after_another_on_one_workspace(b):
    """Each call's later kernels are placed while its first one runs; each call
    takes the one before's output as its queries."""
    k, v, tables, lengths, _ = _group_state([b], [3000], [i * 5 for i in range(b)], 64, 8, 2, 128, False, 121)
    kd, vd, td, ln = k.cuda(), v.cuda(), tables.cuda(), _i32(lengths).cuda()
    sh = _i32([3000]).cuda()
    q = _randn(b, 8, 128, seed=124).cuda()
    ws = torch.empty(pkg.cpattn_decode_shared_workspace_bytes(b, 8, 2, 128), dtype=torch.uint8, device="cuda")

    def chain(sync):
        x, out = q, []
        for _ in range(6):
            x, lse = cpattn_decode_shared(x * 8, kd, vd, td, ln, sh, workspace=ws)
            out += [x, lse]
            if sync:
                torch.cuda.synchronize()
        return out

    want = chain(True)
    for _ in range(20):
        got = chain(False)
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(want, got))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = chain(False)
    for count in (100, 3000, 0):  # counts are read on the device
        sh.fill_(count)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(chain(True), got))


def test_pool_offsets_beyond_32_bits():
    """Pages that start over 2^31 elements into the pools."""
    size, hkv, d = 256, 8, 128
    pages = 9000  # 2.36e9 elements each
    kd, vd = (torch.zeros(pages, size, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tables = _i32([[8999, 8500], [8999, 8300]])
    n, p = [300, 290], 270
    new = _randn(2, 300, 8 + 2 * hkv, d, seed=131)
    new[1, :p] = new[0, :p]  # the tokens in common
    q, k, v = new.cuda().split([8, hkv, hkv], dim=2)
    for i in range(2):
        cpattn_append_paged(k[i:i + 1, :n[i]], v[i:i + 1, :n[i]], kd, vd, tables[i:i + 1].cuda(), _i32([n[i]]).cuda(), rotate=False)
    q1 = new[:, 299, :8].contiguous()
    host_k, host_v = new[..., 8:16, :], new[..., 16:, :]
    flat = torch.arange(2 * 2, dtype=torch.int32).view(2, 2)
    pk, pv = (torch.cat([x, x.new_zeros(2, 212, hkv, d)], 1).view(4, 256, hkv, d) for x in (host_k, host_v))
    for o, lse in (cpattn_decode_paged(q1.cuda(), kd, vd, tables.cuda(), _i32(n).cuda()),
                   cpattn_decode_shared(q1.cuda(), kd, vd, tables.cuda(), _i32(n).cuda(), _i32([p]).cuda())):
        _check(q1, pk, pv, flat, n, 0, 0, None, o, lse)


@pytest.mark.parametrize("hq", [2, 6, 8])
def test_checked_build_is_silent_and_identical(hq):
    """Groups of up to 20, 60 and 80 rows."""
    lib = pkg.checked_library()

    def status():
        st = ctypes.c_int(0)
        lib.cpattn_device_status(None, ctypes.byref(st))
        return st.value

    from test_paged_abi import Pages
    from test_operators_abi import Rotary, Rows

    groups, hkv, d, size = [3, 20, 2], 2, 128, 48
    k, v, tables, lengths, off = _group_state(groups, [333, 1000, 5], [i % 9 for i in range(25)], size, hq, hkv, d, False, 141)
    b = 25
    q, kd, vd, td, ln = _randn(b, hq, d, seed=144).cuda(), k.cuda(), v.cuda(), tables.cuda(), _i32(lengths).cuda()
    sh, od = _i32([333, 1000, 5]).cuda(), off.cuda()
    ptr = lambda t: t.data_ptr()  # noqa: E731

    def pg(kt, vt):
        s = (size * hkv * d, hkv * d, d)
        return Pages(ptr(kt), ptr(vt), kt.shape[0], size, tables.shape[1], ptr(td), tables.shape[1], *s, *s)

    for window, sinks in ((0, 0), (128, 4)):
        o, lse = cpattn_decode_paged(q, kd, vd, td, ln, window, sinks)
        o2, l2 = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
        rc = lib.cpattn_decode_paged(ptr(q), pg(kd, vd), ptr(ln), ptr(o2), ptr(l2), None, 0, b, hq, hkv, d, hq * d, window, sinks,
                                     0.0, None)
        assert rc == 0 and status() == 0
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    o, lse = cpattn_decode_shared(q, kd, vd, td, ln, sh, group_offsets=od, max_group=20)
    o2, l2 = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
    need = lib.cpattn_decode_shared_workspace_bytes(b, hq, hkv, d, 3, 20)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    rc = lib.cpattn_decode_shared(ptr(q), pg(kd, vd), ptr(ln), ptr(sh), ptr(od), 3, 20, ptr(o2), ptr(l2), ptr(ws), need, b, hq, hkv,
                                  d, hq * d, 0.0, None)
    assert rc == 0 and status() == 0
    assert torch.equal(o, o2) and torch.equal(lse, l2)
    # new tokens
    new = _randn(b, 3, hq + 2 * hkv, d, seed=145).cuda()
    freq = pkg.cpattn_rope_frequencies(d)
    parts = new.split([hq, hkv, hkv], dim=2)
    k1, v1, k2, v2 = kd.clone(), vd.clone(), kd.clone(), vd.clone()
    q1 = cpattn_append_paged(parts[1], parts[2], k1, v1, td, ln, q=parts[0], inv_freq=freq)
    q2 = torch.full_like(q1, 7.0)
    row = (hq + 2 * hkv) * d
    rows = [Rows(ptr(p), 3 * row, row) for p in parts]
    plan = Rotary(0, d, 1.0, 0, 0, -1, None, 0, None, 0, freq.data_ptr())
    rc = lib.cpattn_append_paged(rows[1], rows[2], pg(k2, v2), ptr(ln), None, b, rows[0], Rows(ptr(q2), 3 * hq * d, hq * d), b, 3,
                                 hq, hkv, d, plan, None)
    assert rc == 0 and status() == 0
    assert torch.equal(q1, q2) and torch.equal(v1, v2) and torch.equal(k1, k2)


def test_refusals():
    q, pool = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(5, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    t, ln, x = _i32([[0, 1], [2, 3]]).cuda(), _i32([3, 4]).cuda(), torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    one = ln[:1]
    for call in (lambda **kw: cpattn_decode_paged(q, pool, pool, t, ln, **kw),
                 lambda **kw: cpattn_decode_shared(q, pool, pool, t, ln, one, **kw)):
        for kw in ({"scale": -1.0}, {"scale": NAN}):
            with pytest.raises(pkg.CpattnError):
                call(**kw)
    for kw in ({"window": -1}, {"sinks": -1}):
        with pytest.raises(pkg.CpattnError):
            cpattn_decode_paged(q, pool, pool, t, ln, **kw)
    for kw in ({"max_group": 0}, {"max_group": 3}, {"workspace": torch.empty(100, dtype=torch.uint8, device="cuda")}):
        with pytest.raises(pkg.CpattnError):
            cpattn_decode_shared(q, pool, pool, t, ln, one, **kw)
    with pytest.raises(pkg.CpattnError):  # 3 query heads over 2 KV heads
        cpattn_decode_paged(q[:, :3].contiguous(), pool, pool, t, ln)
    with pytest.raises(pkg.CpattnError):  # pages of 15 tokens
        cpattn_decode_paged(q, pool[:, :15], pool[:, :15], t, ln)
    with pytest.raises(pkg.CpattnError):  # one page for all: nothing could be kept in it
        cpattn_append_paged(x, x, pool[:1].expand(5, 16, 2, 64), pool, t, ln)
    with pytest.raises(pkg.CpattnError):  # every sequence the same table
        cpattn_append_paged(x, x, pool, pool, t[:1].expand(2, 2), ln)
    for call in (lambda: cpattn_decode_paged(q, pool, pool, t.long(), ln), lambda: cpattn_decode_paged(q, pool, pool.float(), t, ln),
                 lambda: cpattn_decode_paged(q, pool, pool, t, ln.long()), lambda: cpattn_append_paged(x, x.float(), pool, pool, t, ln),
                 lambda: cpattn_decode_shared(q, pool, pool, t, ln, one.long())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: cpattn_decode_paged(q, pool, pool[:4], t, ln), lambda: cpattn_decode_paged(q, pool, pool, t[:1], ln),
                 lambda: cpattn_decode_paged(q, pool, pool, t, one), lambda: cpattn_decode_paged(q[..., :32], pool, pool, t, ln),
                 lambda: cpattn_decode_paged(q, pool.transpose(2, 3), pool.transpose(2, 3), t, ln),
                 lambda: cpattn_decode_paged(q, pool, pool, t.t(), ln), lambda: cpattn_append_paged(x, x[:, :2], pool, pool, t, ln),
                 lambda: cpattn_append_paged(x, x, pool, pool, t, ln, cu_tokens=one), lambda: cpattn_append_paged(x, x, pool, pool, t, ln, cu_tokens=_i32([0, 2, 3]).cuda()),
                 lambda: cpattn_append_paged(x, x, pool, pool, t, ln, q=q[:, None, :, :].expand(2, 2, 4, 64)),
                 lambda: cpattn_append_paged(x, x, pool, pool, t, ln, q_out=x), lambda: cpattn_append_paged(x[:, :, :1], x[:, :, :1], pool, pool, t, ln),
                 lambda: cpattn_append_paged(x, x, pool, pool, t, ln, layout="other"),
                 lambda: cpattn_decode_shared(q, pool, pool, t, ln, ln), lambda: cpattn_decode_shared(q, pool, pool, t, ln, ln, group_offsets=ln)):
        with pytest.raises(ValueError):
            call()

"""A cache in pages, fp64 on the CPU. TEST INFRASTRUCTURE (see the package
docstring): what a sequence holds, read token by token through its table, and
what a call that appends leaves behind.
"""
import torch

from .qk_norm import rotate

_F64 = torch.float64


def held_tokens(pool, table, length):
    """Tokens 0 .. length - 1 of a sequence, [length, hkv, d], from a pool
    [pages, page_size, hkv, d]; those of an entry that names no page are zeros."""
    pages, size = pool.shape[:2]
    out = torch.zeros(length, *pool.shape[2:], dtype=pool.dtype)
    for t in range(length):
        page = int(table[t // size])
        if 0 <= page < pages:
            out[t] = pool[page, t % size]
    return out


def append_tokens(k, v, q, k_pool, v_pool, tables, lengths, counts, inv_freq=None, layout="half", positions=None,
                  magnitude=1.0):
    """Rows of k, v [rows, hkv, d] and q [rows, hq, d] or None, sequence after
    sequence, counts[i] of sequence i. Returns fp64 (q or None, k_pool, v_pool)
    and two bool tensors: [pages, page_size] slots written, [rows] rows whose
    sequence had a place for them."""
    k_pool, v_pool = k_pool.to(_F64).clone(), v_pool.to(_F64).clone()
    pages, size = k_pool.shape[:2]
    written = torch.zeros(pages, size, dtype=torch.bool)
    rows = int(sum(counts))
    kept = torch.zeros(rows, dtype=torch.bool)
    pos = torch.empty(rows, dtype=torch.int64)
    slots = []
    row = 0
    for table, n, m in zip(tables, lengths, counts):
        for j in range(m):
            place = n - m + j
            pos[row] = place
            page = int(table[place // size]) if 0 <= place < len(table) * size else -1
            if 0 <= page < pages:
                kept[row] = True
                slots.append((row, page, place % size))
            row += 1
    if positions is not None:
        pos = positions.to(torch.int64)
    turn = (lambda x: rotate(x[None], pos[None], inv_freq, layout, magnitude)[0]) if inv_freq is not None else (
        lambda x: x.to(_F64))
    kr = turn(k)
    for r, page, slot in slots:
        k_pool[page, slot], v_pool[page, slot] = kr[r], v[r].to(_F64)
        written[page, slot] = True
    return (None if q is None else turn(q)), k_pool, v_pool, written, kept

"""Tables and groups of calls over a cache in pages that are not cut to the call:
tables with room for a model's whole context, group offsets that reach
outside of the batch, hundreds of groups, long own parts behind a short common
one. Tolerances as in test_paged_gpu.py."""
import pytest
import torch

from context_blockwise_causal_gb300 import cpattn_decode_paged, cpattn_decode_shared
from test_paged_gpu import NAN, _check, _group_state, _hide, _i32, _randn, _status

pytestmark = pytest.mark.gpu


def _wide(tables, tokens, size):
    out = torch.full((tables.shape[0], tokens // size), -1, dtype=torch.int32)
    out[:, :tables.shape[1]] = tables
    return out


def _outputs(b, hq, d):
    return {"o": torch.full((b, hq, d), NAN, dtype=torch.bfloat16, device="cuda"), "lse": torch.full((b, hq), NAN, device="cuda")}


WIDE = [
    # groups, prefix, own, size, hq, hkv, d
    ([8], [300], [i % 9 for i in range(8)], 16, 32, 8, 128),          # 32 rows of 8 heads, another kernel behind a wide table
    ([16], [200], [i * 3 for i in range(16)], 64, 8, 2, 64),          # 64 rows
    ([4], [130], [0, 1, 5, 60], 32, 4, 1, 64),                        # 16 rows: the same kernel
    ([3, 9], [77, 400], [i % 5 for i in range(12)], 48, 12, 2, 128),
    ([1], [500], [411], 16, 24, 2, 64),                               # one sequence, 12 heads to a KV head
]


@pytest.mark.parametrize("groups,prefix,own,size,hq,hkv,d", WIDE)
def test_tables_with_room_for_a_whole_context(groups, prefix, own, size, hq, hkv, d):
    """Runs and kernels follow the tables' room; what they compute does not."""
    k, v, tables, lengths, offsets = _group_state(groups, prefix, own, size, hq, hkv, d, False, 201)
    b = len(lengths)
    q = _randn(b, hq, d, seed=204)
    kd, vd = _hide(k.cuda(), v.cuda(), tables, lengths, 0, 0)
    ln, sh, off = _i32(lengths).cuda(), _i32(prefix).cuda(), offsets.cuda()
    for t in (tables, _wide(tables, 8192, size), _wide(tables, 131072, size), _wide(tables, 1 << 20, size)):
        out = _outputs(b, hq, d)
        cpattn_decode_shared(q.cuda(), kd, vd, t.cuda(), ln, sh, group_offsets=off, max_group=max(groups), **out)
        _check(q, k, v, tables, lengths, 0, 0, None, **out)
        for window, sinks in ((0, 0), (100, 3)):
            out = _outputs(b, hq, d)
            cpattn_decode_paged(q.cuda(), kd, vd, t.cuda(), ln, window, sinks, **out)
            _check(q, k, v, tables, lengths, window, sinks, None, **out)
    assert _status() == 0


@pytest.mark.parametrize("hq", [2, 8, 40])
@pytest.mark.parametrize("offsets", [[-2, 0, 500], [-7, 4, 400], [11, 12, 13], [3, 5, 5, 9], [-1 << 31, 6, (1 << 31) - 1],
                                     [0, 11, 3, 11]])
def test_group_offsets_outside_of_the_batch(offsets, hq):
    """Offsets are clamped to the batch; sequences outside of every group share
    nothing. All of them begin alike, so any grouping gives the same."""
    size, hkv, d = 32, 2, 128
    k, v, tables, lengths, _ = _group_state([11], [300], [20, 5, 0, 60, 1, 2, 3, 4, 5, 7, 9], size, hq, hkv, d, False, 211)
    q = _randn(11, hq, d, seed=214)
    kd, vd = _hide(k.cuda(), v.cuda(), tables, lengths, 0, 0)
    groups = len(offsets) - 1
    for most in (11, 4):
        out = _outputs(11, hq, d)
        cpattn_decode_shared(q.cuda(), kd, vd, tables.cuda(), _i32(lengths).cuda(), _i32([300, 297, 300][:groups]).cuda(),
                             group_offsets=_i32(offsets).cuda(), max_group=most, **out)
        torch.cuda.synchronize()
        assert _status() == 0
        _check(q, k, v, tables, lengths, 0, 0, None, **out)


@pytest.mark.parametrize("count,members,hq", [(110, 5, 4), (230, 5, 4), (230, 2, 40), (1030, 2, 34)])
def test_hundreds_of_groups(count, members, hq):
    """More groups than a warp has lanes many times over: of 20 rows, in either
    kernel, and of 80, and so many that their sequences share nothing."""
    groups, size, hkv, d = [members] * count, 16, 1, 64
    b, prefix = count * members, [(i * 29) % 70 for i in range(count)]
    k, v, tables, lengths, offsets = _group_state(groups, prefix, [i % 4 for i in range(b)], size, hq, hkv, d, False, 221)
    q = _randn(b, hq, d, seed=224)
    kd, vd = _hide(k.cuda(), v.cuda(), tables, lengths, 0, 0)
    for t in (tables, _wide(tables, 131072, size)):
        out = _outputs(b, hq, d)
        cpattn_decode_shared(q.cuda(), kd, vd, t.cuda(), _i32(lengths).cuda(), _i32(prefix).cuda(),
                             group_offsets=offsets.cuda(), max_group=members, **out)
        torch.cuda.synchronize()
        assert _status() == 0
        _check(q, k, v, tables, lengths, 0, 0, None, **out)


@pytest.mark.parametrize("hq,hkv", [(16, 8), (36, 2)])
def test_long_own_parts_behind_a_short_common_one(hq, hkv):
    """One run of 94 and of 63 rounds for each sequence."""
    k, v, tables, lengths, _ = _group_state([5], [64], [6000, 4000, 17, 0, 1500], 128, hq, hkv, 64, True, 231)
    q = _randn(5, hq, 64, seed=234)
    kd, vd = _hide(k.cuda(), v.cuda(), tables, lengths, 0, 0)
    out = _outputs(5, hq, 64)
    cpattn_decode_shared(q.cuda(), kd, vd, tables.cuda(), _i32(lengths).cuda(), _i32([64]).cuda(), **out)
    torch.cuda.synchronize()
    assert _status() == 0
    _check(q, k, v, tables, lengths, 0, 0, None, **out)


@pytest.mark.parametrize("hq,d", [(2, 64), (3, 128), (300, 64)])
def test_units_whose_members_have_finished(hq, d):
    """The first members of a large group have finished, and all of those of a
    later unit of 256 rows; a unit's pages are named by one of its own."""
    b, p, size = (400 if hq < 100 else 6), 200, 32
    k, v, tables, lengths, _ = _group_state([b], [p], [i % 5 for i in range(b)], size, hq, 1, d, False, 241)
    gone = list(range(0, b // 3)) + list(range(b // 2, b - 1))
    for i in gone:
        lengths[i] = (0, p - 1, 7)[i % 3]
        tables[i, -(-lengths[i] // size):] = -1
    q = _randn(b, hq, d, seed=244)
    kd, vd = _hide(k.cuda(), v.cuda(), tables, lengths, 0, 0)
    out = _outputs(b, hq, d)
    cpattn_decode_shared(q.cuda(), kd, vd, tables.cuda(), _i32(lengths).cuda(), _i32([p]).cuda(), **out)
    torch.cuda.synchronize()
    assert _status() == 0
    _check(q, k, v, tables, lengths, 0, 0, None, **out)

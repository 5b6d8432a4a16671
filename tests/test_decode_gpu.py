"""Single-token attention over a cache (cpattn_decode) through the C ABI
against the CPU fp64 oracle, every element.

Tolerance: P is rounded to bf16 before P V (u sum_j P_j |v_j|, u = 2^-8; the
warps' and runs' parts are joined in fp32) and the output once more (u |o|);
fp32 sums and exponentials are under 1/16 of the first. LSE: 1e-4 (scores are
off by at most 2^-17 sum |q k| scale, below 5e-5 here).
"""
import ctypes

import pytest
import torch

import context_blockwise_causal_gb300 as pkg
import oracle
from context_blockwise_causal_gb300 import cpattn_decode

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


def _randn(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)


def _check(q, k, v, lengths, window, sinks, scale, o, lse):
    for i, n in enumerate(lengths):
        n = min(max(n, 0), k.shape[1])
        ref, l_ref, err = oracle.decode_attention(q[i], k[i], v[i], n, window, sinks, scale)
        got = o[i].double().cpu()
        off = (got - ref).abs()
        assert (off <= err * (1 + 1 / 16) + U * ref.abs() + 1e-6).all(), (i, n, off.max().item())
        if n == 0:
            assert (got == 0).all() and (lse[i] == float("-inf")).all()
        else:
            assert (lse[i].double().cpu() - l_ref).abs().max().item() <= 1e-4, (i, n)


CASES = [
    # lengths, cap, hq, hkv, d, window, sinks, scale
    ([1], 1, 1, 1, 128, 0, 0, None),
    ([0, 1, 2, 15, 16, 17, 63, 64, 65, 200], 200, 4, 2, 128, 0, 0, None),
    ([0, 1, 2, 15, 16, 17, 63, 64, 65, 200], 200, 8, 1, 64, 16, 0, None),
    ([200, 199, 150, 20, 19, 18, 17, 3], 201, 8, 8, 64, 16, 4, None),     # one head per group
    ([1000, 900, 17], 1000, 24, 2, 128, 100, 30, 0.3),                    # 12 heads per group
    ([700, 33], 700, 40, 1, 64, 0, 0, None),                             # 40 heads per group: three row tiles
    ([5000], 5003, 4, 2, 128, 0, 0, None),                               # one sequence over many runs
    ([5000, 1], 5003, 4, 2, 64, 4000, 4, None),                          # a sequence shorter than the runs
    ([40000], 40001, 4, 1, 128, 0, 0, None),                             # more runs than a cluster has CTAs
    ([36000, 0, 3], 40001, 4, 1, 64, 35000, 4, None),
    ([300, 300], 300, 2, 1, 128, 1, 0, None),                            # a window of the new token alone
    ([300, 2], 300, 2, 1, 128, 1, 500, None),                            # every key a first token
    ([777] * 90, 800, 16, 8, 64, 500, 1, None),                          # more sequences than places
]


@pytest.mark.parametrize("lengths,cap,hq,hkv,d,window,sinks,scale", CASES)
def test_all_elements_and_what_lies_past_the_lengths(lengths, cap, hq, hkv, d, window, sinks, scale):
    b = len(lengths)
    q, k, v = _randn(b, hq, d, seed=1), _randn(b, cap, hkv, d, seed=2), _randn(b, cap, hkv, d, seed=3)
    kd, vd = k.cuda(), v.cuda()
    for i, n in enumerate(lengths):  # never read
        kd[i, n:] = float("nan")
        vd[i, n:] = float("inf")
        if window:  # nor is what has left the window
            kd[i, min(sinks, max(0, n - window)):max(0, n - window)] = float("nan")
            vd[i, min(sinks, max(0, n - window)):max(0, n - window)] = float("nan")
    ln = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    o = torch.full((b, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((b, hq), float("nan"), device="cuda")
    cpattn_decode(q.cuda(), kd, vd, ln, window, sinks, scale, o=o, lse=lse)
    torch.cuda.synchronize()
    _check(q, k, v, lengths, window, sinks, scale, o, lse)
    # the other cache layout, q inside a wider row: the same bits
    kt, vt = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (kd, vd))
    wide = torch.zeros(b, hq + 3, d, dtype=torch.bfloat16, device="cuda")
    wide[:, :hq] = q.cuda()
    o2, l2 = cpattn_decode(wide[:, :hq], kt, vt, ln, window, sinks, scale)
    assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_lengths_out_of_range_are_clamped():
    q, k, v = _randn(3, 2, 64, seed=4), _randn(3, 50, 1, 64, seed=5), _randn(3, 50, 1, 64, seed=6)
    lengths = [-5, 1 << 30, 50]
    o, lse = cpattn_decode(q.cuda(), k.cuda(), v.cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    _check(q, k, v, lengths, 0, 0, None, o, lse)


def test_long_cache_offsets_beyond_32_bits():
    """Sequences whose rows start over 2^31 elements into the cache."""
    b, cap, hkv, d = 3, 1 << 20, 8, 128  # 2^30 elements each
    k, v = (torch.zeros(b, cap, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = _randn(b, 8, d, seed=7)
    kt, vt = _randn(b, 300, hkv, d, seed=8), _randn(b, 300, hkv, d, seed=9)
    k[:, cap - 300:], v[:, cap - 300:] = kt.cuda(), vt.cuda()
    ln = torch.full((b,), cap, dtype=torch.int32, device="cuda")
    o, lse = cpattn_decode(q.cuda(), k, v, ln, window=300)
    _check(q, kt, vt, [300] * b, 0, 0, None, o, lse)


def test_graph_replays_with_new_lengths():
    """One captured step replayed while the cache grows: the lengths are read
    on the device."""
    b, cap, hq, hkv, d = 2, 600, 4, 2, 128
    q, k, v = _randn(b, hq, d, seed=10), _randn(b, cap, hkv, d, seed=11), _randn(b, cap, hkv, d, seed=12)
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    ln = torch.tensor([1, 500], dtype=torch.int32, device="cuda")
    cpattn_decode(qd, kd, vd, ln, 64, 4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = cpattn_decode(qd, kd, vd, ln, 64, 4)
    for lengths in ([1, 500], [64, 65], [0, 600]):
        ln.copy_(torch.tensor(lengths, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        _check(q, k, v, lengths, 64, 4, None, o, lse)


def test_given_stream_and_two_calls_at_once():
    b, cap, hq, hkv, d = 4, 3000, 8, 2, 64
    q, k, v = _randn(b, hq, d, seed=13).cuda(), _randn(b, cap, hkv, d, seed=14).cuda(), _randn(b, cap, hkv, d, seed=15).cuda()
    ln = torch.tensor([3000, 1, 1500, 77], dtype=torch.int32, device="cuda")
    want = [cpattn_decode(q, k, v, ln, w, 4) for w in (100, 2000)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = [cpattn_decode(q, k, v, ln, w, 4, stream=s) for w, s in ((100, s1), (2000, s2))]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])


def test_checked_build_is_silent_and_identical():
    lib = pkg.checked_library()
    b, cap, hq, hkv, d = 3, 900, 6, 2, 128
    q, k, v = _randn(b, hq, d, seed=16).cuda(), _randn(b, cap, hkv, d, seed=17).cuda(), _randn(b, cap, hkv, d, seed=18).cuda()
    ln = torch.tensor([900, 0, 333], dtype=torch.int32, device="cuda")
    for window, sinks in ((0, 0), (128, 4)):
        o, lse = cpattn_decode(q, k, v, ln, window, sinks)
        o2, l2 = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
        n = lib.cpattn_decode_workspace_bytes(b, hq, hkv, d, cap, window, sinks)
        ws = torch.empty(n + 16, dtype=torch.uint8, device="cuda")
        rc = lib.cpattn_decode(q.data_ptr(), k.data_ptr(), v.data_ptr(), ln.data_ptr(), o2.data_ptr(), l2.data_ptr(),
                               ws.data_ptr(), n, b, hq, hkv, d, cap, hq * d, cap * hkv * d, hkv * d, d, cap * hkv * d,
                               hkv * d, d, window, sinks, 0.0, None)
        assert rc == 0
        torch.cuda.synchronize()
        st = ctypes.c_int(0)
        lib.cpattn_device_status(None, ctypes.byref(st))
        assert st.value == 0, hex(st.value)
        assert torch.equal(o, o2) and torch.equal(lse, l2)


def test_refusals():
    q, k = (torch.zeros(*s, dtype=torch.bfloat16, device="cuda") for s in ((2, 4, 64), (2, 10, 2, 64)))
    ln = torch.ones(2, dtype=torch.int32, device="cuda")
    for kw in ({"window": -1}, {"sinks": -1}, {"scale": -1.0}, {"scale": float("nan")}):
        with pytest.raises(pkg.CpattnError):
            cpattn_decode(q, k, k, ln, **kw)
    with pytest.raises(pkg.CpattnError):
        cpattn_decode(q[:, :3], k, k, ln)  # 3 query heads over 2 KV heads
    with pytest.raises(TypeError):
        cpattn_decode(q, k, k, ln.long())
    with pytest.raises(ValueError):
        cpattn_decode(q, k, k[:, :5], ln)
    with pytest.raises(ValueError):
        cpattn_decode(q, k, k, ln[:1])
    with pytest.raises(TypeError):
        cpattn_decode(q, k.float(), k.float(), ln)
    need = pkg.cpattn_decode_workspace_bytes(1, 4, 2, 64, 100000)
    assert need > 0  # a few long sequences: over 8 runs
    big = torch.zeros(1, 100000, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pkg.CpattnError):
        cpattn_decode(q[:1], big, big, ln[:1], workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


def test_long_decodes_one_after_another_eager_and_captured():
    """More runs than a cluster has CTAs: two kernels a call, the second placed
    while the first still runs. Each call here takes the one before's output as
    its queries, and all of them one workspace."""
    cap, hq, hkv, d = 40001, 4, 1, 64
    k, v = _randn(1, cap, hkv, d, seed=50).cuda(), _randn(1, cap, hkv, d, seed=51).cuda()
    q = _randn(1, hq, d, seed=52).cuda()
    ln = torch.tensor([cap], dtype=torch.int32, device="cuda")
    need = pkg.cpattn_decode_workspace_bytes(1, hq, hkv, d, cap)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def chain(sync):
        x, out = q, []
        for i in range(6):
            x, lse = cpattn_decode(x * 8, k, v, ln, workspace=ws)
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
    for new in (100, cap):
        ln.fill_(new)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(chain(True), got))

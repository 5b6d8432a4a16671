"""Waits of the paged cache's kernels that give up, without a GPU fault: the
copying warps act as if a wait for free room had run out, the kernels record it
in the status word and return, and the same calls afterwards give the bits that
they gave before."""
import ctypes

import pytest
import torch

from context_blockwise_causal_gb300 import cpattn_decode_paged, cpattn_decode_shared, library
from test_paged_abi import Pages
from test_paged_gpu import _i32, _randn, _status


def test_abort_selftest_arguments():
    from context_blockwise_causal_gb300 import build
    from context_blockwise_causal_gb300._build import is_stale

    if is_stale():
        build()
    lib, p = library(), ctypes.c_void_p(4096)  # never dereferenced: the checks come first
    assert lib.cpattn_selftest_abort_paged(p, None, p, None, p, p, p, 1 << 30, 2, 4, 2, 64, 256, 1, None) == -2
    assert lib.cpattn_selftest_abort_paged(None, p, p, p, p, p, p, 1 << 30, 2, 4, 2, 64, 256, 1, None) == -2
    assert lib.cpattn_selftest_abort_paged(p, None, p, p, p, p, p, 1 << 30, 2, 4, 2, 64, 256, 1, None) == -2


CASES = [
    # b, hq, hkv, d, tokens, shared (None: whole sequences), the bit of who gives up first
    (1, 8, 2, 128, 40000, None, 4),      # runs joined by a kernel
    (4, 16, 8, 64, 16000, None, 4),      # clusters
    (64, 32, 8, 128, 1000, None, 4),     # a run for each sequence, 64 KV heads' worth of rows
    (4, 8, 2, 128, 40000, 39000, 4),     # 16 rows: common and own keys in one launch
    (40, 2, 2, 128, 100000, 99900, 0),   # 40 rows: one row tile, key tiles in turn
    (40, 8, 2, 128, 100000, 99900, 0),   # 160 rows: two row tiles
    (40, 8, 2, 64, 100000, 99900, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("b,hq,hkv,d,tokens,shared,bit", CASES)
def test_waits_give_up_and_the_calls_work_afterwards(b, hq, hkv, d, tokens, shared, bit):
    size = 64
    cols = -(-tokens // size)
    tables = torch.arange(cols, dtype=torch.int32)[None].expand(b, cols).contiguous().cuda()
    k, v = (torch.empty(cols, size, hkv, d, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(s))
            for s in (1, 2))
    q, ln = _randn(b, hq, d, seed=3).cuda(), _i32([tokens - i for i in range(b)]).cuda()
    sh = None if shared is None else _i32([shared]).cuda()

    def call():
        return cpattn_decode_paged(q, k, v, tables, ln) if sh is None else cpattn_decode_shared(q, k, v, tables, ln, sh)

    want = call()
    torch.cuda.synchronize()
    assert _status() == 0
    lib = library()
    need = (lib.cpattn_decode_paged_workspace_bytes(b, hq, hkv, d, cols * size, 0, 0) if sh is None else
            lib.cpattn_decode_shared_workspace_bytes(b, hq, hkv, d, 1, b))
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    page, s = size * hkv * d, (hkv * d, d)
    pg = Pages(k.data_ptr(), v.data_ptr(), cols, size, cols, tables.data_ptr(), cols, page, *s, page, *s)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for waits in (0, 1, 3):
        rc = lib.cpattn_selftest_abort_paged(q.data_ptr(), pg, ln.data_ptr(), None if sh is None else sh.data_ptr(),
                                             o.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), b, hq, hkv, d, hq * d,
                                             waits, stream)
        assert rc == 0, lib.cpattn_strerror(rc)
        torch.cuda.synchronize()
        status = _status()
        assert status & (1 << bit), (waits, hex(status))
        # who gave up, and no wait for what was in flight
        assert not status & ~(0b111 | 1 << 4), (waits, hex(status))
        for _ in range(2):
            got = call()
            torch.cuda.synchronize()
            assert _status() == 0
            assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])

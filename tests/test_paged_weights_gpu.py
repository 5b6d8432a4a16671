"""cpattn_decode_paged against the CPU fp64 oracle to the output's own rounding:
probabilities enter their product in two bf16 pieces.

Tolerance: the output's rounding, u |o| with u = 2^-8 (half a step of bf16 relative
to the value), and of sum_j P_j |v_j| what stays before it: 2^-16 (a piece's
rounding, u, of the first piece's, u); 2^-12 for what is fp32: scores that are
off by up to 5e-5 (2^-17 sum |q k| scale) move weight and sum by 1e-4 = 2^-13.3
together, products' and weights' sums of some hundred terms to a warp add under
2^-15, exponentials and joins under 2^-20."""
import pytest
import torch

import oracle
from context_blockwise_causal_gb300 import cpattn_decode_paged
from test_paged_gpu import U, _i32, _pools, _randn, _status, _tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lengths,size,cols,hq,hkv,d,window,sinks", [
    ([2, 3, 5, 17, 63, 64, 200], 16, 13, 4, 2, 128, 0, 0),
    ([2, 3, 5, 17, 63, 64, 200], 48, 5, 8, 1, 64, 16, 4),
    ([1000, 900, 17], 80, 13, 24, 2, 128, 100, 30),      # 12 heads to a KV head
    ([700, 33], 64, 11, 40, 1, 64, 0, 0),
    ([5000], 128, 40, 4, 2, 128, 0, 0),                  # runs joined by a kernel
    ([3000, 1, 2222, 1500], 64, 47, 16, 8, 64, 0, 0),    # clusters
])
def test_weights_keep_sixteen_bits(lengths, size, cols, hq, hkv, d, window, sinks):
    b = len(lengths)
    k, v, kd, vd = _pools(b * cols, size, hkv, d, False, 301)
    tables, q = _tables(b, cols, b * cols, 303), _randn(b, hq, d, seed=304)
    o, lse = cpattn_decode_paged(q.cuda(), kd, vd, tables.cuda(), _i32(lengths).cuda(), window, sinks)
    torch.cuda.synchronize()
    assert _status() == 0
    for i, n in enumerate(lengths):
        ref, _, err = oracle.decode_attention(q[i], oracle.held_tokens(k, tables[i], n), oracle.held_tokens(v, tables[i], n), n,
                                              window, sinks)
        off = (o[i].double().cpu() - ref).abs()  # err: u sum_j P_j |v_j|
        assert (off <= U * ref.abs() + err * (2.0 ** -8 + 2.0 ** -4) + 1e-12).all(), (i, n, off.max().item())

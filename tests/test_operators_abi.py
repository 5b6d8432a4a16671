"""CPU tests of the C boundary of the windowed attention, single-token
attention, rotary and q/k norm calls: argument errors come before any device
work (the pointers are never followed), sizes of workspaces, frequencies."""
import ctypes
import os
import re

import pytest
import torch

import oracle



class Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64)]

    @property
    def _as_parameter_(self):
        return ctypes.byref(self)


class Rotary(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int), ("rot_dim", ctypes.c_int), ("magnitude", ctypes.c_float), ("s", ctypes.c_int),
                ("cp", ctypes.c_int), ("rank", ctypes.c_int), ("cu_seqlens", ctypes.c_void_p), ("nseq", ctypes.c_int),
                ("positions", ctypes.c_void_p), ("positions_batch", ctypes.c_int64), ("inv_freq", ctypes.c_void_p)]

    @property
    def _as_parameter_(self):
        return ctypes.byref(self)


P = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4096 + 8)
ARG, NULL, MISALIGNED, ARCH, SMALL = -1, -2, -3, -4, -5


@pytest.fixture(scope="module")
def lib():
    import context_blockwise_causal_gb300 as pkg
    from context_blockwise_causal_gb300._build import is_stale

    if is_stale():
        pkg.build()
    return pkg.library()


def test_window_arguments(lib):
    def f(ptr=(P,) * 5, b=1, sq=100, skv=200, hq=4, hkv=2, d=64, window=10, sinks=2, scale=0.0):
        return lib.cpattn_fwd_window(*ptr, b, sq, skv, hq, hkv, d, window, sinks, scale, None)

    for i in range(5):
        assert f((P,) * i + (None,) + (P,) * (4 - i)) == NULL
        assert f((P,) * i + (ODD,) + (P,) * (4 - i)) == MISALIGNED
    for bad in ({"b": 0}, {"sq": 0}, {"sq": 201}, {"hq": 3}, {"hkv": 0}, {"d": 96}, {"window": 0}, {"sinks": -1},
                {"scale": -1.0}, {"scale": float("nan")}, {"skv": (1 << 30) + 1}, {"b": 4, "skv": 1 << 29},
                {"b": 1 << 20, "hq": 1 << 12, "hkv": 1 << 12, "skv": 128}):
        assert f(**bad) == ARG, bad

    def g(n, window=10, sinks=2):
        return lib.cpattn_bwd_window(*(P,) * 10, n, 1, 100, 200, 4, 2, 64, window, sinks, 0.0, None)

    need = lib.cpattn_bwd_window_workspace_bytes(1, 100, 200, 4, 2, 64, 10, 2)
    assert need == 2 * 4 * 128 * 4  # L and D of each head's padded rows; no walk is cut
    assert g(need - 1) == SMALL and g(need, window=0) == ARG
    # 8192 queries, a first token: the first tile's 64-tile walk in parts of 8, fp32 dK and dV
    need = lib.cpattn_bwd_window_workspace_bytes(1, 8192, 8192, 4, 2, 64, 10, 1)
    assert need == 2 * 4 * 8192 * 4 + 2 * (2 * 8 * 128 * 64 * 4)
    assert lib.cpattn_bwd_window_workspace_bytes(1, 300, 200, 4, 2, 64, 10, 2) == 0
    # parts cost workspace only where whole walks would not balance: not with
    # many sequences, nor when every key is a first token
    assert lib.cpattn_bwd_window_workspace_bytes(512, 8192, 8192, 4, 2, 64, 10, 1) == 512 * 2 * 4 * 8192 * 4
    assert lib.cpattn_bwd_window_workspace_bytes(1, 32768, 32768, 32, 8, 128, 10, 32768) == 2 * 32 * 32768 * 4
    # at most 64 parts of a walk
    need = lib.cpattn_bwd_window_workspace_bytes(1, 1 << 20, 1 << 20, 4, 2, 64, 10, 1)
    assert need == 2 * 4 * (1 << 20) * 4 + 2 * (2 * 64 * 128 * 64 * 4)


def test_window_packed_arguments(lib):
    def cu(*xs):
        return (ctypes.c_int * len(xs))(*xs)

    def f(c, n, **kw):
        a = {"hq": 4, "hkv": 2, "d": 64, "window": 10, "sinks": 2, "scale": 0.0} | kw
        return lib.cpattn_fwd_window_varlen(*(P,) * 5, c, n, *a.values(), None)

    assert f(None, 1) == NULL
    assert f(cu(0, 10, 5), 2) == ARG and f(cu(1, 10), 1) == ARG and f(cu(0, 10), 0) == ARG
    assert f(cu(0, 10), 1, window=0) == ARG and f(cu(0, 10), 1, hq=5) == ARG and f(cu(0, 0), 1, d=32) == ARG
    assert f(cu(0, 0), 1) == 0  # nothing to do
    assert lib.cpattn_fwd_window_varlen(*(None,) * 5, cu(0, 0), 1, 4, 2, 64, 10, 2, 0.0, None) == 0
    assert lib.cpattn_bwd_window_varlen(*(None,) * 10, 0, cu(0, 0), 1, 4, 2, 64, 10, 2, 0.0, None) == 0
    w = lib.cpattn_bwd_window_varlen_workspace_bytes
    # three samples of up to two tiles: L and D of 256 rows per sample and head
    assert w(cu(0, 100, 300, 301), 3, 4, 2, 64, 10, 2) == 2 * 3 * 4 * 256 * 4
    assert w(cu(0, 10, 5), 2, 4, 2, 64, 10, 2) == 0
    assert lib.cpattn_bwd_window_varlen(*(P,) * 10, 64, cu(0, 100), 1, 4, 2, 64, 10, 2, 0.0, None) == SMALL


def test_decode_arguments(lib):
    def f(ptr=(P,) * 7, n=1 << 30, b=2, hq=4, hkv=2, d=64, cap=100, strides=(256, 12800, 128, 64, 12800, 128, 64), window=0,
          sinks=0, scale=0.0):
        return lib.cpattn_decode(*ptr, n, b, hq, hkv, d, cap, *strides, window, sinks, scale, None)

    for i in range(6):
        assert f((P,) * i + (None,) + (P,) * (6 - i)) == NULL
    for bad in ({"b": 0}, {"hq": 3}, {"d": 80}, {"cap": 0}, {"cap": (1 << 30) + 1}, {"window": -1}, {"sinks": -1},
                {"scale": -2.0}, {"strides": (256, 12800, 129, 64, 12800, 128, 64)},
                {"strides": (256, 12800, 128, 64, -8, 128, 64)}, {"strides": (4, 12800, 128, 64, 12800, 128, 64)},
                {"b": 1 << 20, "hq": 64}):
        assert f(**bad) == ARG, bad
    assert f((ODD,) + (P,) * 6) == MISALIGNED
    assert lib.cpattn_decode_workspace_bytes(2, 3, 2, 64, 100, 0, 0) == 0


def test_rotary_arguments(lib):
    freq = torch.ones(64, dtype=torch.float64)

    def plan(**kw):
        a = {"layout": 0, "rot_dim": 64, "magnitude": 1.0, "s": 10, "cp": 1, "rank": -1, "inv_freq": freq.data_ptr()} | kw
        return Rotary(**a)

    def rows(data=4096, batch=1280, token=128):
        return Rows(data, batch, token)

    def f(x=None, y=None, pl=None, b=2, n=10, h=2, d=64):
        return lib.cpattn_rope_ex(x or rows(), y or rows(), b, n, h, d, pl or plan(), 0, None)

    assert f(x=rows(data=None)) == NULL and f(y=rows(data=None)) == NULL
    assert f(pl=plan(inv_freq=None)) == NULL
    assert lib.cpattn_rope_ex(None, rows(), 2, 10, 2, 64, plan(), 0, None) == NULL
    assert lib.cpattn_rope_ex(rows(), rows(), 2, 10, 2, 64, None, 0, None) == NULL
    assert f(x=rows(data=4104)) == MISALIGNED
    for bad in ({"layout": 2}, {"rot_dim": 24}, {"rot_dim": 0}, {"rot_dim": 80}, {"magnitude": 0.0},
                {"magnitude": float("nan")}, {"s": 11}, {"rank": 1, "s": 20}, {"rank": 0, "s": 20, "cp": 3},
                {"cu_seqlens": 4096, "nseq": 2}, {"positions": 4096, "rank": 0}, {"positions": 4096, "positions_batch": -1},
                {"positions": 4096, "cu_seqlens": 4096, "nseq": 1}):
        assert f(pl=plan(**bad)) == ARG, bad
    for bad in (torch.full((64,), float("nan")), torch.full((64,), -1.0), torch.full((64,), float("inf"))):
        bad = bad.double()
        assert f(pl=plan(inv_freq=bad.data_ptr())) == ARG
    # strides: 16-byte pieces, tokens that do not overlap, outputs whose batch elements do not
    for bad in (rows(token=132), rows(token=64), rows(batch=1284), rows(batch=-1280)):
        assert f(x=bad) == ARG and f(y=bad) == ARG
    assert f(y=rows(batch=640)) == ARG and f(y=rows(batch=0)) == ARG
    args = (P, P, 1, 1e-6)
    q = rows()
    assert lib.cpattn_qk_norm_rope(q, q, None, P, 1, 1e-6, q, q, 2, 10, 2, 2, 64, plan(), None) == NULL
    assert lib.cpattn_qk_norm_rope(q, q, P, P, 1, -1.0, q, q, 2, 10, 2, 2, 64, plan(), None) == ARG
    assert lib.cpattn_qk_norm_rope(q, q, ODD, P, 1, 1e-6, q, q, 2, 10, 2, 2, 64, plan(), None) == MISALIGNED
    assert lib.cpattn_qk_norm_rope(q, q, P, P, 1, 1e-6, q, q, 2, 10, 2, 0, 64, plan(), None) == ARG
    need = lib.cpattn_qk_norm_rope_bwd_workspace_bytes(64)
    assert need > 0 and lib.cpattn_qk_norm_rope_bwd_workspace_bytes(96) == 0
    bwd = lib.cpattn_qk_norm_rope_bwd
    assert bwd(q, q, *args, q, q, q, q, P, P, P, need - 1, 2, 10, 2, 2, 64, plan(), None) == SMALL
    assert bwd(q, q, *args, q, q, q, q, P, None, P, need, 2, 10, 2, 2, 64, plan(), None) == NULL


def test_frequencies(lib):
    from context_blockwise_causal_gb300 import cpattn_rope_frequencies

    for rot, base, kw in ((128, 10000.0, {}), (64, 500000.0, {"scaling": "linear", "factor": 4.0}),
                          (48, 10000.0, {"scaling": "base", "factor": 8.0}),
                          (128, 500000.0, {"scaling": "turns", "factor": 8.0, "original_len": 8192, "low": 1, "high": 4}),
                          (64, 10000.0, {"scaling": "index", "factor": 40.0, "original_len": 4096, "low": 1, "high": 32}),
                          (2, 10.0, {"scaling": "index", "factor": 4.0, "original_len": 100, "low": 1, "high": 2})):
        got = cpattn_rope_frequencies(rot, base, **kw)
        assert torch.allclose(got, oracle.scaled_frequencies(rot, base, **kw), rtol=1e-13, atol=0), (rot, kw)
    f = lib.cpattn_rope_frequencies
    out = (ctypes.c_double * 64)()
    assert f(128, 10000.0, 0, 0.0, 0.0, 0.0, 0.0, None) == NULL
    for bad in ((127, 1e4, 0, 1.0, 0.0, 0.0, 0.0), (0, 1e4, 0, 1.0, 0.0, 0.0, 0.0), (64, 1.0, 0, 1.0, 0.0, 0.0, 0.0),
                (64, 1e4, 5, 1.0, 0.0, 0.0, 0.0), (64, 1e4, 1, 0.9, 0.0, 0.0, 0.0), (2, 1e4, 2, 2.0, 0.0, 0.0, 0.0),
                (64, 1e4, 3, 2.0, 0.0, 1.0, 4.0), (64, 1e4, 3, 2.0, 8192.0, 4.0, 1.0), (64, 1e4, 4, 2.0, 8192.0, 0.0, 1.0),
                (64, float("inf"), 0, 1.0, 0.0, 0.0, 0.0)):
        assert f(*bad, out) == ARG, bad


def test_counts_that_the_call_cannot_take(lib):
    import context_blockwise_causal_gb300 as cp

    # counts beyond int32 are every key, negative ones stay refusable
    assert [cp._keys(n) for n in (0, 5, 1 << 40, -1, -(1 << 32) + 5)] == [0, 5, 0x7FFFFFFF, -1, -1]


def test_binding_refuses_before_it_needs_a_device(lib):
    import context_blockwise_causal_gb300 as cp

    x, w = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16), torch.ones(64)
    q, ln = torch.zeros(1, 2, 64, dtype=torch.bfloat16), torch.ones(1, dtype=torch.int32)
    for call in (lambda: cp.cpattn_rope(x, layout="interleaved"), lambda: cp.cpattn_rope(x.half(), rot_dim=32),
                 lambda: cp.cpattn_rope(None, rot_dim=32), lambda: cp.cpattn_qk_norm_rope(x, x, w, w),
                 lambda: cp.cpattn_qk_norm_rope_bwd(x, x, w, w, x, x), lambda: cp.cpattn_fwd_window(x, x, x, 4),
                 lambda: cp.cpattn_fwd_window(x.half(), x, x, 4), lambda: cp.cpattn_fwd_window(5, x, x, 4),
                 lambda: cp.cpattn_bwd_window(x, x, x, x, w, x, 4), lambda: cp.cpattn_decode(q, x, x, ln),
                 lambda: cp.cpattn_decode(q, x, x, None), lambda: cp.cpattn_fwd_window_varlen(x[0], x[0], x[0], [0, 4], 4)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        cp.cpattn_fwd_window(x[0], x, x, 4)
    # the table of functions is checked, and so is the number of arguments
    for bad in ((), (b"",), (cp.library().calls,), (cp.library().calls, x)):
        with pytest.raises((SystemError, TypeError)):
            cp._native().rope(*bad)


def test_binding_table_names_the_structure_of_the_source():
    import context_blockwise_causal_gb300 as cp

    src = open(os.path.join(os.path.dirname(cp.__file__), "csrc", "binding.cpp")).read()
    body = src[src.index("struct Calls {"):]
    assert tuple(re.findall(r"decltype\(&(\w+)\)", body[:body.index("};")])) == cp._CALLS


def test_rows_of_a_token_stay_below_32_bits(lib):
    """The kernels form a head's offset in 32 bits: a token of 2^31 features or
    more (one tensor's, or q's and k's together) is refused before a launch."""
    freq = torch.ones(64, dtype=torch.float64)

    def f(h, d):
        r = Rows(4096, 0, h * d)
        plan = Rotary(layout=0, rot_dim=64, magnitude=1.0, s=1, cp=1, rank=-1, inv_freq=freq.data_ptr())
        return lib.cpattn_rope_ex(r, r, 1, 1, h, d, plan, 0, None)

    def g(hq, hkv, d):
        q, k = Rows(4096, 0, hq * d), Rows(4096, 0, hkv * d)
        plan = Rotary(layout=0, rot_dim=64, magnitude=1.0, s=1, cp=1, rank=-1, inv_freq=freq.data_ptr())
        fwd = lib.cpattn_qk_norm_rope(q, k, P, P, 1, 1e-6, q, k, 1, 1, hq, hkv, d, plan, None)
        bwd = lib.cpattn_qk_norm_rope_bwd(q, k, P, P, 1, 1e-6, q, k, q, k, P, P, P, 1 << 30, 1, 1, hq, hkv, d, plan, None)
        assert fwd == bwd
        return fwd

    for h, d in ((1 << 24, 128), (1 << 25, 64), (2 ** 31 - 1, 64)):
        assert f(h, d) == ARG and g(h, 1, d) == ARG and g(1, h, d) == ARG, (h, d)
    assert g((1 << 24) - 1, 1, 128) == ARG and g(1, (1 << 25) - 1, 64) == ARG and g(1 << 23, 1 << 23, 128) == ARG
    if not torch.cuda.is_available():  # shapes below it pass the checks (and would be launched on a GPU)
        assert f((1 << 24) - 1, 128) not in (0, ARG) and g((1 << 24) - 2, 1, 128) not in (0, ARG)

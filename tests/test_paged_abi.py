"""CPU tests of the C boundary of the paged cache: argument errors come before
any device work (the pointers are never followed), and the oracle's pins."""
import ctypes

import pytest
import torch

import oracle
from test_operators_abi import ARCH, ARG, MISALIGNED, NULL, ODD, P, SMALL, Rotary, Rows, lib  # noqa: F401


class Pages(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pages", ctypes.c_int), ("page_size", ctypes.c_int),
                ("table_cols", ctypes.c_int), ("tables", ctypes.c_void_p), ("tables_row", ctypes.c_int64)] + [
                    (n, ctypes.c_int64) for n in ("k_page", "k_token", "k_head", "v_page", "v_token", "v_head")]

    @property
    def _as_parameter_(self):
        return ctypes.byref(self)


def pages(hkv=2, d=64, heads_first=False, **kw):
    """10 pages of 32 tokens, 5 to a sequence."""
    token, head = (d, 32 * d) if heads_first else (hkv * d, d)
    a = {"k": 4096, "v": 8192, "pages": 10, "page_size": 32, "table_cols": 5, "tables": 4096, "tables_row": 5}
    for p in "kv":
        a |= {p + "_page": 32 * hkv * d, p + "_token": token, p + "_head": head}
    return Pages(**(a | kw))


BAD_PAGES = [{"pages": 0}, {"page_size": 0}, {"page_size": 8}, {"page_size": 40}, {"table_cols": 0}, {"tables_row": -1},
             {"page_size": 1 << 20, "table_cols": 1025}, {"k_page": 32 * 128 - 8}, {"k_page": 32 * 128 + 4},
             {"v_token": 64}, {"v_token": 127}, {"k_head": 0}, {"k_head": -64}, {"v_head": 60}, {"v_page": 0},
             {"k_page": 1 << 38}, {"v_page": 1 << 37, "pages": 1 << 20}]


def check_pages_of(f, over):
    """f(pages) of any call that takes pages; over: a status other than an argument error."""
    for bad in BAD_PAGES:
        assert f(pages(**bad)) == ARG, bad
    for name in ("k", "v", "tables"):
        assert f(pages(**{name: None})) == NULL
    assert f(pages(k=4104)) == MISALIGNED and f(pages(v=4104)) == MISALIGNED and f(pages(tables=4098)) == MISALIGNED
    if not torch.cuda.is_available():  # these pass the checks (and would be launched on a GPU)
        assert f(pages()) in over and f(pages(heads_first=True)) in over
        assert f(pages(pages=1, k_page=0, v_page=-1)) in over


def test_append_arguments(lib):  # noqa: F811
    freq = torch.ones(64, dtype=torch.float64)

    def plan(**kw):
        return Rotary(**({"layout": 0, "rot_dim": 64, "magnitude": 1.0, "rank": -1, "inv_freq": freq.data_ptr()} | kw))

    kv, qr = Rows(4096, 3 * 128, 128), Rows(4096, 3 * 256, 256)

    def f(k=kv, v=kv, pg=None, lengths=P, cu=None, seqs=2, q=qr, q_out=qr, b=2, n=3, hq=4, hkv=2, d=64, pl=plan()):
        return lib.cpattn_append_paged(k, v, pages() if pg is None else pg, lengths, cu, seqs, q, q_out, b, n, hq, hkv, d,
                                       pl, None)

    check_pages_of(lambda p: f(pg=p), (-4, -8))
    assert f(k=None) == NULL and f(v=None) == NULL and f(lengths=None) == NULL and f(q=None) == NULL
    assert f(q_out=None) == NULL and f(k=Rows(None, 384, 128)) == NULL
    assert lib.cpattn_append_paged(kv, kv, None, P, None, 2, qr, qr, 2, 3, 4, 2, 64, plan(), None) == NULL
    for bad in ({"b": 0}, {"n": 0}, {"seqs": 0}, {"seqs": 3}, {"hq": 0}, {"hkv": 0}, {"d": 96}, {"cu": P},
                {"q": None, "q_out": None}, {"k": Rows(4096, 384, 120)}, {"v": Rows(4096, 380, 128)},
                {"q_out": Rows(4096, 256, 256)}, {"pg": pages(tables_row=4)}, {"pl": plan(rank=0)},
                {"pl": plan(cu_seqlens=4096, nseq=1)}, {"pl": plan(rot_dim=24)}, {"pl": plan(magnitude=0.0)},
                {"pl": plan(layout=2)}, {"pl": plan(positions=4096, positions_batch=-1)}):
        assert f(**bad) == ARG, bad
    assert f(k=Rows(4104, 384, 128)) == MISALIGNED and f(lengths=ctypes.c_void_p(4098)) == MISALIGNED
    assert f(b=1, seqs=1, cu=ctypes.c_void_p(4098)) == MISALIGNED
    assert f(pl=plan(inv_freq=None)) == NULL
    # a token's features stay below 2^31
    big = Rows(4096, 0, 0)
    assert f(k=big, v=big, q=None, q_out=None, b=1, n=1, seqs=1, hq=0, hkv=1 << 24, d=64,
             pg=pages(hkv=1, k_head=64, v_head=64, k_token=1 << 30, v_token=1 << 30, k_page=1 << 36, v_page=1 << 36)) == ARG
    if not torch.cuda.is_available():
        assert f() == ARCH or f() == -8
        for good in ({"pl": None}, {"q": None, "q_out": None, "hq": 0}, {"b": 1, "seqs": 7, "cu": P},
                     {"pl": plan(positions=4096, positions_batch=3)}, {"pl": plan(s=99)}):
            assert f(**good) in (ARCH, -8), good


def test_decode_paged_arguments(lib):  # noqa: F811
    def f(ptr=(P,) * 4, pg=None, ws=P, n=1 << 30, b=2, hq=4, hkv=2, d=64, q_batch=256, window=0, sinks=0, scale=0.0):
        q, ln, o, lse = ptr
        return lib.cpattn_decode_paged(q, pages() if pg is None else pg, ln, o, lse, ws, n, b, hq, hkv, d, q_batch, window,
                                       sinks, scale, None)

    for i in range(4):
        assert f((P,) * i + (None,) + (P,) * (3 - i)) == NULL
    for i in (0, 2):
        assert f((P,) * i + (ODD,) + (P,) * (3 - i)) == MISALIGNED
    assert lib.cpattn_decode_paged(P, None, P, P, P, P, 1, 2, 4, 2, 64, 256, 0, 0, 0.0, None) == NULL
    check_pages_of(lambda p: f(pg=p), (-4, -8))
    for bad in ({"b": 0}, {"hq": 3}, {"hkv": 0}, {"d": 80}, {"window": -1}, {"sinks": -1}, {"scale": -2.0},
                {"scale": float("nan")}, {"q_batch": 4}, {"q_batch": -8}, {"b": 1 << 20, "hq": 64}):
        assert f(**bad) == ARG, bad
    assert lib.cpattn_decode_paged_workspace_bytes(2, 3, 2, 64, 160, 0, 0) == 0


def test_decode_shared_arguments(lib):  # noqa: F811
    def f(ptr=(P,) * 5, pg=None, off=P, groups=2, most=2, ws=P, n=1 << 40, b=3, hq=4, hkv=2, d=64, q_batch=256, scale=0.0):
        q, ln, sh, o, lse = ptr
        return lib.cpattn_decode_shared(q, pages() if pg is None else pg, ln, sh, off, groups, most, o, lse, ws, n, b, hq,
                                        hkv, d, q_batch, scale, None)

    for i in range(5):
        assert f((P,) * i + (None,) + (P,) * (4 - i)) == NULL
    assert f(ws=None) == NULL and f(ws=ODD) == MISALIGNED
    assert f((ODD,) + (P,) * 4) == MISALIGNED and f(off=ctypes.c_void_p(4098)) == MISALIGNED
    assert lib.cpattn_decode_shared(P, None, P, P, P, 2, 2, P, P, P, 1, 3, 4, 2, 64, 256, 0.0, None) == NULL
    check_pages_of(lambda p: f(pg=p), (-4, -8))
    for bad in ({"b": 0}, {"hq": 3}, {"d": 80}, {"groups": 0}, {"groups": 4}, {"most": 0}, {"most": 4}, {"off": None},
                {"scale": -2.0}, {"q_batch": 4}):
        assert f(**bad) == ARG, bad
    # more units than results are numbered for: every sequence a group of all of them
    many = 1 << 15
    if torch.cuda.is_available():
        assert f(b=many, hq=64, hkv=64, groups=many, most=many, pg=pages(hkv=64), q_batch=4096) == ARG
    assert lib.cpattn_decode_shared_workspace_bytes(many, 64, 64, 64, many, many) == 0
    for bad in ((3, 4, 2, 64, 0, 2), (3, 4, 2, 64, 4, 2), (3, 4, 2, 64, 2, 0), (3, 4, 2, 64, 2, 4), (3, 4, 3, 64, 2, 2),
                (0, 4, 2, 64, 1, 1), (3, 4, 2, 96, 2, 2)):
        assert lib.cpattn_decode_shared_workspace_bytes(*bad) == 0
    if torch.cuda.is_available():
        need = lib.cpattn_decode_shared_workspace_bytes(3, 4, 2, 64, 2, 2)
        assert need > 0 and f(n=need - 1) == SMALL


def test_binding_refuses_before_it_needs_a_device(lib):  # noqa: F811
    import context_blockwise_causal_gb300 as cp

    x, q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    pool, t = torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 3, dtype=torch.int32)
    ln = torch.ones(1, dtype=torch.int32)
    for call in (lambda: cp.cpattn_append_paged(x, x, pool, pool, t, ln), lambda: cp.cpattn_append_paged(x.float(), x, pool, pool, t, ln),
                 lambda: cp.cpattn_append_paged(None, x, pool, pool, t, ln), lambda: cp.cpattn_decode_paged(q, pool, pool, t, ln),
                 lambda: cp.cpattn_decode_paged(q.half(), pool, pool, t, ln), lambda: cp.cpattn_decode_shared(q, pool, pool, t, ln, ln),
                 lambda: cp.cpattn_decode_shared(q, None, pool, t, ln, ln)):
        with pytest.raises(TypeError):
            call()


def test_oracle_pages_by_hand():
    pool = torch.arange(4 * 16, dtype=torch.float64).view(4, 16, 1, 1)  # 4 pages of 16 tokens: value 16 page + slot
    got = oracle.held_tokens(pool, [2, 0, 9], 34)[:, 0, 0]
    assert got.tolist() == [32.0 + i for i in range(16)] + [float(i) for i in range(16)] + [0.0, 0.0]
    # two sequences: three tokens that end at 17 (places 14, 15, 16), one without room
    k = torch.tensor([1.0, 2.0, 3.0, 4.0]).view(4, 1, 1)
    q, kp, vp, written, kept = oracle.append_tokens(k, -k, None, pool, pool, [[2, 0, 9], [1, 1, 1]], [17, 0], [3, 1])
    assert q is None and kept.tolist() == [True, True, True, False] and written.sum() == 3
    assert (kp[2, 14, 0, 0], kp[2, 15, 0, 0], kp[0, 0, 0, 0], vp[0, 0, 0, 0]) == (1.0, 2.0, 3.0, -3.0)
    assert torch.equal(kp[~written], pool[~written]) and torch.equal(vp[~written], pool[~written])
    # a quarter turn per token: (1, 0) at place 17 - 1 stays, one place on it is (0, 1)
    x = torch.tensor([1.0, 0.0]).view(1, 1, 2).expand(2, 1, 2)
    wide = torch.zeros(4, 16, 1, 2, dtype=torch.float64)
    q, kp, *_ = oracle.append_tokens(x, x, x, wide, wide, [[3, 1]], [18], [2], torch.tensor([torch.pi / 2], dtype=torch.float64))
    want = torch.tensor([[1.0, 0.0], [0.0, 1.0]], dtype=torch.float64)
    assert torch.allclose(kp[1, :2, 0], want, atol=1e-12) and torch.allclose(q[:, 0], want, atol=1e-12)

"""Refusals of the serving calls, answered on the host without a GPU: the C ABI's argument checks and
the binding's checks of tensors (no launch is made here)."""
import ctypes

import pytest
import torch

import scaled_dot_product_16_b200 as sdpa
from scaled_dot_product_16_b200 import build as sdpa_build
from tests.test_abi import FakeCuda

INVALID, UNSUP, OK = sdpa.ATTN_ERR_INVALID, sdpa.ATTN_ERR_UNSUPPORTED, sdpa.ATTN_OK
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def lib():
    sdpa_build.build()
    return sdpa.load_library()


@pytest.fixture
def on_cuda0(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(sdpa, "_stream", lambda s: 0)


def _call(f, defaults, kw):
    a = dict(defaults)
    assert set(kw) <= set(a), kw
    a.update(kw)
    return f(*a.values())


def test_sinks(lib):
    d = dict(q=16, k=16, v=16, cq=None, ck=None, B=1, Sq=8, Skv=8, Nq=2, Nkv=1, D=64, scale=0.125, window=4,
             sinks=1, dtype=0, layout=0, out=16, m=None, l=None, stream=None)

    def f(**kw):
        return _call(lib.attn_fwd_sinks, d, kw)

    assert f(window=0) == INVALID and f(window=-1) == INVALID and f(sinks=-1) == INVALID
    assert f(D=96) == UNSUP and f(D=769) == INVALID and f(Nq=3, Nkv=2) == INVALID
    assert f(q=None) == INVALID and f(q=18) == INVALID and f(scale=0.0) == INVALID
    assert f(m=16) == INVALID and f(layout=1) == INVALID and f(dtype=7) == INVALID
    assert f(B=0) == OK and f(Sq=0, window=1 << 62, sinks=1 << 62) == OK


def test_a_band_without_limits_is_not_empty(lib):
    """Both limits of a band at 2^30 or more are unbounded; their sum does not wrap round."""
    for pre, nxt in ((1 << 30, 1 << 30), (1 << 40, 1 << 30), ((1 << 63) - 1, (1 << 63) - 1)):
        rc = lib.attn_fwd_masked(16, 16, 16, None, None, 0, 8, 8, 2, 1, 64, 64, 0.125, 3, pre, nxt, None, 0, 0, 1, 0, 16,
                                 None, None, None)
        assert rc == OK, (pre, nxt)


def test_decode(lib):
    n = ctypes.c_int64(0)
    ref = ctypes.byref(n)
    assert lib.attn_decode_workspace_size(32, 8, 128, 0, ref) == OK and n.value > 0
    need = n.value
    assert lib.attn_decode_workspace_size(32, 8, 128, 0, None) == INVALID
    assert lib.attn_decode_workspace_size(32, 8, 257, 1, ref) == UNSUP
    assert lib.attn_decode_workspace_size(32, 5, 128, 0, ref) == INVALID
    assert lib.attn_decode_workspace_size(257, 1, 128, 0, ref) == INVALID
    assert lib.attn_decode_workspace_size(32, 8, 128, 3, ref) == INVALID
    d = dict(q=16, k=16, v=16, table=16, lens=16, B=2, Nq=32, Nkv=8, D=128, num_pages=9, page_size=16, max_pages=4,
             stride=0, scale=0.1, window=8, sinks=0, dtype=0, layout=1, ws=16, ws_bytes=need, out=16, m=None, l=None,
             stream=None)

    def f(**kw):
        return _call(lib.attn_decode_paged, d, kw)

    for bad in (dict(dtype=5), dict(layout=2), dict(B=-1), dict(Nq=12), dict(Nq=0), dict(D=0), dict(num_pages=-1),
                dict(page_size=0), dict(max_pages=-1), dict(stride=16 * 8 * 128 - 1), dict(stride=-1), dict(scale=0.0),
                dict(scale=float("inf")), dict(scale=float("nan")), dict(window=0), dict(sinks=-1), dict(ws=None),
                dict(ws=24), dict(ws_bytes=need - 1), dict(q=None), dict(out=None), dict(k=None), dict(v=None),
                dict(table=None), dict(lens=None), dict(m=16), dict(l=16), dict(Nkv=0), dict(Nq=512, Nkv=1)):
        assert f(**bad) == INVALID, bad
    assert f(D=300) == UNSUP
    assert f(page_size=1 << 20, max_pages=1 << 11) == UNSUP  # more than 2^30 positions a row
    assert f(B=0, q=None, ws=16) == OK


def test_append(lib):
    d = dict(k=16, v=16, table=16, lens=16, cu=None, T=2, B=2, Nkv=8, D=128, num_pages=9, page_size=16, max_pages=4,
             stride=0, dtype=0, layout=1, kc=16, vc=16, stream=None)

    def f(**kw):
        return _call(lib.attn_cache_append, d, kw)

    for bad in (dict(dtype=3), dict(layout=5), dict(T=3), dict(T=-1, cu=16), dict(k=None), dict(v=None), dict(kc=None),
                dict(vc=None), dict(table=None), dict(lens=None), dict(page_size=0), dict(stride=5), dict(Nkv=0),
                dict(D=0), dict(B=0, cu=16)):
        assert f(**bad) == INVALID, bad
    assert f(page_size=1 << 20, max_pages=1 << 11) == UNSUP
    assert f(T=0, B=0) == OK


def test_page_calls(lib):
    fork = dict(table=16, src=16, ref=16, lens=None, rows_in=2, rows_out=3, max_pages=4, num_pages=9, out=32,
                ref_out=16, lens_out=None, stream=None)

    def f(**kw):
        return _call(lib.attn_cache_fork, fork, kw)

    for bad in (dict(rows_in=-1), dict(max_pages=0), dict(num_pages=-1), dict(lens=16), dict(lens_out=16),
                dict(out=16), dict(table=None), dict(src=None), dict(out=None), dict(ref=None), dict(ref_out=None)):
        assert f(**bad) == INVALID, bad
    assert f(rows_in=8193) == UNSUP and f(rows_out=8193) == UNSUP and f(rows_in=4096, max_pages=1 << 18) == UNSUP

    res = dict(table=16, ref=16, lens=16, new=None, B=2, max_pages=4, num_pages=9, page_size=16, copies=16, stream=None)

    def r(**kw):
        return _call(lib.attn_cache_reserve, res, kw)

    for bad in (dict(B=-1), dict(page_size=0), dict(lens=None), dict(copies=None), dict(table=None), dict(ref=None)):
        assert r(**bad) == INVALID, bad
    assert r(B=8193) == UNSUP and r(page_size=1 << 29) == UNSUP and r(B=0) == OK

    com = dict(table=16, ref=16, rows=2, max_pages=4, num_pages=9, out=16, ref_out=16, pmap=16, copies=16, live=16,
               stream=None)

    def c(**kw):
        return _call(lib.attn_cache_compact, com, kw)

    for bad in (dict(rows=-1), dict(table=None), dict(ref=None), dict(out=None), dict(ref_out=None), dict(pmap=None),
                dict(copies=None), dict(live=None), dict(num_pages=-1)):
        assert c(**bad) == INVALID, bad
    assert c(rows=8193) == UNSUP

    ev = dict(table=16, ref=16, lens=16, B=2, max_pages=4, num_pages=9, page_size=16, window=8, sinks=0, stream=None)

    def e(**kw):
        return _call(lib.attn_cache_evict, ev, kw)

    for bad in (dict(B=-1), dict(page_size=0), dict(window=0), dict(sinks=-1), dict(table=None), dict(ref=None),
                dict(lens=None), dict(max_pages=-1)):
        assert e(**bad) == INVALID, bad
    assert e(B=8193) == UNSUP and e(page_size=1 << 29) == UNSUP and e(B=0) == OK

    cp = dict(copies=16, n=2, num_pages=9, page_elems=64, stride=0, dtype=0, k=16, v=16, stream=None)

    def p(**kw):
        return _call(lib.attn_cache_copy, cp, kw)

    for bad in (dict(n=-1), dict(num_pages=-1), dict(page_elems=0), dict(stride=63), dict(dtype=4), dict(copies=None),
                dict(copies=20), dict(k=None), dict(v=None)):
        assert p(**bad) == INVALID, bad
    assert p(n=0) == OK


def test_binding_refuses_wrong_tensors(lib, on_cuda0):
    B, Nq, Nkv, D, ps, mp, n = 2, 4, 2, 64, 16, 3, 5
    ws = sdpa.attn_decode_workspace_size(Nq=Nq, Nkv=Nkv, D=D, dtype=sdpa.ATTN_BF16)
    pool = n * ps * Nkv * D

    def call(**kw):
        a = dict(q=FakeCuda(B * Nq * D, BF), k_cache=FakeCuda(pool, BF), v_cache=FakeCuda(pool, BF),
                 page_table=FakeCuda(B * mp, I32), seq_lens=FakeCuda(B, I32), B=B, Nq=Nq, Nkv=Nkv, D=D, num_pages=n,
                 page_size=ps, max_pages=mp, scale=0.1, dtype=sdpa.ATTN_BF16, layout=sdpa.ATTN_TND,
                 workspace=FakeCuda(ws, torch.uint8), out=FakeCuda(B * Nq * D, BF))
        a.update(kw)
        sdpa.attn_decode_paged(**a)

    for kw, msg in ((dict(q=FakeCuda(B * Nq * D - 1, BF)), "q holds"), (dict(q=FakeCuda(B * Nq * D, F32)), "bfloat16"),
                    (dict(k_cache=FakeCuda(pool - 1, BF)), "k_cache holds"),
                    (dict(v_cache=FakeCuda(pool, BF), page_stride=ps * Nkv * D + 8), "k_cache holds"),
                    (dict(page_table=FakeCuda(B * mp - 1, I32)), "page_table holds"),
                    (dict(page_table=FakeCuda(B * mp, torch.int64)), "int32"),
                    (dict(seq_lens=FakeCuda(B - 1, I32)), "seq_lens holds"),
                    (dict(workspace=FakeCuda(ws, F32)), "uint8"), (dict(out=FakeCuda(1, BF)), "out holds"),
                    (dict(v_cache=FakeCuda(pool, BF, index=1)), "current device")):
        with pytest.raises(ValueError, match=msg):
            call(**kw)
    with pytest.raises(sdpa.AttnError):
        call(workspace=FakeCuda(ws - 1, torch.uint8))

    # sizes and scales of numpy are numbers too (refused by the library here, after the binding took them)
    import numpy as np
    with pytest.raises(sdpa.AttnError, match="invalid"):
        call(B=np.int64(B), Nq=np.int32(Nq), scale=np.float32(0.0))

    class Half:
        """A view [num_pages, ...] of every second page of a pool, on a machine without a GPU."""
        is_cuda, dtype, device = True, BF, torch.device("cuda", 0)

        def __init__(self, pages, elems, stride, dense=True):
            self.shape, self.elems, self.st, self.dense = (pages, elems), elems, stride, dense

        def is_contiguous(self):
            return False

        def dim(self):
            return 2

        def stride(self, i):
            return self.st

        def numel(self):
            return self.shape[0] * self.elems

        def data_ptr(self):
            return 256

        def __getitem__(self, i):
            x = FakeCuda(self.elems, BF)
            x.is_contiguous = lambda: self.dense
            return x

    pe = ps * Nkv * D
    for kw, msg in ((dict(k_cache=Half(n, pe, 2 * pe)), "elements apart"),
                    (dict(k_cache=Half(n - 1, pe, 2 * pe), page_stride=2 * pe), "pages of"),
                    (dict(k_cache=Half(n, pe, 2 * pe, dense=False), page_stride=2 * pe), "contiguous")):
        with pytest.raises(ValueError, match=msg):
            call(**kw)
    with pytest.raises(ValueError, match="copies holds"):
        sdpa.attn_cache_reserve(FakeCuda(B * mp, I32), FakeCuda(n, I32), FakeCuda(B, I32), None, FakeCuda(3, I32), B=B,
                                max_pages=mp, num_pages=n, page_size=ps)
    with pytest.raises(ValueError, match="page_table_out"):
        sdpa.attn_cache_fork(FakeCuda(B * mp, I32), FakeCuda(3, I32), FakeCuda(n, I32), FakeCuda(B * mp, I32),
                             FakeCuda(n, I32), rows_in=B, rows_out=3, max_pages=mp, num_pages=n)

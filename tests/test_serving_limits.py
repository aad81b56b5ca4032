"""Refusals of the serving calls, answered on the host without a GPU: tensors of the CPU, and sizes past the limits
that the header states."""
import pytest
import torch

import scaled_dot_product_16_b200 as sdpa
from scaled_dot_product_16_b200 import build as sdpa_build

BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def lib():
    sdpa_build.build()
    return sdpa.load_library()


def test_tensors_of_the_cpu_are_refused(lib):
    """Whether a device is there or not: the first tensor that is not on it is named."""
    B, Nq, Nkv, D, ps, mp, n = 2, 4, 2, 64, 16, 3, 5
    x, i = torch.zeros(n * ps * Nkv * D, dtype=BF), torch.zeros(64, dtype=I32)
    ws = torch.zeros(sdpa.attn_decode_workspace_size(Nq=Nq, Nkv=Nkv, D=D, dtype=sdpa.ATTN_BF16), dtype=torch.uint8)
    page = dict(Nkv=Nkv, D=D, num_pages=n, page_size=ps, max_pages=mp, dtype=sdpa.ATTN_BF16, layout=sdpa.ATTN_TND)
    calls = [
        lambda: sdpa.attn_fwd_sinks(x, x, x, B=1, Sq=8, Skv=8, Nq=Nq, Nkv=Nkv, D=D, scale=0.1, window_tokens=4,
                                    dtype=sdpa.ATTN_BF16, layout=sdpa.ATTN_BHSD, out=x),
        lambda: sdpa.attn_decode_paged(x, x, x, i, i, B=B, Nq=Nq, scale=0.1, workspace=ws, out=x, **page),
        lambda: sdpa.attn_cache_append(x, x, i, i, x, x, T=B, B=B, **page),
        lambda: sdpa.attn_cache_fork(i, i, i, i, i, rows_in=B, rows_out=B, max_pages=mp, num_pages=n),
        lambda: sdpa.attn_cache_reserve(i, i, i, None, i, B=B, max_pages=mp, num_pages=n, page_size=ps),
        lambda: sdpa.attn_cache_evict(i, i, i, B=B, max_pages=mp, num_pages=n, page_size=ps, window_tokens=4),
        lambda: sdpa.attn_cache_compact(i, i, i, i, i, i, i, rows=B, max_pages=mp, num_pages=n),
        lambda: sdpa.attn_cache_copy(x, x, i, n_copies=2, num_pages=n, page_elems=ps * Nkv * D, dtype=sdpa.ATTN_BF16),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="must be on a CUDA device"):
            call()


UNSUP, MAX32 = sdpa.ATTN_ERR_UNSUPPORTED, 2 ** 31 - 1


def test_pools_of_more_than_2_30_pages(lib):
    """The page kernels step over the pool in 32-bit integers, 8,192 pages at a time."""
    for n in ((1 << 30) + 1, MAX32 - 8192, MAX32):
        assert lib.attn_cache_fork(16, 16, 16, None, 2, 2, 4, n, 32, 32, None, None) == UNSUP
        assert lib.attn_cache_reserve(16, 16, 16, None, 2, 4, n, 16, 16, None) == UNSUP
        assert lib.attn_cache_evict(16, 16, 16, 2, 4, n, 16, 8, 0, None) == UNSUP
        assert lib.attn_cache_compact(16, 16, 2, 4, n, 16, 16, 16, 16, 16, None) == UNSUP


def test_more_than_2_30_rows(lib):
    """decode divides the rows among its threads and append searches them, in 32-bit integers."""
    n = 1 << 40
    for B in ((1 << 30) + 1, MAX32):
        assert lib.attn_decode_paged(16, 16, 16, 16, 16, B, 1, 1, 64, 9, 16, 4, 0, 0.1, 8, 0, 0, 1, 16, n, 16, None,
                                     None, None) == UNSUP
        assert lib.attn_cache_append(16, 16, 16, 16, 16, 8, B, 8, 128, 9, 16, 4, 0, 0, 1, 16, 16, None) == UNSUP


def test_more_than_2_30_new_tokens(lib):
    for T in ((1 << 30) + 1, MAX32):
        assert lib.attn_cache_append(16, 16, 16, 16, 16, T, 8, 8, 128, 9, 16, 4, 0, 0, 1, 16, 16, None) == UNSUP


def test_a_window_over_more_than_2_30_keys(lib):
    """ATTN_WINDOW_ALL is 2^30: it would not be every key there."""
    for sq, sk in ((1, (1 << 30) + 1), (1, MAX32), ((1 << 30) + 1, 8), (MAX32, MAX32)):
        assert lib.attn_fwd_sinks(16, 16, 16, None, None, 1, sq, sk, 1, 1, 1, 0.5, sdpa.ATTN_WINDOW_ALL, 0, 1, 0, 16,
                                  None, None, None) == UNSUP


def test_grow_refuses_what_reserve_does(lib):
    INVALID, OK = sdpa.ATTN_ERR_INVALID, sdpa.ATTN_OK
    d = dict(table=16, ref=16, lens=16, new=None, live=0, B=2, max_pages=4, num_pages=9, page_size=16, copies=16,
             new_lens=32, stream=None)

    def f(**kw):
        return lib.attn_cache_grow(*dict(d, **kw).values())

    for bad in (dict(B=-1), dict(page_size=0), dict(lens=None), dict(copies=None), dict(table=None), dict(ref=None),
                dict(new_lens=None), dict(new_lens=16), dict(new=32), dict(live=2), dict(live=-1)):
        assert f(**bad) == INVALID, bad
    assert f(B=8193) == UNSUP and f(page_size=1 << 29) == UNSUP and f(num_pages=MAX32) == UNSUP and f(B=0) == OK
    i = torch.zeros(64, dtype=I32)
    with pytest.raises(ValueError, match="must be on a CUDA device"):
        sdpa.attn_cache_grow(i, i, i, None, i, i, B=2, max_pages=3, num_pages=5, page_size=4)

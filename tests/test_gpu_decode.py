"""attn_decode_paged on the GPU against the plain float64 form (tests/serving_ref.py).

Tolerances, derived from the kernels' arithmetic (eps = 2^-24, a rounding of fp32):
  * a score is a sum of D exact (16-bit) or rounded (fp32) products in fp32: off by at most
    (D + 1) eps S, with S the largest scale * sum |q_d k_d| of the row; times log2 e, minus the running
    maximum and through exp2 (2 units in the last place) it makes a weight's relative error
    e_w <= (D + 1) eps S + 4 eps (|s| + 1), with |s| <= S;
  * weights go to the products with V in 16 bits where the kernel uses the tensor cores: 2^-11 for fp16,
    2^-16 for bf16 (two terms); the sums over n keys are off by n eps at most;
  * the output is the quotient of two such sums, so its error is at most c A with
    c = 2 e_w + u + 2 n eps and A = sum w |v|, plus half a unit of the output type.
  * softmax max: (D + 2) eps S; softmax sum: relative 2 e_w + n eps.
"""
import numpy as np
import pytest
import torch

import scaled_dot_product_16_b200 as sdpa
from scaled_dot_product_16_b200 import workloads as W
from tests import gpu_util as G
from tests import serving_ref as R

pytestmark = pytest.mark.gpu

BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32
IDS = {BF: "bf16", F16: "f16", F32: "f32"}.get
EPS = 2.0 ** -24
UNIT = {BF: 2.0 ** -16, F16: 2.0 ** -11, F32: 0.0}
ALL = sdpa.ATTN_WINDOW_ALL


class Case:
    """A cache on the CPU in which everything that no row may see is NaN, and the call's arguments."""

    def __init__(self, lens, Nq, Nkv, D, dtype, *, page=16, layout=W.TND, window=ALL, sinks=0, seed=0, extra=3,
                 gap_pages=False):
        rng = np.random.default_rng(seed)
        self.lens, self.page, self.layout, self.window, self.sinks = lens, page, layout, window, sinks
        self.B, self.Nq, self.Nkv, self.D, self.dtype = len(lens), Nq, Nkv, D, dtype
        self.max_pages = max(1, max(-(-n // page) for n in lens)) + 1
        self.num_pages = sum(-(-n // page) for n in lens) + extra
        table, _ = R.live_table(rng, lens, page, self.max_pages, self.num_pages)
        seen = np.zeros((self.num_pages, page), bool)
        for b, n in enumerate(lens):
            for j in range(n):
                if j >= n - window or j < sinks:
                    seen[table[b][j // page], j % page] = True
        if gap_pages:  # pages without a visible position are not in the table any more
            table = [[p if p >= 0 and seen[p].any() else -1 for p in row] for row in table]
        self.table = torch.tensor(table, dtype=torch.int32)
        shape = (self.num_pages, page, Nkv, D)
        mask = torch.from_numpy(seen)[:, :, None, None]
        k = torch.where(mask, W.randn(shape, 7 * seed + 1), torch.nan).to(dtype)
        v = torch.where(mask, W.randn(shape, 7 * seed + 2), torch.nan).to(dtype)
        if layout == W.BHSD:
            k, v = k.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous()
        self.k, self.v = k, v
        self.q = W.randn((self.B, Nq, D), 7 * seed + 3).to(dtype)
        self.scale = D ** -0.5

    def workspace(self):
        n = sdpa.attn_decode_workspace_size(Nq=self.Nq, Nkv=self.Nkv, D=self.D, dtype=W.dtype_code(self.dtype))
        return torch.zeros(n, dtype=torch.uint8, device="cuda")

    def kwargs(self):
        return dict(B=self.B, Nq=self.Nq, Nkv=self.Nkv, D=self.D, num_pages=self.num_pages, page_size=self.page,
                    max_pages=self.max_pages, scale=self.scale, window_tokens=self.window, sink_tokens=self.sinks,
                    dtype=W.dtype_code(self.dtype), layout=self.layout)

    def dev(self):
        return [x.cuda() for x in (self.q, self.k, self.v, self.table)] + [
            torch.tensor(self.lens, dtype=torch.int32, device="cuda")]

    def run(self, ws=None, stats=True, args=None, status=0, **kw):
        out = G.Guarded((self.B, self.Nq, self.D), self.dtype)
        m = G.Guarded((self.B, self.Nq), F32) if stats else None
        l = G.Guarded((self.B, self.Nq), F32) if stats else None
        a = dict(self.kwargs(), **kw)
        sdpa.attn_decode_paged(*(args or self.dev()), workspace=self.workspace() if ws is None else ws, out=out.t,
                               softmax_max=m.t if stats else None, softmax_sum=l.t if stats else None, **a)
        assert sdpa.attn_get_last_error() == status
        for g in (out, m, l):
            if g is not None:
                g.check()
        return out.t.cpu(), (m.t.cpu() if stats else None), (l.t.cpu() if stats else None)

    def check(self, **kw):
        got = self.run(**kw)
        ref = R.decode(self.q, self.k, self.v, self.table, self.lens, layout=self.layout, page_size=self.page,
                       scale=self.scale, window=self.window, sinks=self.sinks)
        hold(got, ref, self.D, self.dtype)
        return got


def hold(got, ref, D, dtype):
    out, m, l = (x.double() for x in got)
    ro, rm, rl, A, S, seen = ref
    n = torch.from_numpy(seen).double()[:, None]
    ew = (D + 1) * EPS * S + 4 * EPS * (S + 1)
    half = torch.exp2(torch.floor(torch.log2(ro.abs().clamp(min=2.0 ** (-14 if dtype == F16 else -126))))) * (
        torch.finfo(dtype).eps / 2)
    tol = half + (2 * ew + UNIT[dtype] + 2 * n * EPS)[..., None] * A
    err = (out - ro).abs()
    assert torch.all(err <= tol), f"out: {float((err / tol.clamp(min=1e-300)).max())} of its bound"
    empty = torch.isneginf(rm)
    assert torch.equal(torch.isneginf(m), empty) and torch.all(l[empty] == 0) and torch.all(out[empty] == 0)
    full = ~empty
    assert torch.all((m - rm).abs()[full] <= ((D + 2) * EPS * S)[full])
    assert torch.all((l / rl - 1).abs()[full] <= (2 * ew + n * EPS)[full])


LENS = [0, 1, 15, 16, 17, 63, 64, 65, 500, 1025]


@pytest.mark.parametrize("dtype", [BF, F16, F32], ids=IDS)
@pytest.mark.parametrize("layout", [W.TND, W.BHSD], ids=["tnd", "bhsd"])
@pytest.mark.parametrize("page", [1, 7, 16, 24, 128])
def test_ragged_lengths_and_pages(dtype, layout, page):
    Case(LENS, 8, 2, 128, dtype, page=page, layout=layout, seed=page).check()


@pytest.mark.parametrize("dtype", [BF, F32], ids=IDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [(1, 1), (3, 3), (2, 1), (6, 2), (5, 1), (8, 1), (9, 1), (32, 2), (40, 1)])
def test_heads(dtype, D, heads):
    Case([70, 3, 333], *heads, D, dtype, seed=D + heads[0]).check()


@pytest.mark.parametrize("dtype", [BF, F16, F32], ids=IDS)
@pytest.mark.parametrize("D", [1, 8, 33, 80, 96, 192, 256])
def test_head_sizes(dtype, D):
    Case([70, 3, 333], 6, 2, D, dtype, seed=D).check()


@pytest.mark.parametrize("dtype", [BF, F16, F32], ids=IDS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 4), (100, 130), (129, 64), (16, 16), (2000, 5), (ALL, 9)])
def test_window_and_sinks(dtype, window, sinks):
    Case([1, 40, 130, 200, 1000, 2000], 4, 2, 64, dtype, window=window, sinks=sinks, seed=sinks, gap_pages=True).check()
    Case([1, 999], 2, 2, 128, dtype, window=window, sinks=sinks, page=24, layout=W.BHSD, seed=sinks,
         gap_pages=True).check()


@pytest.mark.parametrize("dtype", [BF, F32], ids=IDS)
def test_one_long_sequence_among_many_short_ones(dtype):
    rng = np.random.default_rng(1)
    Case([9000] + [int(x) for x in rng.integers(0, 40, 150)], 4, 1, 64, dtype, seed=1).check()


@pytest.mark.parametrize("dtype", [BF, F32], ids=IDS)
def test_more_units_than_blocks(dtype):
    rng = np.random.default_rng(2)
    Case([int(x) for x in rng.integers(0, 200, 300)], 8, 4, 64, dtype, seed=2).check()


def test_more_rows_than_threads():
    rng = np.random.default_rng(3)
    Case([int(x) for x in rng.integers(0, 6, 2500)], 2, 1, 64, BF, seed=3, page=4).check()


@pytest.mark.parametrize("dtype", [BF, F16, F32], ids=IDS)
def test_large_scores(dtype):
    """Scores of hundreds: one key takes nearly all the weight, wherever in the sequence it lies."""
    c = Case([700, 64, 129], 8, 2, 128, dtype, seed=4)
    c.q = c.q * 32
    c.check()


@pytest.mark.parametrize("dtype", [BF, F32], ids=IDS)
def test_interleaved_pools(dtype):
    """K and V as the halves of one [num_pages, 2, ...] tensor."""
    c = Case([70, 0, 333], 8, 2, 128, dtype, seed=5)
    q, k, v, table, lens = c.dev()
    kv = torch.stack([k, v], 1)
    got = c.run(args=[q, kv[:, 0], kv[:, 1], table, lens], page_stride=2 * 16 * 2 * 128)
    for x, y in zip(got, c.run()):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [BF, F16, F32], ids=IDS)
def test_unaligned_tensors(dtype):
    """Addresses off the 16-byte boundary take the path without vector loads."""
    c = Case([70, 0, 333], 8, 2, 128, dtype, seed=6)
    want = c.check()
    args = c.dev()
    for i in range(3):
        args2 = list(args)
        x = args[i]
        buf = torch.empty(x.numel() + 1, dtype=dtype, device="cuda")
        buf[1:] = x.reshape(-1)
        args2[i] = buf[1:].view(x.shape)
        got = c.run(args=args2)
        ref = R.decode(c.q, c.k, c.v, c.table, c.lens, layout=c.layout, page_size=c.page, scale=c.scale,
                       window=c.window, sinks=c.sinks)
        hold(got, ref, c.D, dtype)
        assert want[0].shape == got[0].shape


def test_repeats_and_shared_workspace_are_bit_identical():
    """One workspace through calls of several sizes; each call's result is that of a fresh one."""
    big = Case([9000, 3, 700], 8, 2, 128, BF, seed=7)
    ws = big.workspace()
    cases = [big, Case([65], 8, 2, 128, BF, seed=8), Case([4000] * 5, 8, 2, 128, BF, seed=9),
             Case([0, 1], 4, 1, 64, F32, seed=10)]
    fresh = [c.run() for c in cases]
    for _ in range(3):
        for c, want in zip(cases, fresh):
            for x, y in zip(want, c.run(ws=ws)):
                assert torch.equal(x, y)
    assert torch.equal(big.run(stats=False)[0], fresh[0][0])
    assert int(ws[:4 * 2 * 512].view(torch.int32).abs().sum()) == 0  # the arrival counters


def test_graph_replay_with_new_lengths():
    """A captured call reads the lengths and the table of the moment it is replayed."""
    c = Case([900, 65, 400], 8, 2, 128, BF, seed=11)
    args, ws = c.dev(), c.workspace()
    out = torch.empty((3, 8, 128), dtype=BF, device="cuda")
    sdpa.attn_decode_paged(*args, workspace=ws, out=out, **c.kwargs())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sdpa.attn_decode_paged(*args, workspace=ws, out=out, **c.kwargs())
    for lens in ([900, 65, 400], [1, 0, 399], [16, 65, 17]):
        args[4].copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        c.lens = lens
        assert torch.equal(out.cpu(), c.run()[0])


def test_two_streams_with_a_workspace_each():
    cases = [Case([5000, 100], 8, 2, 128, BF, seed=12), Case([64] * 40, 8, 2, 64, F16, seed=13)]
    want = [c.run()[0] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    args, ws = [c.dev() for c in cases], [c.workspace() for c in cases]
    outs = [torch.empty_like(a[0]) for a in args]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, a, w, o in zip(cases, streams, args, ws, outs):
            with torch.cuda.stream(s):
                sdpa.attn_decode_paged(*a, workspace=w, out=o, **c.kwargs())
    torch.cuda.synchronize()
    for o, x in zip(outs, want):
        assert torch.equal(o.cpu(), x)


@pytest.mark.parametrize("dtype", [BF, F32], ids=IDS)
def test_bad_lengths_and_pages(dtype):
    """A length outside the table: the row is empty. A page outside the pool: its keys are left out."""
    c = Case([70, 300, 40, 33], 8, 2, 128, dtype, seed=14)
    args = c.dev()
    args[4].copy_(torch.tensor([70, -1, c.max_pages * 16 + 1, 33], dtype=torch.int32))
    c.lens = [70, 0, 0, 33]
    got = c.run(args=args, status=sdpa.ATTN_ERR_DATA)
    hold(got, R.decode(c.q, c.k, c.v, c.table, c.lens, layout=c.layout, page_size=16, scale=c.scale, window=ALL,
                       sinks=0), 128, dtype)
    for bad in (-1, c.num_pages, 2 ** 31 - 1):
        d = Case([70, 300, 40, 33], 8, 2, 128, dtype, seed=14)
        d.table[1, 5] = bad
        d.table[3, :] = bad
        hold(d.run(status=sdpa.ATTN_ERR_DATA),
             R.decode(d.q, d.k, d.v, d.table, d.lens, layout=d.layout, page_size=16, scale=d.scale, window=ALL,
                      sinks=0), 128, dtype)


def test_empty_batch_and_rows():
    c = Case([0, 0, 0], 4, 2, 64, BF, seed=15)
    out, m, l = c.run()
    assert not out.any() and torch.all(torch.isneginf(m)) and not l.any()


@pytest.mark.parametrize("dtype", [BF, F32], ids=IDS)
def test_pools_beyond_32_bit_offsets(dtype):
    """A pool of more than 2^31 elements (and bytes past 2^32); the row's pages lie at its end."""
    Nkv, D, page = 8, 128, 64
    per = page * Nkv * D
    num = 2 ** 31 // per + 9
    c = Case([200], 16, Nkv, D, dtype, page=page, seed=16)
    k = torch.empty((num, page, Nkv, D), dtype=dtype, device="cuda")
    v = torch.empty_like(k)
    table = torch.full_like(c.table, -1)
    for i in range(4):
        table[0, i] = num - 1 - i
        k[num - 1 - i].copy_(c.k[c.table[0, i]])
        v[num - 1 - i].copy_(c.v[c.table[0, i]])
    args = [c.q.cuda(), k, v, table.cuda(), torch.tensor([200], dtype=torch.int32, device="cuda")]
    for x, y in zip(c.check(), c.run(args=args, num_pages=num)):
        assert torch.equal(x, y)


def test_scores_of_nan_keys_reach_the_output():
    """NaN in a visible key is not swallowed."""
    for dtype, D in ((BF, 128), (F32, 128), (F16, 80)):
        c = Case([40, 40], 4, 2, D, dtype, seed=17)
        c.k[int(c.table[0, 1]), 3] = float("nan")
        out = c.run()[0]
        assert torch.isnan(out[0]).all() and not torch.isnan(out[1]).any()

"""attn_fwd_sinks on the GPU against the plain float64 form (tests/serving_ref.py). Tolerances are
those of the other forward tests (tests/gpu_util.py); the arithmetic is the same kernels'."""
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


def _run(inp, window, sinks, stats=True, dev=None):
    q, k, v, cq, ck = dev if dev is not None else G.to_dev(inp)
    out = G.Guarded(tuple(q.shape), q.dtype)
    shape = tuple(q.shape[:-1])
    m = G.Guarded(shape, F32) if stats else None
    l = G.Guarded(shape, F32) if stats else None
    sdpa.attn_fwd_sinks(q, k, v, cu_seqlens_q=cq, cu_seqlens_kv=ck, B=inp.B, Sq=inp.Sq, Skv=inp.Skv, Nq=inp.Nq,
                        Nkv=inp.Nkv, D=inp.D, scale=inp.scale, window_tokens=window, sink_tokens=sinks, dtype=inp.dtype,
                        layout=inp.layout, out=out.t, softmax_max=m.t if stats else None,
                        softmax_sum=l.t if stats else None)
    assert sdpa.attn_get_last_error() == 0
    for g in (out, m, l):
        if g is not None:
            g.check()
    return out.t.cpu(), (m.t.cpu() if stats else None), (l.t.cpu() if stats else None)


def _check(inp, window, sinks):
    out, m, l = _run(inp, window, sinks)
    ref, rm, rl, A = R.window_fwd(inp, window, sinks)
    G.check_out(G.f64(out), ref, inp.dtype, abs_ref=A)
    G.check_stats(m.numpy(), l.numpy(), rm, rl)


SPANS = [(1, 0), (1, 3), (64, 4), (127, 130), (128, 128), (129, 1), (300, 7), (5, 100000), (1 << 40, 0)]


@pytest.mark.parametrize("dtype", [BF, F16, F32], ids=IDS)
@pytest.mark.parametrize("window,sinks", SPANS)
def test_dense(dtype, window, sinks):
    inp = W.dense_bhsd(1, 2, 700, 64, causal=False, dtype=dtype, seed=window % 91 + sinks % 17, cfg=72)
    _check(inp, window, sinks)


@pytest.mark.parametrize("dtype", [BF, F32], ids=IDS)
@pytest.mark.parametrize("Sq,Skv", [(1, 900), (130, 1000), (257, 1290), (400, 90), (300, 0), (1, 1)])
@pytest.mark.parametrize("heads", [(2, 2), (4, 1), (6, 2)])
def test_chunks_and_rows_without_keys(dtype, Sq, Skv, heads):
    inp = W.dense_bhsd(2, heads[0], Sq, 128, causal=False, dtype=dtype, seed=Sq + Skv, cfg=73, Skv=Skv, Hkv=heads[1])
    _check(inp, 200, 5)
    _check(inp, 150, 300)


@pytest.mark.parametrize("dtype", [BF, F16, F32], ids=IDS)
@pytest.mark.parametrize("heads", [(8, 2), (3, 3)])
def test_varlen(dtype, heads):
    inp = W.varlen_tnd([0, 700, 1, 257, 513, 0], *heads, 128, causal=False, dtype=dtype, seed=3, cfg=74)
    _check(inp, 100, 4)
    _check(inp, 256, 0)


def test_varlen_with_longer_keys():
    lq, lk = [5, 0, 300, 1], [905, 40, 640, 1]
    a = W.varlen_tnd(lq, 4, 2, 64, causal=False, dtype=BF, seed=5, cfg=75)
    b = W.varlen_tnd(lk, 4, 2, 64, causal=False, dtype=BF, seed=6, cfg=75)
    a.k, a.v, a.Skv, a.cu_kv = b.k, b.v, b.Skv, b.cu_kv
    _check(a, 130, 20)


@pytest.mark.parametrize("dtype", [BF, F16], ids=IDS)
@pytest.mark.parametrize("sinks", [1, 2, 31, 32, 33])
@pytest.mark.parametrize("gain", [0.0, 1.0, -1.0, 30.0, -30.0])
def test_few_sinks_apart_from_the_window(dtype, sinks, gain):
    """A tile that holds only some sinks, whose scores lie at, above or far below those of the window (the row's
    maximum moves after it or never); keys of that tile behind the sinks are NaN and are not seen."""
    inp = W.varlen_tnd([700, 300, 1100], 4, 2, 128, causal=False, dtype=dtype, seed=sinks, cfg=79)
    for b in range(3):
        t = int(inp.cu_kv[b])
        q = inp.q[t:t + 256].float().mean((0, 1))
        inp.k[t:t + sinks] = (gain * (inp.k[t:t + sinks].float().abs() + 0.1) * torch.sign(q)).to(dtype)
    _check(inp, 100, sinks)
    x = _run(inp, 100, sinks)
    for b in range(3):
        t = int(inp.cu_kv[b])
        rows = inp.k[t + sinks:t + 120].clone()
        inp.k[t + sinks:t + 120] = float("nan")
        y = _run(inp, 100, sinks)
        inp.k[t + sinks:t + 120] = rows
        # rows whose window begins behind the NaN
        for u, v in zip(x, y):
            assert torch.equal(u[t + 230:t + 300], v[t + 230:t + 300])


@pytest.mark.parametrize("D", [1, 33, 80, 256])
def test_f32_head_sizes(D):
    _check(W.dense_bhsd(1, 2, 150, D, causal=False, dtype=F32, seed=D, cfg=76), 40, 3)


@pytest.mark.parametrize("dtype", [BF, F16, F32], ids=IDS)
def test_a_window_of_every_key_is_the_causal_forward(dtype):
    """However every key comes to be seen the result is the same, bit for bit; in float32, where both run
    the same loop, it is also attn_fwd's."""
    inp = W.varlen_tnd([300, 0, 513], 4, 2, 128, causal=True, dtype=dtype, seed=4, cfg=77,
                       mask_mode=W.MASK_CAUSAL_BOTTOMRIGHT)
    want = G.run_fwd(inp) if dtype == F32 else _run(inp, sdpa.ATTN_WINDOW_ALL, 0)
    for window, sinks in ((sdpa.ATTN_WINDOW_ALL, 0), (513, 0), (7, 1 << 40)):
        for x, y in zip(want, _run(inp, window, sinks)):
            assert torch.equal(x, y), (window, sinks)
    ref, rm, rl = G.oracle_fwd(inp)
    G.check_out(G.f64(want[0]), ref, inp.dtype, abs_ref=lambda: G.oracle_abs_fwd(inp))
    G.check_stats(want[1].numpy(), want[2].numpy(), rm, rl)


@pytest.mark.parametrize("dtype", [BF, F32], ids=IDS)
def test_keys_left_out_may_hold_anything(dtype):
    """A chunk of 256 rows at positions 2048 .. 2303, window 128, 3 sinks: the key tiles between the
    sinks' tile and the first window are never read."""
    inp = W.dense_bhsd(1, 2, 256, 128, causal=False, dtype=dtype, seed=8, cfg=78, Skv=2304)
    want = _run(inp, 128, 3)
    inp.k[:, :, 128:1920] = float("nan")
    inp.v[:, :, 128:1920] = float("inf")
    inp.k[:, :, 1920:1921] = float("nan")   # position 1920 = 2048 - 128: in a tile that is read, seen by no row
    for x, y in zip(want, _run(inp, 128, 3)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [BF, F16, F32], ids=IDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [(4, 2), (3, 3)])
def test_a_sequence_of_nan_stays_by_itself(dtype, D, heads):
    """NaN and infinities in one sequence of a packed batch leave the others as they were, bit for bit, though
    their last key tiles hold its tokens."""
    inp = W.varlen_tnd([300, 5, 129, 1, 700, 128], *heads, D, causal=False, dtype=dtype, seed=12, cfg=82)
    cu = [0] + list(inp.cu_q)
    for window, sinks in ((100, 4), (sdpa.ATTN_WINDOW_ALL, 0)):
        want = _run(inp, window, sinks)
        for bad in (1, 3, 5):
            k, v = inp.k.clone(), inp.v.clone()
            rows = slice(cu[bad], cu[bad + 1])
            k[rows], v[rows] = float("nan"), float("inf") if bad == 3 else float("nan")
            other = W.AttnInputs(inp.q, k, v, inp.layout, 0, inp.dtype, inp.B, inp.Sq, inp.Skv, inp.Nq, inp.Nkv, D,
                                 inp.scale, inp.cu_q, inp.cu_kv)
            got = _run(other, window, sinks)
            keep = torch.ones(inp.Sq, dtype=torch.bool)
            keep[rows] = False
            for x, y in zip(want, got):
                assert torch.equal(x[keep], y[keep]), (window, bad)
            assert not torch.isfinite(got[0][~keep]).any()


def test_large_scores_and_one_hot_rows():
    inp = W.dense_bhsd(1, 2, 300, 64, causal=False, dtype=BF, seed=9, cfg=79)
    inp.q = inp.q * 64
    _check(inp, 90, 2)


def test_no_statistics_graph_replay_and_two_streams():
    inp = W.varlen_tnd([300, 129, 800], 8, 2, 128, causal=False, dtype=BF, seed=10, cfg=80)
    dev = G.to_dev(inp)
    want = _run(inp, 200, 4, dev=dev)[0]
    assert torch.equal(_run(inp, 200, 4, stats=False, dev=dev)[0], want)
    q, k, v, cq, ck = dev
    kw = dict(cu_seqlens_q=cq, cu_seqlens_kv=ck, B=inp.B, Sq=inp.Sq, Skv=inp.Skv, Nq=8, Nkv=2, D=128, scale=inp.scale,
              window_tokens=200, sink_tokens=4, dtype=inp.dtype, layout=inp.layout)
    outs = [torch.empty_like(q) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s, o in zip(streams, outs):
        with torch.cuda.stream(s):
            for _ in range(3):
                sdpa.attn_fwd_sinks(q, k, v, out=o, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sdpa.attn_fwd_sinks(q, k, v, out=outs[2], **kw)
    outs[2].zero_()
    g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o.cpu(), want)


def test_bad_lengths_are_reported():
    inp = W.varlen_tnd([100, 50], 2, 2, 64, causal=False, dtype=BF, seed=11, cfg=81)
    q, k, v, cq, ck = G.to_dev(inp)
    out = torch.empty_like(q)
    kw = dict(B=2, Sq=150, Skv=150, Nq=2, Nkv=2, D=64, scale=0.125, window_tokens=9, sink_tokens=1, dtype=inp.dtype,
              layout=inp.layout, out=out)
    bad = torch.tensor([120, 100], dtype=torch.int32, device="cuda")
    sdpa.attn_fwd_sinks(q, k, v, cu_seqlens_q=bad, cu_seqlens_kv=ck, **kw)
    assert sdpa.attn_get_last_error() == sdpa.ATTN_ERR_DATA
    sdpa.attn_fwd_sinks(q, k, v, cu_seqlens_q=cq, cu_seqlens_kv=bad, **kw)
    assert sdpa.attn_get_last_error() == sdpa.ATTN_ERR_DATA
    sdpa.attn_fwd_sinks(q, k, v, cu_seqlens_q=cq, cu_seqlens_kv=ck, **kw)
    assert sdpa.attn_get_last_error() == 0


@pytest.mark.parametrize("D", [4, 64, 100, 256])
def test_f32_tiles_at_any_alignment(D):
    """Rows of whole 16-byte chunks come by another kind of copy than those at an odd address: the results
    are the same bits. The keys behind a head's last one are the next head's, here NaN."""
    inp = W.dense_bhsd(1, 3, 75, D, causal=False, dtype=F32, seed=D, cfg=82, Skv=109)
    inp.k[:, 1], inp.v[:, 1] = float("nan"), float("nan")
    q, k, v, cq, ck = G.to_dev(inp)
    want = _run(inp, 50, 5, dev=(q, k, v, cq, ck))
    assert torch.isfinite(want[0][:, ::2]).all() and torch.isnan(want[0][:, 1]).all()

    def shifted(t):
        room = torch.full((t.numel() + 1,), float("nan"), device=t.device)
        room[1:] = t.flatten()
        return room[1:].view(t.shape)

    for c, a, b in ((q, shifted(k), v), (q, k, shifted(v)), (shifted(q), k, v), (shifted(q), shifted(k), shifted(v))):
        for x, y in zip(want, _run(inp, 50, 5, dev=(c, a, b, cq, ck))):
            assert torch.equal(x.nan_to_num(nan=7.0), y.nan_to_num(nan=7.0))

"""attn_fwd_sinks in 16 bits within a bound of the arithmetic, several times below the flat 1e-2 of the other forward
tests: outputs that are means of hundreds of values are about 0.1 themselves.

With eps = 2^-24, S the row's largest scale * sum |q k|, A = sum w |v|, n visible keys in T tiles of 128:
  * a score is off by (D + 1) eps S; times scale * log2 e, less the reference and through exp2 (2^-22 on the special
    function unit, 2.4e-7 < 2^-22 by the polynomial) a weight is off by e_w = (D + 1) eps S + 4 eps (S + 1) + 2^-21;
  * each tile may move the reference: a factor that is off by 2^-21 with its products, T 2^-21 in all;
  * P is rounded to the type (u = 2^-8 for bf16, 2^-11 for fp16); sums over n keys are off by n eps;
  * out: half a unit of the type + (2 e_w + u + 2 n eps + 2 T 2^-21) A; max: (D + 2) eps S;
    sum: relative 2 e_w + n eps + T 2^-21.
"""
import numpy as np
import pytest
import torch

from scaled_dot_product_16_b200 import workloads as W
from tests import serving_ref as R
from tests.test_gpu_sinks import BF, F16, IDS, SPANS, _run

EPS = 2.0 ** -24
UNIT = {BF: 2.0 ** -8, F16: 2.0 ** -11}


def reference(inp, window, sinks, shift=0):
    """out, max, sum, A, S and visible keys, in the call's layout; `shift` moves the window's edge by a key."""
    shape = tuple(inp.q.shape)
    out, A = torch.zeros(shape, dtype=torch.float64), torch.zeros(shape, dtype=torch.float64)
    m, l, S, n = (torch.zeros(shape[:-1], dtype=torch.float64) for _ in range(4))
    eq, ek = ([0] + list(inp.cu_q), [0] + list(inp.cu_kv)) if inp.layout == W.TND else (None, None)
    for b in range(inp.B):
        for h in range(inp.Nq):
            g = h // (inp.Nq // inp.Nkv)
            if inp.layout == W.TND:
                iq, ik = (slice(eq[b], eq[b + 1]), h), (slice(ek[b], ek[b + 1]), g)
            else:
                iq, ik = (b, h), (b, g)
            q, k, v = inp.q[iq], inp.k[ik], inp.v[ik]
            seen = R.window_seen(len(q), len(k), window + shift, sinks)
            out[iq], m[iq], l[iq], A[iq], S[iq] = R.attend(q, k, v, seen, inp.scale)
            n[iq] = seen.sum(1).double()
    return out, m, l, A, S, n


def bounds(ref, D, dtype):
    out, m, l, A, S, n = ref
    T = torch.ceil(n / 128) + 2
    ew = (D + 1) * EPS * S + 4 * EPS * (S + 1) + 2.0 ** -21
    half = torch.exp2(torch.floor(torch.log2(out.abs().clamp(min=2.0 ** (-14 if dtype == F16 else -126))))) * (
        torch.finfo(dtype).eps / 2)
    return (half + (2 * ew + UNIT[dtype] + 2 * n * EPS + 2 * T * 2.0 ** -21)[..., None] * A, (D + 2) * EPS * S,
            2 * ew + n * EPS + T * 2.0 ** -21)


def cases(D, dtype):
    yield W.dense_bhsd(1, 2, 300, D, causal=False, dtype=dtype, seed=11, cfg=94, Skv=700, Hkv=1)
    yield W.dense_bhsd(1, 3, 270, D, causal=False, dtype=dtype, seed=12, cfg=94, Skv=200)
    yield W.varlen_tnd([0, 390, 1, 129, 256], 4, 2, D, causal=False, dtype=dtype, seed=13, cfg=94)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F16], ids=IDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks", SPANS)
def test_within_the_arithmetic(window, sinks, D, dtype):
    for inp in cases(D, dtype):
        out, m, l = (x.double() for x in _run(inp, window, sinks))
        ref = reference(inp, window, sinks)
        tol, tol_m, tol_l = bounds(ref, D, dtype)
        err = (out - ref[0]).abs()
        assert torch.all(err <= tol), f"{float((err / tol.clamp(min=1e-300)).max())} of its bound"
        empty = torch.isneginf(ref[1])
        assert torch.equal(torch.isneginf(m), empty) and not l[empty].any() and not out[empty].any()
        assert torch.all((m - ref[1]).abs()[~empty] <= tol_m[~empty])
        assert torch.all((l / ref[2] - 1).abs()[~empty] <= tol_l[~empty])


@pytest.mark.parametrize("dtype", [BF, F16], ids=IDS)
@pytest.mark.parametrize("window,sinks", [(64, 4), (129, 1), (300, 7)])
def test_the_bound_sees_one_key_too_many(window, sinks, dtype):
    """Outputs of a window one key longer are outside the bound, the softmax sums aside."""
    for inp in cases(64, dtype):
        ref, other = reference(inp, window, sinks), reference(inp, window, sinks, shift=1)
        if not torch.any(other[5] != ref[5]):
            continue
        err = (other[0] - ref[0]).abs()
        assert torch.any(err > bounds(ref, 64, dtype)[0])

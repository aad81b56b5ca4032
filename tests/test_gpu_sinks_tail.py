"""attn_fwd_sinks where one key in 16 takes nearly all the weight and carries no value, so that the output is what
the other keys' small weights make, against the plain float64 form.

Bound: that of the other forward tests (tests/gpu_util.py: half a unit of the output, and (u_P + 2^-13 + 2^-12) A with
u_P = 2^-11 for fp16, 2^-8 for bf16 and A = sum w |v|), and for fp16 the end of its numbers: half a step of its
subnormal ones is 2^-25, P is kept times 2^7, so a weight is off by 2^-32 of the largest at most, wherever that is more.
float32: 2^-11 A holds 512 times what its sums of 700 terms can be off.
"""
import math

import pytest
import torch

from scaled_dot_product_16_b200 import workloads as W
from tests import gpu_util as G
from tests import serving_ref as R
from tests.test_gpu_sinks import BF, F16, F32, IDS, _run

# weights relative to the largest: what fp16 rounds to 0, to 2^-24, by 6 %, and by 2^-9 of itself
TAILS = [0.99 * 2.0 ** -25, 1.49 * 2.0 ** -24, 1.0625 * 2.0 ** -21, 2.0 ** -17 * (1 + 0.99 / 256)]
UNIT = {BF: 2.0 ** -8, F16: 2.0 ** -11, F32: 0.0}


def long_tail(weight, D, dtype, Sq=150, Skv=700, heads=(2, 1)):
    inp = W.dense_bhsd(1, heads[0], Sq, D, causal=False, dtype=dtype, seed=5, cfg=92, Skv=Skv, Hkv=heads[1])
    target = math.log(weight)
    hi = float(torch.tensor(target).to(dtype))
    inp.scale = 1.0
    inp.q.zero_()
    inp.q[..., 0] = inp.q[..., 1] = 1.0
    inp.k.zero_()
    inp.k[..., 0], inp.k[..., 1] = hi, float(torch.tensor(target - hi).to(dtype))
    inp.v = (1000 * (inp.v.float().abs() + 0.5)).to(dtype)
    inp.k[:, :, 8::16] = 0.0
    inp.v[:, :, 8::16] = 0.0
    return inp


def bound(inp, ref, window, sinks, dtype):
    ro, _, rl, A = (torch.from_numpy(x) for x in ref)
    half = torch.exp2(torch.floor(torch.log2(ro.abs().clamp(min=2.0 ** (-14 if dtype == F16 else -126))))) * (
        torch.finfo(dtype).eps / 2)
    tol = half + (UNIT[dtype] + 2.0 ** -13 + 2.0 ** -12) * A
    if dtype == F16:
        seen = R.window_seen(inp.Sq, inp.Skv, window, sinks).double()
        total = torch.stack([seen @ inp.v[0, 0].double().abs()] * inp.Nq)[None]
        tol += 2.0 ** -32 * total / rl[..., None]
    return tol


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F16, BF, F32], ids=IDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1 << 30, 0), (300, 0), (200, 20), (64, 200)])
@pytest.mark.parametrize("weight", TAILS)
def test_small_weights_beside_large_ones(weight, window, sinks, D, dtype):
    inp = long_tail(weight, D, dtype)
    out, m, l = _run(inp, window, sinks)
    ref = R.window_fwd(inp, window, sinks)
    err = (out.double() - torch.from_numpy(ref[0])).abs()
    tol = bound(inp, ref, window, sinks, dtype)
    assert torch.all(err <= tol), f"{float((err / tol).max())} of its bound"
    G.check_stats(m.numpy(), l.numpy(), ref[1], ref[2])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gain", [1.0, 40.0, 2000.0, 60000.0])
def test_float16_scores_of_any_size(D, gain):
    """Scores up to 6e4 * sqrt(D) and more, in steps of their own rounding: weights stay in fp16's range and the output
    is finite. (Where the largest score is far ahead it is that key's value.)"""
    inp = W.dense_bhsd(1, 2, 200, D, causal=False, dtype=F16, seed=6, cfg=93, Skv=400, Hkv=1)
    inp.q = (inp.q.float().clamp(-1, 1) * gain).to(F16)
    inp.k = (inp.k.float().clamp(-1, 1) * min(gain, 2000.0)).to(F16)
    for window, sinks in ((1 << 30, 0), (100, 3)):
        out, _, _ = _run(inp, window, sinks)
        assert torch.isfinite(out).all()
        ro, rm, _, _ = R.window_fwd(inp, window, sinks)
        s = inp.q[0].double() @ inp.k[0].double().transpose(1, 2) * inp.scale
        s[:, ~R.window_seen(200, 400, window, sinks)] = -math.inf
        top = s.topk(2, -1)
        # float32 rounds a score to 2^-24 of sum |q k| a term; 1,000 of these and 30 more apart, nothing else counts
        far = top.values[..., 0] - top.values[..., 1] > 30 + 1000 * 2.0 ** -24 * (
            inp.q[0].double().abs() @ inp.k[0].double().abs().transpose(1, 2)).amax(-1) * inp.scale
        # one key: A = |v|. It is not v to the bit: e^(s - m) of the largest score is 2^x with x what rounding scale s
        # to the reference m left, so its P is not 1; rounding P to fp16 moves the output by u_P of itself, and the
        # sum it is divided by is not rounded. With M the largest score times log2 e, |x| <= d = ulp(M) / 2 =
        # 2^(floor(log2 M) - 24), so P >= 2^-d. Where that is normal in fp16 u_P = 2^-11; below, half a step of
        # 2^-25 is up to 2^(d - 25) of it. (Scores past 2^28 are rounded to 32 and more by float32: there only
        # finite outputs are asked for.)
        M = top.values[..., 0].abs() * math.log2(math.e)
        d = torch.exp2(torch.floor(torch.log2(M.clamp(min=1.0))) - 24)
        u = torch.exp2(d.clamp(max=60.0) - 25).clamp(min=2.0 ** -11)[..., None]
        want = inp.v[0, 0][top.indices[..., 0]].double()
        half = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0 ** -14)))) * 2.0 ** -11
        err, tol = (out[0].double() - want).abs(), half + (u + 2.0 ** -13 + 2.0 ** -12) * want.abs()
        assert torch.all((err <= tol)[far]), f"{float((err / tol)[far].max())} of its bound"
        assert gain < 2000 or bool(far.any())


@pytest.mark.parametrize("weight", TAILS)
def test_the_bound_tells_weights_of_plain_fp16_apart(weight):
    """The same inputs with weights rounded to fp16 relative to the largest, everything else in 64 bits, are outside the
    bound; times 2^7 first they are inside."""
    inp = long_tail(weight, 64, F16)
    ref = R.window_fwd(inp, 1 << 30, 0)
    tol = bound(inp, ref, 1 << 30, 0, F16)[0, 0]
    s = inp.q[0, 0].double() @ inp.k[0, 0].double().T
    w = torch.where(R.window_seen(inp.Sq, inp.Skv, 1 << 30, 0), torch.exp(s), 0.0)
    for bias, good in ((0, False), (7, True)):
        kept = (w * 2.0 ** bias).to(F16).double() * 2.0 ** -bias
        err = ((kept @ inp.v[0, 0].double()) / w.sum(1, keepdim=True) - torch.from_numpy(ref[0][0, 0])).abs()
        assert bool(torch.all(err <= tol)) == good, (bias, float((err / tol).max()))

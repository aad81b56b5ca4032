"""attn_decode_paged where one key in 16 takes nearly all the weight and carries no value, so that the output is what
the other keys' small weights make, against the plain float64 form.

Bound, as in tests/test_gpu_decode.py with eps = 2^-24: a weight is off by e_w <= (D + 1) eps S + 4 eps (S + 1)
relative, the product with V by u (2^-11 for fp16 weights, 2^-16 for bf16's two terms) of each weight, and half a
unit of the output type comes last. The sums over n keys are not one chain of n additions here: n keys of one unit
are cut over the whole GPU, so a warp adds n / (4 x blocks) of them or the 32 of one step, and what the warps and
blocks have is joined in three levels of at most 4, 16 and 32 terms. With 131,072 keys on 100 blocks or more that is
below 400 additions, and CHAIN = 1,024 covers it: 2 CHAIN eps = 1.2e-4 of A = sum w |v|.

Weights kept in fp16 relative to the largest one are outside that bound (also checked here, on the CPU): below 2^-14
fp16 has fewer bits, below 2^-25 none.
"""
import math

import pytest
import torch

from tests import serving_ref as R
from tests.test_gpu_decode import BF, EPS, F16, F32, IDS, UNIT, Case

CHAIN = 1024
# weights relative to the largest: what fp16 rounds to 0, to 2^-24, and down by 2^-9 of itself
TAILS = [0.99 * 2.0 ** -25, 1.49 * 2.0 ** -24, 2.0 ** -17 * (1 + 0.99 / 256)]


def long_tail(weight, D, dtype, n, Nq=4):
    """n keys: every 16th has score 0 and value 0, the others score ln(weight) (scale 1, in two exact terms)."""
    c = Case([n], Nq, 1, D, dtype, page=16, seed=1)
    c.scale = 1.0
    target = math.log(weight)
    hi = torch.tensor(target).to(dtype)
    c.q.zero_()
    c.q[:, :, 0] = c.q[:, :, 1] = 1.0
    row = torch.zeros(D)
    row[0], row[1] = float(hi), float(torch.tensor(target - float(hi)).to(dtype))
    live = ~torch.isnan(c.k[..., :1].float())
    c.k = torch.where(live, row, torch.nan).to(dtype)
    c.v = torch.where(live, 1000 * (c.v.float().abs() + 0.5), torch.nan).to(dtype)
    first = c.table[0][c.table[0] >= 0].long()
    c.k[first, 8] = 0.0
    c.v[first, 8] = torch.where(live[first, 8], 0.0, torch.nan).to(dtype)
    return c


def bounds(ref, D, dtype, unit):
    ro, _, rl, A, S, _ = ref
    ew = (D + 1) * EPS * S + 4 * EPS * (S + 1)
    half = torch.exp2(torch.floor(torch.log2(ro.abs().clamp(min=2.0 ** (-14 if dtype == F16 else -126))))) * (
        torch.finfo(dtype).eps / 2)
    return half + (2 * ew + unit + 2 * CHAIN * EPS)[..., None] * A, 2 * ew + CHAIN * EPS


def reference(c):
    return R.decode(c.q, c.k, c.v, c.table, c.lens, layout=c.layout, page_size=c.page, scale=c.scale, window=c.window,
                    sinks=c.sinks)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F16, BF, F32], ids=IDS)
@pytest.mark.parametrize("D,n", [(64, 2000), (128, 2000), (64, 131072)])
@pytest.mark.parametrize("weight", TAILS)
def test_small_weights_beside_large_ones(weight, D, n, dtype):
    c = long_tail(weight, D, dtype, n)
    out, m, l = (x.double() for x in c.run())
    ref = reference(c)
    tol, tol_l = bounds(ref, D, dtype, UNIT[dtype])
    err = (out - ref[0]).abs()
    assert torch.all(err <= tol), f"{float((err / tol).max())} of its bound"
    assert torch.all((l / ref[2] - 1).abs() <= tol_l)
    assert not m.any()


@pytest.mark.parametrize("weight", TAILS)
def test_the_bound_tells_weights_of_plain_fp16_apart(weight):
    """The same inputs with weights rounded to fp16 relative to the largest, everything else in 64 bits: outside the
    bound, so that the test above sees it; times 2^15 first they are inside."""
    n = 2000
    c = long_tail(weight, 64, F16, n)
    ref = reference(c)
    tol, _ = bounds(ref, 64, F16, UNIT[F16])
    page, off = torch.tensor([(int(c.table[0, j // 16]), j % 16) for j in range(n)]).T
    k, v = c.k[page, off, 0].double(), c.v[page, off, 0].double()
    w = torch.exp(k @ c.q[0, 0].double())
    for bias, good in ((0, False), (15, True)):
        kept = (w * 2.0 ** bias).to(F16).double() * 2.0 ** -bias
        err = ((kept @ v) / w.sum() - ref[0][0, 0]).abs()
        assert bool(torch.all(err <= tol[0, 0])) == good, (bias, float((err / tol[0, 0]).max()))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F16, BF, F32], ids=IDS)
@pytest.mark.parametrize("shift", [0, 1], ids=["aligned", "unaligned"])
@pytest.mark.parametrize("D,heads", [(64, (4, 1)), (128, (4, 1)), (128, (16, 1))])
def test_two_values_that_nearly_cancel(D, heads, shift, dtype):
    """Two keys with nearly the same weight and opposite values: the output is the difference of the weights, so it
    shows how many bits of them reach the product with V. u = 2^-16 for every type and any alignment."""
    c = Case([2] * 40, *heads, D, dtype, seed=3)
    c.q = (c.q.float() * 0.05).to(dtype)
    first = c.table[:, 0].long()
    c.v[first, 1] = -c.v[first, 0]
    args = c.dev()
    if shift:  # an address off the 16-byte boundary takes the kernel without tensor cores
        room = torch.empty(args[0].numel() + 1, dtype=dtype, device="cuda")
        room[1:] = args[0].reshape(-1)
        args[0] = room[1:].view(args[0].shape)
    out, _, _ = c.run(args=args)
    ro, _, _, A, S, _ = reference(c)
    ew = (D + 1) * EPS * S + 4 * EPS * (S + 1)
    half = torch.exp2(torch.floor(torch.log2(ro.abs().clamp(min=2.0 ** (-14 if dtype == F16 else -126))))) * (
        torch.finfo(dtype).eps / 2)
    tol = half + (2 * ew + (0.0 if dtype == F32 else 2.0 ** -16) + 4 * EPS)[..., None] * A
    err = (out.double() - ro).abs()
    assert torch.all(err <= tol), f"{float((err / tol).max())} of its bound"

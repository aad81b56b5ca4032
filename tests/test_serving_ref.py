"""The plain implementations of serving_ref.py against the oracle, against each other and against
what the page bookkeeping must conserve (CPU)."""
import numpy as np
import pytest
import torch

import oracle
from scaled_dot_product_16_b200 import workloads as W
from tests import serving_ref as R


@pytest.mark.parametrize("Sq,Skv", [(9, 9), (5, 23), (23, 5), (1, 40)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 2), (7, 30), (1 << 30, 0)])
def test_window_equals_the_oracle_under_an_explicit_mask(Sq, Skv, window, sinks):
    inp = W.dense_bhsd(2, 4, Sq, 16, causal=False, dtype=torch.float32, seed=Sq, cfg=70, Skv=Skv, Hkv=2)
    out, m, l, _ = R.window_fwd(inp, window, sinks)
    mask = np.ones((Sq, Skv), np.uint8)
    for i in range(Sq):
        p = i + Skv - Sq
        for j in range(Skv):
            if j <= p and (j > p - window or j < sinks):
                mask[i, j] = 0
    ref, rm, rl = oracle.attn_fwd_ext(inp.q, inp.k, inp.v, B=2, Sq=Sq, Skv=Skv, Nq=4, Nkv=2, Dqk=16, Dv=16,
                                      scale=inp.scale, mask_mode=W.MASK_NONE, mask=mask.reshape(-1),
                                      mask_bstride=0, mask_rstride=Skv, layout=W.BHSD)
    np.testing.assert_allclose(out, ref, rtol=1e-12, atol=1e-13)
    assert np.array_equal(np.isneginf(m), np.isneginf(rm))
    np.testing.assert_allclose(l, rl, rtol=1e-12)


@pytest.mark.parametrize("layout", [W.TND, W.BHSD])
def test_decode_equals_the_last_row_of_the_window(layout):
    rng = np.random.default_rng(2)
    n, ps, D = 29, 4, 8
    inp = W.dense_bhsd(1, 4, n, D, causal=False, dtype=torch.float32, seed=3, cfg=71, Hkv=2)
    table = torch.from_numpy(rng.permutation(11)[None, :8].astype(np.int32))
    shape = (11, ps, 2, D) if layout == W.TND else (11, 2, ps, D)
    kc, vc = torch.full(shape, torch.nan), torch.full(shape, torch.nan)
    for j in range(n):
        p, o = int(table[0, j // ps]), j % ps
        for c, x in ((kc, inp.k), (vc, inp.v)):
            if layout == W.TND:
                c[p, o] = x[0, :, j]
            else:
                c[p, :, o] = x[0, :, j]
    out, m, l, A, _, seen = R.decode(inp.q[:, :, n - 1], kc, vc, table, [n], layout=layout, page_size=ps,
                                     scale=inp.scale, window=9, sinks=2)
    ref, rm, rl, rA = R.window_fwd(inp, 9, 2)
    np.testing.assert_allclose(out[0], ref[0, :, n - 1], rtol=1e-12)
    np.testing.assert_allclose(m[0], rm[0, :, n - 1])
    np.testing.assert_allclose(l[0], rl[0, :, n - 1])
    np.testing.assert_allclose(A[0], rA[0, :, n - 1])
    assert seen[0] == 11


def _counts(table, n):
    c = [0] * n
    for row in table:
        for p in row:
            if p >= 0:
                c[p] += 1
    return c


@pytest.mark.parametrize("seed", range(6))
def test_bookkeeping_keeps_the_counts(seed):
    """After every call the counts are the number of holders, new positions are held alone, and the
    contents that a row sees (tracked by page identity) are its parent's."""
    rng = np.random.default_rng(seed)
    ps, mp, n, rows = 4, 12, 200, 9
    lens = [int(x) for x in np.repeat(rng.integers(1, 30, 3), 3)]
    table, ref = R.live_table(rng, lens, ps, mp, n, share=2)
    content = {p: ("page", p) for p in range(n)}
    for step in range(12):
        src = [int(rng.integers(-1, rows)) for _ in range(rows)]
        seen = [[content[p] for p in (table[s] if s >= 0 else []) if p >= 0] for s in src]
        table, ref, lens = R.fork(table, src, ref, lens, n)
        assert ref == _counts(table, n)
        new = [int(rng.integers(0, 6)) if x + 6 <= mp * ps else 0 for x in lens]
        lens = [a + b for a, b in zip(lens, new)]
        table, ref, copies = R.reserve(table, ref, lens, new, ps)
        assert ref == _counts(table, n)
        for a, b in copies:
            if a >= 0:
                content[b] = content[a]
        for b in range(rows):
            whole = -(-(lens[b] - new[b]) // ps)
            got = [content[p] for p in table[b][:whole]]
            assert got == seen[b][:whole]
            for i in range((lens[b] - new[b]) // ps, -(-lens[b] // ps)):
                if new[b]:
                    assert ref[table[b][i]] == 1
                    content[table[b][i]] = ("new", step, b, i)
        table, ref, pmap, moves, live = R.compact(table, ref)
        assert ref == _counts(table, n) and all(r > 0 for r in ref[:live]) and not any(ref[live:])
        moved = dict(content)
        for a, b in moves:
            if a >= 0:
                moved[b] = content[a]
        content = moved

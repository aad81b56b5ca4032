"""attn_cache_grow, append after it, and what PagedCache makes of a step that is refused or whose rows have ended,
against the row-by-row forms of tests/serving_ref.py (whole numbers and copied tokens: equal)."""
import numpy as np
import pytest
import torch

import scaled_dot_product_16_b200 as sdpa
from scaled_dot_product_16_b200 import workloads as W
from scaled_dot_product_16_b200.cache import PagedCache
from tests import gpu_util as G
from tests import serving_ref as R
from tests.test_gpu_cache import BF, F16, F32, IDS, I32, Model, dev, guarded, status

pytestmark = pytest.mark.gpu


def _grow(table, ref, lens, new, page, live_only=False):
    """The call against reserve of the lengths with the new tokens; returns the state afterwards."""
    rows = len(table)
    t, r, n = dev(table), dev(ref), dev(lens)
    c, nl = guarded((rows, 2)), guarded((rows,))
    sdpa.attn_cache_grow(t, r, n, None if new is None else dev(new), nl.t, c.t, B=rows, max_pages=len(table[0]),
                         num_pages=len(ref), page_size=page, live_only=live_only)
    c.check()
    nl.check()
    add = new if new is not None else [int(x > 0) if live_only else 1 for x in lens]
    try:
        if any(x < 0 for x in lens):
            raise R.Refused("data")
        want = R.reserve(table, ref, [a + b for a, b in zip(lens, add)], add, page)
    except R.Refused as e:
        status({"data": sdpa.ATTN_ERR_DATA, "pages": sdpa.ATTN_ERR_PAGES}[e.what])
        want, want_lens, want_new = (table, ref, [[-1, -1]] * rows), lens, [0] * rows
    else:
        status()
        want_lens = [a + b for a, b in zip(lens, add)]
        want_new = [x if b else 0 for x, b in zip(want_lens, add)]
    for x, y in zip((t, r, c.t), want):
        assert x.tolist() == y
    assert n.tolist() == want_lens and nl.t.tolist() == want_new
    return want[0], want[1], want_lens


@pytest.mark.parametrize("seed", range(8))
def test_grow_random(seed):
    """Rows forked at random, growing by several pages, by one token or not at all; at times too few pages."""
    rng = np.random.default_rng(seed)
    rows, mp, page = int(rng.integers(1, 40)), 12, int(rng.choice([1, 4, 5]))
    lens = [int(x) for x in rng.integers(0, 5 * page, rows)]
    num = int(rng.integers(rows * 5, rows * 12)) + 1
    table, ref = R.live_table(rng, lens, page, mp, num)
    for _ in range(6):
        src = [int(x) for x in rng.integers(-1, rows, rows)]
        table, ref, lens = R.fork(table, src, ref, lens, num)
        kind = rng.integers(0, 3)
        new = [int(rng.choice([0, 1, 1, 2, 2 * page + 1])) for _ in lens] if kind == 0 else None
        table, ref, lens = _grow(table, ref, lens, new, page, live_only=bool(kind == 1))


def test_grow_bad_data_and_many_rows():
    table, ref = [[0, -1], [1, -1]], [1, 1, 0, 0]
    _grow(table, ref, [4, 2], [1, -1], 4)
    _grow(table, ref, [-1, 2], [1, 1], 4)
    _grow(table, ref, [-1, 2], [2, 1], 4)
    _grow(table, ref, [8, 2], [1, 1], 4)                 # past the table
    _grow(table, ref, [8, 2], [2 ** 31 - 1, 1], 4)       # the sum passes 32 bits
    _grow([[0, -1], [9, -1]], ref, [4, 2], [1, 1], 4)    # a page outside the pool
    _grow([[0, -1], [2, -1]], ref, [4, 2], [1, 1], 4)    # a held page that counts as free
    rng = np.random.default_rng(9)
    lens = [int(x) for x in rng.integers(0, 60, 2000)]   # more rows than the block has threads
    table, ref = R.live_table(rng, lens, 1, 61, sum(lens) + 2000)
    _grow(table, ref, lens, None, 1)
    _grow(table, ref, lens, None, 1, live_only=True)
    _grow(table, ref[:-2] + [1, 1], lens, None, 1)       # two pages too few


@pytest.mark.parametrize("dtype", [BF, F16, F32], ids=IDS)
def test_append_skips_rows_of_length_0(dtype):
    """One token a row and packed tokens: rows whose length is 0 have none, whatever the packing says."""
    rows, mp, page, Nkv, D, num = 4, 3, 4, 2, 64, 9
    table = [[0, 1, -1], [2, -1, -1], [-1, -1, -1], [3, 4, 5]]
    base = [W.randn((num, page, Nkv, D), s).to(dtype) for s in (1, 2)]
    kw = dict(B=rows, Nkv=Nkv, D=D, num_pages=num, page_size=page, max_pages=mp, dtype=W.dtype_code(dtype), layout=W.TND)
    for lens, new in (([6, 0, 0, 9], None), ([0, 0, 0, 0], None), ([6, 0, 0, 9], [3, 2, 1, 2]), ([0] * 4, [1, 2, 0, 4])):
        n = new or [1] * rows
        k, v = (W.randn((sum(n), Nkv, D), s).to(dtype) for s in (3, 4))
        kd, vd = (x.cuda() for x in base)
        sdpa.attn_cache_append(k.cuda(), v.cuda(), dev(table), dev(lens), kd, vd,
                               cu_seqlens=None if new is None else dev(np.cumsum(n).tolist()), T=sum(n), **kw)
        status()
        want = [x.clone() for x in base]
        t = 0
        for b in range(rows):
            for i in range(n[b]):
                if lens[b]:
                    pos = lens[b] - n[b] + i
                    for w, x in zip(want, (k, v)):
                        w[table[b][pos // page], pos % page] = x[t]
                t += 1
        assert torch.equal(kd.cpu(), want[0]) and torch.equal(vd.cpu(), want[1])


def _full_cache(dtype=BF, layers=2):
    """Two beams that share a partly filled page, in a pool without a free one, and a third row."""
    rows, D = 4, 64
    cache = PagedCache(layers=layers, rows=rows, max_pages=6, num_pages=5, page_size=8, Nq=4, Nkv=2, D=D,
                       dtype=W.dtype_code(dtype))
    cache.pool.zero_()
    model = Model(cache, dtype, 7)
    new = [13, 0, 20, 0]
    cache.reserve(dev(new))
    cu = dev(np.cumsum(new).tolist())
    for layer, (k, v) in enumerate(model.step(new)):
        cache.append(layer, k.cuda(), v.cuda(), cu)
    cache.fork(dev([0, 0, 2, -1]))
    model.fork([0, 0, 2, -1])
    cache.check()
    assert cache.ref_count.tolist() == [2, 2, 1, 1, 1]
    return cache, model


def _attend(cache, model, dtype=BF):
    for layer in range(cache.layers):
        q = model.draw((cache.rows, cache.Nq, cache.D))
        out = torch.full(tuple(q.shape), float("nan"), dtype=dtype, device="cuda")
        cache.attend(layer, q.cuda(), out)
        cache.check()
        ref, A = model.attend(layer, q)
        G.check_out(G.f64(out.cpu()), ref, cache.dtype, abs_ref=A)


@pytest.mark.parametrize("graph", [False, True], ids=["eager", "graph"])
def test_a_refused_step_changes_nothing_and_can_be_repeated(graph):
    """The pool is full: reserve is refused, the tokens of the step are written nowhere (the beams still share their
    last page), lengths and counts stay. With a page free the same step goes through."""
    cache, model = _full_cache()
    rows = cache.rows
    k, v = (torch.ones((rows, cache.Nkv, cache.D), dtype=BF, device="cuda") for _ in range(2))

    def step():
        cache.reserve(live_only=True)
        for layer in range(cache.layers):
            cache.append(layer, k, v)

    if graph:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
    before = [x.clone() for x in (cache.pool, cache.page_table, cache.ref_count, cache.seq_lens)]
    for _ in range(2):
        g.replay() if graph else step()
        with pytest.raises(sdpa.AttnError, match="free pages"):
            cache.check()
        for x, y in zip((cache.pool, cache.page_table, cache.ref_count, cache.seq_lens), before):
            assert torch.equal(x, y)
        assert not cache.new_lens.any()
    _attend(cache, model)
    cache.fork(dev([0, 0, -1, -1]))   # row 2 ends: three pages are free again
    model.fork([0, 0, -1, -1])
    new = model.step([1, 1, 0, 0])
    k[:2].copy_(new[0][0]), v[:2].copy_(new[0][1])
    for layer in range(1, cache.layers):  # the step writes the same tokens in every layer
        for b in range(2):
            model.kv[layer][b][0][-1], model.kv[layer][b][1][-1] = new[0][0][b], new[0][1][b]
    g.replay() if graph else step()
    cache.check()
    assert cache.seq_lens.tolist() == [14, 14, 0, 0] and cache.new_lens.tolist() == [14, 14, 0, 0]
    _attend(cache, model)


def test_rows_that_have_ended_stay_so():
    """The loop of the module's description: ended rows hold no page and answer 0, and the others go on."""
    rows, D = 4, 64
    cache = PagedCache(layers=1, rows=rows, max_pages=8, num_pages=24, page_size=4, Nq=4, Nkv=2, D=D, dtype=W.F16)
    model = Model(cache, F16, 3)
    new = [5, 1, 9, 4]
    cache.reserve(dev(new))
    (k, v), = model.step(new)
    cache.append(0, k.cuda(), v.cuda(), dev(np.cumsum(new).tolist()))
    alive = [1, 1, 1, 1]
    for step in range(8):
        cache.reserve(live_only=True)
        k, v = model.draw((rows, 2, D)), model.draw((rows, 2, D))  # of every row, ended or not
        cache.append(0, k.cuda(), v.cuda())
        for b in range(rows):
            if alive[b]:
                model.kv[0][b][0].append(k[b]), model.kv[0][b][1].append(v[b])
        _attend(cache, model, F16)
        src = [b if alive[b] and b != step else -1 for b in range(rows)] if step < 2 else list(range(rows))
        alive = [a and s >= 0 for a, s in zip(alive, src)]
        cache.fork(dev(src))
        model.fork(src)
        held = (cache.page_table >= 0).sum(1).tolist()
        assert [n > 0 for n in cache.seq_lens.tolist()] == [n > 0 for n in held] == [bool(a) for a in alive]
    assert cache.seq_lens.tolist() == [0, 0, 17, 12]


def test_tokens_for_some_rows_without_packing():
    """new_tokens of 0 and 1 decided on the device, and a key and value for every row."""
    cache, model = _full_cache(layers=1)
    cache.fork(dev([0, 0, -1, -1]))
    model.fork([0, 0, -1, -1])
    k, v = model.draw((4, 2, 64)), model.draw((4, 2, 64))
    cache.reserve(dev([0, 1, 0, 1]))
    cache.append(0, k.cuda(), v.cuda())
    cache.check()
    for b in (1, 3):
        model.kv[0][b][0].append(k[b]), model.kv[0][b][1].append(v[b])
    assert cache.seq_lens.tolist() == [13, 14, 0, 1]
    _attend(cache, model)

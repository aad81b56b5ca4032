"""The page calls on the GPU against the row-by-row forms of tests/serving_ref.py (whole numbers: equal),
and a run of all serving calls together."""
import numpy as np
import pytest
import torch

import scaled_dot_product_16_b200 as sdpa
from scaled_dot_product_16_b200 import workloads as W
from tests import gpu_util as G
from tests import serving_ref as R

pytestmark = pytest.mark.gpu

BF, F16, F32, I32 = torch.bfloat16, torch.float16, torch.float32, torch.int32
IDS = {BF: "bf16", F16: "f16", F32: "f32"}.get


def dev(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def guarded(shape):
    return G.Guarded(shape, I32)


def status(want=0):
    assert sdpa.attn_get_last_error() == want


# ---- append --------------------------------------------------------------------------------------
def _append(lens, new, Nkv, D, dtype, page, layout, one=False, interleave=False, shift=0):
    rng = np.random.default_rng(len(lens))
    mp = max(1, max(-(-n // page) for n in lens))
    table, _ = R.live_table(rng, lens, page, mp, sum(-(-n // page) for n in lens) + 2)
    num = sum(-(-n // page) for n in lens) + 2
    shape = (num, page, Nkv, D) if layout == W.TND else (num, Nkv, page, D)
    T = sum(new)
    kn, vn = (W.randn((T + 1, Nkv, D), s).to(dtype) for s in (1, 2))
    want = [W.randn(shape, s).to(dtype) for s in (3, 4)]
    kd, vd = (x.cuda() for x in want)
    pool = torch.stack([kd, vd], 1) if interleave else None
    if interleave:
        kd, vd = pool[:, 0], pool[:, 1]
    if shift:
        flat = torch.empty(T * Nkv * D + shift, dtype=dtype, device="cuda")
        flat[shift:] = kn[:T].reshape(-1).cuda()
        kn_dev = flat[shift:].view(T, Nkv, D)
    else:
        kn_dev = kn[:T].cuda().contiguous()
    sdpa.attn_cache_append(kn_dev, vn[:T].cuda().contiguous(), dev(table), dev(lens), kd, vd,
                           cu_seqlens=None if one else dev(np.cumsum(new).tolist()), T=T, B=len(lens), Nkv=Nkv, D=D,
                           num_pages=num, page_size=page, max_pages=mp,
                           page_stride=2 * page * Nkv * D if interleave else 0, dtype=W.dtype_code(dtype), layout=layout)
    status()
    t = 0
    for b, (n, a) in enumerate(zip(lens, new)):
        for pos in range(n - a, n):
            p, o = table[b][pos // page], pos % page
            for c, x in zip(want, (kn, vn)):
                if layout == W.TND:
                    c[p, o] = x[t]
                else:
                    c[p, :, o] = x[t]
            t += 1
    assert torch.equal(kd.cpu(), want[0]) and torch.equal(vd.cpu(), want[1])


@pytest.mark.parametrize("dtype", [BF, F16, F32], ids=IDS)
@pytest.mark.parametrize("layout", [W.TND, W.BHSD], ids=["tnd", "bhsd"])
@pytest.mark.parametrize("page", [1, 7, 16])
@pytest.mark.parametrize("Nkv,D", [(1, 64), (3, 128), (2, 33)])
def test_append(dtype, layout, page, Nkv, D):
    _append([5, 40, 0, 16, 1, 100], [5, 17, 0, 0, 1, 33], Nkv, D, dtype, page, layout)
    _append([5, 40, 16, 1, 100], [1] * 5, Nkv, D, dtype, page, layout, one=True)


def test_append_interleaved_and_unaligned():
    _append([5, 40, 100], [5, 17, 33], 2, 64, BF, 16, W.TND, interleave=True)
    _append([5, 40, 100], [5, 17, 33], 2, 64, BF, 16, W.BHSD, shift=1)
    _append([5, 40, 100], [5, 17, 33], 2, 65, F32, 16, W.TND, interleave=True)


def test_append_bad_data_is_skipped_and_reported():
    k = W.randn((6, 2, 64), 5).to(BF).cuda()
    base = W.randn((4, 16, 2, 64), 6).to(BF)
    kw = dict(B=3, Nkv=2, D=64, num_pages=4, page_size=16, max_pages=2, dtype=W.BF16, layout=W.TND)
    for table, lens, cu, good in (
            ([[0, -1], [9, -1], [2, -1]], [2, 2, 2], [2, 4, 6], {0: (0, 1), 2: (4, 5)}),   # a page outside the pool
            ([[0, -1], [-1, -1], [2, -1]], [2, 2, 2], [2, 4, 6], {0: (0, 1), 2: (4, 5)}),  # no page
            ([[0, -1], [1, -1], [2, -1]], [2, 1, 33], [2, 4, 6], {0: (0, 1)}),             # before 0 and past the table
            ([[0, -1], [1, -1], [2, -1]], [2, 2, 2], [2, 4, 5], {0: (0, 1), 1: (2, 3)})):  # lengths that miss T
        kd, vd = base.cuda(), base.cuda()
        sdpa.attn_cache_append(k, k, dev(table), dev(lens), kd, vd, cu_seqlens=dev(cu), T=6, **kw)
        status(sdpa.ATTN_ERR_DATA)
        want = base.clone()
        for p, toks in good.items():
            for o, t in enumerate(toks):
                want[p, o] = k[t].cpu()
        if cu[-1] == 5:
            want[2, 1] = k[4].cpu()  # the third row has one token of its two
        if lens[1] == 1:
            want[1, 0] = k[3].cpu()  # the second of the row's two tokens has a position
        if lens[2] == 33:
            want = want              # positions 31 (page -1) and 32 (past the table) are both skipped
        assert torch.equal(kd.cpu(), want) and torch.equal(vd.cpu(), want)


# ---- fork ----------------------------------------------------------------------------------------
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("rows_in,rows_out,max_pages", [(1, 1, 1), (9, 9, 7), (7, 12, 40), (12, 5, 33), (300, 300, 5)])
def test_fork(in_place, rows_in, rows_out, max_pages):
    if in_place and rows_in != rows_out:
        pytest.skip("in place the table keeps its rows")
    rng = np.random.default_rng(rows_in + max_pages)
    num = rows_in * max_pages + 5
    lens = [int(x) for x in rng.integers(0, 4 * max_pages + 1, rows_in)]
    table, ref = R.live_table(rng, lens, 4, max_pages, num)
    ref = [r + (1 if r and p % 5 == 0 else 0) for p, r in enumerate(ref)]  # some held elsewhere too
    src = [int(x) for x in rng.integers(-1, rows_in, rows_out)]
    t, r, ln = dev(table), dev(ref), dev(lens)
    to, ro = (t, r) if in_place else (guarded((rows_out, max_pages)), guarded((num,)))
    lo = ln if in_place else guarded((rows_out,))
    outs = [x if in_place else x.t for x in (to, ro, lo)]
    sdpa.attn_cache_fork(t, dev(src), r, outs[0], outs[1], rows_in=rows_in, rows_out=rows_out, max_pages=max_pages,
                         num_pages=num, seq_lens=ln, seq_lens_out=outs[2])
    status()
    want = R.fork(table, src, ref, lens, num)
    for x, y in zip(outs, want):
        assert x.tolist() == y
    if not in_place:
        for x in (to, ro, lo):
            x.check()
        assert t.tolist() == table and r.tolist() == ref and ln.tolist() == lens


def test_fork_without_lengths_many_rows_and_bad_data():
    rng = np.random.default_rng(0)
    table, ref = R.live_table(rng, [1] * 8192, 1, 3, 8200)
    src = [int(x) for x in rng.integers(-1, 8192, 8192)]
    t, r = dev(table), dev(ref)
    sdpa.attn_cache_fork(t, dev(src), r, t, r, rows_in=8192, rows_out=8192, max_pages=3, num_pages=8200)
    status()
    want = R.fork(table, src, ref, [0] * 8192, 8200)
    assert t.tolist() == want[0] and r.tolist() == want[1]
    table = [[0, 7], [1, -1]]
    to, ro = dev(table), dev([1, 1, 0])
    sdpa.attn_cache_fork(dev(table), dev([0, 5, 1]), ro, guarded((3, 2)).t, ro, rows_in=2, rows_out=3, max_pages=2, num_pages=3)
    status(sdpa.ATTN_ERR_DATA)
    sdpa.attn_cache_fork(to, dev([0, 0]), ro, to, ro, rows_in=2, rows_out=2, max_pages=2, num_pages=3)
    status(sdpa.ATTN_ERR_DATA)
    assert to.tolist() == [[0, -1], [0, -1]] and ro.tolist() == [2, 0, 0]


# ---- reserve -------------------------------------------------------------------------------------
def _reserve(table, ref, lens, new, page, null_new=False):
    t, r, c = dev(table), dev(ref), guarded((len(table), 2))
    sdpa.attn_cache_reserve(t, r, dev(lens), None if null_new else dev(new), c.t, B=len(table),
                            max_pages=len(table[0]), num_pages=len(ref), page_size=page)
    c.check()
    try:
        want = R.reserve(table, ref, lens, new, page)
    except R.Refused as e:
        status({"data": sdpa.ATTN_ERR_DATA, "pages": sdpa.ATTN_ERR_PAGES}[e.what])
        want = (table, ref, [[-1, -1]] * len(table))
    else:
        status()
    assert t.tolist() == want[0]
    assert r.tolist() == want[1]
    assert c.t.tolist() == want[2]
    return want


@pytest.mark.parametrize("seed", range(8))
def test_reserve_random(seed):
    """Rows forked at random, with new tokens that reach over several pages; at times too few pages."""
    rng = np.random.default_rng(seed)
    rows, mp, page = int(rng.integers(1, 40)), 12, int(rng.choice([1, 4, 5]))
    lens = [int(x) for x in rng.integers(0, 5 * page, rows)]
    num = int(rng.integers(rows * 5, rows * 14)) + 1
    table, ref = R.live_table(rng, lens, page, mp, num)
    src = [int(x) for x in rng.integers(-1, rows, rows)]
    table, ref, lens = R.fork(table, src, ref, lens, num)
    for _ in range(3):
        new = [int(rng.choice([0, 1, 1, 2, 2 * page + 1])) for _ in lens]
        new = [a if n + a <= mp * page else 0 for a, n in zip(new, lens)]
        lens = [n + a for n, a in zip(lens, new)]
        table, ref, _ = _reserve(table, ref, lens, new, page)
        keep = [int(x) for x in rng.integers(-1, rows, rows)]
        table, ref, lens = R.fork(table, keep, ref, lens, num)
        # a refused step leaves rows without pages for their tokens: cut them back
        lens = [min(n, page * sum(p >= 0 for p in row)) for n, row in zip(lens, table)]


def test_reserve_one_token_for_all_rows_many_pages_and_exact_fit():
    rng = np.random.default_rng(9)
    lens = [int(x) for x in rng.integers(1, 60, 2000)]
    table, ref = R.live_table(rng, [n - 1 for n in lens], 1, 61, sum(lens))
    _reserve(table, ref, lens, [1] * 2000, 1, null_new=True)            # exactly as many pages as are needed
    _reserve(table, ref[:-1] + [1], lens, [1] * 2000, 1, null_new=True)  # one too few
    # whole prompts: more slots than the block has threads, in a pool whose free pages are scattered
    ref = [int(x) for x in rng.integers(0, 2, 9000)]
    _reserve([[-1] * 700 for _ in range(6)], ref, [700, 0, 699, 1, 700, 650], [700, 0, 699, 1, 700, 650], 1)


def test_reserve_all_share_one_page():
    """Every row holds the same partly filled page: one keeps it if all write, none if one does not."""
    for rows in (2, 7, 1500):
        num = rows + 3
        table, ref = [[0, -1] for _ in range(rows)], [rows] + [0] * (num - 1)
        _reserve(table, ref, [3] * rows, [1] * rows, 4)
        _reserve(table, ref, [3] * (rows - 1) + [2], [1] * (rows - 1) + [0], 4)
        _reserve(table, [rows + 1] + ref[1:], [3] * rows, [1] * rows, 4)      # held elsewhere too
        _reserve(table, [rows] + [0] * (rows - 2), [3] * rows, [1] * rows, 4)  # one page too few: undone
        _reserve(table, [rows + 2] + [0] * (rows - 2), [3] * rows, [1] * rows, 4)


def test_reserve_bad_data_changes_nothing():
    table, ref = [[0, -1], [1, -1]], [1, 1, 0, 0]
    _reserve(table, ref, [5, 2], [1, 3], 4)            # more new tokens than the length
    _reserve(table, ref, [9, 2], [1, 1], 4)            # past the table
    _reserve(table, ref, [5, 2], [1, -1], 4)
    _reserve([[0, -1], [9, -1]], ref, [5, 2], [1, 1], 4)   # a page outside the pool
    _reserve([[0, -1], [2, -1]], ref, [5, 2], [1, 1], 4)   # a held page that counts as free
    _reserve([[0, -1]] * 3, [2, 0, 0, 0], [3] * 3, [1] * 3, 4)  # more holders than the count
    _reserve([[0, -1]] * 2 + [[-1, 7]], [2, 0, 0, 0], [3, 3, 5], [1] * 3, 4)  # data error beside shared pages
    for count in (1 << 16, (1 << 16) + 1, 1 << 17, (1 << 17) + 5, 2 ** 31 - 1, -1, -5, -(1 << 16)):
        _reserve([[0, -1]] * 2, [count, 0, 0, 0], [3, 3], [1] * 2, 4)   # the largest count, and what is none
        _reserve([[0, -1]] * 2, [count, 0, 0, 0], [3, 3], [1, 0], 4)


# ---- compact and copy ------------------------------------------------------------------------------
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("num,p_live", [(1, 1.0), (1, 0.0), (2, 0.5), (1023, 0.3), (1024, 0.6), (5000, 0.9), (4097, 0.02), (40000, 0.5),
                                        (70000, 0.7)])
def test_compact(num, p_live, in_place):
    rng = np.random.default_rng(num)
    ref = [int(x) for x in (rng.random(num) < p_live) * rng.integers(1, 4, num)]
    live = [p for p in range(num) if ref[p]]
    rng.shuffle(live)
    rows, mp = 3, len(live) // 3 + 2
    flat = live + [-1] * (rows * mp - len(live))
    table = [flat[r * mp:(r + 1) * mp] for r in range(rows)]
    t, r = dev(table), dev(ref)
    to, ro = (t, r) if in_place else (guarded((rows, mp)).t, guarded((num,)).t)
    pmap, copies, n = guarded((num,)), guarded((num // 2, 2)), guarded((1,))
    sdpa.attn_cache_compact(t, r, to, ro, pmap.t, copies.t, n.t, rows=rows, max_pages=mp, num_pages=num)
    status()
    want = R.compact(table, ref)
    for x, y in zip((to, ro, pmap.t, copies.t), want):
        assert x.tolist() == y
    assert n.t.tolist() == [want[4]]
    for g in (pmap, copies, n):
        g.check()


def test_compact_bad_entries():
    t, r = dev([[0, 9, 2]]), dev([1, 0, 0, 1])
    out = [guarded((4,)).t for _ in range(2)]
    sdpa.attn_cache_compact(t, r, t, out[0], out[1], guarded((2, 2)).t, guarded((1,)).t, rows=1, max_pages=3, num_pages=4)
    status(sdpa.ATTN_ERR_DATA)
    assert t.tolist() == [[0, -1, -1]] and out[0].tolist() == [1, 1, 0, 0] and out[1].tolist() == [0, -1, -1, 1]


@pytest.mark.parametrize("dtype", [BF, F32], ids=IDS)
@pytest.mark.parametrize("elems", [1, 33, 1000, 4096, 70000])
@pytest.mark.parametrize("gap", [0, 24])
def test_copy(dtype, elems, gap):
    rng = np.random.default_rng(elems)
    num = 24
    pages = rng.permutation(num)
    copies = [[int(pages[2 * i]), int(pages[2 * i + 1])] if i % 4 else [-1, -1] for i in range(12)]
    base = [W.randn((num, elems + gap), s).to(dtype) for s in (1, 2)]
    d = [x.cuda() for x in base]
    views = [x[:, :elems] for x in d] if gap else d
    sdpa.attn_cache_copy(*views, dev(copies), n_copies=12, num_pages=num, page_elems=elems,
                         page_stride=elems + gap if gap else 0, dtype=W.dtype_code(dtype))
    status()
    for a, b in copies:
        if a >= 0:
            for x in base:
                x[b, :elems] = x[a, :elems]
    for x, y in zip(d, base):
        assert torch.equal(x.cpu(), y)


def test_copy_bad_pairs_are_skipped():
    base = W.randn((4, 64), 1).to(BF)
    k, v = base.cuda(), base.cuda()
    sdpa.attn_cache_copy(k, v, dev([[0, 4], [-1, 1], [1, -1], [9, 2], [0, 3]]), n_copies=5, num_pages=4, page_elems=64,
                         dtype=W.BF16)
    status(sdpa.ATTN_ERR_DATA)
    base[3] = base[0]
    assert torch.equal(k.cpu(), base) and torch.equal(v.cpu(), base)


# ---- evict -----------------------------------------------------------------------------------------
@pytest.mark.parametrize("page", [1, 4, 16])
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 3), (16, 16), (40, 1), (3, 1000), (sdpa.ATTN_WINDOW_ALL, 2)])
def test_evict(page, window, sinks):
    rng = np.random.default_rng(page)
    lens = [0, 1, 15, 16, 17, 64, 100, 100, 100]
    mp = 100 // page + 2
    num = sum(-(-n // page) for n in lens) + 3
    table, ref = R.live_table(rng, lens, page, mp, num)
    table, ref, lens = R.fork(table, [0, 1, 2, 3, 4, 5, 6, 6, 8], ref, lens, num)  # row 7 shares row 6's pages
    t, r = dev(table), dev(ref)
    sdpa.attn_cache_evict(t, r, dev(lens), B=9, max_pages=mp, num_pages=num, page_size=page, window_tokens=window,
                          sink_tokens=sinks)
    status()
    want = R.evict(table, ref, lens, page, window, sinks)
    assert t.tolist() == want[0] and r.tolist() == want[1]


def test_evict_bad_data():
    table, ref = [[0, 1, 9], [2, 3, 4]], [1] * 6
    t, r = dev(table), dev(ref)
    sdpa.attn_cache_evict(t, r, dev([12, 13]), B=2, max_pages=3, num_pages=6, page_size=4, window_tokens=1)
    status(sdpa.ATTN_ERR_DATA)  # row 1 is longer than its table
    assert t.tolist() == [[-1, -1, 9], [2, 3, 4]] and r.tolist() == [0, 0, 1, 1, 1, 1]
    t, r = dev([[0, 7, 2]]), dev(ref)
    sdpa.attn_cache_evict(t, r, dev([12]), B=1, max_pages=3, num_pages=6, page_size=4, window_tokens=1)
    status(sdpa.ATTN_ERR_DATA)
    assert t.tolist() == [[-1, 7, 2]] and r.tolist() == [0, 1, 1, 1, 1, 1]


# ---- all of them together ---------------------------------------------------------------------------
class Model:
    """The keys and values of each row as plain lists, beside a PagedCache of two layers."""

    def __init__(self, cache, dtype, seed):
        self.cache, self.dtype, self.seed = cache, dtype, seed
        self.kv = [[([], []) for _ in range(cache.rows)] for _ in range(cache.layers)]

    def draw(self, shape):
        self.seed += 1
        return W.randn(shape, self.seed).to(self.dtype)

    def step(self, new):
        """Adds new[b] tokens to each row in both layers; returns the packed (k, v) of each."""
        c = self.cache
        out = []
        for layer in range(c.layers):
            k, v = self.draw((sum(new), c.Nkv, c.D)), self.draw((sum(new), c.Nkv, c.D))
            t = 0
            for b, n in enumerate(new):
                for i in range(t, t + n):
                    self.kv[layer][b][0].append(k[i])
                    self.kv[layer][b][1].append(v[i])
                t += n
            out.append((k, v))
        return out

    def fork(self, src):
        for layer in range(self.cache.layers):
            old = self.kv[layer]
            self.kv[layer] = [(list(old[s][0]), list(old[s][1])) if s >= 0 else ([], []) for s in src]

    def attend(self, layer, q):
        c = self.cache
        out, A = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
        for b in range(c.rows):
            ks, vs = self.kv[layer][b]
            if not ks:
                continue
            k, v = torch.stack(ks), torch.stack(vs)
            seen = R.window_seen(1, len(ks), c.window_tokens, c.sink_tokens)
            for h in range(c.Nq):
                g = h // (c.Nq // c.Nkv)
                o, _, _, a, _ = R.attend(q[b, h][None], k[:, g], v[:, g], seen, c.scale)
                out[b, h], A[b, h] = o[0], a[0]
        return out.numpy(), A.numpy()


@pytest.mark.parametrize("dtype,layout,D,window,sinks", [
    (BF, W.TND, 128, sdpa.ATTN_WINDOW_ALL, 0), (F16, W.BHSD, 64, 40, 5), (F32, W.TND, 40, 24, 0),
    (BF, W.BHSD, 64, 30, 40)], ids=["bf16", "f16-window", "f32-window", "bf16-sinks"])
def test_serving_from_prompts_to_beams(dtype, layout, D, window, sinks):
    """Prompts through the windowed forward into the cache, tokens one by one, forks as beam search makes
    them, eviction, compaction and rows that end, in two layers that share the table; after every step
    attention over the pages is that over the rows' own lists of keys and values."""
    from scaled_dot_product_16_b200.cache import PagedCache
    rng = np.random.default_rng(D)
    rows, Nq, Nkv = 6, 8, 2
    cache = PagedCache(layers=2, rows=rows, max_pages=24, num_pages=90, page_size=8, Nq=Nq, Nkv=Nkv, D=D,
                       dtype=W.dtype_code(dtype), layout=layout, window_tokens=window, sink_tokens=sinks)
    cache.pool.fill_(float("nan"))  # nothing that was not written is seen
    model = Model(cache, dtype, 100 * D)

    def attend():
        for layer in range(2):
            q = model.draw((rows, Nq, D))
            out = G.Guarded(tuple(q.shape), dtype)
            cache.attend(layer, q.cuda(), out.t)
            cache.check()
            out.check()
            ref, A = model.attend(layer, q)
            G.check_out(G.f64(out.t.cpu()), ref, W.dtype_code(dtype), abs_ref=A)

    new = [50, 1, 0, 83, 16, 7]
    cache.reserve(dev(new))
    cu = dev(np.cumsum(new).tolist())
    for layer, (k, v) in enumerate(model.step(new)):
        q = model.draw((sum(new), Nq, D))
        out = G.Guarded(tuple(q.shape), dtype)
        cache.prefill(layer, q.cuda(), k.cuda(), v.cuda(), cu, out.t)
        cache.check()
        out.check()
        inp = W.AttnInputs(q, k, v, W.TND, 0, W.dtype_code(dtype), rows, sum(new), sum(new), Nq, Nkv, D, cache.scale,
                           np.cumsum(new).astype(np.int32), np.cumsum(new).astype(np.int32))
        ref, _, _, A = R.window_fwd(inp, window, sinks)
        G.check_out(G.f64(out.t.cpu()), ref, inp.dtype, abs_ref=A)
    attend()
    for step in range(8):
        cache.reserve()
        for layer, (k, v) in enumerate(model.step([1] * rows)):
            cache.append(layer, k.cuda(), v.cuda())
        attend()
        if step == 5:
            src = [0, 1, 2, -1, 4, 4]   # a row ends, one is forked
        else:
            src = [int(x) for x in rng.integers(0, rows, rows)]
        cache.fork(dev(src))
        model.fork(src)
        if step % 3 == 1 and window < 100:
            cache.evict()
        if step % 3 == 2:
            cache.compact()
            cache.check()
            n = int(cache.live_pages)
            assert (cache.ref_count[:n] > 0).all() and not cache.ref_count[n:].any()
        held = cache.page_table[cache.page_table >= 0].long()
        assert torch.equal(torch.bincount(held, minlength=90).int(), cache.ref_count)
        attend()
    cache.fork(dev([-1] * rows))
    cache.check()
    assert not cache.ref_count.any() and not cache.seq_lens.any() and bool((cache.page_table == -1).all())
    cache.reserve(dev([24 * 8] * rows))   # more pages than there are
    with pytest.raises(sdpa.AttnError, match="pages"):
        cache.check()


def test_a_step_captured_into_a_graph():
    """reserve, append and attend recorded once and replayed token by token."""
    from scaled_dot_product_16_b200.cache import PagedCache
    rows, Nq, Nkv, D = 4, 4, 2, 64
    cache = PagedCache(layers=1, rows=rows, max_pages=6, num_pages=30, page_size=4, Nq=Nq, Nkv=Nkv, D=D, dtype=W.BF16)
    model = Model(cache, BF, 5)
    q, k, v = (torch.zeros((rows, n, D), dtype=BF, device="cuda") for n in (Nq, Nkv, Nkv))
    out = torch.empty_like(q)

    def step():
        cache.reserve()
        cache.append(0, k, v)
        cache.attend(0, q, out)

    step()                       # once outside the capture; then from the start again
    cache.fork(dev([-1] * rows))
    cache.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    cache.fork(dev([-1] * rows))
    for i in range(20):
        (kn, vn), = model.step([1] * rows)
        qn = model.draw((rows, Nq, D))
        q.copy_(qn), k.copy_(kn), v.copy_(vn)
        if i == 7:
            cache.fork(dev([0, 0, 2, 1]))
            model.fork([0, 0, 2, 1])
            for b in range(rows):  # the step's own token is the one drawn for the row
                model.kv[0][b] = (model.kv[0][b][0][:-1] + [kn[b]], model.kv[0][b][1][:-1] + [vn[b]])
        g.replay()
        cache.check()
        ref, A = model.attend(0, qn)
        G.check_out(G.f64(out.cpu()), ref, W.BF16, abs_ref=A)
    assert cache.seq_lens.tolist() == [20] * rows

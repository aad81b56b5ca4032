"""Plain float64 implementations of the serving operators, for their tests: windowed attention with
sink tokens, attention of one token over a paged cache, and the page bookkeeping row by row as
include/attn.h states it. No code is shared with the library; test_serving_ref.py holds them against
the oracle and against closed forms."""
from __future__ import annotations

import numpy as np
import torch

from scaled_dot_product_16_b200 import workloads as W


def attend(q, k, v, seen, scale):
    """q [n, D], k, v [m, D], seen [n, m] -> out, max, sum, A (sum of w |v|), S (largest sum |q k| scale)."""
    q, k, v = (x.double() for x in (q, k, v))
    s = torch.where(seen, (q @ k.T) * scale, torch.tensor(-torch.inf, dtype=torch.float64))
    big = torch.where(seen, (q.abs() @ k.abs().T) * scale, torch.tensor(0.0, dtype=torch.float64))
    if k.shape[0] == 0:
        z = torch.zeros(q.shape[0], dtype=torch.float64)
        return torch.zeros_like(q), z - torch.inf, z, torch.zeros_like(q), z
    m = s.amax(1)
    e = torch.exp(s - torch.where(m == -torch.inf, 0.0, m)[:, None])
    l = e.sum(1)
    w = e / torch.where(l == 0, 1.0, l)[:, None]
    v = torch.where(seen.any(0)[:, None], v, 0.0)     # a key that no row sees may hold anything
    return w @ v, m, l, w @ v.abs(), big.amax(1)


def window_seen(sq, sk, window, sinks):
    p = torch.arange(sq)[:, None] + sk - sq
    j = torch.arange(sk)[None, :]
    return (j <= p) & ((j > p - window) | (j < sinks))


def window_fwd(inp: W.AttnInputs, window, sinks):
    """(out, max, sum, A) in the layouts of attn_fwd_sinks."""
    shape = tuple(inp.q.shape)
    out, A = torch.zeros(shape, dtype=torch.float64), torch.zeros(shape, dtype=torch.float64)
    m = torch.zeros(shape[:-1], dtype=torch.float64)
    l = torch.zeros_like(m)
    grp = inp.Nq // inp.Nkv
    if inp.layout == W.TND:
        eq, ek = [0] + list(inp.cu_q), [0] + list(inp.cu_kv)
    for b in range(inp.B):
        for h in range(inp.Nq):
            if inp.layout == W.TND:
                iq, ik = (slice(eq[b], eq[b + 1]), h), (slice(ek[b], ek[b + 1]), h // grp)
            else:
                iq, ik = (b, h), (b, h // grp)
            q, k, v = inp.q[iq], inp.k[ik], inp.v[ik]
            out[iq], m[iq], l[iq], A[iq], _ = attend(q, k, v, window_seen(len(q), len(k), window, sinks), inp.scale)
    return out.numpy(), m.numpy(), l.numpy(), A.numpy()


def decode(q, k_cache, v_cache, table, lens, *, layout, page_size, scale, window, sinks):
    """q [B, Nq, D], caches as attn_decode_paged takes them (CPU tensors) -> out, max, sum, A, S, keys seen."""
    B, Nq, _ = q.shape
    tnd = layout == W.TND
    Nkv = k_cache.shape[2] if tnd else k_cache.shape[1]
    grp = Nq // Nkv
    out, A = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    m = torch.full((B, Nq), -torch.inf, dtype=torch.float64)
    l, S = torch.zeros((B, Nq), dtype=torch.float64), torch.zeros((B, Nq), dtype=torch.float64)
    seen = np.zeros(B, np.int64)
    for b in range(B):
        n = int(lens[b])
        pos = [j for j in range(n) if j >= n - window or j < sinks]
        pos = [j for j in pos if 0 <= int(table[b, j // page_size]) < k_cache.shape[0]]
        seen[b] = len(pos)
        if not pos:
            continue
        page = torch.tensor([int(table[b, j // page_size]) for j in pos])
        off = torch.tensor([j % page_size for j in pos])
        for h in range(Nkv):
            k, v = ((x[page, off, h] if tnd else x[page, h, off]) for x in (k_cache, v_cache))
            r = slice(h * grp, (h + 1) * grp)
            out[b, r], m[b, r], l[b, r], A[b, r], S[b, r] = attend(
                q[b, r], k, v, torch.ones((grp, len(pos)), dtype=torch.bool), scale)
    return out, m, l, A, S, seen


class Refused(Exception):
    """The whole call is refused: `what` is "data" or "pages"."""

    def __init__(self, what):
        super().__init__(what)
        self.what = what


def fork(table, src, ref, lens, num_pages):
    """New table, counts and lengths (lists)."""
    ref = list(ref)
    for row in table:
        for p in row:
            if 0 <= p < num_pages:
                ref[p] -= 1
    width = len(table[0]) if table else 0
    out, ln = [], []
    for s in src:
        ok = 0 <= s < len(table)
        out.append([(p if p < num_pages else -1) for p in table[s]] if ok else [-1] * width)
        ln.append(lens[s] if ok else 0)
        for p in out[-1]:
            if p >= 0:
                ref[p] += 1
    return out, ref, ln


def reserve(table, ref, lens, new, page_size):
    """Table, counts and copies afterwards, or Refused."""
    num_pages, max_pages = len(ref), len(table[0])
    slots = []
    for b, (n, a) in enumerate(zip(lens, new)):
        if a < 0 or n < a or n > max_pages * page_size:
            raise Refused("data")
        if a:
            slots += [(b, i) for i in range((n - a) // page_size, (n - 1) // page_size + 1)]
    asking = {}
    for b, i in slots:
        p = table[b][i]
        if p >= num_pages:
            raise Refused("data")
        if p >= 0 and not 1 <= ref[p] <= 1 << 16:
            raise Refused("data")
        if p >= 0 and ref[p] > 1:
            asking.setdefault(p, []).append((b, i))
    if any(len(a) > ref[p] for p, a in asking.items()):
        raise Refused("data")
    keeps = {a[0] for p, a in asking.items() if len(a) == ref[p]}
    todo = [(b, i) for b, i in slots if table[b][i] < 0 or (table[b][i] in asking and (b, i) not in keeps)]
    free = [p for p in range(num_pages) if ref[p] == 0]
    if len(free) < len(todo):
        raise Refused("pages")
    table, ref = [list(r) for r in table], list(ref)
    copies = [[-1, -1] for _ in table]
    for (b, i), p in zip(todo, free):
        old, start = table[b][i], lens[b] - new[b]
        if old >= 0:
            ref[old] -= 1
            if i == start // page_size and start % page_size:
                copies[b] = [old, p]
        table[b][i] = p
        ref[p] = 1
    return table, ref, copies


def compact(table, ref):
    """Table, counts, page map, copies and the number of live pages afterwards."""
    live = [p for p, r in enumerate(ref) if r > 0]
    n = len(live)
    holes = [p for p in range(n) if ref[p] == 0]
    high = [p for p in live if p >= n]
    pmap = [p if r > 0 else -1 for p, r in enumerate(ref)]
    for p, h in zip(high, holes):
        pmap[p] = h
    out = [0] * len(ref)
    for p in live:
        out[pmap[p]] = ref[p]
    copies = [list(x) for x in zip(high, holes)]
    copies += [[-1, -1]] * (len(ref) // 2 - len(copies))
    return [[pmap[p] if 0 <= p < len(ref) else -1 for p in row] for row in table], out, pmap, copies, n


def live_table(rng, lens, page_size, max_pages, num_pages, share=0):
    """A table whose rows hold what their lengths need, in a random order of the pool, and its counts.
    With share > 0, row r + 1 .. r + share hold the pages of row r (equal lengths are the caller's)."""
    order = list(rng.permutation(num_pages))
    table, ref = [], [0] * num_pages
    for r, n in enumerate(lens):
        need = -(-n // page_size)
        if share and r % (share + 1):
            row = list(table[r - r % (share + 1)])
        else:
            row = [int(order.pop()) for _ in range(need)] + [-1] * (max_pages - need)
        for p in row:
            if p >= 0:
                ref[p] += 1
        table.append(row)
    return table, ref


def evict(table, ref, lens, page_size, window, sinks):
    """Table and counts afterwards."""
    table, ref = [list(r) for r in table], list(ref)
    for row, n in zip(table, lens):
        for i, p in enumerate(row):
            gone = all(sinks <= j < n - window for j in range(i * page_size, (i + 1) * page_size))
            if 0 <= p < len(ref) and gone:
                row[i] = -1
                ref[p] -= 1
    return table, ref

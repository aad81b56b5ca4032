"""Cases for the serving operators: sliding-window attention with sink tokens over a prompt, attention
of one new token over a paged key/value cache, the writes of new tokens into that cache, and the
bookkeeping of its pages (forking, reserving, copying, compacting).

A case is a dict of plain values. prepare() makes what a serving program holds before the call, run()
makes one pass (the plain torch form, or the library's calls where `own` is true), work() counts the
bytes and operations a pass cannot do without, exact() computes the outputs from their definitions in
64 bits.

Ragged lengths are a fixed function of the case (golden-ratio fractions of the longest length), so that
work() does not depend on the seed; values, page orders and beam parents come from the seed.
"""
import math

import torch

own = False

BF16, F32, F16 = 0, 1, 2          # the library's dtype codes
BHSD, TND = 0, 1                  # and its layout codes
DT = {"bf16": torch.bfloat16, "f32": torch.float32, "f16": torch.float16}
CODE = {"bf16": BF16, "f32": F32, "f16": F16}
LAY = {"bhsd": BHSD, "tnd": TND}
NO_WINDOW = 1 << 30               # a window of every key
WORKSPACE_BYTES = 32 << 20        # a decoding program's workspace, made once and zero-filled
GOLD = 0.6180339887498949


# ------------------------------------------------------------------------------------------------
# the cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # a short prompt through a small fp32 model: odd head size, odd length, latency counts
        dict(name="window f32 short", op="window", dtype="f32", layout="bhsd", B=2, Nq=4, Nkv=4, D=80,
             S=333, ctx=0, window=128, sinks=4),
        # an ordinary packed batch of prompts, an empty one among them, grouped heads
        dict(name="window bf16 packed", op="window", dtype="bf16", layout="tnd", B=6, Nq=32, Nkv=8, D=128,
             S=4096, ctx=0, window=1024, sinks=4),
        # one chunk of a long prompt against the keys of the chunks before it (bottom-right aligned)
        dict(name="window f16 chunk", op="window", dtype="f16", layout="bhsd", B=1, Nq=16, Nkv=16, D=64,
             S=2047, ctx=14364, window=4096, sinks=64),
        # one interactive user: the smallest decode call, latency counts
        dict(name="decode bf16 one", op="decode", dtype="bf16", layout="tnd", B=1, Nq=32, Nkv=8, D=128,
             L=1000, page=16, window=0, sinks=0),
        # the ordinary serving batch: ragged lengths, grouped heads, small pages
        dict(name="decode bf16 batch", op="decode", dtype="bf16", layout="tnd", B=64, Nq=32, Nkv=8, D=128,
             L=8192, page=16, window=0, sinks=0),
        # few very long sequences, one key head for all query heads: parallel along the length only
        dict(name="decode bf16 long", op="decode", dtype="bf16", layout="bhsd", B=2, Nq=8, Nkv=1, D=128,
             L=131072, page=64, window=0, sinks=0),
        # a stream that keeps a window and a few sinks of a long history, a key head per query head
        dict(name="decode f16 window", op="decode", dtype="f16", layout="bhsd", B=16, Nq=16, Nkv=16, D=64,
             L=32768, page=64, window=4096, sinks=4),
        # the same call in full precision, an odd page size
        dict(name="decode f32 batch", op="decode", dtype="f32", layout="tnd", B=16, Nq=8, Nkv=2, D=128,
             L=4096, page=24, window=0, sinks=0),
        # one decode step's new keys and values
        dict(name="append step", op="append", dtype="bf16", layout="tnd", B=64, Nkv=8, D=128, L=4096,
             new=1, page=16),
        # the keys and values of whole prompts
        dict(name="append prompts", op="append", dtype="bf16", layout="bhsd", B=16, Nkv=8, D=128, L=4096,
             new=2048, page=16),
        # a beam-search step: rows take their parents' pages, shared last pages are copied for the next token
        dict(name="fork beams", op="fork", dtype="bf16", layout="tnd", groups=16, beams=8, Nkv=8, D=128,
             L=2048, page=16),
        # compaction of a fragmented pool before it shrinks
        dict(name="compact pool", op="compact", dtype="bf16", layout="tnd", pages=8192, live=0.6, rows=64,
             Nkv=8, D=128, page=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["window", "window", "window", "decode", "decode", "decode", "append", "fork", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    layout = rng.choice(["bhsd", "tnd"])
    most = {"window": (2.0e8, 4.0e11), "decode": (1.2e9, 2e10)}
    for _ in range(1000):
        nkv = rng.choice([1, 2, 4, 8, 16])
        D = rng.choice([64, 128]) if dtype != "f32" else rng.choice([64, 128, rng.randint(16, 128)])
        if op == "window":
            c = dict(op=op, dtype=dtype, layout=layout, B=rng.randint(1, 6), Nq=nkv * rng.choice([1, 2, 3, 4, 8]),
                     Nkv=nkv, D=D, S=_log(rng, 1, 4096), ctx=rng.choice([0, 0, _log(rng, 1, 14000)]),
                     window=_log(rng, 1, 8192), sinks=rng.choice([0, rng.randint(1, 8), rng.randint(9, 300)]))
            if c["Nq"] > 32 or c["B"] * c["Nq"] * c["S"] * (c["S"] + c["ctx"]) > 3.3e9:
                continue
            if dtype == "f32" and work(c)["flops"] > 4.0e10:
                continue
        elif op == "decode":
            c = dict(op=op, dtype=dtype, layout=layout, B=_log(rng, 1, 128), Nq=nkv * rng.choice([1, 2, 4, 5, 8]),
                     Nkv=nkv, D=D, L=_log(rng, 1, 131072), page=rng.choice([1, 16, 16, 24, 32, 64, 128]),
                     window=rng.choice([0, _log(rng, 1, 8192)]), sinks=0)
            if c["window"]:
                c["sinks"] = rng.choice([0, rng.randint(1, 8), rng.randint(9, 300)])
            # the plain form gathers every key in fp32; an odd page of one token needs a long table
            if c["Nq"] > 64 or c["B"] * c["L"] * c["Nkv"] * D > 1.1e9 or c["L"] // c["page"] > 32768:
                continue
        elif op == "append":
            new = rng.choice([1, _log(rng, 1, 2048)])
            c = dict(op=op, dtype=dtype, layout=layout, B=_log(rng, 1, 128), Nkv=nkv, D=D,
                     L=max(new, _log(rng, 16, 8192)), new=new, page=rng.choice([1, 16, 24, 64]))
            if c["B"] * c["L"] * nkv * D > 4e8 or c["B"] * new * nkv * D > 1.6e7:
                continue
        elif op == "fork":
            c = dict(op=op, dtype=dtype, layout=layout, groups=_log(rng, 1, 32), beams=rng.randint(1, 8), Nkv=nkv, D=D,
                     L=_log(rng, 8, 4096), page=rng.choice([8, 16, 24, 64]))
            if c["groups"] * c["beams"] * (c["L"] / 4 + 2 * c["page"]) * nkv * D > 1.2e8:
                continue
        else:
            c = dict(op=op, dtype=dtype, layout=layout, pages=_log(rng, 64, 8192), live=round(rng.uniform(0.1, 0.95), 2),
                     rows=_log(rng, 1, 64), Nkv=nkv, D=D, page=rng.choice([8, 16, 24, 64]))
            if c["pages"] * c["page"] * nkv * D > 1.3e8:
                continue
        if op in most:
            w = work(c)
            if w["bytes"] > most[op][0] or w["flops"] > most[op][1]:
                continue
        return c
    return dict(listed()[3], name=None, L=rng.randint(1, 1000))


# ------------------------------------------------------------------------------------------------
# lengths
# ------------------------------------------------------------------------------------------------
def _lens(n, longest, empty=True):
    """n ragged lengths up to `longest`: the first one is the longest, one of four or more is empty."""
    out = [longest] + [1 + int(((i * GOLD) % 1.0) * longest) for i in range(1, n)]
    if empty and n >= 4:
        out[n // 2] = 0
    return [min(x, longest) for x in out]


def _window_lens(c):
    """Query and key lengths of each sequence."""
    q = _lens(c["B"], c["S"]) if c["layout"] == "tnd" else [c["S"]] * c["B"]
    return q, [x + c["ctx"] if x else 0 for x in q]


def _span(c):
    """Window and sinks of a case as the calls take them (0: every key)."""
    return (c["window"], c["sinks"]) if c["window"] else (NO_WINDOW, 0)


def _visible(p, window, sinks):
    """Keys that position p sees: those of the window that ends at p, and the sinks before it."""
    n = min(p + 1, window)
    return n + min(sinks, p + 1 - n)


def _visible_sum(sq, sk, window, sinks):
    """Sum of _visible over the positions sk - sq .. sk - 1."""
    def upto(n):                     # positions 0 .. n - 1
        a = min(n, window)           # those that see every key before them
        total = a * (a + 1) // 2 + (n - a) * window
        m = min(n - a, sinks)        # those whose sinks are still partly in the window
        return total + m * (m + 1) // 2 + (n - a - m) * sinks
    return upto(sk) - upto(sk - sq)


def _step_lens(c):
    return _lens(c["B"], c["L"])


def _append_lens(c):
    """Lengths after the append, and the tokens appended, of each sequence."""
    new = [1] * c["B"] if c["new"] == 1 else _lens(c["B"], c["new"])
    full = _lens(c["B"], c["L"], empty=False)
    return [max(a, n) for a, n in zip(full, new)], new


def _fork_lens(c):
    """Length of each group's rows, their pages, and how many of these all rows of the group share."""
    ln = _lens(c["groups"], c["L"], empty=False)
    used = [-(-x // c["page"]) for x in ln]
    return ln, used, [3 * u // 4 for u in used]


# ------------------------------------------------------------------------------------------------
# the work of a pass
# ------------------------------------------------------------------------------------------------
def work(case):
    c = case
    es = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "window":
        lq, lk = _window_lens(c)
        pairs = sum(_visible_sum(a, b, c["window"], c["sinks"]) for a, b in zip(lq, lk))
        io = (2 * sum(lq) * c["Nq"] + 2 * sum(_keys_read(a, b, c) for a, b in zip(lq, lk)) * c["Nkv"]) * c["D"] * es
        return {"bytes": io + 8 * sum(lq) * c["Nq"], "flops": 4.0 * c["D"] * c["Nq"] * pairs}
    if c["op"] == "decode":
        w, s = _span(c)
        keys = sum(_visible(x - 1, w, s) if x else 0 for x in _step_lens(c))
        io = 2 * keys * c["Nkv"] * c["D"] * es + 2 * c["B"] * c["Nq"] * c["D"] * es
        return {"bytes": io + 8 * c["B"] * c["Nq"] + 4 * (c["B"] + keys // c["page"]),
                "flops": 4.0 * c["D"] * c["Nq"] * keys}
    row = c["Nkv"] * c["D"] * es
    if c["op"] == "append":
        _, new = _append_lens(c)
        return {"bytes": 4 * sum(new) * row, "flops": 0}
    if c["op"] == "fork":
        ln, used, _ = _fork_lens(c)
        rows, cols = c["groups"] * c["beams"], -(-(c["L"] + 1) // c["page"]) + 1
        b = c["beams"]
        # rows of a parent beyond its first child copy the last page, where it is partly filled
        copies = sum(b * (1 - 1 / b) ** b for x in ln[:_live_groups(c)] if x % c["page"])
        return {"bytes": 8 * rows * cols + 4 * copies * c["page"] * row, "flops": 0}
    used = c["live"] * c["pages"]
    return {"bytes": 12 * c["pages"] + 4 * used * (1 - c["live"]) * c["page"] * row, "flops": 0}


def _keys_read(lq, lk, c):
    """Keys of a sequence that some query sees."""
    if lq == 0:
        return 0
    first = max(0, lk - lq - c["window"] + 1)
    return lk - first + min(c["sinks"], first)


def _live_groups(c):
    """A finished request among them, where there are four or more: its rows are freed."""
    return c["groups"] - 1 if c["groups"] >= 4 else c["groups"]


# ------------------------------------------------------------------------------------------------
# what a program holds before the call
# ------------------------------------------------------------------------------------------------
def _cache_shape(c, pages):
    return (pages, c["page"], c["Nkv"], c["D"]) if c["layout"] == "tnd" else (pages, c["Nkv"], c["page"], c["D"])


def _randn(shape, g, dt):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)


def _page_table(lens, page, cols, pool, g):
    """A table whose rows hold pages in a random order of the pool; unused entries are -1."""
    need = torch.tensor([-(-x // page) for x in lens], device="cuda")
    held = torch.arange(cols, device="cuda")[None, :] < need[:, None]
    order = torch.randperm(pool, generator=g, device="cuda")
    at = (held.reshape(-1).cumsum(0) - 1).clamp_(min=0)
    return torch.where(held, order[at].reshape(held.shape), -1).to(torch.int32)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DT[c["dtype"]]
    s = dict(c=c, dtype=CODE[c["dtype"]], layout=LAY[c["layout"]])
    if c["op"] == "window":
        lq, lk = _window_lens(c)
        if c["layout"] == "tnd":
            s.update(Sq=sum(lq), Skv=sum(lk),
                     cu_q=torch.tensor(lq, device="cuda").cumsum(0).to(torch.int32),
                     cu_k=torch.tensor(lk, device="cuda").cumsum(0).to(torch.int32))
            qs, ks, st = (s["Sq"], c["Nq"], c["D"]), (s["Skv"], c["Nkv"], c["D"]), (s["Sq"], c["Nq"])
        else:
            s.update(Sq=lq[0], Skv=lk[0], cu_q=None, cu_k=None)
            qs, ks = (c["B"], c["Nq"], s["Sq"], c["D"]), (c["B"], c["Nkv"], s["Skv"], c["D"])
            st = (c["B"], c["Nq"], s["Sq"])
        s.update(q=_randn(qs, g, dt), k=_randn(ks, g, dt), v=_randn(ks, g, dt),
                 out=torch.empty(qs, device="cuda", dtype=dt), mx=torch.empty(st, device="cuda"),
                 sm=torch.empty(st, device="cuda"))
    elif c["op"] == "decode":
        lens = _step_lens(c)
        cols = -(-c["L"] // c["page"])
        pool = sum(-(-x // c["page"]) for x in lens) + 3
        w, sinks = _span(c)
        table = _page_table(lens, c["page"], cols, pool, g)
        s.update(cols=cols, pool=pool, window=w, sinks=sinks, table=table,
                 lens=torch.tensor(lens, device="cuda", dtype=torch.int32),
                 q=_randn((c["B"], c["Nq"], c["D"]), g, dt), k=_randn(_cache_shape(c, pool), g, dt),
                 v=_randn(_cache_shape(c, pool), g, dt), ws=torch.zeros(WORKSPACE_BYTES, device="cuda", dtype=torch.uint8),
                 out=torch.empty((c["B"], c["Nq"], c["D"]), device="cuda", dtype=dt),
                 mx=torch.empty((c["B"], c["Nq"]), device="cuda"), sm=torch.empty((c["B"], c["Nq"]), device="cuda"))
    elif c["op"] == "append":
        lens, new = _append_lens(c)
        cols = -(-max(lens) // c["page"])
        pool = sum(-(-x // c["page"]) for x in lens) + 3
        s.update(T=sum(new), cols=cols, pool=pool, table=_page_table(lens, c["page"], cols, pool, g),
                 lens=torch.tensor(lens, device="cuda", dtype=torch.int32),
                 cu=None if c["new"] == 1 else torch.tensor(new, device="cuda").cumsum(0).to(torch.int32),
                 k_new=_randn((sum(new), c["Nkv"], c["D"]), g, dt), v_new=_randn((sum(new), c["Nkv"], c["D"]), g, dt),
                 k=_randn(_cache_shape(c, pool), g, dt), v=_randn(_cache_shape(c, pool), g, dt))
    elif c["op"] == "fork":
        ln, used, shared = _fork_lens(c)
        b, rows, cols = c["beams"], c["groups"] * c["beams"], -(-(c["L"] + 1) // c["page"]) + 1
        pool = sum(sh + b * (u - sh + 1) for u, sh in zip(used, shared)) + 3
        # every row holds its own pages behind the ones that its group shares
        own_lens = [(u - sh) * c["page"] for u, sh in zip(used, shared) for _ in range(b)]
        need = torch.tensor(used, device="cuda").repeat_interleave(b)[:, None]
        sh = torch.tensor(shared, device="cuda").repeat_interleave(b)[:, None]
        col = torch.arange(cols, device="cuda")[None, :]
        order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
        first = torch.tensor([0] + shared, device="cuda").cumsum(0)[:-1].repeat_interleave(b)[:, None]
        mine = torch.tensor([0] + [x // c["page"] for x in own_lens], device="cuda").cumsum(0)[:-1][:, None]
        at = torch.where(col < sh, first + col, sum(shared) + mine + col - sh)
        table = torch.where(col < need, order[at.clamp(0, pool - 1)], -1).to(torch.int32)
        ref = torch.zeros(pool + 1, device="cuda", dtype=torch.int32)
        ref.scatter_add_(0, torch.where(table < 0, pool, table).reshape(-1).long(),
                         torch.ones(rows * cols, device="cuda", dtype=torch.int32))
        group = torch.arange(rows, device="cuda") // b
        parent = group * b + torch.randint(0, b, (rows,), generator=g, device="cuda")
        live = group < _live_groups(c)
        s.update(rows=rows, cols=cols, pool=pool, table=table, ref=ref[:pool].contiguous(),
                 lens=torch.tensor([x for x in ln for _ in range(b)], device="cuda", dtype=torch.int32),
                 src=torch.where(live, parent, -1).to(torch.int32), new=live.to(torch.int32),
                 k=_randn(_cache_shape(c, pool), g, dt), v=_randn(_cache_shape(c, pool), g, dt))
        s.update(table_out=torch.empty_like(s["table"]), ref_out=torch.empty_like(s["ref"]),
                 lens_out=torch.empty_like(s["lens"]), copies=torch.empty((rows, 2), device="cuda", dtype=torch.int32))
    else:
        live = int(c["live"] * c["pages"])
        cols = -(-live // c["rows"])
        # the live pages, spread over the rows: row r holds entries r, r + rows, ...
        order = torch.randperm(c["pages"], generator=g, device="cuda")[:live].to(torch.int32)
        at = torch.arange(cols, device="cuda")[None, :] * c["rows"] + torch.arange(c["rows"], device="cuda")[:, None]
        table = torch.where(at < live, order[at.clamp(max=live - 1)], -1).to(torch.int32)
        ref = torch.zeros(c["pages"], device="cuda", dtype=torch.int32)
        ref[order.long()] = 1
        s.update(cols=cols, table=table, ref=ref, k=_randn(_cache_shape(c, c["pages"]), g, dt),
                 v=_randn(_cache_shape(c, c["pages"]), g, dt), table_out=torch.empty_like(table),
                 ref_out=torch.empty_like(ref), page_map=torch.empty_like(ref),
                 copies=torch.empty((c["pages"] // 2, 2), device="cuda", dtype=torch.int32),
                 live=torch.empty(1, device="cuda", dtype=torch.int32))
    return s


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(state):
    if own:
        return OWN[state["c"]["op"]](state)
    return PLAIN[state["c"]["op"]](state)


# ---- the library's calls ------------------------------------------------------------------------
def _own_window(s):
    import scaled_dot_product_16_b200 as sdpa
    c = s["c"]
    sdpa.attn_fwd_sinks(s["q"], s["k"], s["v"], cu_seqlens_q=s["cu_q"], cu_seqlens_kv=s["cu_k"], B=c["B"], Sq=s["Sq"],
                        Skv=s["Skv"], Nq=c["Nq"], Nkv=c["Nkv"], D=c["D"], scale=c["D"] ** -0.5,
                        window_tokens=c["window"], sink_tokens=c["sinks"], dtype=s["dtype"], layout=s["layout"],
                        out=s["out"], softmax_max=s["mx"], softmax_sum=s["sm"])
    return s["out"], s["mx"], s["sm"]


def _own_decode(s):
    import scaled_dot_product_16_b200 as sdpa
    c = s["c"]
    sdpa.attn_decode_paged(s["q"], s["k"], s["v"], s["table"], s["lens"], B=c["B"], Nq=c["Nq"], Nkv=c["Nkv"], D=c["D"],
                           num_pages=s["pool"], page_size=c["page"], max_pages=s["cols"], scale=c["D"] ** -0.5,
                           window_tokens=s["window"], sink_tokens=s["sinks"], dtype=s["dtype"], layout=s["layout"],
                           workspace=s["ws"], out=s["out"], softmax_max=s["mx"], softmax_sum=s["sm"])
    return s["out"], s["mx"], s["sm"]


def _own_append(s):
    import scaled_dot_product_16_b200 as sdpa
    c = s["c"]
    sdpa.attn_cache_append(s["k_new"], s["v_new"], s["table"], s["lens"], s["k"], s["v"], cu_seqlens=s["cu"], T=s["T"],
                           B=c["B"], Nkv=c["Nkv"], D=c["D"], num_pages=s["pool"], page_size=c["page"],
                           max_pages=s["cols"], dtype=s["dtype"], layout=s["layout"])
    return s["k"], s["v"]


def _own_fork(s):
    import scaled_dot_product_16_b200 as sdpa
    c = s["c"]
    sdpa.attn_cache_fork(s["table"], s["src"], s["ref"], s["table_out"], s["ref_out"], rows_in=s["rows"],
                         rows_out=s["rows"], max_pages=s["cols"], num_pages=s["pool"], seq_lens=s["lens"],
                         seq_lens_out=s["lens_out"])
    torch.add(s["lens_out"], s["new"], out=s["lens_out"])
    sdpa.attn_cache_reserve(s["table_out"], s["ref_out"], s["lens_out"], s["new"], s["copies"], B=s["rows"],
                            max_pages=s["cols"], num_pages=s["pool"], page_size=c["page"])
    sdpa.attn_cache_copy(s["k"], s["v"], s["copies"], n_copies=s["rows"], num_pages=s["pool"],
                         page_elems=c["page"] * c["Nkv"] * c["D"], dtype=s["dtype"])
    return s["table_out"], s["ref_out"], s["lens_out"], s["copies"], s["k"], s["v"]


def _own_compact(s):
    import scaled_dot_product_16_b200 as sdpa
    c = s["c"]
    sdpa.attn_cache_compact(s["table"], s["ref"], s["table_out"], s["ref_out"], s["page_map"], s["copies"], s["live"],
                            rows=c["rows"], max_pages=s["cols"], num_pages=c["pages"])
    sdpa.attn_cache_copy(s["k"], s["v"], s["copies"], n_copies=c["pages"] // 2, num_pages=c["pages"],
                         page_elems=c["page"] * c["Nkv"] * c["D"], dtype=s["dtype"])
    return s["table_out"], s["ref_out"], s["page_map"], s["copies"], s["live"], s["k"], s["v"]


OWN = {"window": _own_window, "decode": _own_decode, "append": _own_append, "fork": _own_fork, "compact": _own_compact}


# ---- the plain forms ----------------------------------------------------------------------------
def _softmax(scores, mask, v):
    """softmax over the keys that the mask leaves, times V, with the row's maximum and sum. A row without
    a key gives zeros, -inf and 0."""
    scores = scores.masked_fill(~mask, -math.inf)
    mx = scores.amax(-1)
    p = torch.exp(scores - torch.where(mx == -math.inf, 0.0, mx)[..., None])
    sm = p.sum(-1)
    out = p @ v
    return out / torch.where(sm == 0, 1.0, sm)[..., None], mx, sm


def _plain_window(s):
    c = s["c"]
    grp = c["Nq"] // c["Nkv"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    dev = q.device
    if s["layout"] == TND:
        cq, ck = s["cu_q"].long(), s["cu_k"].long()
        q0, k0 = torch.cat([cq.new_zeros(1), cq[:-1]]), torch.cat([ck.new_zeros(1), ck[:-1]])
        lq, lk = cq - q0, ck - k0
        qi, ki = torch.arange(c["S"], device=dev), torch.arange(c["S"] + c["ctx"], device=dev)
        q = q[(q0[:, None] + qi).clamp(max=max(s["Sq"] - 1, 0))].transpose(1, 2)
        k = k[(k0[:, None] + ki).clamp(max=max(s["Skv"] - 1, 0))].transpose(1, 2)
        v = v[(k0[:, None] + ki).clamp(max=max(s["Skv"] - 1, 0))].transpose(1, 2)
    else:
        lq = torch.full((c["B"],), s["Sq"], device=dev)
        lk = torch.full((c["B"],), s["Skv"], device=dev)
        qi, ki = torch.arange(s["Sq"], device=dev), torch.arange(s["Skv"], device=dev)
    pos = (qi[None, :] + (lk - lq)[:, None])[:, :, None]                       # [B, Sq, 1]
    j = ki[None, None, :]
    mask = (j <= pos) & ((j > pos - c["window"]) | (j < c["sinks"])) & (j < lk[:, None, None])
    B, n, D = c["B"], q.shape[2], c["D"]
    scores = (q.reshape(B, c["Nkv"], grp * n, D) @ k.transpose(-1, -2)) * D ** -0.5
    out, mx, sm = _softmax(scores.view(B, c["Nkv"], grp, n, -1), mask[:, None, None], v[:, :, None])
    out, mx, sm = out.reshape(B, c["Nq"], n, D), mx.reshape(B, c["Nq"], n), sm.reshape(B, c["Nq"], n)
    if s["layout"] == TND:
        t = torch.arange(s["Sq"], device=dev)
        b = torch.searchsorted(cq, t, right=True)
        i = t - q0[b]
        out, mx, sm = out[b, :, i], mx[b, :, i], sm[b, :, i]
    return out.to(s["q"].dtype), mx, sm


def _gather(cache, table, tnd):
    """The pages of each row, one behind the other: [rows, heads, positions, D]."""
    x = cache[table.clamp(min=0).long()]                       # [B, pages, page, N, D] or [B, pages, N, page, D]
    x = x.permute(0, 3, 1, 2, 4) if tnd else x.permute(0, 2, 1, 3, 4)
    return x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])


def _plain_decode(s):
    c = s["c"]
    grp = c["Nq"] // c["Nkv"]
    k, v = (_gather(s[x], s["table"], s["layout"] == TND).float() for x in ("k", "v"))
    j = torch.arange(k.shape[2], device=k.device)[None, :]
    ln = s["lens"].long()[:, None]
    mask = (j < ln) & ((j >= ln - s["window"]) | (j < s["sinks"]))
    q = s["q"].float().view(c["B"], c["Nkv"], grp, c["D"])
    scores = (q @ k.transpose(-1, -2)) * c["D"] ** -0.5
    v = torch.where(mask[:, None, :, None], v, 0.0)
    out, mx, sm = _softmax(scores, mask[:, None, None, :], v)
    return out.reshape(s["q"].shape).to(s["q"].dtype), mx.reshape(c["B"], -1), sm.reshape(c["B"], -1)


def _plain_append(s):
    c = s["c"]
    t = torch.arange(s["T"], device=s["k"].device)
    if s["cu"] is None:
        b, left = t, torch.ones_like(t)
    else:
        cu = s["cu"].long()
        b = torch.searchsorted(cu, t, right=True)
        left = cu[b] - t                                       # tokens of the row from this one on
    pos = s["lens"].long()[b] - left
    page, off = s["table"][b, pos // c["page"]].long(), pos % c["page"]
    if s["layout"] == TND:
        s["k"][page, off], s["v"][page, off] = s["k_new"], s["v_new"]
    else:
        s["k"][page, :, off], s["v"][page, :, off] = s["k_new"], s["v_new"]
    return s["k"], s["v"]


def _counts(pages, n, weight):
    """How often each of n pages stands in `pages` (int64, n for none), weighted."""
    return torch.zeros(n + 1, device=pages.device, dtype=torch.int64).scatter_add_(0, pages.reshape(-1), weight.reshape(-1))[:n]


def _copy_pages(cache, copies):
    """cache[dst] = cache[src] for the pairs that are there; a pair of -1 leaves page 0 to itself last of all."""
    src, dst = copies[:, 0].long(), copies[:, 1].long()
    n = cache.shape[0]
    target = torch.arange(n + 1, device=cache.device)
    target = target.scatter(0, torch.where(dst < 0, n, dst), torch.where(src < 0, n, src))[:n]
    at = target != torch.arange(n, device=cache.device)
    return torch.where(at.view(-1, 1, 1, 1), cache[target], cache)


def _plain_fork(s):
    c, n = s["c"], s["pool"]
    src = s["src"].long()
    table = torch.where(src[:, None] >= 0, s["table"][src.clamp(min=0)], -1).long()
    old = s["table"].long()
    one = torch.ones_like(table)
    ref = s["ref"].long() - _counts(torch.where(old < 0, n, old), n, one) + _counts(torch.where(table < 0, n, table), n, one)
    new = s["new"].long()
    lens = torch.where(src >= 0, s["lens"][src.clamp(min=0)], 0).long() + new
    # the pages that the new tokens of each row go to
    col = torch.arange(s["cols"], device=table.device)[None, :]
    start = lens - new
    wanted = (col >= (start // c["page"])[:, None]) & (col <= ((lens - 1) // c["page"])[:, None]) & (new > 0)[:, None]
    page = torch.where(table < 0, n, table)
    refs = torch.cat([ref, ref.new_zeros(1)])[page]
    shared = wanted & (table >= 0) & (refs > 1)
    asked = _counts(page, n, shared.long())                    # rows that ask for a shared page
    flat = torch.arange(table.numel(), device=table.device).view_as(table)
    first = torch.full((n + 1,), table.numel(), device=table.device).scatter_reduce_(
        0, torch.where(shared, page, n).reshape(-1), flat.reshape(-1), "amin")
    # where every holder of a page asks for it, the first of them keeps it
    all_ask = torch.cat([asked == ref, asked.new_zeros(1, dtype=torch.bool)])[page]
    keeps = shared & all_ask & (flat == first[page])
    leaves = shared & ~keeps
    needs = (wanted & (table < 0)) | leaves
    ref = ref - _counts(page, n, leaves.long())
    # the k-th page that is needed is the k-th free one
    free = ref == 0
    rank = free.long().cumsum(0) - 1
    kth = torch.full((n + 1,), -1, device=table.device).scatter_(
        0, torch.where(free, rank, n), torch.arange(n, device=table.device))
    got = kth[torch.where(needs, needs.reshape(-1).long().cumsum(0).view_as(table) - 1, n)]
    out = torch.where(needs, got, table)
    ref = ref + _counts(torch.where(needs, got, n), n, one)
    # the first of these pages holds earlier tokens, if the row's length is not a whole number of pages
    at = (start // c["page"]).clamp(max=s["cols"] - 1)[:, None]
    moved = (leaves.gather(1, at)[:, 0]) & (start % c["page"] != 0)
    copies = torch.stack([torch.where(moved, table.gather(1, at)[:, 0], -1), torch.where(moved, out.gather(1, at)[:, 0], -1)], 1)
    k, v = _copy_pages(s["k"], copies), _copy_pages(s["v"], copies)
    return out.int(), ref.int(), lens.int(), copies.int(), k, v


def _plain_compact(s):
    c = s["c"]
    n = c["pages"]
    ids = torch.arange(n, device=s["ref"].device)
    live = s["ref"] > 0
    count = live.long().sum()
    high = live & (ids >= count)                               # live pages that move down, in order
    hole = ~live & (ids < count)                               # into the free ones below
    dump = n // 2
    kth_hole = torch.full((dump + 1,), -1, device=ids.device).scatter_(
        0, torch.where(hole, hole.long().cumsum(0) - 1, dump).clamp(max=dump), ids)
    rank = high.long().cumsum(0) - 1
    to = kth_hole[torch.where(high, rank, dump).clamp(max=dump)]
    new = torch.where(high, to, torch.where(live, ids, -1))
    src = torch.full((dump + 1,), -1, device=ids.device).scatter_(0, torch.where(high, rank, dump).clamp(max=dump), ids)
    moves = high.long().sum()
    copies = torch.stack([src[:dump], kth_hole[:dump]], 1)
    copies = torch.where(torch.arange(dump, device=ids.device)[:, None] < moves, copies, -1)
    ref = torch.zeros(n + 1, device=ids.device, dtype=torch.int32).scatter_(0, torch.where(live, new, n), s["ref"])[:n]
    ref = torch.where(ids < count, ref, 0)
    table = torch.where(s["table"] >= 0, new[s["table"].clamp(min=0).long()], -1)
    k, v = _copy_pages(s["k"], copies), _copy_pages(s["v"], copies)
    return table.int(), ref.int(), new.int(), copies.int(), count.int().view(1), k, v


PLAIN = {"window": _plain_window, "decode": _plain_decode, "append": _plain_append, "fork": _plain_fork,
         "compact": _plain_compact}


# ------------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ------------------------------------------------------------------------------------------------
def _attend(q, k, v, seen):
    """Rows q [n, D] over keys k, v [m, D]; seen [n, m]. All in float64."""
    sc = torch.where(seen, (q @ k.T) / math.sqrt(q.shape[1]), -math.inf)
    mx = sc.max(1).values
    e = torch.where(seen, (sc - mx[:, None].nan_to_num(neginf=0.0)).exp(), 0.0)
    sm = e.sum(1)
    return torch.where(sm[:, None] > 0, (e @ v) / sm.clamp(min=1e-300)[:, None], 0.0), mx, sm


def exact(case, seed):
    s = prepare(case, seed)
    return EXACT[case["op"]](s)


def _exact_window(s):
    c = s["c"]
    lq, lk = _window_lens(c)
    tnd = s["layout"] == TND
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    mx = torch.zeros(s["mx"].shape, dtype=torch.float64, device="cuda")
    sm = torch.zeros_like(mx)
    a0 = b0 = 0
    for b in range(c["B"]):
        for h in range(c["Nq"]):
            kv = h // (c["Nq"] // c["Nkv"])
            if tnd:
                q, k, v = s["q"][a0:a0 + lq[b], h], s["k"][b0:b0 + lk[b], kv], s["v"][b0:b0 + lk[b], kv]
            else:
                q, k, v = s["q"][b, h], s["k"][b, kv], s["v"][b, kv]
            for r0 in range(0, lq[b], 1024):
                r1 = min(r0 + 1024, lq[b])
                shift = lk[b] - lq[b]
                lo = max(0, r0 + shift - c["window"] + 1)
                keys = torch.cat([torch.arange(min(c["sinks"], lo), device="cuda"), torch.arange(lo, r1 + shift, device="cuda")])
                p = torch.arange(r0 + shift, r1 + shift, device="cuda")[:, None]
                seen = (keys <= p) & ((p - keys < c["window"]) | (keys < c["sinks"]))
                o, m, l = _attend(q[r0:r1].double(), k[keys].double(), v[keys].double(), seen)
                if tnd:
                    out[a0 + r0:a0 + r1, h], mx[a0 + r0:a0 + r1, h], sm[a0 + r0:a0 + r1, h] = o, m, l
                else:
                    out[b, h, r0:r1], mx[b, h, r0:r1], sm[b, h, r0:r1] = o, m, l
        a0, b0 = a0 + lq[b], b0 + lk[b]
    return out, mx, sm


def _exact_decode(s):
    c = s["c"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    mx = torch.full(s["mx"].shape, -math.inf, dtype=torch.float64, device="cuda")
    sm = torch.zeros_like(mx)
    grp = c["Nq"] // c["Nkv"]
    for b, n in enumerate(_step_lens(c)):
        if n == 0:
            continue
        lo = max(0, n - s["window"])
        pos = torch.cat([torch.arange(min(s["sinks"], lo), device="cuda"), torch.arange(lo, n, device="cuda")])
        page, off = s["table"][b, pos // c["page"]].long(), pos % c["page"]
        for h in range(c["Nkv"]):
            k, v = ((x[page, off, h] if s["layout"] == TND else x[page, h, off]).double() for x in (s["k"], s["v"]))
            r = slice(h * grp, (h + 1) * grp)
            out[b, r], mx[b, r], sm[b, r] = _attend(s["q"][b, r].double(), k, v,
                                                    torch.ones((grp, len(pos)), dtype=torch.bool, device="cuda"))
    return out, mx, sm


def _exact_append(s):
    c = s["c"]
    lens, new = _append_lens(c)
    k, v = s["k"].double(), s["v"].double()
    t = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        pos = torch.arange(n - m, n, device="cuda")
        page, off = s["table"][b, pos // c["page"]].long(), pos % c["page"]
        for cache, x in ((k, s["k_new"]), (v, s["v_new"])):
            if s["layout"] == TND:
                cache[page, off] = x[t:t + m].double()
            else:
                cache[page, :, off] = x[t:t + m].double()
        t += m
    return k, v


def _exact_fork(s):
    """Row by row on the host, as the definition reads."""
    c, n = s["c"], s["pool"]
    old, src, new, lens0 = (s[x].tolist() for x in ("table", "src", "new", "lens"))
    table = [list(old[r]) if r >= 0 else [-1] * s["cols"] for r in src]
    ref = [0] * n
    held = lambda t: [p for row in t for p in row if p >= 0]  # noqa: E731
    for p in held(table):
        ref[p] += 1
    lens = [(lens0[r] if r >= 0 else 0) + m for r, m in zip(src, new)]
    slots = [(r, i) for r in range(len(table)) if new[r]
             for i in range((lens[r] - new[r]) // c["page"], (lens[r] - 1) // c["page"] + 1)]
    asked = {}
    for r, i in slots:
        p = table[r][i]
        if p >= 0 and ref[p] > 1:
            asked.setdefault(p, []).append((r, i))
    keeps = {a[0] for p, a in asked.items() if len(a) == ref[p]}
    copies = [[-1, -1] for _ in table]
    todo = [x for x in slots if table[x[0]][x[1]] < 0 or (table[x[0]][x[1]] in asked and x not in keeps)]
    for r, i in todo:
        if table[r][i] >= 0:
            ref[table[r][i]] -= 1
    free = iter([p for p in range(n) if ref[p] == 0])
    for r, i in todo:
        p = next(free)
        if table[r][i] >= 0 and i == (lens[r] - new[r]) // c["page"] and (lens[r] - new[r]) % c["page"]:
            copies[r] = [table[r][i], p]
        table[r][i] = p
        ref[p] = 1
    k, v = s["k"].double(), s["v"].double()
    for a, b in copies:
        if a >= 0:
            k[b], v[b] = k[a], v[a]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return i32(table), i32(ref), i32(lens), i32(copies), k, v


def _exact_compact(s):
    c = s["c"]
    ref = s["ref"].tolist()
    live = [p for p in range(len(ref)) if ref[p] > 0]
    holes = [p for p in range(len(live)) if ref[p] == 0]
    high = [p for p in live if p >= len(live)]
    new = [-1] * len(ref)
    for p in live:
        new[p] = p
    for p, h in zip(high, holes):
        new[p] = h
    out = [0] * len(ref)
    for p in live:
        out[new[p]] = ref[p]
    copies = [list(x) for x in zip(high, holes)]
    copies += [[-1, -1]] * (c["pages"] // 2 - len(copies))
    table = [[new[p] if p >= 0 else -1 for p in row] for row in s["table"].tolist()]
    k, v = s["k"].double(), s["v"].double()
    if high:
        a, b = torch.tensor(high, device="cuda"), torch.tensor(holes, device="cuda")
        k[b], v[b] = k[a], v[a]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return i32(table), i32(out), i32(new), i32(copies).view(-1, 2), i32([len(live)]), k, v


EXACT = {"window": _exact_window, "decode": _exact_decode, "append": _exact_append, "fork": _exact_fork,
         "compact": _exact_compact}

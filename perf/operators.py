"""Timing cases of the paged-cache and sliding-window operators.

Each case is one call (or the calls that belong together) a serving program
makes per step, with inputs like the ones it meets: a page pool in the
scattered order of a long-running server, ragged sequence lengths, grouped
query heads.  `run` computes a case in plain torch operations when `own` is
false and through the library when it is true.

Operators:
    decode   one new token per sequence over a paged KV cache (optionally a
             sliding window with a few first tokens that stay visible)
    window   causal grouped-query prefill with a sliding window and sinks
    append   new K/V rows into the pages of their sequences
    pages    the page allocator: fork + copy, compact + copy, free + reserve
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one chat session, a short context: the launch and the joining of the splits count
        dict(name="decode_one_short", op="decode", dtype="bf16", B=1, Hq=32, Hkv=8, D=128, S=16,
             lo=700, hi=700, window=0, sinks=0, order="head"),
        # the contiguous decode workload of the benchmark, in pages of 16 tokens
        dict(name="decode_batch8_4096", op="decode", dtype="bf16", B=8, Hq=32, Hkv=8, D=128, S=16,
             lo=4096, hi=4096, window=0, sinks=0, order="head"),
        # streaming sessions of very different ages, each bounded by its window
        dict(name="decode_window_ragged", op="decode", dtype="f16", B=48, Hq=16, Hkv=4, D=64, S=32,
             lo=1, hi=9000, window=1024, sinks=4, order="token"),
        # long documents, ragged, a group of 8 query heads
        dict(name="decode_long_ragged", op="decode", dtype="bf16", B=12, Hq=64, Hkv=8, D=128, S=64,
             lo=9000, hi=60000, window=0, sinks=0, order="head"),
        # an exact fp32 prefill of a short prompt
        dict(name="window_f32_short", op="window", dtype="f32", B=2, Hq=8, Hkv=2, D=64, Nq=515,
             Nkv=515, window=128, sinks=4, order="head"),
        # a prompt of the causal prefill's benchmark length
        dict(name="window_4096", op="window", dtype="bf16", B=1, Hq=32, Hkv=8, D=128, Nq=4096,
             Nkv=4096, window=1024, sinks=4, order="head"),
        # a long document through a windowed layer
        dict(name="window_32768", op="window", dtype="bf16", B=1, Hq=32, Hkv=8, D=128, Nq=32768,
             Nkv=32768, window=4096, sinks=4, order="token"),
        # every sequence of a batch gets its next token
        dict(name="append_step", op="append", dtype="bf16", B=64, Hkv=8, D=128, S=16, T=1, lo=1,
             hi=1500),
        # prompts of different lengths into the cache, read from the packed projection
        dict(name="append_prompts", op="append", dtype="bf16", B=6, Hkv=8, D=128, S=16, T=8000,
             lo=0, hi=40),
        # parallel samples of prompts: full pages shared, last pages copied in 2 layers
        dict(name="pages_fork", op="fork", dtype="bf16", B=32, n=16, Hkv=8, D=128, S=16, lo=900,
             hi=4000, layers=2),
        # a pool emptied of two fifths of its pages is closed up
        dict(name="pages_compact", op="compact", dtype="bf16", B=32, Hkv=8, D=128, S=16, P=6000,
             M=256, live=0.6, layers=2),
        # finished sequences give back their pages, new prompts and the next tokens get theirs
        dict(name="pages_admit", op="admit", B=256, S=16, P=140000, M=2048, lo=1, hi=16000,
             new=16, add=9000),
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "window", "window", "append", "fork", "compact", "admit"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 7, 8, 16])
    S = rng.choice([8, 16, 32, 48, 64, 128])
    dtype = rng.choice(["bf16", "f16"])
    order = rng.choice(["head", "token"])
    if op == "decode":
        B = _log(rng, 1, 64)
        hi = _log(rng, 4, min(60000, 300000 // B))
        window, sinks = rng.choice([(0, 0), (0, 0), (_log(rng, 1, hi), rng.choice([0, 4, 33]))])
        return dict(op=op, dtype=dtype, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, S=S, lo=rng.choice([0, 1, hi]),
                    hi=hi, window=window, sinks=sinks, order=order)
    if op == "window":
        dtype = rng.choice(["bf16", "f16", "f32"])
        nkv = _log(rng, 1, 3000 if dtype == "f32" else 20000)
        nq = rng.choice([nkv, nkv, max(1, nkv // 3), 1])
        hq = min(Hkv * G, 32) // Hkv * Hkv
        return dict(op=op, dtype=dtype, B=1 if nkv > 5000 else rng.choice([1, 2, 3]), Hq=hq,
                    Hkv=Hkv, D=rng.choice([32, 64, 128]) if dtype == "f32" else D, Nq=nq, Nkv=nkv,
                    window=_log(rng, 1, min(nkv, 4096)), sinks=rng.choice([0, 1, 4, 130]),
                    order=order)
    if op == "append":
        B = _log(rng, 1, 100)
        return dict(op=op, dtype=rng.choice(["bf16", "f16", "f32"]), B=B, Hkv=Hkv, D=D, S=S,
                    T=rng.choice([1, _log(rng, 1, 20000 // B)]), lo=0, hi=_log(rng, 1, 2000))
    if op == "fork":
        B = _log(rng, 2, 100)
        return dict(op=op, dtype=dtype, B=B, n=rng.randint(1, B - 1), Hkv=Hkv, D=D, S=S,
                    lo=rng.choice([0, 1, 300]), hi=_log(rng, 400, max(500, 60000 // B)),
                    layers=rng.choice([1, 2]))
    if op == "compact":
        B = _log(rng, 1, 32)
        P = _log(rng, 100, 2500)
        return dict(op=op, dtype=dtype, B=B, Hkv=Hkv, D=D, S=rng.choice([8, 16, 32]), P=P,
                    M=P // B + rng.randint(1, 50), live=rng.uniform(0.2, 0.95),
                    layers=rng.choice([1, 2]))
    B = _log(rng, 2, 256)
    hi = _log(rng, 10, 12000)
    add = _log(rng, 1, 9000)
    M = -(-(hi + add) // S) + rng.randint(0, 30)
    return dict(op=op, B=B, S=S, P=B * (-(-hi // S) + 1) + B * (-(-add // S) + 1), M=M, lo=1, hi=hi,
                new=rng.randint(1, B - 1), add=add)


# ---------------------------------------------------------------- inputs

def _generators(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h = torch.Generator()
    h.manual_seed(seed + 1)
    return g, h


def _lengths(h, n, lo, hi):
    """n lengths in [lo, hi], spread over their logarithm."""
    u = torch.rand(n, generator=h, dtype=torch.float64)
    a, b = math.log(lo + 1), math.log(hi + 1)
    return ((a + (b - a) * u).exp() - 1).round().clamp(lo, hi).long()


def _pool(g, P, Hkv, S, D, dtype, order, layers=None):
    """K and V pages as the [P, Hkv, S, D] views of either memory order."""
    lead = () if layers is None else (layers,)
    out = []
    for _ in range(2):
        if order == "token":
            x = torch.empty(lead + (P, S, Hkv, D), dtype=dtype, device="cuda").normal_(generator=g)
            out.append(x.transpose(-3, -2))
        else:
            out.append(torch.empty(lead + (P, Hkv, S, D), dtype=dtype, device="cuda")
                       .normal_(generator=g))
    return out


def _tables(h, lens, S, P, M):
    """A page table of scattered, exclusively owned pages, and the reference counts."""
    perm = torch.randperm(P, generator=h)
    table = torch.full((len(lens), M), -1, dtype=torch.int32)
    refs = torch.zeros(P, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens.tolist()):
        k = -(-n // S)
        table[b, :k] = perm[at:at + k].int()
        refs[perm[at:at + k]] = 1
        at += k
    return table, refs


def prepare(case, seed):
    g, h = _generators(seed)
    op = case["op"]
    st = dict(case=case)
    if op == "window":
        dt = DTYPES[case["dtype"]]
        B, Hq, Hkv, D = case["B"], case["Hq"], case["Hkv"], case["D"]

        def proj(heads, n):
            if case["order"] == "token":     # a [B, N, heads, D] projection, seen heads-major
                x = torch.empty(B, n, heads, D, dtype=dt, device="cuda").normal_(generator=g)
                return x.transpose(1, 2)
            return torch.empty(B, heads, n, D, dtype=dt, device="cuda").normal_(generator=g)

        st.update(q=proj(Hq, case["Nq"]), k=proj(Hkv, case["Nkv"]), v=proj(Hkv, case["Nkv"]))
        return st
    if op in ("fork", "admit"):
        return _prepare_tables(case, g, h, st)
    dt = DTYPES[case["dtype"]]
    Hkv, D, S = case["Hkv"], case["D"], case["S"]
    if op == "compact":
        P, M, B, L = case["P"], case["M"], case["B"], case["layers"]
        n_live = min(int(P * case["live"]), B * M)
        per = torch.full((B,), n_live // B, dtype=torch.long)
        per[:n_live - int(per.sum())] += 1
        table, refs = _tables(h, per * S, S, P, M)
        st["k"], st["v"] = _pool(g, P, Hkv, S, D, dt, "head", L)
        st["table"], st["refs"] = table.cuda(), refs.cuda()
        return st
    lens = _lengths(h, case["B"], case["lo"], case["hi"])
    total, most = lens, case["hi"]
    if op == "append":
        T = case["T"]
        news = torch.full_like(lens, T) if T == 1 else _lengths(h, case["B"], max(1, T // 8), T)
        total, most = lens + news, most + T
    M = -(-most // S) + 2
    P = case["B"] * -(-most // S) + 8
    table, _ = _tables(h, total, S, P, M)
    st.update(table=table.cuda(), seq_len=lens.int().cuda(), lens=lens.tolist())
    if op == "decode":
        st["k"], st["v"] = _pool(g, P, Hkv, S, D, dt, case["order"])
        st["q"] = torch.empty(case["B"], case["Hq"], D, dtype=dt, device="cuda").normal_(generator=g)
        if own:
            import transformer_attention_tcgen05_gb300 as ta
            st["ws"] = torch.zeros(ta.decode_paged_workspace_bytes(case["B"], case["Hq"], Hkv, D),
                                   dtype=torch.uint8, device="cuda")
    else:
        st["k"], st["v"] = _pool(g, P, Hkv, S, D, dt, "head")
        # the K and V columns of a packed [B, T, 2, Hkv, D] projection, seen heads-major
        packed = torch.empty(case["B"], T, 2, Hkv, D, dtype=dt, device="cuda").normal_(generator=g)
        st["kn"], st["vn"] = packed[:, :, 0].transpose(1, 2), packed[:, :, 1].transpose(1, 2)
        st["new_len"], st["news"] = news.int().cuda(), news.tolist()
    return st


def _prepare_tables(case, g, h, st):
    B, S = case["B"], case["S"]
    lens = _lengths(h, B, case["lo"], case["hi"])
    rows = torch.randperm(B, generator=h)
    if case["op"] == "fork":
        n = case["n"]
        dst, rest = rows[:n], rows[n:]
        src = rest[torch.randint(len(rest), (n,), generator=h)]
        M = -(-case["hi"] // S) + 4
        P = B * -(-case["hi"] // S) + n + 16
        table, refs = _tables(h, lens, S, P, M)
        st.update(src=src.int().cuda(), dst=dst.int().cuda())
        st["k"], st["v"] = _pool(g, P, case["Hkv"], S, case["D"], DTYPES[case["dtype"]], "head",
                                 case["layers"])
    else:
        P, M, n = case["P"], case["M"], case["new"]
        add = torch.ones(B, dtype=torch.long)
        add[rows[:n]] = _lengths(h, n, max(1, case["add"] // 8), case["add"])
        # a server admits no more than its pool holds
        room = P - int((-(-lens // S)).sum()) - B
        while int((-(-add // S)).sum()) > room and int(add.max()) > 1:
            add = (add // 2).clamp(min=1)
        table, refs = _tables(h, lens, S, P, M)
        lens = lens.clone()
        lens[rows[:n]] = 0                     # finished: their pages are still held
        st["add"] = add.int().cuda()
    st.update(table=table.cuda(), refs=refs.cuda(), seq_len=lens.int().cuda())
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    return (_run_own if own else _run_plain)(op, st["case"], st)


def _run_own(op, c, st):
    import transformer_attention_tcgen05_gb300 as ta
    if op == "decode":
        return ta.decode_gqa_paged(st["q"], st["k"], st["v"], st["table"], st["seq_len"],
                                   window=c["window"], sinks=c["sinks"], workspace=st["ws"])
    if op == "window":
        return ta.causal_gqa_window_fwd(st["q"], st["k"], st["v"], window=c["window"],
                                        sinks=c["sinks"])
    if op == "append":
        ta.kv_append_paged(st["k"], st["v"], st["kn"], st["vn"], st["table"], st["seq_len"],
                           new_len=st["new_len"], advance=False)
        return [st["k"], st["v"]]
    if op == "fork":
        cs, cd = ta.kv_pages_fork(st["table"], st["seq_len"], st["refs"], st["src"], st["dst"],
                                  page_size=c["S"])
        ta.kv_pages_copy(st["k"], st["v"], cs, cd)
        return [st["table"], st["seq_len"], st["refs"], st["k"], st["v"]]
    if op == "compact":
        table, refs = torch.empty_like(st["table"]), torch.empty_like(st["refs"])
        cs, cd, n = ta.kv_pages_compact(st["table"], st["refs"], new_table=table, new_refs=refs)
        ta.kv_pages_copy(st["k"], st["v"], cs, cd, count=n)
        return [table, refs, st["k"], st["v"]]
    ta.kv_pages_free(st["table"], st["seq_len"], st["refs"], page_size=c["S"])
    ta.kv_pages_reserve(st["table"], st["seq_len"], st["add"], st["refs"], page_size=c["S"])
    return [st["table"], st["refs"]]


def _run_plain(op, c, st):
    return {"decode": _plain_decode, "window": _plain_window, "append": _plain_append,
            "fork": _plain_fork, "compact": _plain_compact, "admit": _plain_admit}[op](c, st)


def _plain_decode(c, st):
    S, G = c["S"], c["Hq"] // c["Hkv"]
    out = torch.zeros_like(st["q"])
    scale = 1.0 / math.sqrt(c["D"])
    for b, n in enumerate(st["lens"]):
        if n == 0:
            continue
        pos = torch.arange(n, device="cuda")
        if c["window"] > 0:
            pos = pos[max(0, n - c["window"]):] if c["sinks"] == 0 else torch.cat(
                [pos[:min(c["sinks"], max(0, n - c["window"]))], pos[max(0, n - c["window"]):]])
        pages, rows = st["table"][b][pos // S].long(), pos % S
        k = st["k"][pages, :, rows].float().transpose(0, 1)          # [Hkv, n, D]
        v = st["v"][pages, :, rows].float().transpose(0, 1)
        q = st["q"][b].float().view(c["Hkv"], G, c["D"])
        s = q @ k.transpose(1, 2) * scale
        p = torch.exp(s - s.amax(-1, keepdim=True))
        o = (p @ v) / p.sum(-1, keepdim=True)
        out[b] = o.view(c["Hq"], c["D"]).to(out.dtype)
    return out


def _blocks(c):
    """Query blocks of a windowed pass: (first, last + 1, key positions, visibility)."""
    off = c["Nkv"] - c["Nq"]
    size = 2048 if c["Nq"] * c["Hq"] * c["B"] > 100000 else 8192
    for i0 in range(0, c["Nq"], size):
        i1 = min(i0 + size, c["Nq"])
        lo = max(0, off + i0 - c["window"] + 1)
        ns = min(c["sinks"], lo)
        key = torch.cat([torch.arange(ns, device="cuda"),
                         torch.arange(lo, off + i1, device="cuda")])
        p = torch.arange(off + i0, off + i1, device="cuda")[:, None]
        see = (key <= p) & ((key > p - c["window"]) | (key < c["sinks"]))
        yield i0, i1, key, see


def _plain_window(c, st):
    G = c["Hq"] // c["Hkv"]
    out = torch.empty(c["B"], c["Hq"], c["Nq"], c["D"], dtype=st["q"].dtype, device="cuda")
    scale = 1.0 / math.sqrt(c["D"])
    for i0, i1, key, see in _blocks(c):
        for h in range(c["Hkv"]):
            q = st["q"][:, h * G:(h + 1) * G, i0:i1].float()
            k = st["k"][:, h, key].float()[:, None]
            v = st["v"][:, h, key].float()[:, None]
            s = (q @ k.transpose(-1, -2) * scale).masked_fill(~see, float("-inf"))
            p = torch.exp(s - s.amax(-1, keepdim=True))
            o = (p @ v) / p.sum(-1, keepdim=True)
            out[:, h * G:(h + 1) * G, i0:i1] = o.to(out.dtype)
    return out


def _plain_append(c, st):
    S = c["S"]
    for b, (n, m) in enumerate(zip(st["lens"], st["news"])):
        pos = torch.arange(n, n + m, device="cuda")
        pages, rows = st["table"][b][pos // S].long(), pos % S
        st["k"][pages, :, rows] = st["kn"][b, :, :m].transpose(0, 1)
        st["v"][pages, :, rows] = st["vn"][b, :, :m].transpose(0, 1)
    return [st["k"], st["v"]]


def _take_free(refs, n):
    """The free pages, lowest first (at least n entries), without a count on the host."""
    order = torch.argsort((refs != 0).to(torch.int8), stable=True)
    return order[:n]


def _plain_fork(c, st):
    S, table, refs, lens = c["S"], st["table"], st["refs"], st["seq_len"]
    src, dst = st["src"].long(), st["dst"].long()
    P = refs.numel()
    spare = torch.cat([refs, refs.new_zeros(1)])

    def count(rows, by):
        rows = torch.where(rows < 0, P, rows).reshape(-1).long()
        spare.index_add_(0, rows, torch.full_like(rows, by, dtype=torch.int32))

    count(table[dst], -1)
    n = lens[src]
    M = table.shape[1]
    idx = torch.arange(M, device="cuda")
    full = idx[None] < (n // S)[:, None]
    new = torch.where(full, table[src], -1)
    count(new, 1)
    refs.copy_(spare[:P])
    part = (n % S) != 0
    rank = torch.cumsum(part.int(), 0) - 1
    page = _take_free(refs, len(src))[rank.clamp(min=0).long()]
    tail = (n // S).clamp(max=M - 1).long()
    old = table[src].gather(1, tail[:, None])[:, 0].long()
    at = torch.nonzero(part)[:, 0]
    new[at, tail[at]] = page[at].int()
    refs[page[at]] = 1
    table[dst] = new
    lens[dst] = n
    st["k"][:, page[at]] = st["k"][:, old[at]]
    st["v"][:, page[at]] = st["v"][:, old[at]]
    return [table, lens, refs, st["k"], st["v"]]


def _plain_compact(c, st):
    refs, table = st["refs"], st["table"]
    live = refs > 0
    n = live.sum()
    idx = torch.arange(refs.numel(), device="cuda")
    src = torch.nonzero(live & (idx >= n))[:, 0]
    dst = torch.nonzero(~live & (idx < n))[:, 0]
    to = idx.clone()
    to[src] = dst
    new_table = torch.where(table < 0, table, to[table.clamp(min=0).long()].int())
    new_refs = refs.clone()
    new_refs[dst] = refs[src]
    new_refs[src] = 0
    st["k"][:, dst] = st["k"][:, src]
    st["v"][:, dst] = st["v"][:, src]
    return [new_table, new_refs, st["k"], st["v"]]


def _plain_admit(c, st):
    S, table, refs, lens = c["S"], st["table"], st["refs"], st["seq_len"]
    P, M = refs.numel(), table.shape[1]
    idx = torch.arange(M, device="cuda")[None]
    gone = (table >= 0) & (idx * S >= lens[:, None])
    spare = torch.cat([refs, refs.new_zeros(1)])
    rows = torch.where(gone, table, P).reshape(-1).long()
    spare.index_add_(0, rows, torch.full_like(rows, -1, dtype=torch.int32))
    refs.copy_(spare[:P])
    table.masked_fill_(gone, -1)
    need = (table < 0) & (idx >= (lens // S)[:, None]) & (idx * S < (lens + st["add"])[:, None])
    rank = torch.cumsum(need.reshape(-1).int(), 0).view_as(need) - 1
    free = _take_free(refs, P)
    page = free[rank.clamp(min=0, max=P - 1).long()].int()
    table.copy_(torch.where(need, page, table))
    spare = torch.cat([refs, refs.new_zeros(1)])
    rows = torch.where(need, page, P).reshape(-1).long()
    spare.index_add_(0, rows, torch.ones_like(rows, dtype=torch.int32))
    refs.copy_(spare[:P])
    return [table, refs]


# ---------------------------------------------------------------- work

def _visible(n, window, sinks):
    if window <= 0 or n <= window:
        return n
    return window + min(sinks, n - window)


def work(case):
    c = case
    if c["op"] == "decode":
        # the mean length of a sequence drawn over the logarithm of [lo, hi]
        steps = 64
        lens = [int(round((c["lo"] + 1) * ((c["hi"] + 1) / (c["lo"] + 1)) ** ((i + .5) / steps))) - 1
                for i in range(steps)]
        seen = sum(_visible(n, c["window"], c["sinks"]) for n in lens) / steps * c["B"]
        es = ESIZE[c["dtype"]]
        return dict(bytes=2 * seen * c["Hkv"] * c["D"] * es + 2 * c["B"] * c["Hq"] * c["D"] * es
                    + 4 * seen / c["S"],
                    flops=4 * c["Hq"] * c["D"] * seen)
    if c["op"] == "window":
        off = c["Nkv"] - c["Nq"]
        pairs = sum(_visible(off + i + 1, c["window"], c["sinks"]) for i in range(c["Nq"]))
        es = ESIZE[c["dtype"]]
        keys = c["Nkv"] if off - c["window"] < 0 else c["Nq"] + c["window"] - 1 + c["sinks"]
        keys = min(keys, c["Nkv"])
        return dict(bytes=2 * es * c["B"] * c["D"] * (c["Hq"] * c["Nq"] + c["Hkv"] * keys),
                    flops=4 * c["B"] * c["Hq"] * c["D"] * pairs)
    if c["op"] == "append":
        mean = 1 if c["T"] == 1 else _log_mean(max(1, c["T"] // 8), c["T"])
        return dict(bytes=4 * c["B"] * mean * c["Hkv"] * c["D"] * ESIZE[c["dtype"]], flops=0)
    if c["op"] == "fork":
        # the counts, the rows that are read and written, and the last pages
        mean = _log_mean(c["lo"], c["hi"])
        page = c["Hkv"] * c["S"] * c["D"] * ESIZE[c["dtype"]]
        part = c["n"] * (c["S"] - 1) / c["S"] * (mean > 0)
        return dict(bytes=12 * c["n"] * mean / c["S"] + 4 * c["B"] * mean / c["S"]
                    + 4 * part * page * c["layers"], flops=0)
    if c["op"] == "compact":
        page = c["Hkv"] * c["S"] * c["D"] * ESIZE[c["dtype"]]
        moves = c["P"] * c["live"] * (1 - c["live"])
        return dict(bytes=8 * c["P"] + 8 * c["B"] * c["M"] + 4 * moves * page * c["layers"], flops=0)
    mean = _log_mean(max(1, c["add"] // 8), c["add"]) * c["new"] / c["S"]
    return dict(bytes=4 * c["P"] + 4 * c["B"] * c["M"] + 8 * mean, flops=0)


def _log_mean(lo, hi):
    if hi <= lo:
        return lo
    return (hi - lo) / math.log((hi + 1) / (lo + 1)) - 1 if hi > 0 else 0


# ---------------------------------------------------------------- exact values

def exact(case, seed):
    """The attention outputs in 64 bits; pages and tables are copies and whole numbers."""
    c = case
    if c["op"] not in ("decode", "window"):
        return None
    st = prepare(case, seed)
    G = c["Hq"] // c["Hkv"]
    if c["op"] == "decode":
        out = torch.zeros(c["B"], c["Hq"], c["D"], dtype=torch.float64, device="cuda")
        for b, n in enumerate(st["lens"]):
            if n == 0:
                continue
            m = -(-n // c["S"])
            pages = st["table"][b, :m].long()
            see = torch.ones(n, dtype=torch.bool, device="cuda")
            if c["window"] > 0:
                see[:max(0, n - c["window"])] = False
                see[:c["sinks"]] = True
            for h in range(c["Hkv"]):
                k = st["k"][pages, h].reshape(-1, c["D"])[:n][see].double()
                v = st["v"][pages, h].reshape(-1, c["D"])[:n][see].double()
                q = st["q"][b, h * G:(h + 1) * G].double()
                w = torch.softmax(torch.einsum("gd,nd->gn", q, k) / c["D"] ** 0.5, -1)
                out[b, h * G:(h + 1) * G] = torch.einsum("gn,nd->gd", w, v)
        return out
    out = torch.empty(c["B"], c["Hq"], c["Nq"], c["D"], dtype=torch.float64, device="cuda")
    off, step = c["Nkv"] - c["Nq"], 1024
    for b in range(c["B"]):
        for hq in range(c["Hq"]):
            k, v = st["k"][b, hq // G], st["v"][b, hq // G]
            for i0 in range(0, c["Nq"], step):
                q = st["q"][b, hq, i0:i0 + step].double()
                first, last = off + i0, off + i0 + len(q) - 1
                a = max(0, first - c["window"] + 1)
                at = list(range(min(a, c["sinks"]))) if c["sinks"] else []
                kk = torch.cat([k[:len(at)], k[a:last + 1]]).double()
                vv = torch.cat([v[:len(at)], v[a:last + 1]]).double()
                key = torch.cat([torch.arange(len(at)), torch.arange(a, last + 1)]).cuda()
                at_q = torch.arange(first, last + 1).cuda()
                gap = at_q[:, None] - key[None, :]
                hide = (gap < 0) | ((gap >= c["window"]) & (key[None, :] >= c["sinks"]))
                s = torch.einsum("id,jd->ij", q, kk) / c["D"] ** 0.5
                w = torch.softmax(s.masked_fill(hide, -math.inf), -1)
                out[b, hq, i0:i0 + len(q)] = torch.einsum("ij,jd->id", w, vv)
    return out

"""Timing cases of the packed-prompt and 4-bit-cache operators.

A server takes the tokens of many sequences as one packed projection.  Each case
is one call (or the calls that belong together) of such a step, with scattered
pages, ragged lengths and grouped query heads.  `run` computes a case in plain
torch operations when `own` is false and through the library when it is true.

Operators:
    rope     rotary positions of packed or heads-major rows, either pair layout,
             part of the head, frequencies scaled for long contexts; also the
             transposed rotation (the gradient)
    append   new K/V rows into the pages of a 16-bit cache, K rotated on the way,
             the queries of the same tokens rotated by the same call
    store4   the same into a cache held in 4 bits, and rows read back from it, as
             the attention of a continued prompt takes them
    decode4  one new token per sequence over the 4-bit cache
    varlen   causal grouped-query attention over packed sequences of different
             lengths, optionally behind cached keys, with a window and sinks

The 4-bit cache keeps a token's K and V of one KV head in a row of D + D / 8
bytes: groups of 32 channels, x = s (n - 8) with n of 4 bits and s of 16.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f16": 2, "f32": 4}
THETA = 500000.0


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the queries of a packed prompt far inside a long context, frequencies scaled by parts
        dict(name="rope_prompt", op="rope", dtype="bf16", B=1, H=32, N=8192, D=128, rot=128, pairs="half",
             scaling="by_parts", far=900000, order="token", inverse=False),
        # the gradient of half-rotated fp32 heads of a small batch
        dict(name="rope_grad_f32", op="rope", dtype="f32", B=2, H=8, N=515, D=64, rot=32, pairs="interleaved",
             scaling="none", far=4000, order="head", inverse=True),
        # every sequence of a batch gets its next token: one call for its query, key and value
        dict(name="append_step", op="append", dtype="bf16", B=64, Hq=32, Hkv=8, D=128, S=16, T=1, lo=1,
             hi=1500, rot=128, pairs="half"),
        # prompts of different lengths, read from the packed projection
        dict(name="append_prompts", op="append", dtype="bf16", B=6, Hq=32, Hkv=8, D=128, S=16, T=8000, lo=1,
             hi=40, rot=128, pairs="half"),
        # the next tokens of a batch into the 4-bit cache, and what it holds of them
        dict(name="store4_step", op="store4", dtype="bf16", B=64, Hq=32, Hkv=8, D=128, S=16, T=1, lo=1,
             hi=1500, rot=128, pairs="half", past=False),
        # chunks of prompts behind cached ones: stored, and the whole sequences read for their attention
        dict(name="store4_chunks", op="store4", dtype="bf16", B=6, Hq=32, Hkv=8, D=128, S=16, T=2000, lo=500,
             hi=9000, rot=128, pairs="half", past=True),
        # one chat session, a short context: the launch and the joining of the splits count
        dict(name="decode4_one_short", op="decode4", dtype="bf16", B=1, Hq=32, Hkv=8, D=128, S=16, lo=700,
             hi=700, window=0, sinks=0),
        # the decode workload of the benchmark over 4-bit pages of 16 tokens
        dict(name="decode4_batch8_4096", op="decode4", dtype="bf16", B=8, Hq=32, Hkv=8, D=128, S=16, lo=4096,
             hi=4096, window=0, sinks=0),
        # long documents, ragged, a group of 8 query heads
        dict(name="decode4_long_ragged", op="decode4", dtype="bf16", B=12, Hq=64, Hkv=8, D=128, S=64, lo=9000,
             hi=60000, window=0, sinks=0),
        # prompts of very different lengths in one pass
        dict(name="varlen_mixed", op="varlen", dtype="bf16", B=16, Hq=32, Hkv=8, D=128, lo=1, hi=6000, past=0,
             window=0, sinks=0),
        # chunks of prompts behind their cached keys in a windowed layer, a group of 3 query heads
        dict(name="varlen_chunks_window", op="varlen", dtype="f16", B=7, Hq=24, Hkv=8, D=64, lo=100, hi=2000,
             past=5000, window=1024, sinks=4),
        # an exact fp32 pass over short prompts
        dict(name="varlen_f32_short", op="varlen", dtype="f32", B=5, Hq=8, Hkv=2, D=64, lo=3, hi=515, past=0,
             window=0, sinks=0),
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "store4", "decode4", "decode4", "varlen", "varlen"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 7, 8, 16])
    S = rng.choice([8, 16, 32, 48, 64, 128])
    dtype = rng.choice(["bf16", "f16"])
    pairs = rng.choice(["half", "interleaved"])
    if op == "rope":
        D = rng.choice([32, 64, 128])
        dtype = rng.choice(["bf16", "f16", "f32"])
        B, H = rng.choice([1, 1, 2, 3]), rng.choice([1, 2, 5, 8, 16, 32])
        return dict(op=op, dtype=dtype, B=B, H=H, N=_log(rng, 1, 8000 // B), D=D,
                    rot=max(16, rng.choice([D, D, D // 2, D // 4])), pairs=pairs,
                    scaling=rng.choice(["none", "linear", "ntk", "by_parts"]), far=_log(rng, 1, 1000000),
                    order=rng.choice(["token", "head"]), inverse=rng.choice([False, True]))
    if op in ("append", "store4"):
        if op == "append":
            D, dtype = rng.choice([32, 64, 128]), rng.choice(["bf16", "f16", "f32"])
        B = _log(rng, 1, 100)
        case = dict(op=op, dtype=dtype, B=B, Hq=Hkv * min(G, 8), Hkv=Hkv, D=D, S=S,
                    T=rng.choice([1, _log(rng, 1, 12000 // B)]), lo=rng.choice([1, 7]), hi=_log(rng, 8, 2000),
                    rot=rng.choice([D, D, D // 2]), pairs=pairs)
        if op == "store4":
            case["past"] = rng.choice([False, True])
        return case
    if op == "decode4":
        B = _log(rng, 1, 64)
        hi = _log(rng, 4, min(60000, 300000 // B))
        window, sinks = rng.choice([(0, 0), (0, 0), (_log(rng, 1, hi), rng.choice([0, 4, 33]))])
        return dict(op=op, dtype=dtype, B=B, Hq=Hkv * G, Hkv=Hkv, D=D, S=S, lo=rng.choice([1, 1, hi]), hi=hi,
                    window=window, sinks=sinks)
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    B = _log(rng, 1, 40)
    top = min(800, 3000 // B) if dtype == "f32" else int(math.sqrt(1e7 / B))
    hi = _log(rng, 2, top)
    window, sinks = rng.choice([(0, 0), (_log(rng, 1, 4000), rng.choice([0, 1, 4, 130]))])
    return dict(op=op, dtype=dtype, B=B, Hq=min(Hkv * G, 32) // Hkv * Hkv, Hkv=Hkv,
                D=rng.choice([32, 64, 128]) if dtype == "f32" else D, lo=rng.choice([1, hi]), hi=hi,
                past=rng.choice([0, 0, _log(rng, 1, top)]), window=window, sinks=sinks)


# ---------------------------------------------------------------- inputs

def _spread(lo, hi, n):
    """n lengths spread evenly over the logarithm of [lo, hi]."""
    return [min(hi, max(lo, int(round(lo * (hi / lo) ** ((i + 0.5) / n))))) for i in range(n)]


def _chunk(case):
    """The tokens that each sequence of an append brings."""
    return [1] * case["B"] if case["T"] == 1 else _spread(max(1, case["T"] // 8), case["T"], case["B"])


def _past(case):
    """The cached tokens in front of each sequence of a packed pass."""
    return _spread(max(1, case["past"] // 8), case["past"], case["B"]) if case["past"] else [0] * case["B"]


def _shuffled(values, h):
    return [values[i] for i in torch.randperm(len(values), generator=h).tolist()]


def _starts(lens):
    """The first row of each packed sequence, and the rows of all."""
    return torch.tensor([0] + lens).cumsum(0).int().cuda()


def _rates(case):
    """Radians per position of each rotated pair."""
    r = case["rot"]
    at = torch.arange(0, r, 2, dtype=torch.float64) / r
    f = THETA ** -at
    scaling = case.get("scaling", "none")
    if scaling == "linear":
        f = f / 4
    elif scaling == "ntk":
        f = (THETA * 4 ** (r / (r - 2))) ** -at
    elif scaling == "by_parts":
        share = ((8192 * f / (2 * math.pi) - 1) / (32 - 1)).clamp(0, 1)
        f = (1 - share) * f / 4 + share * f
    return f.cuda()


def _size(case):
    """The factor of the rotated rows (a by-parts scaling makes scores a little sharper)."""
    return 0.1 * math.log(4) + 1 if case.get("scaling") == "by_parts" else 1.0


def _rows(g, n, heads, D, dt):
    return torch.empty(n, heads, D, dtype=dt, device="cuda").normal_(generator=g)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    h = torch.Generator()
    h.manual_seed(seed + 1)
    op, dt, D = case["op"], DTYPES[case["dtype"]], case["D"]
    st = dict(case=case)
    if op == "rope":
        B, H, N = case["B"], case["H"], case["N"]
        if case["order"] == "token":         # a packed [B, N, H, D] projection, seen heads-major
            st["x"] = _rows(g, B * N, H, D, dt).view(B, N, H, D).transpose(1, 2)
        else:
            st["x"] = _rows(g, B * H, N, D, dt).view(B, H, N, D)
        first = torch.randint(0, case["far"], (B, 1), generator=h)
        st["pos"] = (first + torch.arange(N)[None]).int().cuda()
        _keep_rates(case, st)
        return st
    if op == "varlen":
        lens = _shuffled(_spread(case["lo"], case["hi"], case["B"]), h)
        total = [n + m for n, m in zip(lens, _shuffled(_past(case), h))]
        st.update(lens=lens, total=total, cu_q=_starts(lens), cu_k=_starts(total))
        Nq, Nk, Hq, Hkv = sum(lens), sum(total), case["Hq"], case["Hkv"]
        # the queries come rotated from their projection, keys and values as one packed [N, 2, Hkv, D]
        st["q"] = _rows(g, Nq, Hq, D, dt)
        kv = _rows(g, Nk, 2 * Hkv, D, dt).view(Nk, 2, Hkv, D)
        st["k"], st["v"] = kv[:, 0], kv[:, 1]
        return st
    # the paged operators: scattered pages, exclusively owned
    B, Hkv, S = case["B"], case["Hkv"], case["S"]
    lens = _shuffled(_spread(case["lo"], case["hi"], B), h)
    news = [0] * B if op == "decode4" else _shuffled(_chunk(case), h)
    total = [n + m for n, m in zip(lens, news)]
    pages = [-(-n // S) for n in total]
    P, M = sum(pages) + 8, max(pages) + 2
    perm = torch.randperm(P, generator=h).int()
    table = torch.full((B, M), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    st.update(table=table.cuda(), seq_len=torch.tensor(lens).int().cuda(), lens=lens, news=news)
    if op == "append":
        st["k"], st["v"] = (torch.empty(P, Hkv, S, D, dtype=dt, device="cuda").normal_(generator=g) for _ in "kv")
    else:
        st["pages"] = _pool4(g, P, Hkv, S, D, dt)
    if op == "decode4":
        st["q"] = _rows(g, B, case["Hq"], D, dt)
        if own:
            import transformer_attention_tcgen05_gb300 as ta
            st["ws"] = torch.zeros(ta.decode_paged_q4_workspace_bytes(B, case["Hq"], Hkv, D), dtype=torch.uint8,
                                   device="cuda")
        return st
    # queries, keys and values are columns of one packed projection
    N, Hq = sum(news), case["Hq"]
    qkv = _rows(g, N, Hq + 2 * Hkv, D, dt)
    st["q"], st["kn"], st["vn"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    st["cu"] = None if case["T"] == 1 else _starts(news)
    # sequence and place in it of every new row
    st["seq"] = torch.repeat_interleave(torch.arange(B), torch.tensor(news)).cuda()
    st["pos"] = torch.cat([torch.arange(n, n + m) for n, m in zip(lens, news)]).cuda()
    if op == "store4":
        first, count = ([0] * B, total) if case["past"] else (lens, news)
        st["first"], st["cu_read"] = torch.tensor(first).int().cuda(), _starts(count)
        st["read_seq"] = torch.repeat_interleave(torch.arange(B), torch.tensor(count)).cuda()
        st["read_pos"] = torch.cat([torch.arange(n, n + m) for n, m in zip(first, count)]).cuda()
        st["k_out"], st["v_out"] = (torch.empty(sum(count), Hkv, D, dtype=dt, device="cuda") for _ in "kv")
    _keep_rates(case, st)
    return st


def _keep_rates(case, st):
    st["rates"] = _rates(case)
    if own:
        import transformer_attention_tcgen05_gb300 as ta
        scaling = case.get("scaling", "none")
        st["freq"] = ta.rope_frequencies(case["rot"], THETA, scaling=None if scaling == "none" else scaling,
                                         factor=4.0, original_len=8192, alpha=1.0, beta=32.0, device="cuda")


def _pool4(g, P, Hkv, S, D, dt):
    """Pages of 4-bit rows as a server's past left them: any codes, scales of normal values."""
    pages = torch.randint(0, 256, (P, Hkv, S, D + D // 8), generator=g, dtype=torch.uint8, device="cuda")
    scale = torch.empty(P, Hkv, S, D // 16, device="cuda").normal_(generator=g) * 0.05
    scale = (0.25 + scale.clamp(-0.2, 0.2)) * (1 - 2 * torch.randint(0, 2, scale.shape, generator=g, device="cuda"))
    pages[..., D:] = scale.to(dt).contiguous().view(torch.uint8).view(P, Hkv, S, D // 8)
    return pages


# ---------------------------------------------------------------- one pass

def run(st):
    return (_run_own if own else _run_plain)(st["case"], st)


def _run_own(c, st):
    import transformer_attention_tcgen05_gb300 as ta
    op = c["op"]
    pairs = c.get("pairs") == "interleaved"
    if op == "rope":
        return ta.rope_fwd(st["x"], st["freq"], st["pos"], interleaved=pairs, inverse=c["inverse"], mscale=_size(c))
    if op == "append":
        q = ta.kv_append_paged_rope(st["k"], st["v"], st["kn"], st["vn"], st["table"], st["seq_len"], st["freq"],
                                    cu_new=st["cu"], q=st["q"], interleaved=pairs, advance=False)
        return [q, st["k"], st["v"]]
    if op == "store4":
        q = ta.kv_append_paged_q4(st["pages"], st["kn"], st["vn"], st["table"], st["seq_len"], st["freq"],
                                  cu_new=st["cu"], q=st["q"], interleaved=pairs, advance=False)
        k, v = ta.kv_gather_paged_q4(st["pages"], st["table"], st["cu_read"], st["k_out"], st["v_out"],
                                     start=st["first"])
        return [q, k, v]
    if op == "decode4":
        return ta.decode_gqa_paged_q4(st["q"], st["pages"], st["table"], st["seq_len"], window=c["window"],
                                      sinks=c["sinks"], workspace=st["ws"])
    return ta.causal_gqa_varlen_fwd(st["q"], st["k"], st["v"], st["cu_q"], st["cu_k"], window=c["window"],
                                    sinks=c["sinks"])


def _run_plain(c, st):
    return {"rope": _plain_rope, "append": _plain_append, "store4": _plain_store4, "decode4": _plain_decode4,
            "varlen": _plain_varlen}[c["op"]](c, st)


def _turn(x, pos, rates, c, back=False):
    """x [..., D] in fp32, rotated by its positions [...] (64-bit angles)."""
    angle = pos.double()[..., None] * rates
    cos, sin = (torch.cos(angle) * _size(c)).float(), (torch.sin(angle) * _size(c)).float()
    sin = -sin if back else sin
    r = c["rot"]
    y = x.float()
    if c["pairs"] == "half":
        a, b = y[..., :r // 2], y[..., r // 2:r]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., r:]], -1)
    a, b = y[..., 0:r:2], y[..., 1:r:2]
    turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, y[..., r:]], -1)


def _plain_rope(c, st):
    x = st["x"]
    return _turn(x, st["pos"][:, None].expand(x.shape[:3]), st["rates"], c, c["inverse"]).to(x.dtype)


def _plain_append(c, st):
    S, pos = c["S"], st["pos"]
    pages, rows = st["table"][st["seq"], pos // S].long(), pos % S
    k = _turn(st["kn"], pos[:, None].expand(st["kn"].shape[:2]), st["rates"], c)
    q = _turn(st["q"], pos[:, None].expand(st["q"].shape[:2]), st["rates"], c)
    st["k"][pages, :, rows] = k.to(st["k"].dtype)
    st["v"][pages, :, rows] = st["vn"]
    return [q.to(st["q"].dtype), st["k"], st["v"]]


def _codes(x, dt):
    """Codes [..., D] and scales [..., D / 32] (as fp32) of fp32 rows."""
    y = x.unflatten(-1, (-1, 32))
    top, low = y.amax(-1), y.amin(-1)
    s = (torch.where(top >= -low, top, low) / -8).to(dt).float()
    inv = torch.where(s == 0, s, 1 / s)
    n = (torch.round(y * inv[..., None]) + 8).clamp(0, 15)
    return n.flatten(-2).int(), s


def _halves(n):
    """16-bit words [..., 2 bytes] of four codes [..., 4]: code i at bit 4 i, rotated right by two bits."""
    w = n[..., 0] | n[..., 1] << 4 | n[..., 2] << 8 | n[..., 3] << 12
    w = (w >> 2 | w << 14) & 0xffff
    return torch.stack([w & 255, w >> 8], -1).to(torch.uint8)


def _pack(k, v, dt):
    """Rows of D + D / 8 bytes."""
    D = k.shape[-1]
    (kn, ks), (vn, vs) = _codes(k, dt), _codes(v, dt)
    lead = k.shape[:-1]
    # K: eight channels (two words) of lane p and group g at p D / 8 + 4 g
    kb = _halves(kn.reshape(*lead, D // 32, 4, 2, 4)).transpose(-4, -3).reshape(*lead, D // 2)
    # V: four channels of lane q and group g at q D / 16 + 2 g
    vb = _halves(vn.reshape(*lead, D // 32, 8, 4)).transpose(-3, -2).reshape(*lead, D // 2)
    sb = torch.cat([ks, vs], -1).to(dt).view(torch.uint8)
    return torch.cat([kb, vb, sb], -1)


def _values(rows, dt):
    """K and V rows in fp32 of rows of D + D / 8 bytes."""
    D = rows.shape[-1] // 9 * 8
    lead = rows.shape[:-1]
    w = rows[..., :D].reshape(*lead, D // 2, 2).int()
    w = w[..., 0] | w[..., 1] << 8
    w = (w << 2 | w >> 14) & 0xffff
    n = torch.stack([w & 15, w >> 4 & 15, w >> 8 & 15, w >> 12], -1) - 8      # [..., D / 2 words, 4]
    k = n[..., :D // 4, :].reshape(*lead, 4, D // 32, 8).transpose(-3, -2).reshape(*lead, D // 32, 32)
    v = n[..., D // 4:, :].reshape(*lead, 8, D // 32, 4).transpose(-3, -2).reshape(*lead, D // 32, 32)
    s = rows[..., D:].contiguous().view(dt).float()
    return ((k * s[..., :D // 32, None]).flatten(-2), (v * s[..., D // 32:, None]).flatten(-2))


def _plain_store4(c, st):
    S, pos, dt = c["S"], st["pos"], DTYPES[c["dtype"]]
    pages, rows = st["table"][st["seq"], pos // S].long(), pos % S
    k = _turn(st["kn"], pos[:, None].expand(st["kn"].shape[:2]), st["rates"], c)
    q = _turn(st["q"], pos[:, None].expand(st["q"].shape[:2]), st["rates"], c)
    st["pages"][pages, :, rows] = _pack(k, st["vn"].float(), dt)
    pos = st["read_pos"]
    k, v = _values(st["pages"][st["table"][st["read_seq"], pos // S].long(), :, pos % S], dt)
    st["k_out"].copy_(k)
    st["v_out"].copy_(v)
    return [q.to(st["q"].dtype), st["k_out"], st["v_out"]]


def _plain_decode4(c, st):
    B, G, Hkv, S = c["B"], c["Hq"] // c["Hkv"], c["Hkv"], c["S"]
    out = torch.empty_like(st["q"])
    for b, n in enumerate(st["lens"]):
        lo = max(0, n - c["window"]) if c["window"] > 0 else 0
        pos = torch.arange(lo, n, device="cuda")
        pos = torch.cat([torch.arange(min(c["sinks"], lo), device="cuda"), pos])
        rows = st["pages"][st["table"][b, pos // S].long(), :, pos % S]
        k, v = _values(rows, st["q"].dtype)                          # [n, Hkv, D]
        q = st["q"][b].float().view(Hkv, G, c["D"])
        s = q @ k.permute(1, 2, 0) / math.sqrt(c["D"])
        p = torch.exp(s - s.amax(-1, keepdim=True))
        o = (p @ v.transpose(0, 1)) / p.sum(-1, keepdim=True)
        out[b] = o.view(c["Hq"], c["D"]).to(out.dtype)
    return out


def _seen(first, n, last, window, sinks):
    """Whether queries at positions [first, first + n) see keys [0, last)."""
    p, j = torch.arange(first, first + n, device="cuda")[:, None], torch.arange(last, device="cuda")[None]
    see = j <= p
    return see & ((j > p - window) | (j < sinks)) if window > 0 else see


def _plain_varlen(c, st):
    out = torch.empty_like(st["q"])
    G, scale = c["Hq"] // c["Hkv"], 1 / math.sqrt(c["D"])
    q0 = k0 = 0
    for n, t in zip(st["lens"], st["total"]):
        k = st["k"][k0:k0 + t].float().permute(1, 2, 0)[:, None]     # [Hkv, 1, D, t]
        v = st["v"][k0:k0 + t].float().transpose(0, 1)[:, None]      # [Hkv, 1, t, D]
        for i in range(0, n, 2048):
            m = min(2048, n - i)
            last = t - n + i + m
            q = st["q"][q0 + i:q0 + i + m].float().transpose(0, 1).unflatten(0, (-1, G))
            s = q @ k[..., :last] * scale
            s = s.masked_fill(~_seen(last - m, m, last, c["window"], c["sinks"]), float("-inf"))
            p = torch.exp(s - s.amax(-1, keepdim=True))
            o = (p @ v[..., :last, :]) / p.sum(-1, keepdim=True)
            out[q0 + i:q0 + i + m] = o.flatten(0, 1).transpose(0, 1).to(out.dtype)
        q0, k0 = q0 + n, k0 + t
    return out


# ---------------------------------------------------------------- work

def _pairs(first, n, window, sinks):
    """Keys that queries at positions [first, first + n) see, all together."""
    if window <= 0:
        return n * first + n * (n + 1) // 2
    return sum(p + 1 if p < window else window + min(sinks, p + 1 - window) for p in range(first, first + n))


def work(case):
    c = case
    es, D = ESIZE[c["dtype"]], c["D"]
    if c["op"] == "rope":
        return dict(bytes=2 * c["B"] * c["H"] * c["N"] * D * es + 4 * c["B"] * c["N"],
                    flops=3 * c["B"] * c["H"] * c["N"] * c["rot"])
    if c["op"] == "varlen":
        lens, past = _spread(c["lo"], c["hi"], c["B"]), _past(c)
        # the mean over the ways lengths and pasts can meet
        many = [(n, past[(i + k) % c["B"]]) for i, n in enumerate(lens) for k in range(min(c["B"], 4))]
        share = c["B"] / len(many)
        pairs = share * sum(_pairs(m, n, c["window"], c["sinks"]) for n, m in many)
        keys = share * sum(n + (m if c["window"] <= 0 else min(m, c["window"] - 1 + c["sinks"])) for n, m in many)
        return dict(bytes=2 * es * D * (c["Hq"] * sum(lens) + c["Hkv"] * keys), flops=4 * c["Hq"] * D * pairs)
    if c["op"] == "decode4":
        seen = sum(_pairs(n - 1, 1, c["window"], c["sinks"]) for n in _spread(c["lo"], c["hi"], c["B"]))
        return dict(bytes=seen * c["Hkv"] * (D + D // 8) + 2 * c["B"] * c["Hq"] * D * es + 4 * seen / c["S"],
                    flops=4 * c["Hq"] * D * seen)
    new = sum(_chunk(c))
    if c["op"] == "append":
        return dict(bytes=2 * new * (c["Hq"] + 2 * c["Hkv"]) * D * es,
                    flops=3 * new * (c["Hq"] + c["Hkv"]) * c["rot"])
    read = new + (sum(_spread(c["lo"], c["hi"], c["B"])) if c["past"] else 0)
    row = c["Hkv"] * (D + D // 8)
    return dict(bytes=new * (2 * c["Hq"] + 2 * c["Hkv"]) * D * es + new * row
                + read * (row + 2 * c["Hkv"] * D * es), flops=3 * new * (c["Hq"] + c["Hkv"]) * c["rot"])


# ---------------------------------------------------------------- exact values

def _exact_turn(x, pos, case, sign):
    """Complex numbers turned in 64 bits: x [rows, heads, D], pos [rows]."""
    r, i = case["rot"], torch.arange(case["rot"] // 2, dtype=torch.float64)
    f = torch.exp(-2 * i / r * math.log(THETA))
    kind = case.get("scaling", "none")
    if kind == "linear":
        f = 0.25 * f
    if kind == "ntk":
        f = torch.exp(-2 * i / r * (math.log(THETA) + r / (r - 2) * math.log(4.0)))
    if kind == "by_parts":
        turns = 8192 * f / (2 * math.pi)
        f = torch.where(turns > 32, f, torch.where(turns < 1, f / 4, f / 4 + (turns - 1) / 31 * 0.75 * f))
    angle = sign * torch.outer(pos.double(), f.cuda())
    w = torch.polar(torch.full_like(angle, _size(case)), angle)[:, None]
    y = x.double().clone()
    if case["pairs"] == "half":
        z = torch.complex(y[..., :r // 2], y[..., r // 2:r].clone()) * w
        y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
    else:
        z = torch.view_as_complex(y[..., :r].reshape(*y.shape[:-1], r // 2, 2)) * w
        y[..., :r] = torch.view_as_real(z).flatten(-2)
    return y


def _exact_quant(x, dt):
    """What a 4-bit row stands for: x [rows, heads, D] in 64 bits."""
    y = x.reshape(*x.shape[:-1], -1, 32)
    big, least = y.max(-1, keepdim=True).values, y.min(-1, keepdim=True).values
    ref = torch.where(big + least >= 0, big, least)
    s = (-ref / 8).to(dt).double()
    return (torch.where(s == 0, s, (y / s).round().clamp(-8, 7)) * s).reshape(x.shape)


def _exact_rows(raw, dt):
    """64-bit K and V of raw rows [n, heads, D + D / 8], channel by channel from the layout."""
    D = raw.shape[-1] // 9 * 8
    c = torch.arange(D, device="cuda")
    g, i = c // 32, c % 32
    at_k = (i // 8) * (D // 8) + 4 * g + 2 * (i // 4 % 2)            # the word's first byte
    at_v = D // 2 + (i // 4) * (D // 16) + 2 * g
    s = raw[..., D:].contiguous().view(dt).double()
    out = []
    for at, scale in ((at_k, s[..., :D // 32]), (at_v, s[..., D // 32:])):
        word = raw[..., at].long() + 256 * raw[..., at + 1].long()
        word = torch.div(word, 16384, rounding_mode="floor") + 4 * (word % 16384)
        n = torch.div(word, 16 ** (c % 4), rounding_mode="floor") % 16
        out.append((n - 8).double() * scale[..., g])
    return out


def exact(case, seed):
    """What `run` returns, in 64 bits (None for the pages of a 16-bit cache, which are copies)."""
    c, dt = case, DTYPES[case["dtype"]]
    st = prepare(case, seed)
    if c["op"] == "rope":
        x = st["x"]
        y = [_exact_turn(x[b].transpose(0, 1), st["pos"][b], c, -1 if c["inverse"] else 1).transpose(0, 1)
             for b in range(c["B"])]
        return torch.stack(y)
    if c["op"] == "append":
        return [_exact_turn(st["q"], st["pos"], c, 1), None, None]
    if c["op"] == "store4":
        S, M = c["S"], st["table"].shape[1]
        flat = st["table"].long().reshape(-1)
        old = st["pages"][flat[st["read_seq"] * M + st["read_pos"] // S].long(), :, st["read_pos"] % S]
        k, v = _exact_rows(old, dt)
        # where the read rows are new ones: found by (sequence, position)
        far = 1 << 31
        spot = {key: n for n, key in enumerate((st["read_seq"] * far + st["read_pos"]).tolist())}
        at = torch.tensor([spot[x] for x in (st["seq"] * far + st["pos"]).tolist()], device="cuda")
        k[at] = _exact_quant(_exact_turn(st["kn"], st["pos"], c, 1), dt)
        v[at] = _exact_quant(st["vn"].double(), dt)
        return [_exact_turn(st["q"], st["pos"], c, 1), k, v]
    G = c["Hq"] // c["Hkv"]
    if c["op"] == "decode4":
        out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(st["lens"]):
            m = -(-n // c["S"])
            raw = st["pages"][st["table"][b, :m].long()].transpose(1, 2).flatten(0, 1)[:n]
            if c["window"] > 0:
                age = torch.arange(n - 1, -1, -1, device="cuda")
                raw = raw[(age < c["window"]) | (torch.arange(n, device="cuda") < c["sinks"])]
            k, v = _exact_rows(raw, dt)
            for hq in range(c["Hq"]):
                w = torch.softmax(k[:, hq // G] @ st["q"][b, hq].double() / c["D"] ** 0.5, 0)
                out[b, hq] = w @ v[:, hq // G]
        return out
    out = torch.empty(st["q"].shape, dtype=torch.float64, device="cuda")
    cq, ck = st["cu_q"].tolist(), st["cu_k"].tolist()
    for b in range(c["B"]):
        q, k, v = st["q"][cq[b]:cq[b + 1]], st["k"][ck[b]:ck[b + 1]], st["v"][ck[b]:ck[b + 1]]
        n, t = len(q), len(k)
        key = torch.arange(t, device="cuda")
        for i in range(0, n, 1024):
            at = torch.arange(i, min(i + 1024, n), device="cuda") + t - n
            gap = at[:, None] - key[None]
            hide = gap < 0
            if c["window"] > 0:
                hide = hide | ((gap >= c["window"]) & (key[None] >= c["sinks"]))
            for hq in range(c["Hq"]):
                s = torch.einsum("id,jd->ij", q[i:i + 1024, hq].double(), k[:, hq // G].double()) / c["D"] ** 0.5
                w = torch.softmax(s.masked_fill(hide, -math.inf), -1)
                out[cq[b] + i:cq[b] + i + len(at), hq] = w @ v[:, hq // G].double()
    return out

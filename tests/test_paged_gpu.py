"""Paged KV cache: decode against a 64-bit softmax over exactly the visible
positions (everything else in the pool is NaN), append and the page allocator
against a Python model."""
import numpy as np
import pytest
import torch

from tests.paged_ref import DT, Pool, attend, bound, visible

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ta():
    from transformer_attention_tcgen05_gb300.build import build
    build()
    import transformer_attention_tcgen05_gb300 as ta
    torch.cuda.set_device(0)
    return ta


def empty_pool(P, Hkv, S, D, dt, order, fill=float("nan"), device="cuda"):
    def one():
        if order == "token":
            return torch.full((P, S, Hkv, D), fill, dtype=DT[dt], device=device).transpose(1, 2)
        return torch.full((P, Hkv, S, D), fill, dtype=DT[dt], device=device)
    return one(), one()


def build_case(dt, lens, Hq, Hkv, D, S, window, sinks, order, seed, spare=5):
    """Contiguous K/V per sequence, and a NaN-filled pool in which only the visible
    rows exist; entries of pages without one are -1."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    M = max(1, max(-(-n // S) for n in lens)) + 1
    P = sum(-(-n // S) for n in lens) + spare
    kp, vp = empty_pool(P, Hkv, S, D, dt, order, device="cpu")
    table = torch.full((B, M), -1, dtype=torch.int32)
    perm = torch.randperm(P, generator=g).tolist()
    q = torch.randn(B, Hq, D, generator=g).to(DT[dt])
    ks, vs = [], []
    for b, n in enumerate(lens):
        k = torch.randn(Hkv, n, D, generator=g).to(DT[dt])
        v = torch.randn(Hkv, n, D, generator=g).to(DT[dt])
        see = visible(n, [n - 1], window, sinks)[0] if n else torch.zeros(0, dtype=torch.bool)
        for i in range(-(-n // S)):
            s = see[i * S:(i + 1) * S]
            if not s.any():
                continue
            page = perm.pop()
            table[b, i] = page
            at = torch.nonzero(s)[:, 0]
            kp[page][:, at] = k[:, i * S:(i + 1) * S][:, at]
            vp[page][:, at] = v[:, i * S:(i + 1) * S][:, at]
        ks.append(k)
        vs.append(v)
    sl = torch.tensor(lens, dtype=torch.int32)
    # the views keep their memory order on the device
    dev = (lambda x: x.transpose(1, 2).contiguous().cuda().transpose(1, 2)) if order == "token" \
        else (lambda x: x.cuda())
    return q.cuda(), dev(kp), dev(vp), table.cuda(), sl.cuda(), ks, vs


def check(dt, q, ks, vs, lens, o, window, sinks, only=None):
    B, Hq, D = q.shape
    for b, n in enumerate(lens):
        if only is not None and b not in only:
            continue
        if n == 0:
            assert (o[b] == 0).all()
            continue
        Hkv = ks[b].shape[0]
        G = Hq // Hkv
        see = visible(n, [n - 1], window, sinks).expand(G, n)
        for hk in range(Hkv):
            ref, A, E, s1 = attend(q[b, hk * G:(hk + 1) * G].double().cpu(), ks[b][hk].double(),
                                   vs[b][hk].double(), see)
            got = o[b, hk * G:(hk + 1) * G].double().cpu()
            # P enters as a sum of two 16-bit terms: bf16 keeps 2^-18 of it, f16 more
            lim = bound(dt, ref, A, E, s1, n, 2.0 ** -17)
            bad = ~((got - ref).abs() <= lim)
            assert not bad.any(), (b, hk, torch.nonzero(bad)[:4].tolist(),
                                   ((got - ref).abs() / lim).max().item())


CASES = [
    # dt, lens, Hq, Hkv, D, S, window, sinks, order
    ("bf16", [1], 1, 1, 64, 16, 0, 0, "head"),
    ("bf16", [0, 1, 31, 32, 33, 0], 4, 1, 128, 16, 0, 0, "head"),
    ("f16", [64, 5, 200], 8, 2, 64, 8, 0, 0, "token"),
    ("bf16", [127, 128, 129], 12, 4, 128, 48, 0, 0, "token"),      # pages end inside a chunk
    ("bf16", [100, 700], 14, 2, 128, 24, 0, 0, "head"),            # 7 heads per KV head
    ("f16", [333, 0, 65], 16, 2, 128, 64, 0, 0, "head"),
    ("bf16", [1000, 3], 32, 2, 64, 16, 0, 0, "head"),              # 16 heads per KV head
    ("f16", [500, 77], 27, 3, 128, 32, 0, 0, "token"),             # 9 heads per KV head
    ("bf16", [5000, 40, 1], 4, 2, 128, 128, 0, 0, "head"),         # a unit over many CTAs
    ("bf16", [20000], 8, 1, 64, 16, 0, 0, "head"),                 # one unit over all of them
    ("bf16", [300, 90, 5, 1], 4, 2, 128, 16, 64, 4, "head"),
    ("f16", [1000, 64, 65], 4, 1, 64, 32, 1, 0, "token"),          # the newest token alone
    ("bf16", [1000, 100], 4, 1, 128, 16, 70, 40, "token"),         # sinks past a chunk
    ("bf16", [200, 131, 129], 4, 1, 128, 8, 100, 30, "head"),      # sinks meet the window
    ("f16", [900, 20], 2, 1, 128, 16, 100000, 4, "head"),          # window beyond the length
    ("bf16", [900, 20], 2, 1, 64, 16, 16, 5000, "head"),           # sinks beyond it
    ("bf16", [3, 9, 30] * 70, 2, 2, 64, 16, 0, 0, "head"),         # more rows than threads
    ("bf16", [250, 7, 0, 100] * 25, 16, 8, 128, 16, 0, 0, "head"), # units dealt out warp by warp
    ("f16", [250, 1, 0, 33, 64, 0] * 50, 12, 4, 64, 8, 0, 0, "token"),
    ("bf16", [900, 40, 0, 129] * 30, 27, 3, 128, 48, 100, 20, "head"),
    ("bf16", [1200, 300, 700] * 12, 8, 4, 64, 16, 0, 0, "head"),   # ranges that end inside units
    ("bf16", [3000, 1, 0, 40, 257, 256, 7], 8, 8, 64, 16, 0, 0, "head"),   # short units beside long ones
    ("f16", ([1] * 40 + [900, 0]) * 4, 4, 2, 128, 32, 0, 0, "token"),
    ("bf16", [5000, 3] + [300, 64] * 30, 3, 3, 64, 8, 200, 10, "head"),
]


@pytest.mark.parametrize("dt,lens,Hq,Hkv,D,S,window,sinks,order", CASES)
def test_decode_paged_parity(ta, dt, lens, Hq, Hkv, D, S, window, sinks, order):
    q, kp, vp, table, sl, ks, vs = build_case(dt, lens, Hq, Hkv, D, S, window, sinks, order, len(lens))
    n0 = ta.launch_count("decode_paged")
    o = ta.decode_gqa_paged(q, kp, vp, table, sl, window=window, sinks=sinks)
    assert ta.launch_count("decode_paged") == n0 + 1
    assert ta.device_status() == 0
    check(dt, q, ks, vs, lens, o, window, sinks)


@pytest.mark.parametrize("dt,lens,Hq,Hkv,D,S,window,sinks", [
    ("bf16", [700], 16, 8, 128, 16, 0, 0),
    ("f16", [700, 0, 650], 8, 8, 64, 16, 0, 0),
    ("bf16", [1024, 1023, 1025, 993, 600, 289, 1100, 800], 16, 8, 128, 32, 0, 0),
    ("bf16", [2000] * 8, 8, 8, 64, 16, 0, 0),
    ("bf16", [1500, 20, 1400, 0, 3], 12, 4, 128, 16, 0, 0),      # short units beside them
    ("bf16", [5000, 900, 700], 8, 8, 64, 24, 650, 33),
])
def test_decode_paged_ranges_fitted_to_units(ta, dt, lens, Hq, Hkv, D, S, window, sinks):
    """A few long units: a range holds part of one of them."""
    q, kp, vp, table, sl, ks, vs = build_case(dt, lens, Hq, Hkv, D, S, window, sinks, "head", 5)
    o = ta.decode_gqa_paged(q, kp, vp, table, sl, window=window, sinks=sinks)
    assert ta.device_status() == 0
    check(dt, q, ks, vs, lens, o, window, sinks)


def test_decode_paged_workspace_is_left_ready_and_results_repeat(ta):
    lens = [3000, 1, 0, 777]
    q, kp, vp, table, sl, ks, vs = build_case("bf16", lens, 8, 2, 128, 16, 0, 0, "head", 3)
    ws = torch.zeros(ta.decode_paged_workspace_bytes(4, 8, 2, 128), dtype=torch.uint8, device="cuda")
    first = ta.decode_gqa_paged(q, kp, vp, table, sl, workspace=ws)
    check("bf16", q, ks, vs, lens, first, 0, 0)
    for _ in range(20):
        assert torch.equal(ta.decode_gqa_paged(q, kp, vp, table, sl, workspace=ws), first)


@pytest.mark.parametrize("dt,D,S,order,G", [("bf16", 128, 16, "head", 2), ("f16", 64, 32, "token", 1),
                                            ("bf16", 128, 8, "head", 9)])
def test_decode_paged_ring_wraps_in_back_to_back_launches(ta, dt, D, S, order, G):
    """Ten chunks and more per CTA: every ring slot is used several times, and the
    next launch starts while the last CTAs finish."""
    lens = [6000, 5500, 33, 7100]
    q, kp, vp, table, sl, ks, vs = build_case(dt, lens, 4 * G, 4, D, S, 0, 0, order, 9)
    ws = torch.zeros(ta.decode_paged_workspace_bytes(4, 4 * G, 4, D), dtype=torch.uint8, device="cuda")
    outs = [ta.decode_gqa_paged(q, kp, vp, table, sl, workspace=ws) for _ in range(30)]
    assert ta.device_status() == 0
    check(dt, q, ks, vs, lens, outs[0], 0, 0)
    assert all(torch.equal(o, outs[0]) for o in outs)


def test_one_workspace_serves_calls_of_several_sizes(ta):
    sizes = [([2000, 5], 4, 2, 128), ([900] * 9, 16, 1, 64), ([3000], 8, 8, 128), ([70, 800, 9], 27, 3, 128)]
    ws = torch.zeros(ta.decode_paged_workspace_bytes(9, 64, 8, 128), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        for i, (lens, Hq, Hkv, D) in enumerate(sizes):
            q, kp, vp, table, sl, ks, vs = build_case("bf16", lens, Hq, Hkv, D, 16, 0, 0, "head", 30 + i)
            o = ta.decode_gqa_paged(q, kp, vp, table, sl, workspace=ws)
            check("bf16", q, ks, vs, lens, o, 0, 0)
    assert ta.device_status() == 0


def test_empty_fork_list_and_zero_rows(ta):
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    refs, sl = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (8, 2))
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    cs, cd = ta.kv_pages_fork(table, sl, refs, none, none, 8)
    assert cs.numel() == cd.numel() == 0
    k = torch.zeros(8, 1, 8, 64, dtype=torch.bfloat16, device="cuda")
    ta.kv_pages_copy(k, k.clone(), cs, cd)
    ta.kv_pages_reserve(table, sl, sl, refs, 8)
    assert ta.device_status() == 0 and (table == -1).all() and (refs == 0).all()
    with pytest.raises(ta.AttnError):
        ta.decode_gqa_paged(k[:0, 0, :1], k, k.clone(), table[:0], sl[:0])


def test_decode_paged_strided_query_output_and_table(ta):
    lens = [50, 400, 33]
    q, kp, vp, table, sl, ks, vs = build_case("bf16", lens, 6, 2, 64, 16, 0, 0, "head", 4)
    packed = torch.zeros(3, 10, 64, dtype=torch.bfloat16, device="cuda")
    packed[:, 2:8] = q
    wide = torch.full((3, 8, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    big = torch.full((3, table.shape[1] + 9), 123456789, dtype=torch.int32, device="cuda")
    big[:, :table.shape[1]] = table
    ta.decode_gqa_paged(packed[:, 2:8], kp, vp, big[:, :table.shape[1]], sl, o=wide[:, 1:7])
    assert ta.device_status() == 0
    check("bf16", q, ks, vs, lens, wide[:, 1:7], 0, 0)
    assert (wide[:, 0] == 5).all() and (wide[:, 7] == 5).all()


def test_decode_paged_nan_and_infinite_inputs_reach_their_own_heads_only(ta):
    lens = [100, 700]
    q, kp, vp, table, sl, ks, vs = build_case("bf16", lens, 4, 2, 64, 16, 0, 0, "head", 5)
    page, row = table[1, 600 // 16].item(), 600 % 16
    kp[page, 1, row, 3] = float("nan")
    o = ta.decode_gqa_paged(q, kp, vp, table, sl)
    assert torch.isnan(o[1, 2:]).all() and torch.isfinite(o[1, :2]).all()
    check("bf16", q, ks, vs, lens, o, 0, 0, only=[0])
    # a sequence whose only key is NaN
    sl1 = torch.tensor([1, 1], dtype=torch.int32, device="cuda")
    kp[table[0, 0].item(), 0, 0, 0] = float("nan")
    o = ta.decode_gqa_paged(q, kp, vp, table, sl1)
    assert torch.isnan(o[0, :2]).all() and torch.isfinite(o[0, 2:]).all()


def test_decode_paged_bad_pages_and_lengths_are_reported_per_sequence(ta):
    lens = [40, 3000, 80, 500]
    for entry in (-1, 10 ** 6):
        q, kp, vp, table, sl, ks, vs = build_case("bf16", lens, 4, 2, 128, 16, 0, 0, "head", 6)
        table[1, 100] = entry
        sl[2] = table.shape[1] * 16 + 1
        sl[0] = -3
        o = torch.full_like(q, 9.0)
        ws = torch.zeros(ta.decode_paged_workspace_bytes(4, 4, 2, 128), dtype=torch.uint8, device="cuda")
        ta.decode_gqa_paged(q, kp, vp, table, sl, o=o, workspace=ws)
        assert ta.device_status() == 6
        assert (o[:3] == 9).all()
        check("bf16", q, ks, vs, lens, o, 0, 0, only=[3])
        # units dealt out warp by warp
        lens2 = [40, 100, 250, 16] * 40
        q, kp, vp, table, sl, ks, vs = build_case("bf16", lens2, 8, 4, 128, 16, 0, 0, "head", 8)
        table[1, 3] = entry
        sl[2] = -1
        o = torch.full_like(q, 9.0)
        ta.decode_gqa_paged(q, kp, vp, table, sl, o=o)
        assert ta.device_status() == 6
        assert (o[1:3] == 9).all()
        check("bf16", q, ks, vs, lens2, o, 0, 0, only=[0] + list(range(3, 160, 9)))
        # the workspace serves the next call
        q, kp, vp, table, sl, ks, vs = build_case("bf16", lens, 4, 2, 128, 16, 0, 0, "head", 7)
        o = ta.decode_gqa_paged(q, kp, vp, table, sl, workspace=ws)
        assert ta.device_status() == 0
        check("bf16", q, ks, vs, lens, o, 0, 0)


def test_offsets_beyond_32_bits(ta):
    """Pages whose element offsets pass 2^31: decode, append and copy."""
    Hkv, S, D = 8, 128, 128
    P = 2 ** 31 // (Hkv * S * D) + 40
    kp = torch.zeros(P, Hkv, S, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    g = torch.Generator().manual_seed(1)
    n = 200
    k, v = (torch.randn(1, Hkv, n, D, generator=g).bfloat16() for _ in range(2))
    q = torch.randn(1, Hkv, D, generator=g).bfloat16().cuda()
    table = torch.tensor([[P - 1, P - 7]], dtype=torch.int32, device="cuda")
    sl = torch.zeros(1, dtype=torch.int32, device="cuda")
    ta.kv_append_paged(kp, vp, k.cuda(), v.cuda(), table, sl)
    assert sl.item() == n
    assert torch.equal(kp[P - 1].cpu(), k[0, :, :S]) and torch.equal(vp[P - 7, :, :n - S].cpu(), v[0, :, S:])
    o = ta.decode_gqa_paged(q, kp, vp, table, sl)
    check("bf16", q, [k[0]], [v[0]], [n], o, 0, 0)
    src = torch.tensor([P - 1, P - 7], dtype=torch.int32, device="cuda")
    ta.kv_pages_copy(kp, vp, src, src - 20)
    o2 = ta.decode_gqa_paged(q, kp, vp, table - 20, sl)
    assert ta.device_status() == 0 and torch.equal(o, o2)


# ------------------------------------------------------------------- append

@pytest.mark.parametrize("dt,D,S,order,B,T", [("bf16", 128, 16, "head", 3, 1), ("f16", 64, 8, "token", 5, 1),
                                              ("f32", 32, 24, "head", 2, 7), ("bf16", 128, 16, "token", 3, 16),
                                              ("bf16", 64, 48, "head", 4, 100), ("f32", 128, 16, "head", 2, 333),
                                              ("bf16", 32, 16, "token", 2, 17)])
@pytest.mark.parametrize("advance", [True, False])
def test_append_paged(ta, dt, D, S, order, B, T, advance):
    g = torch.Generator().manual_seed(T)
    Hkv = 3
    start = torch.randint(0, 70, (B,), generator=g, dtype=torch.int32)
    new = torch.randint(0, T + 1, (B,), generator=g, dtype=torch.int32) if T > 1 else None
    cnt = new if new is not None else torch.full((B,), T, dtype=torch.int32)
    M = int((start + cnt).max()) // S + 3
    P = B * M + 3
    table = torch.randperm(P, generator=g)[:B * M].view(B, M).int()
    kp, vp = empty_pool(P, Hkv, S, D, dt, order, fill=3.0)
    kw, vw = kp.clone(), vp.clone()
    packed = torch.randn(B, T, 2, Hkv, D, generator=g).to(DT[dt]).cuda()
    kn, vn = packed[:, :, 0].transpose(1, 2), packed[:, :, 1].transpose(1, 2)
    for b in range(B):
        for t in range(int(cnt[b])):
            pos = int(start[b]) + t
            kw[table[b, pos // S], :, pos % S] = kn[b, :, t]
            vw[table[b, pos // S], :, pos % S] = vn[b, :, t]
    sl = start.cuda()
    ta.kv_append_paged(kp, vp, kn, vn, table.cuda(), sl, None if new is None else new.cuda(), advance=advance)
    assert ta.device_status() == 0
    assert torch.equal(kp, kw) and torch.equal(vp, vw)
    assert torch.equal(sl.cpu(), start + cnt if advance else start)


@pytest.mark.parametrize("T", [1, 5, 40])
def test_append_paged_requests_that_do_not_fit(ta, T):
    S, D, B, M = 8, 64, 5, 6
    table = torch.arange(B * M, dtype=torch.int32).view(B, M).cuda()
    kp, vp = empty_pool(B * M, 1, S, D, "bf16", "head", fill=0.0)
    table[1, 0] = -1
    table[2, 0] = B * M
    start = torch.tensor([0, 0, 0, M * S - T + 1, -1], dtype=torch.int32).cuda()
    sl = start.clone()
    new = torch.ones(B, 1, T, D, dtype=torch.bfloat16, device="cuda")
    ta.kv_append_paged(kp, vp, new, new.clone(), table, sl)
    assert ta.device_status() == 6
    assert sl.tolist() == [T, 0, 0, M * S - T + 1, -1]
    written = (kp != 0).any(-1).any(1).sum().item()     # rows: sequence 0, and what fell in good pages of 1, 2
    assert written == T + 2 * max(0, T - S)
    # more rows than given, or a negative count, is refused as well
    sl = torch.zeros(B, dtype=torch.int32, device="cuda")
    n = torch.tensor([T + 1, -1, 0, 0, 0], dtype=torch.int32, device="cuda")
    ta.kv_append_paged(kp, vp, new, new.clone(), table, sl, n)
    assert ta.device_status() == 6 and sl.tolist() == [0] * B


# ---------------------------------------------------------------- allocator

class Model:
    """The Python allocator, the token each position holds, and the device state."""

    def __init__(self, ta, B, M, P, S, layers=2, Hkv=2, D=64, dt="bf16", seed=0):
        self.ta, self.S = ta, S
        self.pool = Pool(B, M, P, S)
        self.tok = [[] for _ in range(B)]
        self.next = 1
        self.table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(P, dtype=torch.int32, device="cuda")
        self.len = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.k = torch.zeros(layers, P, Hkv, S, D, dtype=DT[dt], device="cuda")
        self.v = torch.zeros_like(self.k)

    def i32(self, x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def row(self, ids):
        """K rows [layers, Hkv, T, D] that stand for token ids (exact in 16 bits)."""
        L, _, Hkv, _, D = self.k.shape
        x = torch.tensor([[i % 251, i // 251] for i in ids], dtype=self.k.dtype).view(1, 1, -1, 2)
        y = x.repeat(L, Hkv, 1, D // 2)
        y = y + torch.arange(L).view(L, 1, 1, 1) * 0
        return y.cuda()

    def reserve(self, add):
        ok = self.pool.reserve(add)
        self.ta.kv_pages_reserve(self.table, self.len, self.i32(add), self.refs, self.S)
        assert self.ta.device_status() == (0 if ok else 6)
        return ok

    def append(self, add):
        T = max(1, max(add))
        L, _, Hkv, _, D = self.k.shape
        kn = torch.zeros(L, len(add), Hkv, T, D, dtype=self.k.dtype, device="cuda")
        for b, n in enumerate(add):
            ids = list(range(self.next, self.next + n))
            self.next += n
            self.tok[b] += ids
            if n:
                kn[:, b, :, :n] = self.row(ids)
        for l in range(L):
            self.ta.kv_append_paged(self.k[l], self.v[l], kn[l] + l, kn[l] - l, self.table, self.len,
                                    self.i32(add), advance=l == L - 1)
        self.pool.len += np.array(add, dtype=np.int32)

    def fork(self, src, dst):
        pairs = self.pool.fork(src, dst)
        cs, cd = self.ta.kv_pages_fork(self.table, self.len, self.refs, self.i32(src), self.i32(dst), self.S)
        assert self.ta.device_status() == (0 if pairs is not None else 6)
        if pairs is None:
            assert cs.tolist() == cd.tolist() == [-1] * len(src)
            return False
        assert list(zip(cs.tolist(), cd.tolist())) == pairs
        self.ta.kv_pages_copy(self.k, self.v, cs, cd)
        for s, d in zip(src, dst):
            self.tok[d] = list(self.tok[s])
        return True

    def free(self, window=0, sinks=0):
        self.pool.free(window, sinks)
        self.ta.kv_pages_free(self.table, self.len, self.refs, self.S, window, sinks)

    def drop(self, rows):
        for b in rows:
            self.tok[b] = []
            self.pool.len[b] = 0
            self.len[b] = 0
        self.free()

    def compact(self, in_place):
        pairs = self.pool.compact()
        if in_place:
            cs, cd, n = self.ta.kv_pages_compact(self.table, self.refs)
        else:
            old_t, old_r = self.table.clone(), self.refs.clone()
            t, r = torch.full_like(self.table, 77), torch.full_like(self.refs, 77)
            cs, cd, n = self.ta.kv_pages_compact(self.table, self.refs, new_table=t, new_refs=r)
            assert torch.equal(old_t, self.table) and torch.equal(old_r, self.refs)
            self.table, self.refs = t, r
        assert n.item() == len(pairs)
        assert list(zip(cs.tolist(), cd.tolist())) == pairs + [(-1, -1)] * (len(self.refs) // 2 - len(pairs))
        self.ta.kv_pages_copy(self.k, self.v, cs, cd, count=n)

    def check(self):
        assert self.ta.device_status() == 0
        assert np.array_equal(self.table.cpu().numpy(), self.pool.table)
        assert np.array_equal(self.refs.cpu().numpy(), self.pool.refs)
        assert np.array_equal(self.len.cpu().numpy(), self.pool.len)
        # every token whose page is held reads back as appended, in every layer
        for b, ids in enumerate(self.tok):
            if not ids:
                continue
            pos = torch.arange(len(ids))
            pages = torch.from_numpy(self.pool.table[b]).long()[pos // self.S]
            held = pages >= 0
            if not held.any():
                continue
            got_k = self.k[:, pages[held].cuda(), :, (pos % self.S)[held].cuda()]
            got_v = self.v[:, pages[held].cuda(), :, (pos % self.S)[held].cuda()]
            # [n, layers, Hkv, D] (advanced indices apart) -> [layers, Hkv, n, D]
            want = self.row([i for i, h in zip(ids, held.tolist()) if h])
            off = torch.arange(want.shape[0], device="cuda").view(-1, 1, 1, 1).to(want.dtype)
            assert torch.equal(got_k.permute(1, 2, 0, 3), want + off)
            assert torch.equal(got_v.permute(1, 2, 0, 3), want - off)


@pytest.mark.parametrize("S,P,B,seed", [(8, 60, 6, 0), (16, 41, 5, 1), (24, 200, 9, 2), (8, 1300, 40, 3),
                                        (8, 20011, 7, 4), (8, 17003, 1100, 5)])
def test_allocator_against_the_model(ta, S, P, B, seed):
    rng = np.random.default_rng(seed)
    m = Model(ta, B, M=min(2000, max(12, P // 8)), P=P, S=S, seed=seed, layers=1 if P > 5000 else 2)
    refused = 0
    long_row = 500 * S if P > 5000 else 4 * S     # several entries per thread in a large pool
    for step in range(40 if B < 100 else 12):
        op = rng.choice(["grow", "grow", "grow", "fork", "drop", "slide", "compact"])
        if op == "grow":
            room = m.table.shape[1] * S - m.pool.len
            add = [int(min(room[b], rng.integers(0, long_row if b < 8 else 4 * S) if rng.random() < 0.6 else 0)) for b in range(B)]
            if m.reserve(add):
                m.append(add)
            else:
                refused += 1
        elif op == "fork":
            rows = rng.permutation(B)
            n = int(rng.integers(1, max(2, B // 2)))
            src = [int(rng.choice(rows[n:])) for _ in range(n)]
            refused += not m.fork(src, [int(r) for r in rows[:n]])
        elif op == "drop":
            m.drop([int(rng.integers(B))])
        elif op == "slide":
            m.free(int(rng.integers(1, 3 * S)), int(rng.choice([0, 1, S, 2 * S + 1])))
        else:
            m.compact(bool(rng.integers(2)))
        m.check()


@pytest.mark.parametrize("P", [262143, 600001])
def test_allocator_on_pools_of_several_spans(ta, P):
    """More pages than the CTAs of a call hold at once: numbers run on from one
    span of the pool to the next."""
    rng = np.random.default_rng(P)
    B, S, M = 40, 8, P // 16
    held = rng.permutation(P)[:P * 3 // 5].astype(np.int32)
    per = len(held) // B
    table = np.full((B, M), -1, dtype=np.int32)
    table[:, :per] = held[:per * B].reshape(B, per)
    refs = np.zeros(P, dtype=np.int32)
    refs[table[:, :per].ravel()] = 1
    length = np.full(B, per * S, dtype=np.int32)
    dt, dr, dl = (torch.from_numpy(x.copy()).cuda() for x in (table, refs, length))
    # compact, out of place
    L = int((refs > 0).sum())
    src, dst = L + np.flatnonzero(refs[L:] > 0), np.flatnonzero(refs[:L] == 0)
    place = np.where(refs > 0, np.arange(P), -1)
    place[src] = dst
    nt, nr = torch.empty_like(dt), torch.empty_like(dr)
    cs, cd, n = ta.kv_pages_compact(dt, dr, new_table=nt, new_refs=nr)
    assert n.item() == len(src) == len(dst)
    assert np.array_equal(cs.cpu().numpy()[:len(src)], src) and np.array_equal(cd.cpu().numpy()[:len(src)], dst)
    assert (cs[len(src):] == -1).all() and (cd[len(src):] == -1).all()
    want = np.where(table >= 0, place[table], -1)
    assert np.array_equal(nt.cpu().numpy(), want)
    assert np.array_equal(nr.cpu().numpy(), (np.arange(P) < L).astype(np.int32))
    # reserve nine tenths of what is free, some rows nothing
    free = np.flatnonzero(refs == 0)
    add = np.zeros(B, dtype=np.int32)
    add[1::2] = len(free) * 9 // 10 // (B // 2) * S
    for b in range(1, B, 2):
        k = add[b] // S
        table[b, per:per + k] = free[:k]
        free = free[k:]
    refs[table[table >= 0]] = 1
    ta.kv_pages_reserve(dt, dl, torch.from_numpy(add).cuda(), dr, S)
    assert ta.device_status() == 0
    assert np.array_equal(dt.cpu().numpy(), table) and np.array_equal(dr.cpu().numpy(), refs)
    # one page more than there are
    add[:] = 0
    add[0] = (len(free) + 1) * S
    assert per + len(free) + 1 <= M
    ta.kv_pages_reserve(dt, dl, torch.from_numpy(add).cuda(), dr, S)
    assert ta.device_status() == 6
    assert np.array_equal(dt.cpu().numpy(), table) and np.array_equal(dr.cpu().numpy(), refs)
    # fork: row 2 (its last page partly filled) over row 4, whose pages are let go
    dl[2] -= 3
    ta.kv_pages_fork(dt, dl, dr, torch.tensor([2], dtype=torch.int32, device="cuda"),
                     torch.tensor([4], dtype=torch.int32, device="cuda"), S)
    assert ta.device_status() == 0
    refs[table[4, :per]] -= 1
    refs[table[2, :per - 1]] += 1
    table[4, :per - 1] = table[2, :per - 1]
    table[4, per - 1] = np.flatnonzero(refs == 0)[0]
    refs[table[4, per - 1]] = 1
    assert np.array_equal(dt.cpu().numpy(), table) and np.array_equal(dr.cpu().numpy(), refs)


def test_reserve_is_all_or_nothing(ta):
    m = Model(ta, 3, 8, 10, 8)
    assert m.reserve([30, 0, 20])               # 4 + 3 pages
    m.append([30, 0, 20])
    assert not m.reserve([1, 40, 10])           # 5 + 1 > 3
    m.check()
    assert m.reserve([1, 24, 0])
    m.append([1, 24, 0])
    m.check()
    # a length or an addition that is out of range
    for add in ([0, -1, 0], [0, 8 * 8 - 24 + 1, 0]):
        t = m.table.clone()
        ta.kv_pages_reserve(m.table, m.len, m.i32(add), m.refs, 8)
        assert ta.device_status() == 6 and torch.equal(t, m.table)
    m.check()


def test_fork_refuses_what_it_cannot_do(ta):
    m = Model(ta, 6, 8, 16, 8)
    m.reserve([20, 8, 5, 0, 0, 0])
    m.append([20, 8, 5, 0, 0, 0])
    for src, dst in (([0, 1], [3, 3]), ([0, 3], [3, 4]), ([0, 6], [3, 4]), ([0, 1], [3, -1]), ([2], [2])):
        before = (m.table.clone(), m.refs.clone(), m.len.clone())
        cs, cd = ta.kv_pages_fork(m.table, m.len, m.refs, m.i32(src), m.i32(dst), 8)
        assert ta.device_status() == 6
        assert cs.tolist() == cd.tolist() == [-1] * len(src)
        assert all(torch.equal(a, b) for a, b in zip(before, (m.table, m.refs, m.len)))
    assert m.fork([0, 0, 2], [3, 4, 5])         # one parent twice; tails at 20 and 5 tokens
    m.check()
    assert m.fork([0, 0, 2], [3, 4, 5])         # again, over themselves
    m.check()
    # a table entry that is no counted page
    bad = m.table.clone()
    bad[0, 1] = 15
    refs = m.refs.clone()
    assert refs[15] == 0
    ta.kv_pages_fork(bad, m.len, refs, m.i32([0]), m.i32([3]), 8)
    assert ta.device_status() == 6 and torch.equal(refs, m.refs)


def test_fork_without_pages_for_the_copies_changes_nothing(ta):
    m = Model(ta, 4, 8, 6, 8)
    m.reserve([20, 16, 0, 0])                   # 3 + 2 of 6 pages
    m.append([20, 16, 0, 0])
    assert not m.fork([0, 0], [2, 3])           # two copies, one free page
    m.check()
    assert m.fork([0, 1], [2, 3])
    m.check()


def test_free_reports_pages_that_are_not_counted(ta):
    table = torch.tensor([[0, 1, 2, 7]], dtype=torch.int32, device="cuda")
    refs = torch.tensor([1, 0, 2, 0], dtype=torch.int32, device="cuda")
    sl = torch.zeros(1, dtype=torch.int32, device="cuda")
    ta.kv_pages_free(table, sl, refs, 8)
    assert ta.device_status() == 6
    assert table.tolist() == [[-1, 1, -1, 7]] and refs.tolist() == [0, 0, 1, 0]


@pytest.mark.parametrize("M", [3, 1500])           # tables written by the call's first and second kernel
def test_compact_of_the_smallest_pools(ta, M):
    for P, live in ((1, [0]), (1, []), (2, [1]), (3, [2]), (5, [1, 3, 4])):
        table = torch.full((2, M), -1, dtype=torch.int32, device="cuda")
        refs = torch.zeros(P, dtype=torch.int32, device="cuda")
        for i, page in enumerate(live):
            table[i % 2, M - 1 - i // 2] = page
            refs[page] = 1
        place = {}
        holes = [x for x in range(len(live)) if x not in live]
        for page in live:
            place[page] = page if page < len(live) else holes.pop(0)
        want = torch.tensor([[place.get(x, -1) for x in row] for row in table.tolist()], dtype=torch.int32)
        cs, cd, n = ta.kv_pages_compact(table, refs)
        assert ta.device_status() == 0
        moves = [(x, y) for x, y in place.items() if x != y]
        assert len(cs) == len(cd) == P // 2 and n.tolist() == [len(moves)]
        assert list(zip(cs.tolist(), cd.tolist()))[:len(moves)] == moves
        assert torch.equal(table.cpu(), want)
        assert refs.tolist() == [1] * len(live) + [0] * (P - len(live))


def test_free_leaves_rows_of_impossible_lengths(ta):
    table = torch.tensor([[0, 1], [2, -1], [3, 4]], dtype=torch.int32, device="cuda")
    refs = torch.ones(5, dtype=torch.int32, device="cuda")
    sl = torch.tensor([17, 0, -1], dtype=torch.int32, device="cuda")     # 16 positions per row
    ta.kv_pages_free(table, sl, refs, 8, window=1)
    assert ta.device_status() == 6
    assert table.tolist() == [[0, 1], [-1, -1], [3, 4]] and refs.tolist() == [1, 1, 0, 1, 1]


def test_copy_reports_a_pair_of_equal_numbers_outside_the_pool(ta):
    k, v = torch.randn(2, 1, 8, 64, device="cuda"), torch.randn(2, 1, 8, 64, device="cuda")
    k0 = k.clone()
    pair = torch.tensor([2], dtype=torch.int32, device="cuda")
    ta.kv_pages_copy(k, v, pair, pair)
    assert ta.device_status() == 6
    assert torch.equal(k, k0)


def test_compact_drops_entries_of_free_pages(ta):
    # 4 and 1 name free pages (1 below the live count: another page moves there)
    table = torch.tensor([[5, 3, -1, 4, 99, 1]], dtype=torch.int32, device="cuda")
    refs = torch.tensor([0, 0, 0, 1, 0, 1], dtype=torch.int32, device="cuda")
    cs, cd, n = ta.kv_pages_compact(table, refs)
    assert ta.device_status() == 6
    assert n.item() == 2 and cs.tolist() == [3, 5, -1] and cd.tolist() == [0, 1, -1]
    assert table.tolist() == [[1, 0, -1, -1, -1, -1]] and refs.tolist() == [1, 1, 0, 0, 0, 0]


@pytest.mark.parametrize("order", ["head", "token", "packed"])
def test_copy_pages_layouts_and_bad_pairs(ta, order):
    P, Hkv, S, D = 9, 3, 24, 64
    g = torch.Generator().manual_seed(2)
    if order == "packed":                        # K and V side by side in one page
        both = torch.randn(P, 2, Hkv, S, D, generator=g).bfloat16().cuda()
        k, v = both[:, 0], both[:, 1]
    else:
        k, v = (torch.randn(P, S, Hkv, D, generator=g).bfloat16().cuda().transpose(1, 2)
                if order == "token" else torch.randn(P, Hkv, S, D, generator=g).bfloat16().cuda()
                for _ in range(2))
    k0, v0 = k.clone(), v.clone()
    src = torch.tensor([0, -1, 3, 4, 9, 6], dtype=torch.int32, device="cuda")
    dst = torch.tensor([1, -1, 2, 4, 5, -7], dtype=torch.int32, device="cuda")
    ta.kv_pages_copy(k, v, src, dst)
    assert ta.device_status() == 6               # pairs 4 and 5 name no page
    for x, x0 in ((k, k0), (v, v0)):
        want = x0.clone()
        want[1], want[2] = x0[0], x0[3]
        assert torch.equal(x, want)
    n = torch.tensor([1], dtype=torch.int32, device="cuda")
    k1 = k.clone()
    ta.kv_pages_copy(k, v, src[2:4], dst[:2].abs() + 6, count=n)     # one pair only
    assert ta.device_status() == 0
    k1[7] = k1[3]
    assert torch.equal(k, k1)


# ------------------------------------------------------------ used together

def test_serving_steps_in_a_captured_graph(ta):
    """reserve, append, decode with window and sinks, free: captured once and
    replayed as the sequences grow past the pool's size."""
    B, Hq, Hkv, D, S, P, M = 3, 4, 2, 64, 8, 24, 100
    window, sinks, steps = 20, 3, 150
    g = torch.Generator().manual_seed(5)
    kv = [torch.randn(B, Hkv, steps + 1, D, generator=g).bfloat16() for _ in range(2)]
    qs = torch.randn(steps + 1, B, Hq, D, generator=g).bfloat16()
    kp, vp = empty_pool(P, Hkv, S, D, "bf16", "token")
    table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    sl = torch.zeros(B, dtype=torch.int32, device="cuda")
    one = torch.ones(B, dtype=torch.int32, device="cuda")
    kn, vn = (torch.zeros(B, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(B, Hq, D, dtype=torch.bfloat16, device="cuda")
    o = torch.zeros_like(q)
    ws = torch.zeros(ta.decode_paged_workspace_bytes(B, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    pws = torch.empty(ta.kv_pages_workspace_bytes(P), dtype=torch.uint8, device="cuda")

    def step():
        ta.kv_pages_reserve(table, sl, one, refs, S, workspace=pws)
        ta.kv_append_paged(kp, vp, kn, vn, table, sl)
        ta.decode_gqa_paged(q, kp, vp, table, sl, o=o, window=window, sinks=sinks, workspace=ws)
        ta.kv_pages_free(table, sl, refs, S, window, sinks)

    def feed(t):
        kn.copy_(kv[0][:, :, t])
        vn.copy_(kv[1][:, :, t])
        q.copy_(qs[t])

    feed(0)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in range(1, steps):
        feed(t)
        graph.replay()
        if t % 13 == 0 or t > steps - 3:
            assert ta.device_status() == 0
            assert sl.tolist() == [t + 1] * B
            check("bf16", qs[t], [kv[0][b, :, :t + 1] for b in range(B)],
                  [kv[1][b, :, :t + 1] for b in range(B)], [t + 1] * B, o, window, sinks)
    assert int((refs > 0).sum()) <= B * (-(-window // S) + 1 + 1)


def test_prefill_append_fork_decode(ta):
    """A prompt through the windowed prefill in two parts, its K/V into pages, two
    forked samples, one token each: the decode agrees with the prefill's row."""
    Hq, Hkv, D, S, N, window, sinks = 8, 2, 128, 16, 333, 100, 4
    g = torch.Generator().manual_seed(8)
    q, k, v = (torch.randn(1, N, h, D, generator=g).bfloat16().cuda().transpose(1, 2) for h in (Hq, Hkv, Hkv))
    whole = ta.causal_gqa_window_fwd(q, k, v, window, sinks)
    cut = 200
    part = ta.causal_gqa_window_fwd(q[:, :, cut:], k, v, window, sinks)
    # the parts tile the queries differently; the same sums in another order
    A = v.double().abs().amax().item()
    assert (part.double() - whole[:, :, cut:].double()).abs().max() <= A * 2 * 2.0 ** -8
    B, P, M = 3, 64, 30
    kp, vp = empty_pool(P, Hkv, S, D, "bf16", "head")
    table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    sl = torch.zeros(B, dtype=torch.int32, device="cuda")
    n = torch.tensor([N - 1, 0, 0], dtype=torch.int32, device="cuda")
    ta.kv_pages_reserve(table, sl, n, refs, S)
    ta.kv_append_paged(kp, vp, k.repeat(B, 1, 1, 1), v.repeat(B, 1, 1, 1), table, sl, n)
    cs, cd = ta.kv_pages_fork(table, sl, refs, n.new_tensor([0, 0]), n.new_tensor([1, 2]), S)
    ta.kv_pages_copy(kp, vp, cs, cd)
    assert refs.max() == 3
    ta.kv_pages_reserve(table, sl, torch.ones_like(sl), refs, S)
    last = [x[:, :, -1].expand(B, -1, -1).contiguous() for x in (k, v)]
    last[0][2] = 0                                # the third sample takes another token
    ta.kv_append_paged(kp, vp, last[0], last[1], table, sl)
    qd = q[:, :, -1].expand(B, -1, -1).contiguous()
    o = ta.decode_gqa_paged(qd, kp, vp, table, sl, window=window, sinks=sinks)
    assert ta.device_status() == 0
    k2 = k[0].cpu().clone()
    k2[:, -1] = 0
    check("bf16", qd, [k[0].cpu(), k[0].cpu(), k2], [v[0].cpu()] * 3, [N] * 3, o, window, sinks)
    assert torch.equal(o[0], o[1]) and not torch.equal(o[0], o[2])


def test_calls_on_two_streams_with_their_own_workspaces(ta):
    cases = [build_case("bf16", [900, 30], 4, 2, 128, 16, 0, 0, "head", 20 + i) for i in range(2)]
    want = [ta.decode_gqa_paged(*c[:5]) for c in cases]
    ws = [torch.zeros(ta.decode_paged_workspace_bytes(2, 4, 2, 128), dtype=torch.uint8, device="cuda")
          for _ in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(10):
        for i, (c, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                got[i].append(ta.decode_gqa_paged(*c[:5], workspace=ws[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i]) for i in range(2) for x in got[i])


@pytest.mark.parametrize("dt,Hq,Hkv,D,lens", [
    ("bf16", 32, 8, 128, [700, 0, 128] + [0] * 60),
    ("f16", 27, 3, 64, [0] * 400 + [5] + [0] * 400 + [300, 40]),     # more slots than CTAs
    ("bf16", 4, 4, 128, [0] * 7),
])
def test_idle_slots_write_zeros_and_nothing_else(ta, dt, Hq, Hkv, D, lens):
    q, kp, vp, table, sl, ks, vs = build_case(dt, lens, Hq, Hkv, D, 16, 0, 0, "head", 11)
    wide = torch.full((len(lens), Hq + 2, D), 5.0, dtype=DT[dt], device="cuda")
    ta.decode_gqa_paged(q, kp, vp, table, sl, o=wide[:, 1:-1])
    assert ta.device_status() == 0
    check(dt, q, ks, vs, lens, wide[:, 1:-1], 0, 0)
    assert (wide[:, 0] == 5).all() and (wide[:, -1] == 5).all()


def graph_us(fn, n=40):
    """Best of several replays of n calls, per call."""
    fn()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(n):
            fn()
    best = 1e9
    for _ in range(10):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        g.replay()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) / n * 1e3)
    return best


def decode_us(ta, lens, Hq=32, Hkv=8, D=128):
    q, kp, vp, table, sl, _, _ = build_case("bf16", lens, Hq, Hkv, D, 16, 0, 0, "head", 13)
    ws = torch.zeros(ta.decode_paged_workspace_bytes(len(lens), Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    o = torch.empty_like(q)
    return graph_us(lambda: ta.decode_gqa_paged(q, kp, vp, table, sl, o=o, workspace=ws))


def test_idle_slots_cost_little(ta):
    """60 idle slots are 0.5 MB of zeros, under a microsecond at the HBM rate, beside
    a call of 8 to 9: the limit leaves them four."""
    busy = [700, 300, 512, 128]
    assert decode_us(ta, busy + [0] * 60) < 1.5 * decode_us(ta, busy)


@pytest.mark.parametrize("a,b,Hq,Hkv", [([2048], [200] * 24, 32, 8), ([2000], [300] * 100, 16, 2)])
def test_one_longer_sequence_does_not_hold_up_the_others(ta, a, b, Hq, Hkv):
    """One call over both batches takes no longer than a call for each of them."""
    assert decode_us(ta, a + b, Hq, Hkv) < decode_us(ta, a, Hq, Hkv) + decode_us(ta, b, Hq, Hkv)


@pytest.mark.parametrize("lens,Hq,Hkv", [([2000] + [300] * 12, 16, 8), ([170 + i * 830 // 39 for i in range(40)], 8, 2),
                                         ([2000] + [500] * 15, 8, 8), ([2048] + [200] * 24, 8, 8)])
def test_decode_paged_ranges_of_mixed_units(ta, lens, Hq, Hkv):
    q, kp, vp, table, sl, ks, vs = build_case("bf16", lens, Hq, Hkv, 128, 16, 0, 0, "head", 17)
    o = ta.decode_gqa_paged(q, kp, vp, table, sl)
    assert ta.device_status() == 0
    check("bf16", q, ks, vs, lens, o, 0, 0)


@pytest.mark.parametrize("P", [300, 30000])         # one CTA, a cluster
@pytest.mark.parametrize("what", ["tail", "full", "two targets"])
def test_fork_refuses_pages_counted_too_low_every_time(ta, P, what):
    """A page that a source and a target row name but that is counted once is let go
    by the target: it must not be handed out, whichever thread comes first."""
    S, M, B = 8, 40, 6
    table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    n = [20 * 8 + 3, 0, 0, 0, 9 * 8, 0]
    table[0, :21] = torch.arange(21, dtype=torch.int32)
    table[4, :9] = torch.arange(50, 59, dtype=torch.int32)
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    refs[:21] = 1
    refs[50:59] = 1
    if what == "tail":                               # row 0's last page, partly filled
        table[1, 2] = 20
    elif what == "full":
        table[1, 0] = 7
    else:
        table[1, 5] = table[2, 39] = 55
    sl = torch.tensor(n, dtype=torch.int32, device="cuda")
    src, dst = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 4], [1, 2]))
    before = [x.clone() for x in (table, refs, sl)]
    for _ in range(50):
        cs, cd = ta.kv_pages_fork(table, sl, refs, src, dst, S)
        assert ta.device_status() == 6
        assert cs.tolist() == cd.tolist() == [-1, -1]
        assert all(torch.equal(a, b) for a, b in zip(before, (table, refs, sl)))

"""Rotary positions, appends of packed rows, the 4-bit paged cache and attention
over packed sequences, against 64-bit forms."""
import pytest
import torch

from tests.paged_ref import DT, attend, bound, visible
from tests.q4_ref import layout, pack, quantise, rates, rotate, rotate_bound, unpack

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ta():
    from transformer_attention_tcgen05_gb300.build import build
    build()
    import transformer_attention_tcgen05_gb300 as ta
    torch.cuda.set_device(0)
    return ta


def randn(g, *shape):
    return torch.randn(*shape, generator=g)


def starts(lens, gaps=None):
    return torch.tensor([0] + list(lens)).cumsum(0).int().cuda()


# ------------------------------------------------------------------- rope

def rope_case(ta, dt, x, pos, rot, inter, inverse, m, kw, o=None):
    f = rates(rot, **kw)
    y = ta.rope_fwd(x, ta.rope_frequencies(rot, **kw), pos, interleaved=inter, inverse=inverse, mscale=m, o=o)
    assert ta.device_status() == 0
    return f, y


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("B,H,N,D,rot,inter,order", [
    (1, 1, 1, 32, 16, False, "head"), (2, 3, 5, 64, 64, False, "head"), (2, 5, 33, 64, 32, True, "token"),
    (1, 40, 1, 128, 128, False, "token"), (3, 2, 130, 128, 48, False, "token"), (1, 7, 257, 32, 32, True, "head"),
    (2, 1, 1000, 128, 128, True, "head"), (1, 64, 70, 128, 112, False, "head"),
])
def test_rope(ta, dt, B, H, N, D, rot, inter, order):
    g = torch.Generator().manual_seed(B * 100 + H)
    x = randn(g, B, N, H, D).to(DT[dt]).cuda().transpose(1, 2) if order == "token" else \
        randn(g, B, H, N, D).to(DT[dt]).cuda()
    pos = torch.randint(-5000, 2 ** 20, (B, N), generator=g).int()
    pos[0, 0] = 2 ** 31 - 1
    for inverse, m, kw in ((False, 1.0, {}), (True, 1.1386, dict(scaling="by_parts", factor=4.0, original_len=4096))):
        f, y = rope_case(ta, dt, x, pos.cuda(), rot, inter, inverse, m, kw)
        want = rotate(x.double().cpu(), pos[:, None], f, inter, inverse, m)
        lim = rotate_bound(dt, x.cpu(), want, f, inter, m)
        assert y.is_contiguous() and ((y.double().cpu() - want).abs() <= lim).all()
        assert torch.equal(y[..., rot:], x[..., rot:])


def test_rope_packed_rows_shared_positions_in_place_and_views(ta):
    g = torch.Generator().manual_seed(1)
    qkv = randn(g, 77, 12, 64).bfloat16().cuda()
    pos = torch.arange(77).int().cuda()
    f, f64 = ta.rope_frequencies(64), rates(64)
    x = qkv[:, 2:7].cpu()
    want = rotate(x.double(), pos.cpu()[:, None], f64)
    lim = rotate_bound("bf16", x, want, f64, False, 1.0)
    y = ta.rope_fwd(qkv[:, 2:7], f, pos)
    assert ((y.double().cpu() - want).abs() <= lim).all()
    before = qkv.clone()
    assert ta.rope_fwd(qkv[:, 2:7], f, pos, o=qkv[:, 2:7]).data_ptr() == qkv[:, 2:7].data_ptr()     # in place
    assert torch.equal(qkv[:, 2:7], y) and torch.equal(qkv[:, :2], before[:, :2])
    assert torch.equal(qkv[:, 7:], before[:, 7:])
    # positions shared by the batches of a 4-D tensor, and an output view
    x4 = randn(g, 3, 4, 77, 64).cuda()
    wide = torch.full((3, 4, 80, 64), 7.0).cuda()
    ta.rope_fwd(x4, f, pos, o=wide[:, :, 1:78])
    again = ta.rope_fwd(x4, f, pos[None].expand(3, 77).contiguous())
    assert torch.equal(wide[:, :, 1:78], again) and (wide[:, :, 0] == 7).all() and (wide[:, :, 78:] == 7).all()


@pytest.mark.parametrize("inter", [False, True])
def test_rope_inverse_is_the_gradient(ta, inter):
    """<dy, rope(x + h e)> - <dy, rope(x - h e)> over 2 h against the inverse call."""
    g = torch.Generator().manual_seed(2)
    x, dy, e = (randn(g, 1, 3, 9, 64).cuda() for _ in range(3))
    pos, f = torch.arange(9).int().cuda() * 1001, ta.rope_frequencies(32)
    dx = ta.rope_fwd(dy, f, pos, interleaved=inter, inverse=True, mscale=1.25)
    h = 0.5                                              # the call is linear: any step is exact but for roundings
    up, dn = (ta.rope_fwd(x + s * h * e, f, pos, interleaved=inter, mscale=1.25) for s in (1, -1))
    num = ((up - dn).double() * dy.double()).sum() / (2 * h)
    size = (e.double().norm() * dy.double().norm() + x.double().norm() * dy.double().norm()) * 2
    assert abs(num - (dx.double() * e.double()).sum()) <= size * 2.0 ** -20


def test_rope_nan_stays_in_its_pair(ta):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16).cuda()
    x[1, 1, 5] = float("nan")
    y = ta.rope_fwd(x, ta.rope_frequencies(32), torch.arange(4).int().cuda())
    assert torch.nonzero(torch.isnan(y.float())).tolist() == [[1, 1, 5], [1, 1, 21]]


# ----------------------------------------------------------------- appends

class Cache:
    """A pool of scattered pages in which every sequence has room for its tokens."""

    def __init__(self, lens, news, S, seed, spare=3):
        g = torch.Generator().manual_seed(seed)
        self.S, self.lens, self.news = S, list(lens), list(news)
        need = [-(-(n + m) // S) for n, m in zip(lens, news)]
        self.P, self.M = sum(need) + spare, max(max(need), 1) + 1
        perm = torch.randperm(self.P, generator=g).tolist()
        self.table = torch.full((len(lens), self.M), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            for i in range(n):
                self.table[b, i] = perm.pop()
        self.dev = self.table.cuda()
        self.sl = torch.tensor(self.lens).int().cuda()

    def rows(self, b, lo, hi):
        """(page, row) of positions [lo, hi) of sequence b."""
        p = torch.arange(lo, hi)
        return self.table[b, p // self.S].long(), p % self.S


def new_rows(g, news, Hq, Hkv, D, dt, lead=0, tail=0):
    """Column blocks of a packed projection [N, Hq + 2 Hkv, D], with rows before and
    behind the sequences'."""
    N = lead + sum(news) + tail
    x = randn(g, N, Hq + 2 * Hkv, D).to(DT[dt]).cuda()
    cu = (torch.tensor([0] + list(news)).cumsum(0) + lead).int().cuda()
    return x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], cu


@pytest.mark.parametrize("dt,lens,news,Hq,Hkv,D,S,rot,inter,order", [
    ("bf16", [0], [1], 1, 1, 64, 8, 64, False, "head"),
    ("bf16", [5, 0, 100, 16], [1, 1, 1, 1], 8, 2, 128, 16, 128, False, "head"),
    ("f16", [5, 0, 33, 16], [7, 0, 150, 1], 6, 2, 64, 24, 32, True, "token"),
    ("f32", [1, 2, 3], [40, 1, 0], 3, 3, 32, 8, 16, False, "head"),
    ("bf16", [0, 17], [1000, 333], 5, 5, 128, 48, 48, False, "token"),
    ("f32", [0, 250], [300, 2], 16, 2, 128, 64, 128, True, "head"),
])
@pytest.mark.parametrize("with_q", [True, False])
def test_append_paged_rope(ta, dt, lens, news, Hq, Hkv, D, S, rot, inter, order, with_q):
    g = torch.Generator().manual_seed(len(lens))
    c = Cache(lens, news, S, 3)
    one = all(n == 1 for n in news)
    lead, tail = (0, 0) if one else (3, 70)
    q, kn, vn, cu = new_rows(g, news, Hq, Hkv, D, dt, lead, tail)
    shape = (c.P, S, Hkv, D) if order == "token" else (c.P, Hkv, S, D)
    kp, vp = (randn(g, *shape).to(DT[dt]).cuda() for _ in "kv")
    if order == "token":
        kp, vp = kp.transpose(1, 2), vp.transpose(1, 2)
    k0, v0 = kp.clone(), vp.clone()
    qo = torch.full((len(q), Hq, D), 9.0, dtype=DT[dt]).cuda()
    f, f64 = ta.rope_frequencies(rot, theta=500000.0), rates(rot, theta=500000.0)
    r = ta.kv_append_paged_rope(kp, vp, kn, vn, c.dev, c.sl, f, cu_new=None if one else cu,
                                q=q if with_q else None, q_out=qo if with_q else None, interleaved=inter,
                                mscale=1.25)
    assert ta.device_status() == 0 and (r is qo if with_q else r is None)
    assert c.sl.tolist() == [n + m for n, m in zip(lens, news)]
    for b, (n, m) in enumerate(zip(lens, news)):
        at = slice(cu[b], cu[b + 1])
        pos = torch.arange(n, n + m)[:, None]
        pages, rows = c.rows(b, n, n + m)
        assert torch.equal(vp[pages, :, rows], vn[at])
        pairs = [(kn[at], kp[pages, :, rows])] + ([(q[at], qo[at])] if with_q else [])
        for x, y in pairs:
            x, y = x.cpu(), y.double().cpu()
            want = rotate(x.double(), pos, f64, inter, False, 1.25)
            assert ((y - want).abs() <= rotate_bound(dt, x, want, f64, inter, 1.25)).all()
        k0[pages, :, rows], v0[pages, :, rows] = kp[pages, :, rows], vp[pages, :, rows]
    assert torch.equal(k0, kp) and torch.equal(v0, vp)               # nothing else was touched
    assert (qo[:lead] == 9).all() and (qo[len(q) - tail:] == 9).all()


def test_append_rotates_queries_in_place_and_agrees_with_rope(ta):
    g = torch.Generator().manual_seed(8)
    c = Cache([4, 30], [9, 40], 16, 4)
    q, kn, vn, cu = new_rows(g, c.news, 4, 2, 128, "bf16")
    kp, vp = (torch.zeros(c.P, 2, 16, 128, dtype=torch.bfloat16).cuda() for _ in "kv")
    f = ta.rope_frequencies(128)
    pos = torch.cat([torch.arange(4, 13), torch.arange(30, 70)]).int().cuda()
    want = ta.rope_fwd(q, f, pos)
    ta.kv_append_paged_rope(kp, vp, kn, vn, c.dev, c.sl, f, cu_new=cu, q=q, q_out=q, advance=False)
    assert torch.equal(q, want) and c.sl.tolist() == [4, 30]
    k = ta.rope_fwd(kn, f, pos)
    for b in range(2):
        pages, rows = c.rows(b, c.lens[b], c.lens[b] + c.news[b])
        assert torch.equal(kp[pages, :, rows], k[cu[b]:cu[b + 1]])


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("one", [False, True])
def test_append_requests_that_do_not_fit_are_reported_per_sequence(ta, q4, one):
    """A bad page, a length outside the table, a table that is too short: the other
    sequences are served, what those hold stays."""
    g = torch.Generator().manual_seed(9)
    news = [1] * 5 if one else [3, 4, 5, 6, 2]
    c = Cache([10, 20, 16, 7, 30], news, 8, 5)
    c.dev[1, 2] = c.P                                     # its page is none of the pool
    c.sl[2] = c.M * 8                                     # no room behind it
    c.sl[3] = -2
    q, kn, vn, cu = new_rows(g, news, 2, 2, 64, "bf16")
    qo = torch.full((len(q), 2, 64), 9.0, dtype=torch.bfloat16).cuda()
    f = ta.rope_frequencies(64)
    kp, vp = (torch.full((c.P, 2, 8, 64), 5.0, dtype=torch.bfloat16).cuda() for _ in "kv")
    pages = torch.full((c.P, 2, 8, 72), 5, dtype=torch.uint8).cuda()
    before = c.sl.tolist()
    cu_arg = None if one else cu
    if q4:
        ta.kv_append_paged_q4(pages, kn, vn, c.dev, c.sl, f, cu_new=cu_arg, q=q, q_out=qo)
    else:
        ta.kv_append_paged_rope(kp, vp, kn, vn, c.dev, c.sl, f, cu_new=cu_arg, q=q, q_out=qo)
    assert ta.device_status() == 6
    assert c.sl.tolist() == [before[0] + news[0], before[1], before[2], before[3], before[4] + news[4]]
    touched = torch.zeros(c.P, 8, dtype=torch.bool)
    for b in (0, 4):
        touched[c.rows(b, c.lens[b], c.lens[b] + news[b])] = True
        assert not (qo[cu[b]:cu[b + 1]] == 9).all(-1).any()
    for b in (2, 3):
        assert (qo[cu[b]:cu[b + 1]] == 9).all()
    # of sequence 1 the tokens on its other pages may be written
    for t in range(20, 20 + news[1]):
        if t // 8 != 2:
            touched[c.table[1, t // 8], t % 8] = True
    x = (pages == 5).all(-1) if q4 else (kp == 5).all(-1) & (vp == 5).all(-1)
    assert torch.equal(x.all(1).cpu(), ~touched)


def test_append_starts_that_do_not_rise_are_reported(ta):
    g = torch.Generator().manual_seed(10)
    c = Cache([0, 0, 0], [4, 4, 4], 8, 6)
    q, kn, vn, _ = new_rows(g, [12], 1, 1, 64, "f16")
    kp, vp = (torch.zeros(c.P, 1, 8, 64, dtype=torch.float16).cuda() for _ in "kv")
    cu = torch.tensor([0, 4, 3, 13]).int().cuda()         # the second falls, the third passes the rows
    ta.kv_append_paged_rope(kp, vp, kn, vn, c.dev, c.sl, ta.rope_frequencies(64), cu_new=cu)
    assert ta.device_status() == 6 and c.sl.tolist() == [4, 0, 0]
    assert int((vp != 0).any(-1).sum()) == 4


@pytest.mark.parametrize("q4", [False, True])
def test_append_sequences_that_overlap_stay_in_the_table(ta, q4):
    """Starts that fall let others claim the same rows: the call reports it, and what it
    writes lies on pages of the sequences that rise."""
    g = torch.Generator().manual_seed(41)
    c = Cache([0, 0, 30, 0, 0], [32] * 5, 8, 6)
    q, kn, vn, _ = new_rows(g, [32], 1, 1, 64, "bf16")
    cu = torch.tensor([0, 32, 0, 2, 1, 32]).int().cuda()
    f = ta.rope_frequencies(64)
    kp, vp = (torch.full((c.P, 1, 8, 64), 5.0, dtype=torch.bfloat16).cuda() for _ in "kv")
    pages = torch.full((c.P, 1, 8, 72), 5, dtype=torch.uint8).cuda()
    if q4:
        ta.kv_append_paged_q4(pages, kn, vn, c.dev, c.sl, f, cu_new=cu)
    else:
        ta.kv_append_paged_rope(kp, vp, kn, vn, c.dev, c.sl, f, cu_new=cu)
    assert ta.device_status() == 6
    x = (pages == 5).all(-1) if q4 else (kp == 5).all(-1) & (vp == 5).all(-1)
    own = torch.zeros(c.P, dtype=torch.bool)
    own[[int(i) for b in (0, 2, 4) for i in c.table[b] if i < c.P]] = True
    assert x.all(-1).all(-1).cpu()[~own].all()
    assert c.sl.tolist()[1] == 0 and c.sl.tolist()[3] == 0


# ------------------------------------------------------------- 4-bit cache

@pytest.mark.parametrize("dt,lens,news,Hkv,D,S", [
    ("bf16", [0], [1], 1, 64, 8), ("bf16", [5, 0, 100], [1, 1, 1], 4, 128, 16),
    ("f16", [5, 0, 33, 16], [7, 0, 150, 1], 2, 64, 24), ("bf16", [0, 17], [700, 33], 3, 128, 48),
    ("f16", [0, 250], [300, 2], 8, 128, 64),
])
@pytest.mark.parametrize("heads_first", [True, False])
def test_append_q4_bytes_and_gather(ta, dt, lens, news, Hkv, D, S, heads_first):
    """Without a rotation every byte is known; the reader gives back what it stands for."""
    g = torch.Generator().manual_seed(len(lens) + D)
    c = Cache(lens, news, S, 7)
    lead = 0 if all(n == 1 for n in news) else 2
    q, kn, vn, cu = new_rows(g, news, 2, Hkv, D, dt, lead, lead)
    kn[::7] *= 30
    vn[1::5, :, 3] = 0
    kn[-lead - 1, 0, :32] = 0
    vn[-lead - 1, 0, 32:64] = -1.5
    R = D + D // 8
    pages = torch.randint(0, 256, (c.P, Hkv, S, R), generator=g, dtype=torch.uint8).cuda()
    if not heads_first:                                   # pages inside heads: [Hkv, P, S, R]
        pages = pages.transpose(0, 1).contiguous().transpose(0, 1)
    want = pages.clone()
    qo = ta.kv_append_paged_q4(pages, kn, vn, c.dev, c.sl, cu_new=cu if lead else None, q=q)
    assert ta.device_status() == 0
    assert c.sl.tolist() == [n + m for n, m in zip(lens, news)]
    for b, (n, m) in enumerate(zip(lens, news)):
        at = slice(cu[b], cu[b + 1])
        p, r = c.rows(b, n, n + m)
        want[p, :, r] = pack(kn[at].float().cpu(), vn[at].float().cpu(), dt).cuda()
        assert torch.equal(qo[at], q[at])
    assert torch.equal(pages, want)
    # the new rows alone, behind an offset, and rows around them left as they are
    total = sum(news) + 9
    k, v = (torch.full((total, 2 * Hkv, D), 3.0, dtype=DT[dt]).cuda() for _ in "kv")
    start = torch.tensor(lens).int().cuda()
    cu2 = starts(news) + 4
    out = ta.kv_gather_paged_q4(pages, c.dev, cu2, k[:, Hkv:], v[:, :Hkv], start=start)
    assert ta.device_status() == 0 and out[0].data_ptr() == k[:, Hkv:].data_ptr()
    for b, (n, m) in enumerate(zip(lens, news)):
        p, r = c.rows(b, n, n + m)
        x, y = unpack(want[p, :, r].cpu(), dt)
        at = slice(cu2[b], cu2[b + 1])
        assert torch.equal(k[at, Hkv:].cpu(), x.to(DT[dt])) and torch.equal(v[at, :Hkv].cpu(), y.to(DT[dt]))
    for x in (k[:4], k[total - 5:], v[:4], v[total - 5:], k[:, :Hkv], v[:, Hkv:]):
        assert (x == 3).all()


@pytest.mark.parametrize("dt,D,rot,inter", [("bf16", 128, 128, False), ("f16", 64, 32, True), ("bf16", 64, 64, False)])
def test_append_q4_rotated_keys(ta, dt, D, rot, inter):
    """Rotated in fp32 before the codes are made: within half a step and what the
    rotation's error adds."""
    g = torch.Generator().manual_seed(11)
    c = Cache([1000, 0], [50, 30], 16, 8)
    q, kn, vn, cu = new_rows(g, c.news, 3, 2, D, dt)
    pages = torch.zeros(c.P, 2, 16, D + D // 8, dtype=torch.uint8).cuda()
    f, f64 = ta.rope_frequencies(rot), rates(rot)
    qo = ta.kv_append_paged_q4(pages, kn, vn, c.dev, c.sl, f, cu_new=cu, q=q, interleaved=inter, mscale=1.5)
    half = torch.finfo(DT[dt]).eps / 2
    for b, (n, m) in enumerate(zip(c.lens, c.news)):
        at = slice(cu[b], cu[b + 1])
        pos = torch.arange(n, n + m)[:, None]
        p, r = c.rows(b, n, n + m)
        rows = pages[p, :, r].cpu()
        got, v = unpack(rows, dt)
        want = rotate(kn[at].double().cpu(), pos, f64, inter, False, 1.5)
        s = rows[..., D:D + D // 16].contiguous().view(DT[dt]).double()
        top = want.unflatten(-1, (-1, 32))
        ref = torch.where(top.amax(-1) >= -top.amin(-1), top.amax(-1), top.amin(-1))
        err = 2.0 ** -20 * 1.5 * kn[at].double().abs().amax().cpu()
        assert ((s + ref / 8).abs() <= half * ref.abs() / 8 + err).all()
        step = s.abs().repeat_interleave(32, -1)
        n_exact = want / s.repeat_interleave(32, -1) + 8
        inside = (n_exact > 0.5) & (n_exact < 14.5)
        assert ((got - want).abs() <= step * 0.5 + err)[inside].all()
        edge = torch.where(n_exact <= 0.5, -8.0, 7.0) * s.repeat_interleave(32, -1)
        assert ((got - edge).abs() <= step + err)[~inside].all()
        wq = rotate(q[at].double().cpu(), pos, f64, inter, False, 1.5)
        assert ((qo[at].double().cpu() - wq).abs() <= rotate_bound(dt, q[at].cpu(), wq, f64, inter, 1.5)).all()
        n_v, s_v = quantise(vn[at].float().cpu(), dt)
        assert torch.equal(v, (n_v - 8).double() * s_v.double().repeat_interleave(32, -1))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_append_q4_extreme_groups(ta, dt):
    """Infinite, NaN, vanishing and huge values spoil or vanish with their group alone."""
    top = float(torch.finfo(DT[dt]).max)
    tiny = float(torch.finfo(DT[dt]).tiny)
    x = torch.ones(6, 1, 128)
    x[0, 0, 40], x[1, 0, 70], x[2, 0, 100] = float("inf"), float("nan"), float("-inf")
    x[3, 0, :32] = tiny * torch.arange(1, 33) / 64        # subnormal values
    x[4, 0, ::2], x[4, 0, 1::2] = top, -top
    x[5] = 0
    x = x.to(DT[dt])
    c = Cache([0], [6], 8, 9)
    pages = torch.zeros(c.P, 1, 8, 144, dtype=torch.uint8).cuda()
    kn = x.cuda()
    ta.kv_append_paged_q4(pages, kn, kn.clone(), c.dev, c.sl, cu_new=starts([6]))
    k, v = (torch.zeros(6, 1, 128, dtype=DT[dt]).cuda() for _ in "kv")
    ta.kv_gather_paged_q4(pages, c.dev, starts([6]), k, v)
    assert ta.device_status() == 0
    for got in (k.float().cpu()[:, 0], v.float().cpu()[:, 0]):
        spoiled = torch.isnan(got)
        want = torch.zeros(6, 128, dtype=torch.bool)
        want[0, 32:64] = want[1, 64:96] = want[2, 96:] = True
        assert torch.equal(spoiled, want)
        n, s = quantise(x[:, 0], dt)
        ref = ((n - 8).float() * s.float().repeat_interleave(32, -1)).to(DT[dt]).float()
        assert torch.equal(got[~want], ref[~want])
        assert (got[4].abs() >= 0.8 * top).all() and (got[5] == 0).all()


def test_gather_reports_pages_that_are_none(ta):
    c = Cache([20, 9], [0, 0], 8, 10)
    c.dev[0, 1] = -1
    pages = torch.randint(0, 256, (c.P, 1, 8, 72), dtype=torch.uint8).cuda()
    pages[..., 64:] = torch.ones(c.P, 1, 8, 4, dtype=torch.bfloat16).view(torch.uint8).cuda()
    k, v = (torch.full((31, 1, 64), 9.0, dtype=torch.bfloat16).cuda() for _ in "kv")
    ta.kv_gather_paged_q4(pages, c.dev, torch.tensor([0, 20, 29]).int().cuda(), k, v)
    assert ta.device_status() == 6
    left = (k == 9).all(-1)[:, 0].cpu()
    assert left[8:16].all() and left[29:].all() and not left[:8].any() and not left[16:29].any()
    ta.kv_gather_paged_q4(pages, c.dev, torch.tensor([0, 20, 32]).int().cuda(), k, v,
                          start=torch.tensor([0, 0]).int().cuda())
    assert ta.device_status() == 6
    ta.kv_gather_paged_q4(pages, c.dev, torch.tensor([0, 2, 4]).int().cuda(), k, v,
                          start=torch.tensor([-1, c.M * 8 - 1]).int().cuda())
    assert ta.device_status() == 6


@pytest.mark.parametrize("layers", [0, 3])
@pytest.mark.parametrize("D,S,Hkv,split", [(64, 8, 1, False), (128, 16, 3, False), (128, 48, 2, True)])
def test_copy_q4(ta, layers, D, S, Hkv, split):
    g = torch.Generator().manual_seed(12)
    shape = ((layers,) if layers else ()) + (9, Hkv, S, D + D // 8)
    pages = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8).cuda()
    if split:                                             # heads outside pages
        pages = pages.transpose(-4, -3).contiguous().transpose(-4, -3)
    want = pages.clone()
    src = torch.tensor([0, 3, -1, 5, 7]).int().cuda()
    dst = torch.tensor([8, 1, -1, 2, 4]).int().cuda()
    for a, b in ((0, 8), (3, 1), (5, 2)):
        want[..., b, :, :, :] = pages[..., a, :, :, :]
    ta.kv_pages_copy_q4(pages, src, dst, count=torch.tensor([4]).int().cuda())
    assert ta.device_status() == 0 and torch.equal(pages, want)
    ta.kv_pages_copy_q4(pages, torch.tensor([9]).int().cuda(), torch.tensor([0]).int().cuda())
    assert ta.device_status() == 6 and torch.equal(pages, want)


def build_q4(dt, lens, Hq, Hkv, D, S, window, sinks, seed, spread=0.0, spare=4):
    """Pages whose visible rows are known and whose other bytes are all ones (NaN scales)."""
    g = torch.Generator().manual_seed(seed)
    c = Cache(lens, [0] * len(lens), S, seed, spare)
    R = D + D // 8
    pages = torch.full((c.P, Hkv, S, R), 255, dtype=torch.uint8)
    q = randn(g, len(lens), Hq, D).to(DT[dt])
    ks, vs = [], []
    for b, n in enumerate(lens):
        size = torch.exp(spread * randn(g, Hkv, n, 1))
        rows = pack(randn(g, Hkv, n, D), randn(g, Hkv, n, D) * size, dt)
        k, v = unpack(rows, dt)
        ks.append(k)
        vs.append(v)
        see = visible(n, [n - 1], window, sinks)[0] if n else torch.zeros(0, dtype=torch.bool)
        for i in range(-(-n // S)):
            on = torch.nonzero(see[i * S:(i + 1) * S])[:, 0]
            if len(on) == 0:
                c.table[b, i] = -1                        # pages without a visible row may be gone
                continue
            pages[c.table[b, i]][:, on] = rows[:, i * S:(i + 1) * S][:, on]
    return q.cuda(), pages.cuda(), c.table.cuda(), c.sl, ks, vs


def check_q4(dt, q, ks, vs, lens, o, window, sinks, only=None, scale=None):
    """On top of bound(): scores are sums of (code + 16 or 256) q scaled by s (at most
    3 roundings of 2^-22 of the largest partial sum per group); a weight times its
    value's scale is rounded to f16 (2^-11, below 2^-14 of the largest in steps of
    2^-25); the sums of weights times (code + 256) are rounded at 2^-23 of themselves,
    one rounding per 16 positions of a warp (64 here at most, in both signs)."""
    B, Hq, D = q.shape
    sc = 1 / D ** 0.5 if scale is None else scale
    for b, n in enumerate(lens):
        if only is not None and b not in only:
            continue
        if n == 0:
            assert (o[b] == 0).all()
            continue
        Hkv = ks[b].shape[0]
        G = Hq // Hkv
        see = visible(n, [n - 1], window, sinks)
        on = see[0]
        for hk in range(Hkv):
            qq = q[b, hk * G:(hk + 1) * G].double().cpu()
            k, v = ks[b][hk], vs[b][hk]
            ref, A, E, s1 = attend(qq, k, v, see.expand(G, n), scale=sc)
            sk = k[on].abs().unflatten(-1, (-1, 32)).amax(-1) / 8     # |s| of K (its extreme value is 8 s)
            sv = v[on].abs().unflatten(-1, (-1, 32)).amax(-1) / 8
            E = E + (3 * 2.0 ** -22 * 272 * sc * (qq.abs().unflatten(-1, (-1, 32)).sum(-1) @ sk.T)).amax(-1, keepdim=True)
            p = torch.softmax(qq @ k[on].T * sc, -1)
            Sv = (p @ sv).repeat_interleave(32, -1)       # mean scale of a group's values
            top = (p * sv.amax(-1)).amax(-1, keepdim=True)
            lim = bound(dt, ref, A, E, s1, n, 2.0 ** -11) + Sv * 272 * 2.0 ** -23 * 128 + int(on.sum()) * 2.0 ** -22 * top
            got = o[b, hk * G:(hk + 1) * G].double().cpu()
            bad = ~((got - ref).abs() <= lim)
            assert not bad.any(), (b, hk, torch.nonzero(bad)[:4].tolist(), ((got - ref).abs() / lim).max().item())


Q4_CASES = [
    # dt, lens, Hq, Hkv, D, S, window, sinks
    ("bf16", [1], 1, 1, 64, 16, 0, 0),
    ("bf16", [0, 1, 31, 32, 33, 0], 4, 1, 128, 16, 0, 0),
    ("f16", [64, 5, 200], 8, 2, 64, 8, 0, 0),
    ("bf16", [127, 128, 129], 12, 4, 128, 48, 0, 0),               # pages end inside a chunk
    ("f16", [100, 700], 14, 2, 128, 24, 0, 0),                     # 7 heads per KV head
    ("bf16", [333, 0, 65], 16, 2, 128, 64, 0, 0),
    ("bf16", [1000, 3], 32, 2, 64, 16, 0, 0),                      # 16 heads per KV head
    ("f16", [500, 77], 27, 3, 128, 32, 0, 0),                      # 9 heads per KV head
    ("bf16", [5000, 40, 1], 4, 2, 128, 128, 0, 0),                 # a unit over many CTAs
    ("f16", [20000], 8, 1, 64, 16, 0, 0),                          # one unit over all of them
    ("bf16", [300, 90, 5, 1], 4, 2, 128, 16, 64, 4),
    ("f16", [1000, 64, 65], 4, 1, 64, 32, 1, 0),                   # the newest token alone
    ("bf16", [1000, 100], 4, 1, 128, 16, 70, 40),                  # sinks past a chunk
    ("bf16", [200, 131, 129], 4, 1, 128, 8, 100, 30),              # sinks meet the window
    ("f16", [900, 20], 2, 1, 128, 16, 100000, 4),
    ("bf16", [900, 20], 2, 1, 64, 16, 16, 5000),
    ("bf16", [3, 9, 30] * 70, 2, 2, 64, 16, 0, 0),                 # more rows than threads
    ("bf16", [250, 7, 0, 100] * 25, 16, 8, 128, 16, 0, 0),         # units dealt out warp by warp
    ("f16", [250, 1, 0, 33, 64, 0] * 30, 12, 4, 64, 8, 0, 0),
    ("bf16", [1200, 300, 700] * 8, 8, 4, 64, 16, 0, 0),            # ranges that end inside units
    ("bf16", [3000, 1, 0, 40, 257, 256, 7], 8, 8, 64, 16, 0, 0),   # short units beside long ones
    ("bf16", [2000] * 6, 32, 4, 128, 16, 0, 0),
    ("bf16", [7000, 40, 0, 300, 1], 32, 2, 128, 16, 0, 0),         # 16 heads of 128 channels
    ("f16", [1500, 129] * 3, 48, 3, 128, 24, 500, 4),
]


@pytest.mark.parametrize("dt,lens,Hq,Hkv,D,S,window,sinks", Q4_CASES)
def test_decode_q4_parity(ta, dt, lens, Hq, Hkv, D, S, window, sinks):
    q, pages, table, sl, ks, vs = build_q4(dt, lens, Hq, Hkv, D, S, window, sinks, len(lens))
    n0 = ta.launch_count("decode_paged")
    o = ta.decode_gqa_paged_q4(q, pages, table, sl, window=window, sinks=sinks)
    assert ta.launch_count("decode_paged") == n0 + 1
    assert ta.device_status() == 0
    check_q4(dt, q, ks, vs, lens, o, window, sinks)


@pytest.mark.parametrize("dt,D,G", [("bf16", 128, 4), ("f16", 64, 9)])
def test_decode_q4_scales_of_very_different_size(ta, dt, D, G):
    """Values whose scales span many powers of two, and queries far from one."""
    lens = [700, 64, 3]
    q, pages, table, sl, ks, vs = build_q4(dt, lens, 2 * G, 2, D, 16, 0, 0, 13, spread=2.0)
    for mult in (1.0, 2.0 ** -10, 24.0):
        qm = (q.float() * mult).to(DT[dt])
        o = ta.decode_gqa_paged_q4(qm, pages, table, sl, scale=0.05 / mult)
        assert ta.device_status() == 0
        check_q4(dt, qm, ks, vs, lens, o, 0, 0, scale=0.05 / mult)


def test_decode_q4_values_of_zero_and_one_large_token(ta):
    """A token of zero values takes the weight; then one with a scale 2^40 times the others'."""
    g = torch.Generator().manual_seed(14)
    n, D = 200, 128
    k, v = randn(g, 1, n, D), randn(g, 1, n, D)
    q = randn(g, 1, 2, D).bfloat16()
    v[:, 50] = 0
    k[:, 50] = q[0, 0].float() * 4
    for big in (1.0, 2.0 ** 40):
        v2 = v.clone()
        v2[:, 120] *= big
        c = Cache([n], [0], 16, 15)
        rows = pack(k, v2, "bf16")
        pages = torch.zeros(c.P, 1, 16, 144, dtype=torch.uint8)
        p, r = c.rows(0, 0, n)
        pages[p, :, r] = rows.transpose(0, 1)
        kk, vv = unpack(rows, "bf16")
        o = ta.decode_gqa_paged_q4(q.cuda(), pages.cuda(), c.dev, c.sl)
        check_q4("bf16", q.cuda(), [kk], [vv], [n], o, 0, 0)


@pytest.mark.parametrize("where", ["k", "v"])
def test_decode_q4_nan_reaches_its_own_head_and_channels(ta, where):
    lens = [300, 300]
    q, pages, table, sl, ks, vs = build_q4("bf16", lens, 4, 2, 128, 16, 0, 0, 16)
    clean = ta.decode_gqa_paged_q4(q, pages, table, sl)
    at = 128 + 2 * 2 if where == "k" else 136 + 2 * 2             # the scale of channels 64 .. 95
    row = pages[table[1, 100 // 16], 1, 100 % 16]
    row[at:at + 2] = 255
    o = ta.decode_gqa_paged_q4(q, pages, table, sl)
    assert ta.device_status() == 0
    assert torch.equal(o[0], clean[0]) and torch.equal(o[1, :2], clean[1, :2])
    if where == "k":
        assert torch.isnan(o[1, 2:]).all()
    else:
        assert torch.isnan(o[1, 2:, 64:96]).all() and torch.isfinite(o[1, 2:, :64].float()).all()
    # behind the sequence's end or its window it changes nothing
    short = torch.tensor([300, 100]).int().cuda()
    a = ta.decode_gqa_paged_q4(q, pages, table, short)
    b = ta.decode_gqa_paged_q4(q, pages, table, sl, window=150, sinks=20)
    row[at:at + 2] = 0
    assert torch.equal(a, ta.decode_gqa_paged_q4(q, pages, table, short))
    assert torch.equal(b, ta.decode_gqa_paged_q4(q, pages, table, sl, window=150, sinks=20))
    assert torch.isfinite(a.float()).all() and torch.isfinite(b.float()).all()


def test_decode_q4_infinite_and_nan_queries(ta):
    lens = [100, 100]
    q, pages, table, sl, ks, vs = build_q4("bf16", lens, 4, 2, 64, 16, 0, 0, 17)
    clean = ta.decode_gqa_paged_q4(q, pages, table, sl)
    q[0, 1, 3], q[1, 2, 60] = float("inf"), float("nan")
    o = ta.decode_gqa_paged_q4(q, pages, table, sl)
    for b, h in ((0, 0), (0, 2), (0, 3), (1, 0), (1, 1), (1, 3)):
        assert torch.equal(o[b, h], clean[b, h])
    assert not torch.isfinite(o[0, 1].float()).any() and not torch.isfinite(o[1, 2].float()).any()


def test_decode_q4_bad_pages_and_lengths_are_reported_per_sequence(ta):
    lens = [900, 40, 33, 700, 64]
    q, pages, table, sl, ks, vs = build_q4("bf16", lens, 8, 2, 128, 16, 0, 0, 18)
    table[0, 20] = len(pages)
    table[2, 1] = -7
    sl[4] = table.shape[1] * 16 + 1
    ws = torch.zeros(ta.decode_paged_q4_workspace_bytes(5, 8, 2, 128), dtype=torch.uint8).cuda()
    o = torch.full_like(q, 3.0)
    ta.decode_gqa_paged_q4(q, pages, table, sl, o=o, workspace=ws)
    assert ta.device_status() == 6
    assert (o[0] == 3).all() and (o[2] == 3).all() and (o[4] == 3).all()
    check_q4("bf16", q, ks, vs, lens, o, 0, 0, only=[1, 3])
    # the workspace is as good as new
    sl[:] = torch.tensor([300, 40, 10, 700, 64]).int()
    o = ta.decode_gqa_paged_q4(q, pages, table, sl, workspace=ws)
    assert ta.device_status() == 0
    check_q4("bf16", q, [k[:, :n] for k, n in zip(ks, sl.tolist())], [v[:, :n] for v, n in zip(vs, sl.tolist())],
             sl.tolist(), o, 0, 0)


def test_decode_q4_repeats_and_one_workspace_serves_all_sizes(ta):
    cases = [("bf16", [3000, 200, 1], 8, 2, 128, 16), ("f16", [900] * 9, 18, 2, 64, 32), ("bf16", [64], 1, 1, 64, 8)]
    ws = torch.zeros(ta.decode_paged_q4_workspace_bytes(9, 18, 2, 128), dtype=torch.uint8).cuda()
    made = [(c, build_q4(*c, 0, 0, 19)) for c in cases]
    first = [ta.decode_gqa_paged_q4(*m[:4], workspace=ws) for _, m in made]
    for _ in range(4):
        for (c, m), x in zip(made, first):
            assert torch.equal(ta.decode_gqa_paged_q4(*m[:4], workspace=ws), x)
    for (c, m), x in zip(made, first):
        check_q4(c[0], m[0], m[4], m[5], c[1], x, 0, 0)
    assert ta.device_status() == 0


def test_decode_q4_strided_query_output_and_pages(ta):
    lens = [130, 77]
    q, pages, table, sl, ks, vs = build_q4("f16", lens, 6, 3, 64, 16, 0, 0, 20)
    wide = torch.zeros(2, 10, 64, dtype=torch.float16).cuda()
    wide[:, 2:8] = q
    out = torch.full((2, 9, 64), 5.0, dtype=torch.float16).cuda()
    heads = pages.transpose(0, 1).contiguous().transpose(0, 1)            # [Hkv, P, S, R] in memory
    ta.decode_gqa_paged_q4(wide[:, 2:8], heads, table, sl, o=out[:, 1:7])
    check_q4("f16", q, ks, vs, lens, out[:, 1:7], 0, 0)
    assert (out[:, 0] == 5).all() and (out[:, 7:] == 5).all()
    assert torch.equal(out[:, 1:7], ta.decode_gqa_paged_q4(q, pages, table, sl))


def test_q4_offsets_beyond_32_bits(ta):
    """Pages more than 2^32 bytes apart, from 34 000 pages of 8 heads x 128 tokens."""
    P, Hkv, S, D = 34000, 8, 128, 128
    pages = torch.empty(P, Hkv, S, 144, dtype=torch.uint8, device="cuda")
    assert P * Hkv * S * 144 > 2 ** 32
    lens = [300, 40]
    q, small, table, sl, ks, vs = build_q4("bf16", lens, 16, Hkv, D, S, 0, 0, 21)
    used = torch.unique(table[table >= 0]).tolist()
    far = table.clone()
    for i, p in enumerate(used):
        far[table == p] = P - 1 - i
        pages[P - 1 - i] = small[p]
    o = ta.decode_gqa_paged_q4(q, pages, far, sl)
    assert torch.equal(o, ta.decode_gqa_paged_q4(q, small, table, sl))
    x = torch.randn(2, Hkv, D).bfloat16().cuda()
    ta.kv_append_paged_q4(pages, x, x.clone(), far, sl)
    ta.kv_append_paged_q4(small, x, x.clone(), table, sl, advance=False)   # one further: then compare rows
    k, v = (torch.zeros(340, Hkv, D, dtype=torch.bfloat16).cuda() for _ in "kv")
    ta.kv_gather_paged_q4(pages, far, starts([300, 40]), k, v)
    for b, n in enumerate(lens):
        at = slice(300 * b, 300 * b + n)
        assert torch.equal(k[at].cpu(), ks[b].transpose(0, 1).bfloat16())
    ta.kv_pages_copy_q4(pages, torch.tensor([P - 1]).int().cuda(), torch.tensor([3]).int().cuda())
    assert torch.equal(pages[3], pages[P - 1]) and ta.device_status() == 0


# ------------------------------------------------------ packed attention

def packed(g, dt, lens, heads, D, lead=0, tail=0, cols=None):
    """Rows of all sequences, as a column block of a wider tensor, NaN around them."""
    N = lead + sum(lens) + tail
    x = torch.full((N, heads + 2, D), float("nan")).to(DT[dt])
    x[lead:N - tail, 1:1 + heads] = randn(g, sum(lens), heads, D).to(DT[dt])
    cu = (torch.tensor([0] + list(lens)).cumsum(0) + lead).int().cuda()
    return x.cuda()[:, 1:1 + heads], cu


def check_varlen(dt, q, k, v, cu_q, cu_k, o, window, sinks, rows=None):
    D, G = q.shape[2], q.shape[1] // k.shape[1]
    p_eps = torch.finfo(DT[dt]).eps / 2 if dt != "f32" and D != 32 else 0.0
    cq, ck = cu_q.tolist(), cu_k.tolist()
    for b in range(len(cq) - 1):
        n, t = cq[b + 1] - cq[b], ck[b + 1] - ck[b]
        if n == 0:
            continue
        at = list(range(n)) if rows is None or n <= len(rows) else sorted({r % n for r in rows})
        see = visible(t, [t - n + r for r in at], window, sinks)
        for h in range(q.shape[1]):
            x = q[cq[b]:cq[b + 1], h][at].double().cpu()
            ref, A, E, s1 = attend(x, k[ck[b]:ck[b + 1], h // G].double().cpu(), v[ck[b]:ck[b + 1], h // G].double().cpu(),
                                   see)
            got = o[cq[b]:cq[b + 1], h][at].double().cpu()
            lim = bound(dt, ref, A, E, s1, int(see.sum(1).max()), p_eps)
            bad = ~((got - ref).abs() <= lim)
            assert not bad.any(), (b, h, torch.nonzero(bad)[:5].tolist(), ((got - ref).abs() / lim).max().item())


ROWS = [0, 1, 31, 32, 63, 64, 126, 127, 128, 129, 255, 256, 257, 300, -1, -2]

VARLEN_CASES = [
    # dt, queries, keys before them, Hq, Hkv, D, window, sinks
    ("bf16", [1], [0], 1, 1, 64, 0, 0),
    ("bf16", [1, 0, 2, 130, 0], [0, 5, 0, 0, 0], 2, 1, 128, 0, 0),
    ("f16", [128, 129, 127, 256], [0, 0, 0, 0], 4, 2, 64, 0, 0),
    ("bf16", [300, 5, 77], [200, 1000, 0], 6, 2, 128, 0, 0),           # groups of 3: pairs of row tiles
    ("bf16", [1] * 70, list(range(0, 700, 10)), 4, 1, 128, 0, 0),      # single queries, more than 64 sequences
    ("f16", [17, 400, 3, 257], [90, 0, 500, 130], 5, 5, 64, 100, 3),
    ("bf16", [700, 129], [0, 600], 4, 2, 128, 128, 4),
    ("bf16", [513, 260], [300, 77], 2, 1, 64, 255, 130),               # sinks past a key tile
    ("bf16", [300, 300], [0, 9], 2, 2, 128, 1, 0),
    ("bf16", [150, 64], [0, 900], 2, 1, 128, 3, 1000),                 # sinks cover everything
    ("f16", [2000, 1, 900], [0, 0, 1100], 8, 8, 128, 0, 0),
    ("bf16", [40, 500, 1, 200] * 20, [0, 3, 300, 77] * 20, 2, 1, 64, 0, 0),
    ("f32", [1, 40, 0, 200, 33], [0, 0, 7, 0, 100], 4, 2, 64, 0, 0),
    ("f32", [65, 130], [200, 0], 3, 1, 128, 64, 70),
    ("f32", [5] * 80, [0] * 80, 2, 2, 32, 0, 0),
    ("bf16", [70, 31], [0, 40], 2, 1, 32, 33, 1),                      # D = 32: SIMT kernel
    ("f16", [90, 32, 200], [0, 1, 0], 4, 4, 32, 0, 0),
]


@pytest.mark.parametrize("dt,lens,past,Hq,Hkv,D,window,sinks", VARLEN_CASES)
def test_varlen_parity(ta, dt, lens, past, Hq, Hkv, D, window, sinks):
    g = torch.Generator().manual_seed(len(lens) + D)
    total = [n + m for n, m in zip(lens, past)]
    q, cu_q = packed(g, dt, lens, Hq, D, 2, 150)
    k, cu_k = packed(g, dt, total, Hkv, D, 5, 3)
    v, _ = packed(g, dt, total, Hkv, D, 5, 3)
    o = torch.full((len(q), Hq + 1, D), 7.0, dtype=DT[dt]).cuda()[:, 1:]
    fam = "simt" if dt == "f32" or D == 32 else "tc_flash"
    n0 = ta.launch_count(fam)
    assert ta.causal_gqa_varlen_fwd(q, k, v, cu_q, cu_k, window=window, sinks=sinks, o=o) is o
    assert ta.launch_count(fam) == n0 + 1 and ta.device_status() == 0
    check_varlen(dt, q, k, v, cu_q, cu_k, o, window, sinks, ROWS)
    assert (o[:2] == 7).all() and (o[len(q) - 150:] == 7).all()        # rows behind the last sequence


@pytest.mark.parametrize("dt,D,Hq", [("bf16", 128, 4), ("f16", 64, 3), ("f32", 64, 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 6)])
def test_varlen_agrees_with_one_sequence_at_a_time(ta, dt, D, Hq, window, sinks):
    """The same bits as the windowed entry gives for each sequence by itself, whatever
    (infinite, NaN) stands in the neighbours' rows."""
    g = torch.Generator().manual_seed(30)
    lens, past = [200, 1, 333, 90], [0, 400, 100, 39]
    total = [n + m for n, m in zip(lens, past)]
    q, cu_q = packed(g, dt, lens, Hq, D)
    k, cu_k = packed(g, dt, total, 1, D)
    v, _ = packed(g, dt, total, 1, D)
    cq, ck = cu_q.tolist(), cu_k.tolist()
    for spoil in (None, float("nan"), float("inf")):
        if spoil is not None:                             # all of sequences 0 and 2
            for b in (0, 2):
                q[cq[b]:cq[b + 1]] = spoil
                k[ck[b]:ck[b + 1]] = spoil
                v[ck[b]:ck[b + 1]] = spoil
        o = ta.causal_gqa_varlen_fwd(q, k, v, cu_q, cu_k, window=window, sinks=sinks)
        for b in range(4) if spoil is None else (1, 3):
            one = [x[None, s].transpose(1, 2) for x, s in ((q, slice(cq[b], cq[b + 1])), (k, slice(ck[b], ck[b + 1])),
                                                           (v, slice(ck[b], ck[b + 1])))]
            want = ta.causal_gqa_window_fwd(*one, window, sinks)[0].transpose(0, 1)
            got = o[cq[b]:cq[b + 1]]
            assert torch.isfinite(got.float()).all() and torch.equal(got, want)
    assert ta.device_status() == 0


@pytest.mark.parametrize("dt,D,spot", [("bf16", 128, 100), ("bf16", 64, 2), ("f16", 128, 499), ("f32", 64, 300)])
def test_varlen_infinite_values_reach_the_rows_that_see_them(ta, dt, D, spot):
    g = torch.Generator().manual_seed(31)
    lens = [60, 500, 130]
    q, cu = packed(g, dt, lens, 2, D)
    k, _ = packed(g, dt, lens, 1, D)
    v, _ = packed(g, dt, lens, 1, D)
    clean = ta.causal_gqa_varlen_fwd(q, k, v, cu, window=90, sinks=3)
    v[60 + spot, 0, 5] = float("inf")
    o = ta.causal_gqa_varlen_fwd(q, k, v, cu, window=90, sinks=3)
    sees = torch.zeros(690, dtype=torch.bool)
    sees[60:560] = visible(500, range(500), 90, 3)[:, spot]
    assert torch.equal(o[~sees], clean[~sees])
    assert not torch.isfinite(o[sees][..., 5].float()).any()
    other = [c for c in range(D) if c != 5]
    assert torch.isfinite(o[sees][..., other].float()).all()
    assert ta.device_status() == 0


def test_varlen_sequences_that_cannot_be_are_reported(ta):
    g = torch.Generator().manual_seed(32)
    for dt, D in (("bf16", 128), ("f32", 64)):
        q, _ = packed(g, dt, [100], 2, D)
        k, _ = packed(g, dt, [100], 2, D)
        v, _ = packed(g, dt, [100], 2, D)
        o = torch.full((100, 2, D), 7.0, dtype=DT[dt]).cuda()
        # more queries than keys; starts that fall; starts that pass the rows
        cu_q = torch.tensor([0, 20, 40, 60, 50, 70, 101]).int().cuda()
        cu_k = torch.tensor([0, 20, 35, 60, 61, 81, 100]).int().cuda()
        ta.causal_gqa_varlen_fwd(q, k, v, cu_q, cu_k, o=o)
        assert ta.device_status() == 6
        assert (o[20:40] == 7).all() and (o[70:] == 7).all()
        check_varlen(dt, q, k, v, cu_q[:2], cu_k[:2], o, 0, 0)
        # rows 50 to 59 are claimed by the third sequence too
        check_varlen(dt, q, k, v, cu_q[4:6], cu_k[4:6], o, 0, 0, list(range(10, 20)))
        empty = torch.zeros(4, dtype=torch.int32).cuda()
        o.fill_(7.0)
        ta.causal_gqa_varlen_fwd(q, k, v, empty, o=o)
        assert ta.device_status() == 0 and (o == 7).all()


@pytest.mark.parametrize("dt,Hq,Hkv,D,window", [("bf16", 4, 2, 128, 0), ("f16", 3, 1, 64, 60), ("f32", 2, 1, 64, 0)])
def test_varlen_more_sequences_than_a_warp_holds(ta, dt, Hq, Hkv, D, window):
    """Empty ones at either end and in runs, long ones among them, rows before and behind;
    a bad one at the far end leaves the others as they were."""
    g = torch.Generator().manual_seed(44)
    lens = ([0] * 40 + [1, 700, 0, 33, 128, 129, 0, 0, 5] + [17, 0, 64] * 30 + [300, 0, 31] + [0] * 35) * 2
    past = [(3 * i) % 50 if n else 0 for i, n in enumerate(lens)]
    q, cu_q = packed(g, dt, lens, Hq, D, 140, 70)
    k, cu_k = packed(g, dt, [n + m for n, m in zip(lens, past)], Hkv, D, 3, 2)
    v, _ = packed(g, dt, [n + m for n, m in zip(lens, past)], Hkv, D, 3, 2)
    o = torch.full_like(q, 7.0)
    ta.causal_gqa_varlen_fwd(q, k, v, cu_q, cu_k, window=window, o=o)
    assert ta.device_status() == 0 and (o[:140] == 7).all() and (o[-70:] == 7).all()
    check_varlen(dt, q, k, v, cu_q, cu_k, o, window, 0, [0, 15, 16, 31, 32, 127, 128, 129, 511, 512, -1])
    bad, again = cu_q.clone(), torch.full_like(q, 7.0)
    bad[-1] += 1000                                      # past the rows, and more queries than keys
    ta.causal_gqa_varlen_fwd(q, k, v, bad, cu_k, window=window, o=again)
    assert ta.device_status() == 6 and torch.equal(again, o)


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("f32", 64)])
def test_varlen_sequences_that_overlap(ta, dt, D):
    """The same rows claimed over and over: more blocks than the rows can have.  What is
    written is right, and the call reports it."""
    g = torch.Generator().manual_seed(42)
    n = 300
    q, _ = packed(g, dt, [n], 2, D)
    k, _ = packed(g, dt, [n], 1, D)
    v, _ = packed(g, dt, [n], 1, D)
    once = ta.causal_gqa_varlen_fwd(q, k, v, starts([n]))
    assert ta.device_status() == 0
    o = torch.full_like(q, 7.0)
    ta.causal_gqa_varlen_fwd(q, k, v, torch.tensor([0, n] * 150).int().cuda(), o=o)
    assert ta.device_status() == 6
    same = (o == once).all(-1)
    assert (same | (o == 7).all(-1)).all() and same.any()


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f16", 64)])
def test_varlen_rows_on_16_byte_boundaries(ta, dt, D):
    """Rows of q, k, v and o that start between two sectors."""
    g = torch.Generator().manual_seed(43)
    lens, H = [130, 1, 260], 4
    n = sum(lens)
    q, k, v = (randn(g, n, h * D + 8).to(DT[dt]).cuda()[:, 8:].unflatten(1, (h, D)) for h in (H, 2, 2))
    wide = torch.full((n, H * D + 24), 7.0, dtype=DT[dt]).cuda()
    cu = starts(lens)
    o = ta.causal_gqa_varlen_fwd(q, k, v, cu, window=140, sinks=3, o=wide[:, 8:-16].unflatten(1, (H, D)))
    assert o.data_ptr() % 32 == 16 and (wide[:, :8] == 7).all() and (wide[:, -16:] == 7).all()
    assert torch.equal(o, ta.causal_gqa_varlen_fwd(q, k, v, cu, window=140, sinks=3)) and ta.device_status() == 0
    check_varlen(dt, q, k, v, cu, cu, o, 140, 3, [0, 127, 128, 129, 130, 131, 258, -1])


@pytest.mark.parametrize("D", [64, 128])
def test_rows_beyond_32_bit_offsets(ta, D):
    """Tokens 2 M elements apart: rope in place and attention on views of one buffer."""
    g = torch.Generator().manual_seed(45)
    lens = [300, 1, 799]
    n = sum(lens)
    far = torch.empty(n, 2 ** 21, dtype=torch.bfloat16, device="cuda")
    assert far.numel() > 2 ** 31
    q, k, v, o = (far[:, i * 512:i * 512 + h * D].unflatten(1, (h, D)) for i, h in enumerate((2, 1, 1, 2)))
    for x in (q, k, v):
        x.copy_(randn(g, *x.shape))
    o.fill_(7.0)
    cu, f = starts(lens), ta.rope_frequencies(D)
    pos = torch.cat([torch.arange(m) for m in lens]).int().cuda()
    near = [ta.rope_fwd(x.contiguous(), f, pos) for x in (q, k)]
    for x, y in zip((q, k), near):
        assert torch.equal(ta.rope_fwd(x, f, pos, o=x), y)
    want = ta.causal_gqa_varlen_fwd(*near, v.contiguous(), cu)
    assert torch.equal(ta.causal_gqa_varlen_fwd(q, k, v, cu, o=o), want)
    assert ta.device_status() == 0 and not (o == 7).all(-1).any()


def test_varlen_long_and_many(ta):
    g = torch.Generator().manual_seed(33)
    lens = [9000, 3, 700, 1, 2500]
    q, cu = packed(g, "bf16", lens, 8, 128)
    k, _ = packed(g, "bf16", lens, 2, 128)
    v, _ = packed(g, "bf16", lens, 2, 128)
    o = ta.causal_gqa_varlen_fwd(q, k, v, cu)
    assert all(torch.equal(ta.causal_gqa_varlen_fwd(q, k, v, cu), o) for _ in range(3))
    check_varlen("bf16", q, k, v, cu, cu, o, 0, 0, [0, 127, 128, 2047, 5000, 8191, 8999])
    lens = [(i * 37) % 90 for i in range(1500)]
    q, cu = packed(g, "f16", lens, 2, 64)
    k, _ = packed(g, "f16", lens, 2, 64)
    v, _ = packed(g, "f16", lens, 2, 64)
    o = ta.causal_gqa_varlen_fwd(q, k, v, cu)
    assert ta.device_status() == 0
    pick = [0, 1, 63, 64, 65, 700, 1498, 1499]
    c = cu.tolist()
    for b in pick:
        check_varlen("f16", q, k, v, cu[b:b + 2], cu[b:b + 2], o, 0, 0)
    assert torch.isfinite(o.float()).all() and c[-1] == len(q)


@pytest.mark.parametrize("dt,D,Hq", [("bf16", 128, 2), ("f16", 64, 1), ("bf16", 64, 8)])
def test_varlen_last_round_of_items(ta, dt, D, Hq):
    """Around whole rounds of the SMs: pairs of the last round are split or not."""
    g = torch.Generator().manual_seed(34)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    rows = 128 if Hq % 2 == 0 else 256
    hp = max(1, Hq // 2)
    for items in (sms - 1, sms, sms + 1, sms + sms // 2, sms + sms // 2 + hp):
        n = max(1, items // hp) * rows
        lens = [n // 3, 1, n - n // 3 - 60]
        q, cu = packed(g, dt, lens, Hq, D)
        k, _ = packed(g, dt, lens, 1, D)
        v, _ = packed(g, dt, lens, 1, D)
        o = ta.causal_gqa_varlen_fwd(q, k, v, cu, window=200)
        check_varlen(dt, q, k, v, cu, cu, o, 200, 0, [0, 1, 127, 128, 255, 256, -1, -70, -128, -129])
    assert ta.device_status() == 0


# ------------------------------------------------------------- together

@pytest.mark.parametrize("q4", [True, False])
def test_serving_step_in_a_captured_graph(ta, q4):
    """Prompts in one packed pass, then decode steps from one captured graph: append
    (keys and queries rotated), decode; every step against 64-bit attention over what
    the cache holds."""
    g = torch.Generator().manual_seed(40)
    lens, Hq, Hkv, D, S, steps = [50, 1, 133], 8, 2, 128, 16, 4
    B = len(lens)
    f, f64 = ta.rope_frequencies(D), rates(D)
    P, M = 64, 16
    table = torch.full((B, M), -1, dtype=torch.int32).cuda()
    refs, sl = torch.zeros(P, dtype=torch.int32).cuda(), torch.zeros(B, dtype=torch.int32).cuda()
    ta.kv_pages_reserve(table, sl, torch.tensor([n + steps for n in lens]).int().cuda(), refs, S)
    # prompts: rotate, attend packed, append
    qkv = randn(g, sum(lens), Hq + 2 * Hkv, D).bfloat16().cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    cu = starts(lens)
    pos = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    kr = ta.rope_fwd(k, f, pos)
    if q4:
        pages = torch.zeros(P, Hkv, S, 144, dtype=torch.uint8).cuda()
        qr = ta.kv_append_paged_q4(pages, k, v, table, sl, f, cu_new=cu, q=q)
    else:
        kp, vp = (torch.zeros(P, Hkv, S, D, dtype=torch.bfloat16).cuda() for _ in "kv")
        qr = ta.kv_append_paged_rope(kp, vp, k, v, table, sl, f, cu_new=cu, q=q)
    assert torch.equal(qr, ta.rope_fwd(q, f, pos)) and sl.tolist() == lens
    o = ta.causal_gqa_varlen_fwd(qr, kr, v, cu)
    check_varlen("bf16", qr, kr, v, cu, cu, o, 0, 0, ROWS)
    # one captured step, replayed
    step = torch.zeros(B, Hq + 2 * Hkv, D, dtype=torch.bfloat16).cuda()
    qn, kn, vn = step[:, :Hq], step[:, Hq:Hq + Hkv], step[:, Hq + Hkv:]
    qd, od = torch.empty(B, Hq, D, dtype=torch.bfloat16).cuda(), torch.empty(B, Hq, D, dtype=torch.bfloat16).cuda()
    need = ta.decode_paged_q4_workspace_bytes if q4 else ta.decode_paged_workspace_bytes
    ws = torch.zeros(need(B, Hq, Hkv, D), dtype=torch.uint8).cuda()

    def once():
        if q4:
            ta.kv_append_paged_q4(pages, kn, vn, table, sl, f, q=qn, q_out=qd)
            ta.decode_gqa_paged_q4(qd, pages, table, sl, o=od, workspace=ws)
        else:
            ta.kv_append_paged_rope(kp, vp, kn, vn, table, sl, f, q=qn, q_out=qd)
            ta.decode_gqa_paged(qd, kp, vp, table, sl, o=od, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            once()
    torch.cuda.current_stream().wait_stream(s)
    assert sl.tolist() == lens
    for i in range(steps):
        step.copy_(randn(g, B, Hq + 2 * Hkv, D).bfloat16())
        graph.replay()
        assert ta.device_status() == 0 and sl.tolist() == [n + i + 1 for n in lens]
        now = sl.tolist()
        want = rotate(qn.double().cpu(), torch.tensor(now)[:, None] - 1, f64)
        assert ((qd.double().cpu() - want).abs() <= rotate_bound("bf16", qn.cpu(), want, f64, False, 1.0)).all()
        ks, vs = [], []
        for b, n in enumerate(now):
            p = torch.arange(n)
            at = table[b].cpu()[p // S].long()
            if q4:
                x, y = unpack(pages[at, :, p % S].cpu(), "bf16")
            else:
                x, y = kp[at, :, p % S].double().cpu(), vp[at, :, p % S].double().cpu()
            ks.append(x.transpose(0, 1))
            vs.append(y.transpose(0, 1))
        if q4:
            check_q4("bf16", qd, ks, vs, now, od, 0, 0)
        else:
            for b, n in enumerate(now):
                for hk in range(Hkv):
                    r, A, E, s1 = attend(qd[b, 4 * hk:4 * hk + 4].double().cpu(), ks[b][hk], vs[b][hk],
                                         torch.ones(4, n, dtype=torch.bool))
                    got = od[b, 4 * hk:4 * hk + 4].double().cpu()
                    assert ((got - r).abs() <= bound("bf16", r, A, E, s1, n, 2.0 ** -17)).all()


def test_continued_prompt_over_the_4_bit_cache(ta):
    """A second chunk of each prompt: appended, the whole past gathered, attended packed;
    pages forked and copied on the way."""
    g = torch.Generator().manual_seed(41)
    first, more, Hq, Hkv, D, S = [40, 7, 90], [30, 100, 1], 6, 2, 64, 8
    P, M, B = 128, 24, 3
    f = ta.rope_frequencies(64)
    table = torch.full((B + 1, M), -1, dtype=torch.int32).cuda()
    refs, sl = torch.zeros(P, dtype=torch.int32).cuda(), torch.zeros(B + 1, dtype=torch.int32).cuda()
    pages = torch.zeros(P, Hkv, S, 72, dtype=torch.uint8).cuda()
    for lens in (first, more):
        ta.kv_pages_reserve(table, sl, torch.tensor(lens + [0]).int().cuda(), refs, S)
        x = randn(g, sum(lens), Hq + 2 * Hkv, D).half().cuda()
        cu = starts(lens + [0])
        q = ta.kv_append_paged_q4(pages, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], table, sl, f, cu_new=cu, q=x[:, :Hq])
    total = [a + b for a, b in zip(first, more)]
    assert sl.tolist() == total + [0]
    # row 3 becomes a copy of row 0
    cs, cd = ta.kv_pages_fork(table, sl, refs, torch.tensor([0]).int().cuda(), torch.tensor([3]).int().cuda(), S)
    ta.kv_pages_copy_q4(pages, cs, cd)
    cu_k = starts(total + [total[0]])
    k, v = (torch.empty(sum(total) + total[0], Hkv, D, dtype=torch.float16).cuda() for _ in "kv")
    ta.kv_gather_paged_q4(pages, table, cu_k, k, v)
    assert ta.device_status() == 0
    assert torch.equal(k[:total[0]], k[sum(total):]) and torch.equal(v[:total[0]], v[sum(total):])
    o = ta.causal_gqa_varlen_fwd(q, k, v, cu, cu_k)       # the fourth sequence has no queries
    check_varlen("f16", q, k, v, cu, cu_k, o, 0, 0, ROWS)
    # the last query of each is what decode gives
    last = torch.stack([q[cu[b + 1] - 1] for b in range(B)] + [q[cu[1] - 1]])
    d = ta.decode_gqa_paged_q4(last, pages, table, sl)
    assert ta.device_status() == 0
    assert torch.equal(d[3], d[0])
    for b in range(B):
        assert (d[b].float() - o[cu[b + 1] - 1].float()).abs().max() <= 2.0 ** -8 * v.float().abs().max()


def test_other_streams_and_devices_do_not_matter(ta):
    g = torch.Generator().manual_seed(42)
    lens = [70, 300]
    q, cu = packed(g, "bf16", lens, 4, 128)
    k, _ = packed(g, "bf16", lens, 2, 128)
    v, _ = packed(g, "bf16", lens, 2, 128)
    f, pos = ta.rope_frequencies(128), torch.arange(370).int().cuda()
    q4 = build_q4("bf16", [100, 900], 4, 2, 128, 16, 0, 0, 43)
    want = (ta.rope_fwd(q, f, pos), ta.causal_gqa_varlen_fwd(q, k, v, cu), ta.decode_gqa_paged_q4(*q4[:4]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append((ta.rope_fwd(q, f, pos), ta.causal_gqa_varlen_fwd(q, k, v, cu),
                            ta.decode_gqa_paged_q4(*q4[:4])))
    torch.cuda.synchronize()
    for x in got:
        assert all(torch.equal(a, b) for a, b in zip(x, want))
    assert ta.device_status() == 0


def test_packed_calls_side_by_side_and_replayed(ta):
    """Two calls that each fill the GPU, on two streams, one of them a replayed graph that
    meets other lengths: each takes its own items."""
    g = torch.Generator().manual_seed(46)
    lens = [2500, 1, 1800, 700]
    n = sum(lens)
    sets = []
    for D, dt in ((128, "bf16"), (64, "f16")):
        q, k, v = (randn(g, n, h, D).to(DT[dt]).cuda() for h in (16, 4, 4))
        sets.append((q, k, v))
    cus = [starts(lens), starts([n]), starts([5] * 70 + [n - 350 - 900] + [30] * 30)]
    want = [[ta.causal_gqa_varlen_fwd(*x, cu) for cu in cus] for x in sets]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    held, o = starts(lens), torch.empty_like(sets[0][0])
    graphs = {}
    for B, cu in ((4, held), (1, cus[1]), (101, cus[2])):    # the number of sequences is an argument
        graphs[B] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[B], stream=a):
            ta.causal_gqa_varlen_fwd(*sets[0], cu, o=o)
    for i, B in enumerate((4, 1, 101) * 2):
        with torch.cuda.stream(a):
            graphs[B].replay()
        with torch.cuda.stream(b):
            got = [ta.causal_gqa_varlen_fwd(*sets[1], cu) for cu in cus]
        torch.cuda.synchronize()
        assert torch.equal(o, want[0][(4, 1, 101).index(B)])
        assert all(torch.equal(x, y) for x, y in zip(got, want[1]))
    held.copy_(starts([700, 1800, 1, 2500]))             # the captured call with other lengths
    graphs[4].replay()
    torch.cuda.synchronize()
    assert torch.equal(o, ta.causal_gqa_varlen_fwd(*sets[0], held)) and ta.device_status() == 0


def test_layout_of_the_tests_is_the_headers():
    k, v, bit = layout(128)
    assert k[:9] == [0, 0, 0, 0, 2, 2, 2, 2, 16] and v[:9] == [64, 64, 64, 64, 72, 72, 72, 72, 80]
    assert (k[32], v[32], k[127], v[127]) == (4, 66, 62, 126) and bit[:5] == [0, 4, 8, 12, 0]

"""Causal prefill with a sliding window and sinks against a 64-bit softmax over
exactly the keys each query sees."""
import pytest
import torch

from tests.paged_ref import DT, attend, bound, visible

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ta():
    from transformer_attention_tcgen05_gb300.build import build
    build()
    import transformer_attention_tcgen05_gb300 as ta
    torch.cuda.set_device(0)
    return ta


def make(dt, B, heads, N, D, order, seed):
    g = torch.Generator().manual_seed(seed)
    if order == "token":
        return torch.randn(B, N, heads, D, generator=g).to(DT[dt]).cuda().transpose(1, 2)
    return torch.randn(B, heads, N, D, generator=g).to(DT[dt]).cuda()


def p_eps(dt, D):
    """Rounding of P before the P V product: to 16 bits on the tensor cores."""
    return torch.finfo(DT[dt]).eps / 2 if dt != "f32" and D != 32 else 0.0


def check(ta, dt, q, k, v, o, window, sinks, rows=None):
    B, Hq, Nq, D = q.shape
    Hkv, Nkv = k.shape[1], k.shape[2]
    rows = list(range(Nq)) if rows is None else rows
    see = visible(Nkv, [Nkv - Nq + r for r in rows], window, sinks)
    for b in range(B):
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            ref, A, E, s1 = attend(q[b, h, rows].double().cpu(), k[b, hk].double().cpu(),
                                   v[b, hk].double().cpu(), see)
            got = o[b, h, rows].double().cpu()
            lim = bound(dt, ref, A, E, s1, int(see.sum(1).max()), p_eps(dt, D))
            bad = ~((got - ref).abs() <= lim)
            assert not bad.any(), (b, h, torch.nonzero(bad)[:5].tolist(),
                                   ((got - ref).abs() / lim).max().item())


CASES = [
    # dt, B, Hq, Hkv, Nq, Nkv, D, window, sinks, order
    ("bf16", 1, 2, 1, 1, 1, 128, 1, 0, "head"),
    ("bf16", 2, 3, 3, 1, 300, 64, 17, 2, "token"),
    ("bf16", 1, 4, 2, 129, 129, 128, 1, 0, "head"),
    ("bf16", 1, 4, 2, 300, 300, 128, 128, 4, "token"),
    ("f16", 2, 4, 1, 300, 300, 64, 128, 4, "head"),
    ("bf16", 1, 2, 1, 700, 700, 128, 100, 0, "head"),
    ("bf16", 1, 2, 1, 700, 700, 64, 100, 130, "token"),     # sinks past a key tile
    ("bf16", 1, 2, 2, 700, 700, 128, 256, 256, "head"),     # whole sink tiles
    ("bf16", 1, 2, 1, 513, 1000, 128, 255, 3, "head"),      # queries continue a prompt
    ("f16", 1, 2, 1, 130, 777, 128, 129, 1, "token"),
    ("bf16", 1, 7, 1, 257, 900, 64, 384, 5, "head"),
    ("bf16", 1, 2, 1, 400, 400, 128, 400, 0, "head"),       # the window covers everything
    ("bf16", 1, 2, 1, 400, 400, 64, 100000, 7, "head"),
    ("bf16", 1, 2, 1, 400, 500, 128, 0, 0, "head"),         # no window
    ("bf16", 1, 2, 1, 400, 400, 64, 3, 1000, "head"),       # sinks cover everything
    ("f32", 1, 4, 2, 200, 200, 64, 50, 4, "token"),
    ("f32", 2, 2, 1, 65, 333, 128, 64, 70, "head"),
    ("f32", 1, 1, 1, 1, 1, 32, 5, 5, "head"),
    ("bf16", 1, 2, 1, 150, 150, 32, 33, 1, "head"),         # D = 32: SIMT kernel
    ("f16", 1, 2, 2, 90, 200, 32, 70, 0, "token"),
]


@pytest.mark.parametrize("dt,B,Hq,Hkv,Nq,Nkv,D,window,sinks,order", CASES)
def test_window_parity(ta, dt, B, Hq, Hkv, Nq, Nkv, D, window, sinks, order):
    q = make(dt, B, Hq, Nq, D, order, 1)
    k, v = make(dt, B, Hkv, Nkv, D, order, 2), make(dt, B, Hkv, Nkv, D, order, 3)
    fam = "simt" if dt == "f32" or D == 32 else "tc_flash"
    n0 = ta.launch_count(fam)
    o = ta.causal_gqa_window_fwd(q, k, v, window, sinks)
    assert ta.launch_count(fam) == n0 + 1
    assert ta.device_status() == 0
    check(ta, dt, q, k, v, o, window, sinks)


def test_window_long_sampled_rows(ta):
    q = make("bf16", 1, 8, 9000, 128, "token", 4)
    k, v = make("bf16", 1, 2, 9000, 128, "token", 5), make("bf16", 1, 2, 9000, 128, "token", 6)
    o = ta.causal_gqa_window_fwd(q, k, v, 2048, 4)
    check(ta, "bf16", q, k, v, o, 2048, 4, rows=[0, 1, 127, 128, 2047, 2048, 2051, 2052, 5000, 8191, 8999])


@pytest.mark.parametrize("dt,B,Hq,Hkv,Nq,Nkv,D,window,sinks", [
    ("bf16", 2, 40, 8, 1200, 1200, 128, 300, 4),     # several pairs per CTA and single tiles behind them
    ("f16", 3, 36, 4, 1100, 1500, 64, 130, 140),
    ("bf16", 1, 152, 8, 300, 300, 128, 64, 0),       # whole rounds, a second tile of 44 rows
    ("bf16", 1, 77, 7, 520, 520, 64, 0, 0)])         # a last pair whose second tile is empty
def test_window_persistent_items(ta, dt, B, Hq, Hkv, Nq, Nkv, D, window, sinks):
    q = make(dt, B, Hq, Nq, D, "token", 50)
    k, v = make(dt, B, Hkv, Nkv, D, "head", 51), make(dt, B, Hkv, Nkv, D, "head", 52)
    o = ta.causal_gqa_window_fwd(q, k, v, window, sinks)
    again = [ta.causal_gqa_window_fwd(q, k, v, window, sinks) for _ in range(5)]
    assert ta.device_status() == 0
    assert all(torch.equal(a, o) for a in again)
    check(ta, dt, q, k, v, o, window, sinks,
          rows=sorted({0, 1, 127, 128, 255, 256, Nq // 2, Nq - 2, Nq - 1} & set(range(Nq))))


def test_window_scores_far_above_the_running_maximum(ta):
    """Keys that grow along the sequence move the maximum in every tile."""
    q = make("bf16", 1, 2, 600, 128, "head", 7)
    k, v = make("bf16", 1, 2, 600, 128, "head", 8), make("bf16", 1, 2, 600, 128, "head", 9)
    k = (k.float() * torch.linspace(0.1, 12, 600).cuda()[None, None, :, None]).bfloat16()
    o = ta.causal_gqa_window_fwd(q, k, v, 300, 2)
    check(ta, "bf16", q, k, v, o, 300, 2)


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f16", 64), ("f32", 64), ("bf16", 32)])
@pytest.mark.parametrize("what", ["v_nan", "v_inf", "k_nan", "k_inf"])
def test_what_a_row_does_not_see_does_not_reach_it(ta, dt, D, what):
    N, window, sinks, spots = 500, 90, 3, [200, 333, 499]
    q = make(dt, 1, 2, N, D, "head", 10)
    k, v = make(dt, 1, 1, N, D, "head", 11), make(dt, 1, 1, N, D, "head", 12)
    clean = ta.causal_gqa_window_fwd(q, k, v, window, sinks)
    x = k if what[0] == "k" else v
    x[:, :, spots, 5] = float("nan") if what.endswith("nan") else float("inf")
    o = ta.causal_gqa_window_fwd(q, k, v, window, sinks)
    assert ta.device_status() == 0
    sees = visible(N, range(N), window, sinks)[:, spots].any(1).cuda()
    check(ta, dt, q, k, v, o, window, sinks, rows=torch.nonzero(~sees)[:, 0].tolist())
    if what.endswith("nan"):
        assert torch.isnan(o[:, :, sees].float()).any(-1).all()
    else:
        # an infinite value: the rows that see it have it (or NaN) in channel 5
        if what == "v_inf":
            assert not torch.isfinite(o[:, :, sees, 5].float()).any()
            other = [c for c in range(D) if c != 5]
            assert torch.isfinite(o[:, :, sees][..., other].float()).all()
    assert torch.isfinite(clean.float()).all()


@pytest.mark.parametrize("dt,B,Hq,Hkv,Nq,Nkv,D,window,sinks,order", [
    ("bf16", 1, 4, 2, 300, 1300, 128, 200, 32, "head"),     # 32 sinks: the widest narrow tile
    ("bf16", 1, 4, 2, 300, 1300, 64, 200, 33, "token"),     # 33: a whole one
    ("f16", 1, 2, 1, 260, 1300, 128, 128, 1, "token"),
    ("f16", 2, 6, 2, 260, 700, 64, 129, 31, "head"),        # an odd group: pairs of row tiles
    ("bf16", 1, 24, 8, 520, 520, 128, 100, 5, "token"),
    ("f32", 1, 4, 2, 130, 900, 128, 140, 70, "token"),
    ("f32", 1, 3, 3, 33, 97, 32, 31, 1, "head"),
    ("f16", 1, 4, 4, 65, 300, 32, 64, 64, "token"),
])
def test_window_few_sinks(ta, dt, B, Hq, Hkv, Nq, Nkv, D, window, sinks, order):
    q = make(dt, B, Hq, Nq, D, order, 1)
    k, v = make(dt, B, Hkv, Nkv, D, order, 2), make(dt, B, Hkv, Nkv, D, order, 3)
    o = ta.causal_gqa_window_fwd(q, k, v, window, sinks)
    assert ta.device_status() == 0
    check(ta, dt, q, k, v, o, window, sinks)


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f16", 64), ("f32", 64)])
@pytest.mark.parametrize("spot", [0, 3, 4, 20, 40])
def test_window_sinks_of_extreme_values(ta, dt, D, spot):
    """A sink (0, 3) or a key behind the sinks in their tile (4, 20, 40), far from
    the others: scores of its own scale, or values that no row may see."""
    N, window, sinks = 400, 60, 4
    q = make(dt, 1, 2, N, D, "head", 20)
    k, v = make(dt, 1, 1, N, D, "head", 21), make(dt, 1, 1, N, D, "head", 22)
    k[:, :, spot] *= 8
    rows = [r for r in range(N) if spot < sinks or r < spot or r >= spot + window]
    if spot >= sinks:
        v[:, :, spot] = float("nan")
    o = ta.causal_gqa_window_fwd(q, k, v, window, sinks)
    assert ta.device_status() == 0
    check(ta, dt, q, k, v, o, window, sinks, rows=rows)


@pytest.mark.parametrize("which", ["q", "k", "v"])
def test_window_of_nothing_but_nan(ta, which):
    t = dict(q=make("bf16", 1, 2, 2000, 128, "head", 10), k=make("bf16", 1, 1, 2000, 128, "head", 11),
             v=make("bf16", 1, 1, 2000, 128, "head", 12))
    t[which].fill_(float("nan"))
    o = ta.causal_gqa_window_fwd(t["q"], t["k"], t["v"], 0)
    assert ta.device_status() == 0
    assert torch.isnan(o).all()


def test_window_output_view_and_sentinels(ta):
    B, Hq, N, D = 2, 4, 200, 64
    q, k, v = (make("bf16", B, h, N, D, "token", 20 + i) for i, h in enumerate((Hq, 2, 2)))
    wide = torch.full((B, N, Hq + 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    o = wide[:, :, 1:1 + Hq].transpose(1, 2)
    ta.causal_gqa_window_fwd(q, k, v, 33, 2, o=o)
    assert torch.equal(o, ta.causal_gqa_window_fwd(q, k, v, 33, 2))
    assert (wide[:, :, 0] == 7).all() and (wide[:, :, -1] == 7).all()


def test_window_on_another_stream_and_in_a_graph(ta):
    q, k, v = (make("bf16", 1, h, 300, 128, "head", 30 + i) for i, h in enumerate((4, 2, 2)))
    want = ta.causal_gqa_window_fwd(q, k, v, 64, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = ta.causal_gqa_window_fwd(q, k, v, 64, 1)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    o = torch.zeros_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ta.causal_gqa_window_fwd(q, k, v, 64, 1, o=o)
    q.copy_(q.flip(2))
    g.replay()
    assert torch.equal(o, ta.causal_gqa_window_fwd(q, k, v, 64, 1))


def test_no_window_agrees_with_the_causal_entry(ta):
    q, k, v = (make("bf16", 1, h, 500, 128, "head", 40 + i) for i, h in enumerate((4, 2, 2)))
    a, b = ta.causal_gqa_fwd(q, k, v), ta.causal_gqa_window_fwd(q, k, v, 0)
    check(ta, "bf16", q, k, v, a, 0, 0)
    check(ta, "bf16", q, k, v, b, 0, 0)


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f16", 128), ("bf16", 64), ("f16", 64), ("f32", 64), ("bf16", 32)])
@pytest.mark.parametrize("Hq,Nq,Nkv,window,sinks", [
    (2, 700, 700, 90, 3),          # pairs of heads; a narrow tile of sinks
    (3, 700, 777, 300, 40),        # pairs of row tiles, queries off the tiles' grid
    (3, 600, 600, 130, 0),
    (1, 333, 700, 200, 130),       # a second tile of sinks
])
@pytest.mark.parametrize("what", ["v_nan", "v_inf", "k_nan", "k_inf"])
def test_what_a_row_does_not_see_leaves_every_bit_of_it(ta, dt, D, Hq, Nq, Nkv, window, sinks, what):
    """Not within a tolerance: the output row is the same row.  An infinite or NaN
    value spoils its own channel of the rows that see it and nothing else."""
    q = make(dt, 1, Hq, Nq, D, "head", 60)
    k, v = make(dt, 1, 1, Nkv, D, "head", 61), make(dt, 1, 1, Nkv, D, "head", 62)
    clean = ta.causal_gqa_window_fwd(q, k, v, window, sinks)
    bad = float("nan") if what.endswith("nan") else float("inf")
    for spots in ([Nkv - 1], [Nkv - 200], [Nkv - 256, Nkv - 129, Nkv - 127], [sinks], [sinks + 5, 127], [129],
                  [0] if sinks else [Nkv // 2], [Nkv - 300, 20, Nkv - 64]):
        k2, v2 = k.clone(), v.clone()
        (k2 if what[0] == "k" else v2)[:, :, spots, 5] = bad
        o = ta.causal_gqa_window_fwd(q, k2, v2, window, sinks)
        assert ta.device_status() == 0
        see = visible(Nkv, range(Nkv - Nq, Nkv), window, sinks)[:, spots].any(1).cuda()
        assert torch.equal(o[:, :, ~see], clean[:, :, ~see]), spots
        if what[0] == "v":
            assert not torch.isfinite(o[:, :, see, 5].float()).any(), spots
            assert torch.equal(o[:, :, see, :5], clean[:, :, see, :5])
            assert torch.equal(o[:, :, see, 6:], clean[:, :, see, 6:])
        else:
            # an infinite key: infinite scores of either sign; +inf makes the row NaN
            lost = see if what == "k_nan" else see & (q[0, :, :, 5].float() > 0).all(0)
            assert torch.isnan(o[:, :, lost].float()).all(), spots


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f16", 64)])
def test_infinite_values_cost_little(ta, dt, D):
    """One infinite channel of a sink that nearly every row sees, or of a key behind
    the sinks that none of them sees, over a long prompt: the rows are not
    computed again key by key.  The work is that of the clean call and, for the
    row blocks with the value in a tile on an edge, one more look at such tiles
    (a few of hundreds of steps): less than three times the clean call."""
    N, window, sinks = 16384, 2048, 4
    q = make(dt, 1, 8, N, D, "head", 70)
    k, v = make(dt, 1, 2, N, D, "head", 71), make(dt, 1, 2, N, D, "head", 72)
    clean = ta.causal_gqa_window_fwd(q, k, v, window, sinks)

    def took():
        best = 1e9
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            o = ta.causal_gqa_window_fwd(q, k, v, window, sinks)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best, o

    limit = 3 * took()[0]
    for spot in (2, 20, N // 2):
        keep = v[:, :, spot].clone()
        v[:, :, spot, 5] = float("inf")
        ms, o = took()
        v[:, :, spot] = keep
        assert ta.device_status() == 0
        see = torch.arange(N, device="cuda")
        see = (see >= spot) & ((see < spot + window) | (spot < sinks))
        assert not torch.isfinite(o[:, :, see, 5].float()).any()
        o[:, :, see, 5] = clean[:, :, see, 5]
        assert torch.equal(o, clean)
        assert ms < limit, (spot, ms, limit / 3)


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f16", 128), ("bf16", 64), ("f16", 64)])
@pytest.mark.parametrize("Hq", [2, 3])
@pytest.mark.parametrize("spot", [100, 271, 400, 530, 599])
def test_a_key_that_other_rows_see_leaves_every_bit_of_a_row(ta, dt, D, Hq, spot):
    """Keys that grow along the sequence, so that maxima are due to move, and a NaN
    among them: rows next to those that see it keep theirs as without it."""
    N, window = 600, 300
    q = make(dt, 1, Hq, N, D, "head", 63)
    k, v = make(dt, 1, 1, N, D, "head", 64), make(dt, 1, 1, N, D, "head", 65)
    k = (k.float() * torch.linspace(0.1, 9, N).cuda()[None, None, :, None]).to(DT[dt])
    clean = ta.causal_gqa_window_fwd(q, k, v, window, 2)
    k[:, :, spot, 5] = float("nan")
    o = ta.causal_gqa_window_fwd(q, k, v, window, 2)
    see = visible(N, range(N), window, 2)[:, spot].cuda()
    assert torch.isnan(o[:, :, see].float()).all()
    assert torch.equal(o[:, :, ~see], clean[:, :, ~see])


@pytest.mark.parametrize("dt,D", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("rest", ["split", "whole", "none", "odd group"])
def test_window_last_round_of_items(ta, dt, D, rest):
    """Items are pairs of query tiles, one per CTA; those of a last round that takes
    at most half of the SMs go out as single tiles.  Chosen by the SM count: a
    remainder that is split, one that is not, none, and (pairs of row tiles, split)
    a last pair whose second tile lies behind the queries."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    N, window, sinks = 129, 40, 3
    if rest == "odd group":
        # three heads per KV head, one pair of row tiles each, 100 queries: the second is empty
        Hkv = next(h for h in range(1, 400) if 0 < 2 * (3 * h % sms) <= sms and 3 * h > sms)
        Hq, N = 3 * Hkv, 100
        pairs = Hq
    else:
        want = {"split": lambda r: 0 < 2 * r <= sms, "whole": lambda r: 2 * r > sms, "none": lambda r: r == 0}[rest]
        # two row blocks, two heads per KV head: two pairs per KV head
        Hkv = next(h for h in range(1, 2 * sms) if want(2 * h % sms) and (rest != "split" or 2 * h > sms))
        Hq, pairs = 2 * Hkv, 2 * Hkv
    r = pairs % sms
    assert (0 < 2 * r <= sms) == (rest in ("split", "odd group"))
    q = make(dt, 1, Hq, N, D, "head", 80)
    k, v = make(dt, 1, Hkv, N, D, "head", 81), make(dt, 1, Hkv, N, D, "head", 82)
    wide = torch.full((1, Hq, N + 60, D), 7.0, dtype=DT[dt], device="cuda")
    o = wide[:, :, :N]
    ta.causal_gqa_window_fwd(q, k, v, window, sinks, o=o)
    assert ta.device_status() == 0
    assert (wide[:, :, N:] == 7).all()
    heads = sorted({0, 1, 2, Hq // 2, Hq - 3, Hq - 2, Hq - 1})
    g = Hq // Hkv
    for h in heads:
        check(ta, dt, q[:, h:h + 1], k[:, h // g:h // g + 1], v[:, h // g:h // g + 1], o[:, h:h + 1], window, sinks)
    # the other heads: each as it comes out of a call of its own
    for h in range(0, Hkv, 7):
        one = ta.causal_gqa_window_fwd(q[:, h * g:(h + 1) * g], k[:, h:h + 1], v[:, h:h + 1], window, sinks)
        assert torch.equal(one, o[:, h * g:(h + 1) * g])

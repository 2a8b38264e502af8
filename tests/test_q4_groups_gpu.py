"""Decode over the cache held in 4 bits where the groups of a token have scales of very
different size: every group of channels is as exact as its own values allow."""
import pytest
import torch

from tests.paged_ref import DT, attend, visible
from tests.q4_ref import pack, unpack
from tests.test_packed_gpu import Cache, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ta():
    from transformer_attention_tcgen05_gb300.build import build
    build()
    import transformer_attention_tcgen05_gb300 as ta
    torch.cuda.set_device(0)
    return ta


def limit(dt, q, k, v, sc, ref, A, E, n):
    """The bound of a head's errors, channel by channel, from its own group's values:
    half a step of the output; A times (both scores' errors in exp, 2^-11 for the f16
    product of weight and scale, the fp32 roundings of n weights and sums, the
    exponential's); products below f16's normal range, half a step of 2^-24 where the
    group's largest is 2^7 (less 2^-8 of it) or more, times a code of at most 8; and the
    matrix instructions' roundings of sums of weights times (code + 256 or 264), 2^-23 of
    them each, 4 per chunk of 32 positions, 8 chunks per warp at most here.
    Scores: sums of (code + 16 or 256) q, at most 3 roundings of 2^-22 of the largest
    partial sum per group."""
    s_k, s_v = (x.abs().unflatten(-1, (-1, 32)).amax(-1) / 8 for x in (k, v))    # (the extreme value is 8 s)
    E = E + (3 * 2.0 ** -22 * 272 * sc * (q.abs().unflatten(-1, (-1, 32)).sum(-1) @ s_k.T)).amax(-1, keepdim=True)
    p = torch.softmax(q @ k.T * sc, -1)
    mean = (p @ s_v).repeat_interleave(32, -1)
    top = (p[:, :, None] * s_v).amax(1).repeat_interleave(32, -1)
    half = torch.finfo(DT[dt]).eps / 2
    tiny = torch.finfo(DT[dt]).tiny * half                     # (outputs below the type's normal range)
    return half * ref.abs() + A * (2 * E + 2.0 ** -11 + (n + 64) * 2.0 ** -24 + 2.0 ** -20) * (1 + half) + \
        n * 8 * 2.0 ** -32 * (1 + 2.0 ** -8) * top + mean * 272 * 2.0 ** -23 * 32 + tiny


def run(ta, dt, lens, G, D, ups, seed, change):
    """ups: the groups' scales as powers of two; change(b, q, k, v) sets what is special."""
    g = torch.Generator().manual_seed(seed)
    c = Cache(lens, [0] * len(lens), 16, seed)
    up = (2.0 ** torch.tensor(ups).double()).repeat_interleave(32).float()
    assert len(up) == D and sum(lens) <= 64000
    pages = torch.zeros(c.P, 1, 16, D + D // 8, dtype=torch.uint8)
    q = randn(g, len(lens), G, D).to(DT[dt])
    ks, vs = [], []
    for b, n in enumerate(lens):
        k, v = randn(g, 1, n, D), randn(g, 1, n, D) * up
        change(b, q, k, v)
        rows = pack(k, v, dt)
        page, row = c.rows(b, 0, n)
        pages[page, :, row] = rows.transpose(0, 1)
        kk, vv = unpack(rows, dt)
        ks.append(kk[0])
        vs.append(vv[0])
    o = ta.decode_gqa_paged_q4(q.cuda(), pages.cuda(), c.dev, c.sl)
    assert ta.device_status() == 0
    for b, n in enumerate(lens):
        x = q[b].double()
        ref, A, E, _ = attend(x, ks[b], vs[b], visible(n, [n - 1], 0, 0).expand(G, n))
        off = (o[b].double().cpu() - ref).abs() / limit(dt, x, ks[b], vs[b], D ** -0.5, ref, A, E, n)
        assert (off <= 1).all(), (b, off.unflatten(-1, (-1, 32)).amax((0, 2)).tolist())
    return o.float().cpu()


@pytest.mark.parametrize("dt,D,G,ups", [
    ("bf16", 128, 4, [0, -10, -14, -26]), ("bf16", 128, 2, [-8, 0, -16, -40]), ("f16", 128, 8, [8, -2, -8, -10]),
    ("bf16", 64, 9, [-20, 0]), ("f16", 64, 3, [6, -8]), ("bf16", 128, 16, [60, 0, -12, -60]),
])
def test_groups_of_a_token_far_apart(ta, dt, D, G, ups):
    """Long and ragged; in some sequences one token with most of the first head's weight
    (2^8 of the others' at D 128)."""
    for lens, peaks, seed in (([50000, 3000, 33], [777, 2999, None], 1), ([2100, 7, 640], [None, 0, 0], 2)):
        def peak(b, q, k, v):
            if peaks[b] is not None:
                k[0, peaks[b]] = q[b, 0].float() * 0.5

        run(ta, dt, lens, G, D, ups, seed, peak)


@pytest.mark.parametrize("ups", [[0, 0, 0, 0], [0, -20, 30, -40]])
def test_a_token_that_outweighs_all_without_values(ta, ups):
    """The last token takes the weight of every head (2^40 and more of each other one) and
    has values in its first group alone; those of the others are what is left."""
    def last(b, q, k, v):
        q[b] = q[b].abs()
        k *= 0.1
        k[0, :, :32] = 1.0
        k[0, -1, :32] = 16.0
        v[0, -1, 32:] = 0
        weight = torch.softmax(q[b].double() @ k[0].double().T / 128 ** 0.5, -1)
        assert (weight[:, :-1] < 2.0 ** -40).all()

    o = run(ta, "bf16", [40, 700], 4, 128, ups, 3, last)
    assert (o[..., 32:].abs().amax(-1) > 0).all()


@pytest.mark.parametrize("dt,G", [("bf16", 2), ("f16", 8), ("bf16", 12)])
def test_tiny_scales_and_queries_of_zero(ta, dt, G):
    """Scores that vanish weigh every visible token alike, and the others not at all."""
    g = torch.Generator().manual_seed(5)
    lens = [45, 700]
    c = Cache(lens, [0, 0], 16, 6)
    pages = torch.full((c.P, 1, 16, 144), 255, dtype=torch.uint8)          # (unseen scales are NaN)
    vs = []
    for b, n in enumerate(lens):
        rows = pack(randn(g, 1, n, 128), randn(g, 1, n, 128), dt)
        page, row = c.rows(b, 0, n)
        pages[page, :, row] = rows.transpose(0, 1)
        vs.append(unpack(rows, dt)[1][0])
    q = randn(g, 2, G, 128).to(DT[dt])
    q[:, 0] = 0
    q[:, -1] *= torch.finfo(DT[dt]).tiny
    for scale in (1e-20, 1e-30, 1e-38):
        o = ta.decode_gqa_paged_q4(q.cuda(), pages.cuda(), c.dev, c.sl, scale=scale).double().cpu()
        for b, n in enumerate(lens):
            # half a step, weights of one in f16 times a scale (2^-11), and fp32 sums
            lim = 2.0 ** -8 * vs[b].mean(0).abs() + (2.0 ** -11 + n * 2.0 ** -22) * vs[b].abs().mean(0)
            lim = lim + 272 * 2.0 ** -23 * 32 * vs[b].abs().unflatten(-1, (-1, 32)).amax(-1).mean(0).repeat_interleave(32) / 8
            assert ((o[b] - vs[b].mean(0)).abs() <= lim).all(), (scale, b, o[b, :, 0])
    assert ta.device_status() == 0


def test_products_near_the_least_fp32_numbers(ta):
    """Weights of 2^-45 times scales of 2^-77 are 2^3 and more above 2^-126."""
    def last(b, q, k, v):
        q[b, :, :32] = 1
        k *= 0.1
        k[0, :, :32] = 1.0
        k[0, -1, :32] = 12.0
        v.abs_().clamp_(0.25 * 2.0 ** -75)
        v[0, -1, 32:] = 0
        p = torch.softmax(q[b].double() @ k[0].double().T / 128 ** 0.5, -1)[:, :-1]
        assert (p > 2.0 ** -46).all() and (p < 2.0 ** -44).all()

    o = run(ta, "bf16", [40, 700], 4, 128, [0, -75, -60, -70], 7, last)
    assert (o[..., 32:].abs().amax(-1) > 0).all()


@pytest.mark.parametrize("dt,D,G", [("bf16", 128, 4), ("f16", 128, 4), ("f16", 64, 8), ("f16", 128, 12)])
def test_a_token_with_all_the_weight_is_given_back_exactly(ta, dt, D, G):
    """Values of few bits, so that nothing but the output is rounded where the weight is 1:
    whatever the scores' size and the scale of a group."""
    g = torch.Generator().manual_seed(8)
    n, B = 300, 12
    c = Cache([n] * B, [0] * B, 16, 9)
    s = (1 + torch.randint(0, 32, (B, n, D // 32), generator=g) / 32) * 2.0 ** torch.randint(-9, 3, (B, n, D // 32), generator=g)
    code = torch.randint(0, 16, (B, n, D), generator=g)
    code[..., ::32] = 0                                        # the value that the scale comes from
    v = (code - 8) * s.repeat_interleave(32, -1)
    k = torch.zeros(B, n, D)
    at = torch.randint(0, n, (B,), generator=g)
    q = randn(g, B, G, D).abs().to(DT[dt])
    k[torch.arange(B), at] = torch.rand(B, 1, generator=g) * 10 + 20
    p = torch.softmax(q.double() @ k.to(DT[dt]).double().transpose(1, 2) / D ** 0.5, -1)
    p[torch.arange(B), :, at] = 0
    assert p.max() < 2.0 ** -60
    pages = torch.zeros(c.P, 1, 16, D + D // 8, dtype=torch.uint8)
    for b in range(B):
        rows = pack(k[b][None], v[b][None], dt)
        page, row = c.rows(b, 0, n)
        pages[page, :, row] = rows.transpose(0, 1)
        assert torch.equal(unpack(rows, dt)[1][0], v[b].double())
    o = ta.decode_gqa_paged_q4(q.cuda(), pages.cuda(), c.dev, c.sl)
    assert ta.device_status() == 0
    # a scale of 6 bits times a code of 3 has up to 9: f16 holds them, bf16 (8) rounds some
    want = v[torch.arange(B), at][:, None].expand(B, G, D)
    fits = want.to(DT[dt]).float() == want
    assert fits.all() or dt == "bf16"
    assert ((o.float().cpu() - want).abs() <= torch.where(fits, 0.0, torch.finfo(DT[dt]).eps / 2 * want.abs())).all()

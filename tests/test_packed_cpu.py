"""Argument checks of the rotary, 4-bit-cache and packed entry points (no device is
touched: validation fails first), the frequency tables, and the plain 4-bit rows."""
import ctypes
import math

import pytest
import torch

from tests.q4_ref import layout, pack, quantise, rates, rotate, unpack

P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(12)]   # never dereferenced
ODD = ctypes.c_void_p(0x10004)
S2, S3 = ctypes.c_int64 * 2, ctypes.c_int64 * 3
INVALID, UNSUPPORTED, RESOURCE = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    from transformer_attention_tcgen05_gb300.build import build
    build()
    import transformer_attention_tcgen05_gb300 as ta
    return ta.lib()


def rope(L, **kw):
    a = dict(x=P[0], y=P[1], f=P[2], pos=P[3], ps=0, B=2, H=4, N=5, D=64, rot=32, m=1.0, xs=None, ys=None, dt=1)
    a.update(kw)
    return L.attn_rope_fwd(a["x"], a["y"], a["f"], a["pos"], a["ps"], a["B"], a["H"], a["N"], a["D"], a["rot"], 0,
                           0, a["m"], a["xs"], a["ys"], a["dt"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(f=None), INVALID), (dict(pos=None), INVALID),
    (dict(x=ODD), INVALID), (dict(f=ctypes.c_void_p(0x30004)), INVALID), (dict(pos=ctypes.c_void_p(0x40002)), INVALID),
    (dict(B=0), INVALID), (dict(H=0), INVALID), (dict(N=0), INVALID), (dict(D=48), INVALID), (dict(dt=3), INVALID),
    (dict(rot=0), INVALID), (dict(rot=24), INVALID), (dict(rot=80), INVALID), (dict(rot=-16), INVALID),
    (dict(m=math.nan), INVALID), (dict(m=math.inf), INVALID), (dict(ps=3), INVALID), (dict(ps=-5), INVALID),
    (dict(xs=S3(1280, 320, 60)), INVALID), (dict(ys=S3(1280, 320, 32)), INVALID),   # output rows overlap
    (dict(y=P[0], xs=S3(1280, 64, 256)), INVALID),                                  # in place, other strides
    (dict(y=P[3]), INVALID),
])
def test_rope_refusals(L, kw, want):
    assert rope(L, **kw) == want


def append(L, q4, **kw):
    a = dict(k=P[0], v=P[1], kn=P[2], vn=P[3], q=P[4], qo=P[5], t=P[6], sl=P[7], cu=P[8], f=P[9], B=3, N=7, Hq=4,
             Hkv=2, D=64, rot=64, m=1.0, P=10, S=16, M=4, ts=4, ks=None, vs=None, kns=None, vns=None, qs=None,
             qos=None, dt=1)
    a.update(kw)
    tail = [a["kns"], a["vns"], a["qs"], a["qos"], a["dt"], 1, None]
    head = [a["kn"], a["vn"], a["q"], a["qo"], a["t"], a["sl"], a["cu"], a["f"], a["B"], a["N"], a["Hq"], a["Hkv"],
            a["D"], a["rot"], 0, a["m"], a["P"], a["S"], a["M"], a["ts"], a["ks"]]
    if q4:
        return L.attn_kv_append_paged_q4(a["k"], *head, *tail)
    return L.attn_kv_append_paged_rope(a["k"], a["v"], *head, a["vs"], *tail)


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("kw,want", [
    (dict(k=None), INVALID), (dict(kn=None), INVALID), (dict(vn=None), INVALID), (dict(t=None), INVALID),
    (dict(sl=None), INVALID), (dict(qo=None), INVALID), (dict(k=ODD), INVALID), (dict(kn=ODD), INVALID),
    (dict(q=ODD), INVALID), (dict(cu=ctypes.c_void_p(0x90002)), INVALID), (dict(cu=P[7]), INVALID),
    (dict(kn=P[0]), INVALID), (dict(qo=P[2]), INVALID), (dict(qo=P[0]), INVALID), (dict(q=P[0]), INVALID),
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(cu=None), INVALID),       # 7 rows for 3 sequences
    (dict(Hkv=0), INVALID), (dict(Hq=0), INVALID), (dict(D=40), INVALID), (dict(dt=7), INVALID),
    (dict(rot=8), INVALID), (dict(rot=128), INVALID), (dict(m=math.nan), INVALID), (dict(S=12), INVALID),
    (dict(ts=3), INVALID), (dict(P=0), INVALID), (dict(kns=S2(128, 60)), INVALID), (dict(qos=S2(64, 64)), INVALID),
    (dict(q=P[4], qo=P[4], qs=S2(512, 64)), INVALID),                           # in place, other strides
    (dict(Hkv=70000), UNSUPPORTED), (dict(M=1 << 28, ts=1 << 28), UNSUPPORTED),
])
def test_append_refusals(L, q4, kw, want):
    assert append(L, q4, **kw) == want


def test_append_refusals_of_one_form(L):
    assert append(L, False, f=None) == INVALID
    assert append(L, False, v=P[0]) == INVALID
    assert append(L, False, ks=S3(1024, 1024, 64)) == INVALID                   # heads overlap the next page
    assert append(L, True, f=None) == INVALID                                   # rotary_dim without a table
    assert append(L, True, D=32, rot=32) == UNSUPPORTED
    assert append(L, True, dt=0) == UNSUPPORTED
    assert append(L, True, ks=S2(2 * 16 * 72, 16 * 72 - 16)) == INVALID         # pages overlap
    assert append(L, True, ks=S2(2 * 16 * 72 + 8, 16 * 72)) == INVALID          # not 16 bytes


def gather(L, **kw):
    a = dict(p=P[0], t=P[1], st=P[2], cu=P[3], k=P[4], v=P[5], B=2, N=9, Hkv=2, D=128, P=10, S=8, M=4, ts=4,
             ps=None, ks=None, vs=None, dt=2)
    a.update(kw)
    return L.attn_kv_gather_paged_q4(a["p"], a["t"], a["st"], a["cu"], a["k"], a["v"], a["B"], a["N"], a["Hkv"],
                                     a["D"], a["P"], a["S"], a["M"], a["ts"], a["ps"], a["ks"], a["vs"], a["dt"],
                                     None)


@pytest.mark.parametrize("kw,want", [
    (dict(p=None), INVALID), (dict(t=None), INVALID), (dict(cu=None), INVALID), (dict(k=None), INVALID),
    (dict(k=ODD), INVALID), (dict(st=ctypes.c_void_p(0x30002)), INVALID), (dict(N=0), INVALID), (dict(v=P[4]), INVALID),
    (dict(k=P[0]), INVALID), (dict(S=4), INVALID), (dict(D=100), INVALID), (dict(dt=0), UNSUPPORTED),
    (dict(D=32), UNSUPPORTED), (dict(ks=S2(128, 128)), INVALID), (dict(ps=S2(100, 1152)), INVALID),
])
def test_gather_refusals(L, kw, want):
    assert gather(L, **kw) == want


def test_copy_q4_refusals(L):
    def copy(p=P[0], src=P[1], dst=P[2], n=2, layers=1, pages=10, Hkv=2, S=8, D=64, st=None):
        return L.attn_kv_pages_copy_q4(p, src, dst, n, None, layers, pages, Hkv, S, D, st, None)
    assert copy(p=None) == copy(src=None) == copy(dst=None) == copy(n=0) == copy(layers=0) == copy(S=7) == INVALID
    assert copy(D=80) == copy(p=ODD) == copy(st=S3(16, 100, 576)) == copy(st=S3(1, 1152, 560)) == INVALID
    assert copy(D=32) == copy(layers=70000) == UNSUPPORTED


def decode(L, **kw):
    a = dict(q=P[0], p=P[1], t=P[2], sl=P[3], o=P[4], B=2, Hq=8, Hkv=2, D=128, P=10, S=16, M=4, ts=4, qs=None,
             ps=None, os=None, window=0, sinks=0, dt=1, ws=ctypes.c_void_p(0x90000), nbytes=1 << 30)
    a.update(kw)
    return L.attn_decode_gqa_paged_q4(a["q"], a["p"], a["t"], a["sl"], a["o"], a["B"], a["Hq"], a["Hkv"], a["D"],
                                      a["P"], a["S"], a["M"], a["ts"], a["qs"], a["ps"], a["os"], a["window"],
                                      a["sinks"], a["dt"], 0.0, a["ws"], a["nbytes"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(p=None), INVALID), (dict(t=None), INVALID), (dict(sl=None), INVALID),
    (dict(ws=None), INVALID), (dict(ws=ctypes.c_void_p(0x90010)), INVALID), (dict(q=ODD), INVALID),
    (dict(B=0), INVALID), (dict(Hq=9), INVALID), (dict(D=48), INVALID), (dict(S=12), INVALID), (dict(ts=3), INVALID),
    (dict(sinks=-1), INVALID), (dict(dt=5), INVALID), (dict(o=P[0]), INVALID), (dict(o=P[1]), INVALID),
    (dict(dt=0), UNSUPPORTED), (dict(D=32), UNSUPPORTED), (dict(Hq=34), UNSUPPORTED), (dict(nbytes=100), RESOURCE),
    (dict(qs=S2(1024, 4)), INVALID), (dict(os=S2(1024, 64)), INVALID), (dict(ps=S2(4608, 2300)), INVALID),
])
def test_decode_q4_refusals(L, kw, want):
    assert decode(L, **kw) == want


def varlen(L, **kw):
    a = dict(q=P[0], k=P[1], v=P[2], o=P[3], cq=P[4], ck=P[5], B=2, Nq=9, Nkv=12, Hq=4, Hkv=2, D=64, st=[None] * 4,
             sinks=0, dt=1)
    a.update(kw)
    return L.attn_causal_gqa_varlen_fwd(a["q"], a["k"], a["v"], a["o"], a["cq"], a["ck"], a["B"], a["Nq"], a["Nkv"],
                                        a["Hq"], a["Hkv"], a["D"], *a["st"], 0, a["sinks"], a["dt"], 0.0, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(o=P[0]), INVALID), (dict(cq=None), INVALID), (dict(ck=None), INVALID),
    (dict(k=ODD), INVALID), (dict(cq=ctypes.c_void_p(0x50002)), INVALID), (dict(B=0), INVALID), (dict(Nq=0), INVALID),
    (dict(Nkv=0), INVALID), (dict(Hq=3), INVALID), (dict(D=96), INVALID), (dict(sinks=-1), INVALID), (dict(dt=3), INVALID),
    (dict(B=65536), UNSUPPORTED), (dict(Hq=70000, Hkv=2), UNSUPPORTED), (dict(Nkv=(1 << 30) + 1), UNSUPPORTED),
    (dict(st=[S2(256, 60), None, None, None]), INVALID), (dict(st=[None, None, None, S2(64, 64)]), INVALID),
])
def test_varlen_refusals(L, kw, want):
    assert varlen(L, **kw) == want


@pytest.mark.parametrize("kw", [
    dict(), dict(theta=500000.0), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
    dict(scaling="by_parts", factor=4.0, original_len=8192), dict(scaling="by_parts", factor=32.0, original_len=4096,
                                                                 alpha=2.0, beta=8.0)])
@pytest.mark.parametrize("rot", [16, 48, 64, 128])
def test_frequency_tables(L, rot, kw):
    import transformer_attention_tcgen05_gb300 as ta
    t = ta.rope_frequencies(rot, device="cpu", **kw)
    assert t.dtype == torch.int64 and t.shape == (rot // 2,)
    want = rates(rot, **kw)
    # a few roundings of 2^-53 in pow and the products, and half a unit of 2^-64 turns
    assert ((t.double() / 2.0 ** 64 * 2 * math.pi - want).abs() <= want * 2.0 ** -48 + 2.0 ** -62).all()
    # angles modulo a turn of far positions: the integer product against 64-bit floats
    for pos in (1, 1000003, -7, 2 ** 31 - 1):
        turn = [((pos * int(f)) % 2 ** 64) / 2.0 ** 64 for f in t]
        a = pos * want
        assert (torch.tensor([math.cos(2 * math.pi * x) for x in turn], dtype=torch.float64) - torch.cos(a)).abs().max() <= \
            abs(pos) * 2.0 ** -48 + 2.0 ** -40


def test_frequency_refusals(L):
    import transformer_attention_tcgen05_gb300 as ta
    for kw in (dict(rotary_dim=24), dict(rotary_dim=40), dict(theta=0.0), dict(theta=math.nan), dict(factor=0.0),
               dict(scaling="by_parts", factor=2.0), dict(scaling="by_parts", original_len=8, alpha=3.0, beta=3.0),
               dict(factor=1e-3, scaling="linear")):
        with pytest.raises(ta.AttnError):
            ta.rope_frequencies(**{"rotary_dim": 64, "device": "cpu", **kw})
    for kw in (dict(rotary_dim=0), dict(rotary_dim=144), dict(scaling="cubic")):
        with pytest.raises(ValueError):
            ta.rope_frequencies(**{"rotary_dim": 64, "device": "cpu", **kw})


def test_binding_refuses_wrong_tensors(L):
    import transformer_attention_tcgen05_gb300 as ta
    x, pages = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(4, 4, 8, 72, dtype=torch.uint8)
    f = ta.rope_frequencies(64, device="cpu")
    t = torch.zeros(3, 2, dtype=torch.int32)
    one = torch.zeros(3, dtype=torch.int32)
    kv = torch.zeros(4, 4, 8, 64, dtype=torch.bfloat16)
    for call in (lambda: ta.rope_fwd(x, f, one), lambda: ta.causal_gqa_varlen_fwd(x, x, x, one),
                 lambda: ta.kv_append_paged_rope(kv, kv.clone(), x, x, t, one, f),
                 lambda: ta.kv_append_paged_q4(pages, x, x, t, one),
                 lambda: ta.kv_gather_paged_q4(pages, t, one, x, x.clone()),
                 lambda: ta.kv_pages_copy_q4(pages, one, one), lambda: ta.decode_gqa_paged_q4(x, pages, t, one)):
        with pytest.raises(ValueError):
            call()


def test_workspace_and_row_sizes(L):
    import transformer_attention_tcgen05_gb300 as ta
    assert [ta.kv_q4_row_bytes(d) for d in (32, 64, 96, 128)] == [0, 72, 0, 144]
    n = ta.decode_paged_q4_workspace_bytes(8, 32, 8, 128)
    assert n > 0 and n % 256 == 0
    assert n == ta.decode_paged_q4_workspace_bytes(8, 8, 8, 64)          # tickets at one place
    assert ta.decode_paged_q4_workspace_bytes(1, 34, 2, 128) == 0
    assert ta.decode_paged_q4_workspace_bytes(1, 4, 2, 32) == 0


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
def test_plain_rows_round_trip(dt, D):
    """What the tests' own rows stand for: every code at its place, within half a step."""
    k_at, v_at, bit = layout(D)
    assert len({(a, b) for a, b in zip(k_at, bit)} | {(a, b) for a, b in zip(v_at, bit)}) == 2 * D
    g = torch.Generator().manual_seed(3)
    k, v = torch.randn(5, D, generator=g), torch.randn(5, D, generator=g) * 3
    v[0, :32] = 0
    v[1, 32:64] = -2.5
    rows = pack(k, v, dt)
    assert rows.shape == (5, D + D // 8)
    for x, y in zip((k, v), unpack(rows, dt)):
        n, s = quantise(x, dt)
        step = s.double().abs().repeat_interleave(32, -1)
        inside = (n > 0) & (n < 15)
        assert ((y - x.double()).abs() <= step * (0.5 + 2.0 ** -20) + 1e-30)[inside].all()
        assert ((y - x.double()).abs() <= step * (1 + 2.0 ** -6)).all()
    assert (unpack(rows, dt)[1][0, :32] == 0).all() and (unpack(rows, dt)[1][1, 32:64] == -2.5).all()


def test_plain_rotation_is_orthogonal():
    f = rates(32)
    x = torch.randn(4, 64, dtype=torch.float64)
    p = torch.tensor([0, 1, -5, 100000])
    for inter in (False, True):
        y = rotate(x, p, f, inter)
        assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1)) and torch.equal(y[:, 32:], x[:, 32:])
        assert torch.allclose(rotate(y, p, f, inter, inverse=True), x) and torch.equal(y[0], x[0])

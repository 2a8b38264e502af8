"""Argument checks of the paged-cache and windowed entry points (no device is
touched: validation fails first), and the Python model of the allocator."""
import ctypes

import numpy as np
import pytest

from tests.paged_ref import Pool, visible

A, Bp, Cp, Dp, Ep, Fp = (ctypes.c_void_p(0x10000 * i) for i in range(1, 7))   # never dereferenced
S2, S3, S4 = ctypes.c_int64 * 2, ctypes.c_int64 * 3, ctypes.c_int64 * 4
INVALID, UNSUPPORTED, RESOURCE = 1, 2, 3


@pytest.fixture(scope="module")
def L():
    from transformer_attention_tcgen05_gb300.build import build
    build()
    import transformer_attention_tcgen05_gb300 as ta
    return ta.lib()


def decode(L, **kw):
    a = dict(q=A, k=Bp, v=Cp, table=Dp, sl=Ep, o=Fp, B=2, Hq=8, Hkv=2, D=128, P=10, S=16, M=4, ts=4, qs=None,
             ks=None, vs=None, os=None, window=0, sinks=0, dt=1, ws=ctypes.c_void_p(0x90000), nbytes=1 << 30)
    a.update(kw)
    return L.attn_decode_gqa_paged(a["q"], a["k"], a["v"], a["table"], a["sl"], a["o"], a["B"], a["Hq"],
                                   a["Hkv"], a["D"], a["P"], a["S"], a["M"], a["ts"], a["qs"], a["ks"],
                                   a["vs"], a["os"], a["window"], a["sinks"], a["dt"], 0.0, a["ws"],
                                   a["nbytes"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(table=None), INVALID), (dict(sl=None), INVALID), (dict(ws=None), INVALID),
    (dict(q=ctypes.c_void_p(0x10008)), INVALID), (dict(k=ctypes.c_void_p(0x10002)), INVALID),
    (dict(table=ctypes.c_void_p(0x10002)), INVALID), (dict(ws=ctypes.c_void_p(0x90010)), INVALID),
    (dict(B=0), INVALID), (dict(Hq=9), INVALID), (dict(Hkv=0), INVALID), (dict(D=48), INVALID),
    (dict(P=0), INVALID), (dict(S=0), INVALID), (dict(S=12), INVALID), (dict(S=4), INVALID),
    (dict(M=0), INVALID), (dict(ts=3), INVALID), (dict(sinks=-1), INVALID), (dict(dt=5), INVALID),
    (dict(o=A), INVALID), (dict(o=Bp), INVALID), (dict(o=Cp), INVALID),
    (dict(dt=0), UNSUPPORTED), (dict(D=32), UNSUPPORTED), (dict(Hq=34), UNSUPPORTED),
    (dict(M=1 << 28, ts=1 << 28), UNSUPPORTED), (dict(B=(1 << 20) + 1), UNSUPPORTED),
    (dict(nbytes=100), RESOURCE),
    (dict(qs=S2(0, 128)), INVALID), (dict(qs=S2(1024, 4)), INVALID),
    (dict(ks=S3(4096, 2048, 127)), INVALID), (dict(ks=S3(-4096, 2048, 128)), INVALID),
    (dict(vs=S3(4096, 2044, 128)), INVALID),
    (dict(os=S2(1024, 64)), INVALID),            # output rows overlap
    (dict(os=S2(512, 128)), INVALID),
])
def test_decode_paged_refusals(L, kw, want):
    assert decode(L, **kw) == want


def append(L, **kw):
    a = dict(k=A, v=Bp, kn=Cp, vn=Dp, table=Ep, sl=Fp, nl=None, B=2, T=3, Hkv=2, D=64, P=10, S=16, M=4, ts=4,
             ks=None, vs=None, kns=None, vns=None, dt=1)
    a.update(kw)
    return L.attn_kv_append_paged(a["k"], a["v"], a["kn"], a["vn"], a["table"], a["sl"], a["nl"], a["B"],
                                  a["T"], a["Hkv"], a["D"], a["P"], a["S"], a["M"], a["ts"], a["ks"],
                                  a["vs"], a["kns"], a["vns"], a["dt"], 1, None)


@pytest.mark.parametrize("kw,want", [
    (dict(k=None), INVALID), (dict(sl=None), INVALID), (dict(table=None), INVALID),
    (dict(kn=ctypes.c_void_p(0x30004)), INVALID), (dict(T=0), INVALID), (dict(D=96), INVALID),
    (dict(S=20), INVALID), (dict(v=A), INVALID), (dict(kn=A), INVALID), (dict(vn=A), INVALID),
    (dict(nl=Fp), INVALID), (dict(ts=2), INVALID), (dict(dt=3), INVALID),
    (dict(ks=S3(1024, 1024, 64)), INVALID),      # heads overlap the next page
    (dict(ks=S3(2048, 512, 64)), INVALID),
    (dict(kns=S3(0, 64, 128)), INVALID),
])
def test_append_paged_refusals(L, kw, want):
    assert append(L, **kw) == want


def test_allocator_refusals(L):
    ws, big = ctypes.c_void_p(0x90000), 1 << 20

    def reserve(t=A, sl=Bp, add=Cp, refs=Dp, B=2, P=10, S=8, M=4, ts=4, w=ws, n=big):
        return L.attn_kv_pages_reserve(t, sl, add, refs, B, P, S, M, ts, w, n, None)
    assert reserve(t=None) == reserve(sl=None) == reserve(add=None) == reserve(refs=None) == INVALID
    assert reserve(refs=ctypes.c_void_p(0x40004)) == reserve(S=9) == reserve(ts=3) == INVALID
    assert reserve(w=None) == reserve(w=ctypes.c_void_p(0x90004)) == INVALID
    assert reserve(n=8) == RESOURCE
    assert reserve(B=20000) == UNSUPPORTED
    assert reserve(B=16384, M=1 << 17, ts=1 << 17) == UNSUPPORTED      # 2^31 entries

    def free(t=A, sl=Bp, refs=Cp, sinks=0, B=2, S=8):
        return L.attn_kv_pages_free(t, sl, refs, B, 10, S, 4, 4, 5, sinks, None)
    assert free(t=None) == free(sl=None) == free(refs=None) == free(sinks=-1) == free(B=0) == free(S=1) == INVALID

    def fork(src=Dp, dst=Ep, n=1, cs=Fp, cd=ctypes.c_void_p(0x70000), B=2, w=ws, nb=big):
        return L.attn_kv_pages_fork(A, Bp, Cp, src, dst, n, cs, cd, B, 10, 8, 4, 4, w, nb, None)
    assert fork(src=None) == fork(dst=None) == fork(n=0) == fork(n=3) == fork(cs=None) == INVALID
    assert fork(cd=Fp) == fork(cs=Dp) == fork(cd=Ep) == INVALID
    assert fork(B=20000) == UNSUPPORTED
    assert fork(nb=8) == RESOURCE

    def compact(nt=Cp, ns=4, cs=Ep, cd=Fp, cnt=ctypes.c_void_p(0x70000), t=A, ts=4):
        return L.attn_kv_pages_compact(t, Bp, nt, Dp, cs, cd, cnt, 2, 10, 4, ts, ns, ws, big, None)
    assert compact(nt=None) == compact(ns=3) == compact(cs=None) == compact(cnt=None) == INVALID
    assert compact(cd=Ep) == compact(nt=A, ns=5) == INVALID

    def copy(k=A, v=Bp, n=2, layers=1, P=10, Hkv=2, S=8, D=64, ks=None, dt=1):
        return L.attn_kv_pages_copy(k, v, Cp, Dp, n, None, layers, P, Hkv, S, D, ks, None, dt, None)
    assert copy(k=None) == copy(v=A) == copy(n=0) == copy(layers=0) == copy(S=7) == copy(D=80) == INVALID
    assert copy(dt=4) == copy(ks=S4(1, 1024, 512, 48)) == copy(ks=S4(10240, 512, 512, 64)) == INVALID
    assert copy(layers=70000) == UNSUPPORTED


def window(L, **kw):
    a = dict(q=A, k=Bp, v=Cp, o=Dp, B=1, Hq=4, Hkv=2, Nq=8, Nkv=16, D=64, st=[None] * 4, sinks=0, dt=1)
    a.update(kw)
    return L.attn_causal_gqa_window_fwd(a["q"], a["k"], a["v"], a["o"], a["B"], a["Hq"], a["Hkv"], a["Nq"],
                                        a["Nkv"], a["D"], *a["st"], 4, a["sinks"], a["dt"], 0.0, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(o=A), INVALID), (dict(Nq=17), INVALID), (dict(Nq=0), INVALID),
    (dict(Hq=3), INVALID), (dict(D=40), INVALID), (dict(sinks=-2), INVALID), (dict(dt=9), INVALID),
    (dict(k=ctypes.c_void_p(0x20008)), INVALID), (dict(B=70000), UNSUPPORTED),
    (dict(Nkv=(1 << 30) + 1), UNSUPPORTED),
    (dict(st=[S3(1, 512, 63), None, None, None]), INVALID),
    (dict(st=[None, None, None, S3(2048, 64, 64)]), INVALID),
])
def test_window_refusals(L, kw, want):
    assert window(L, **kw) == want


def test_workspace_sizes(L):
    import transformer_attention_tcgen05_gb300 as ta
    assert ta.decode_paged_workspace_bytes(8, 32, 8, 128) % 256 == 0
    assert ta.decode_paged_workspace_bytes(8, 32, 8, 128) > 0
    assert ta.decode_paged_workspace_bytes(1, 34, 2, 128) == 0       # 17 heads per KV head
    assert ta.decode_paged_workspace_bytes(1, 4, 3, 128) == 0
    assert ta.decode_paged_workspace_bytes(1, 4, 2, 32) == 0
    assert ta.kv_pages_workspace_bytes(0) == 0
    assert ta.kv_pages_workspace_bytes(1000) >= 4000
    # the tickets lie behind the partials, at one place for all sizes
    assert ta.decode_paged_workspace_bytes(8, 32, 8, 128) == ta.decode_paged_workspace_bytes(8, 8, 8, 64)


def test_binding_refuses_cpu_tensors_and_wrong_shapes(L):
    import torch

    import transformer_attention_tcgen05_gb300 as ta
    x = torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16)
    t = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        ta.causal_gqa_window_fwd(x, x, x, 4)
    with pytest.raises(ValueError):
        ta.decode_gqa_paged(x[:, 0], x, x, t, t[:, 0])
    with pytest.raises(ValueError):
        ta.kv_append_paged(x, x.clone(), x, x, t, t[:, 0])
    with pytest.raises(ValueError):
        ta.kv_pages_free(t, t[:, 0], t[0], 8)
    with pytest.raises(ValueError):
        ta.kv_pages_copy(x[0], x[0], t[0], t[0])


def test_model_visibility_and_pool():
    see = visible(6, [5], 2, 1)[0].tolist()
    assert see == [True, False, False, False, True, True]
    assert visible(4, [1], 0, 0)[0].tolist() == [True, True, False, False]
    p = Pool(3, 4, 6, 8)
    assert p.reserve([9, 0, 8]) and p.table[0, :2].tolist() == [0, 1] and p.table[2, 0] == 2
    p.len += np.array([9, 0, 8], dtype=np.int32)
    assert p.fork([0], [1]) == [(1, 3)] and p.refs.tolist() == [2, 1, 1, 1, 0, 0]
    p.len[0] = 0
    p.free()
    assert p.refs.tolist() == [1, 0, 1, 1, 0, 0]
    assert p.compact() == [(3, 1)] and p.table[1].tolist() == [0, 1, -1, -1]

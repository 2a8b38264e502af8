"""Plain forms of rotary positions and of rows held in 4 bits for the tests:
64-bit rotation, and the row layout written out code by code."""
import math

import torch

from tests.paged_ref import DT


def rates(rot, theta=10000.0, scaling=None, factor=1.0, original_len=0, alpha=1.0, beta=32.0):
    """Radians per position of each pair, 64 bits."""
    f = [theta ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "ntk":
        f = [(theta * factor ** (rot / (rot - 2))) ** (-2.0 * i / rot) for i in range(rot // 2)]
    elif scaling == "by_parts":
        g = [min(1.0, max(0.0, (original_len * x / (2 * math.pi) - alpha) / (beta - alpha))) for x in f]
        f = [(1 - a) * x / factor + a * x for a, x in zip(g, f)]
    return torch.tensor(f, dtype=torch.float64)


def rotate(x, pos, f, interleaved=False, inverse=False, m=1.0):
    """x [..., D] float64, pos [...] (broadcast): the rotated rows, float64."""
    r = 2 * len(f)
    a = pos.double()[..., None] * f
    c, s = m * torch.cos(a), m * torch.sin(a) * (-1 if inverse else 1)
    y = x.double().clone()
    i, j = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    p, q = x[..., i].double(), x[..., j].double()
    y[..., i] = p * c - q * s
    y[..., j] = q * c + p * s
    return y


def rotate_bound(dt, x, y, f, interleaved, m):
    """Half a step of the type, and per rotated channel the errors of cos and sin
    (at most 2^-22 each), of the products and of their sum, all relative to the
    pair's two channels."""
    r = 2 * len(f)
    z = torch.zeros_like(y)
    i, j = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    t = (x[..., i].double().abs() + x[..., j].double().abs()) * abs(m)
    z[..., i] = t
    z[..., j] = t
    half = torch.finfo(DT[dt]).eps / 2
    tiny = torch.finfo(DT[dt]).tiny * torch.finfo(DT[dt]).eps / 2
    return half * y.abs() + z * 2.0 ** -21 * (1 + half) + tiny


def quantise(x, dt):
    """Codes [..., D] (int64) and scales [..., D / 32] (of type dt) of fp32 rows,
    with the fp32 operations that the definition names."""
    g = x.float().unflatten(-1, (-1, 32))
    hi, lo = g.amax(-1), g.amin(-1)
    s = torch.where(hi >= -lo, hi, lo) * -0.125
    s = torch.where(torch.isfinite(g).all(-1), s, torch.full_like(s, float("nan"))).to(DT[dt])
    s = torch.where(s.float().abs() < 2.0 ** -126, torch.zeros_like(s), s)
    inv = torch.where(s == 0, torch.zeros_like(s.float()), 1.0 / s.float())
    n = torch.round(g * inv[..., None]) + 8
    n = torch.nan_to_num(n, nan=0.0).clamp(0, 15)
    return n.flatten(-2).long(), s


def layout(D):
    """Of channel c: (byte of K's word, byte of V's word, bit of its code within the
    16-bit word before the rotation)."""
    k, v, bit = [], [], []
    for c in range(D):
        g, r = divmod(c, 32)
        k.append((r // 8) * (D // 8) + 4 * g + 2 * (r // 4 % 2))
        v.append(D // 2 + (r // 4) * (D // 16) + 2 * g)
        bit.append(4 * (c % 4))
    return k, v, bit


def pack(k, v, dt):
    """uint8 rows [..., D + D / 8] of fp32 K and V rows [..., D]."""
    D = k.shape[-1]
    at_k, at_v, bit = layout(D)
    (kn, ks), (vn, vs) = quantise(k, dt), quantise(v, dt)
    words = torch.zeros(*k.shape[:-1], D // 2, dtype=torch.int64)
    for c in range(D):
        words[..., at_k[c] // 2] |= kn[..., c].cpu() << bit[c]
        words[..., at_v[c] // 2] |= vn[..., c].cpu() << bit[c]
    words = (words >> 2 | words << 14) & 0xffff
    rows = torch.stack([words & 255, words >> 8], -1).flatten(-2).to(torch.uint8)
    scales = torch.cat([ks, vs], -1).cpu().contiguous().view(torch.uint8)
    return torch.cat([rows, scales], -1)


def unpack(rows, dt):
    """K and V [..., D] in float64 of rows (CPU)."""
    D = rows.shape[-1] // 9 * 8
    at_k, at_v, bit = layout(D)
    w = rows[..., 0:D:2].long() | rows[..., 1:D:2].long() << 8
    w = (w << 2 | w >> 14) & 0xffff
    s = rows[..., D:].contiguous().view(DT[dt]).double()
    g = torch.arange(D) // 32
    out = []
    for at, sc in ((at_k, s[..., :D // 32]), (at_v, s[..., D // 32:])):
        n = (w[..., torch.tensor(at) // 2] >> torch.tensor(bit)) & 15
        out.append((n - 8).double() * sc[..., g])
    return out

"""The table of rotary positions against 80-digit arithmetic."""
from decimal import Decimal as Dec, getcontext

import pytest


@pytest.fixture(scope="module")
def ta():
    from transformer_attention_tcgen05_gb300.build import build
    build()
    import transformer_attention_tcgen05_gb300 as ta
    return ta


def arctan_of_inverse(n):
    total, k = Dec(0), 0
    while True:
        term = Dec(1) / ((2 * k + 1) * Dec(n) ** (2 * k + 1))
        if term < Dec(10) ** -78:
            return total
        total += -term if k % 2 else term
        k += 1


def turns(rot, theta=10000.0, scaling=None, factor=1.0, original_len=0, alpha=1.0, beta=32.0):
    """Turns per position of each pair."""
    getcontext().prec = 80
    two_pi = 2 * (16 * arctan_of_inverse(5) - 4 * arctan_of_inverse(239))
    out = []
    for i in range(rot // 2):
        e = -Dec(2 * i) / rot
        f = Dec(theta) ** e
        if scaling == "linear":
            f /= Dec(factor)
        elif scaling == "ntk":
            f = (Dec(theta) * Dec(factor) ** (Dec(rot) / (rot - 2))) ** e
        elif scaling == "by_parts":
            g = (Dec(original_len) * f / two_pi - Dec(alpha)) / (Dec(beta) - Dec(alpha))
            g = min(Dec(1), max(Dec(0), g))
            f = (1 - g) * f / Dec(factor) + g * f
        out.append(f / two_pi)
    return out


@pytest.mark.parametrize("kw", [
    dict(), dict(theta=500000.0), dict(theta=1e6, scaling="linear", factor=4.1), dict(theta=0.9), dict(theta=1.0),
    dict(theta=1e300), dict(scaling="ntk", factor=8.0), dict(theta=10000.5, scaling="ntk", factor=0.37),
    dict(scaling="by_parts", factor=4.0, original_len=8192), dict(theta=500000.0, scaling="by_parts", factor=32.0,
                                                                 original_len=4096, alpha=1.7, beta=8.3)])
@pytest.mark.parametrize("rot", [16, 48, 64, 112, 128])
def test_every_entry_is_the_nearest_integer(ta, rot, kw):
    table = ta.rope_frequencies(rot, device="cpu", **kw)
    for got, f in zip(table.tolist(), turns(rot, **kw)):
        # (numbers of some 100 bits: relative errors of 2^-90 at most, 2^-27 of the last unit)
        assert abs(Dec(got) - f * 2 ** 64) <= Dec(0.5) + Dec(2) ** -27
        # so the angle at the last position, modulo a turn
        far = (got * (2 ** 31 - 1)) % 2 ** 64 - (f * (2 ** 31 - 1)) % 1 * 2 ** 64
        assert min(abs(far), 2 ** 64 - abs(far)) <= 2 ** 30 * (1 + Dec(2) ** -26)

"""Refusals of the packed entry points at the edges of their ranges (no device is touched)."""
import pytest

from tests.test_packed_cpu import INVALID, UNSUPPORTED, P, rope


@pytest.fixture(scope="module")
def L():
    from transformer_attention_tcgen05_gb300.build import build
    build()
    import transformer_attention_tcgen05_gb300 as ta
    return ta.lib()


@pytest.mark.parametrize("H", [2 ** 30 + 1, 2 ** 31 - 1])
@pytest.mark.parametrize("y", [0, 1])
def test_rope_refuses_heads_that_could_not_be_counted(L, H, y):
    """Also in place: 2^31 - 1 heads of 32 bf16 channels would fit the memory."""
    assert rope(L, y=P[y], B=1, N=1, H=H, D=32, rot=16) == UNSUPPORTED
    assert rope(L, y=P[y], B=1, N=1, H=H, D=32, rot=24) == INVALID

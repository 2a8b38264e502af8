"""Rotary positions, appends of packed rows and the 4-bit cache at the edges of what
their documentation allows."""
import pytest
import torch

from tests.test_packed_gpu import Cache, new_rows, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ta():
    from transformer_attention_tcgen05_gb300.build import build
    build()
    import transformer_attention_tcgen05_gb300 as ta
    torch.cuda.set_device(0)
    return ta


@pytest.mark.parametrize("axes", [2, 4, 5, 6, 7, 9])
def test_new_rows_of_other_ranks_are_refused(ta, axes):
    """Also as views with more strides than a packed row tensor has."""
    c = Cache([3], [2], 8, 1)
    kp, vp = (torch.zeros(c.P, 2, 8, 64, dtype=torch.bfloat16).cuda() for _ in "kv")
    pages = torch.zeros(c.P, 2, 8, 72, dtype=torch.uint8).cuda()
    good = torch.zeros(2, 2, 64, dtype=torch.bfloat16).cuda()
    rows = torch.zeros(*[2] * (axes - 1), 64, dtype=torch.bfloat16).cuda()
    rows = rows.transpose(0, axes - 2)
    assert rows.is_contiguous() == (axes == 2) and rows.stride(-1) == 1
    cu, f = torch.tensor([0, 2]).int().cuda(), ta.rope_frequencies(64)
    for kn, vn in ((rows, rows), (good, rows), (rows, good)):
        with pytest.raises(ValueError):
            ta.kv_append_paged_rope(kp, vp, kn, vn, c.dev, c.sl, f, cu_new=cu)
        with pytest.raises(ValueError):
            ta.kv_append_paged_q4(pages, kn, vn, c.dev, c.sl, f, cu_new=cu)
    assert c.sl.tolist() == [3] and ta.device_status() == 0


@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("advance", [False, True])
@pytest.mark.parametrize("wrong", [-2, "past the table"])
def test_lengths_of_sequences_without_new_tokens_are_looked_at(ta, q4, advance, wrong):
    """Whether lengths advance or not; the other sequences are served."""
    news = [2, 0, 3, 0]
    c = Cache([5, 4, 0, 16], news, 8, 2)
    g = torch.Generator().manual_seed(3)
    q, kn, vn, cu = new_rows(g, news, 2, 1, 64, "bf16")
    f = ta.rope_frequencies(64)
    pages = torch.zeros(c.P, 1, 8, 72, dtype=torch.uint8).cuda()
    kp, vp = (torch.zeros(c.P, 1, 8, 64, dtype=torch.bfloat16).cuda() for _ in "kv")

    def append():
        if q4:
            return ta.kv_append_paged_q4(pages, kn, vn, c.dev, c.sl, f, cu_new=cu, q=q, advance=advance)
        return ta.kv_append_paged_rope(kp, vp, kn, vn, c.dev, c.sl, f, cu_new=cu, q=q, advance=advance)

    c.sl[3] = c.M * 8                                     # a full table is no error
    want = append()
    assert ta.device_status() == 0
    c.sl[:] = torch.tensor([5, 4, 0, 16]).int()
    c.sl[1] = c.M * 8 + 1 if isinstance(wrong, str) else wrong
    before = c.sl.tolist()
    assert torch.equal(append(), want) and ta.device_status() == 6
    assert c.sl.tolist() == [n + m * advance for n, m in zip(before, news)]

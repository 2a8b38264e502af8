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


@pytest.mark.parametrize("advance", [False, True])
def test_4_bit_rows_in_pages_beyond_32_bit_offsets(ta, advance):
    """New rows' bytes, and what the reader gives back of K and V, in pages more than 2^32
    bytes from the pool's start against the same call on a small pool."""
    Hkv, S, D, P = 8, 128, 128, 34000
    assert (P - 20) * Hkv * S * (D + D // 8) > 2 ** 32
    g = torch.Generator().manual_seed(7)
    news = [200, 1, 40]
    c = Cache([300, 40, 127], news, S, 8)
    q, kn, vn, cu = new_rows(g, news, 2, Hkv, D, "bf16", 3, 2)
    small = torch.randint(0, 256, (c.P, Hkv, S, D + D // 8), generator=g, dtype=torch.uint8).cuda()
    small[..., D:] = torch.ones(c.P, Hkv, S, D // 16, dtype=torch.bfloat16).view(torch.uint8).cuda()
    pages = torch.empty(P, Hkv, S, D + D // 8, dtype=torch.uint8, device="cuda")
    pages[P - c.P:] = small
    far = torch.where(c.dev >= 0, c.dev + (P - c.P), c.dev)
    f, lens = ta.rope_frequencies(D), c.sl.clone()
    first = small.clone()
    a = ta.kv_append_paged_q4(small, kn, vn, c.dev, c.sl, f, cu_new=cu, q=q, advance=advance)
    b = ta.kv_append_paged_q4(pages, kn, vn, far, lens, f, cu_new=cu, q=q, advance=advance)
    assert torch.equal(a[3:-2], b[3:-2]) and torch.equal(c.sl, lens)
    assert torch.equal(pages[P - c.P:], small)
    changed = (small != first).flatten(2).any(-1).any(-1).cpu()
    for i, (n, m) in enumerate(zip(c.lens, news)):
        assert changed[c.rows(i, n, n + m)[0]].all()
    total = [n + m for n, m in zip(c.lens, news)]
    to = torch.tensor([0] + total).cumsum(0).int().cuda()
    out = [torch.zeros(2, sum(total), Hkv, D, dtype=torch.bfloat16).cuda() for _ in range(2)]
    ta.kv_gather_paged_q4(small, c.dev, to, *out[0])
    ta.kv_gather_paged_q4(pages, far, to, *out[1])
    assert torch.equal(*out) and (out[0] != 0).flatten(2).any(-1).all() and ta.device_status() == 0
    last = torch.tensor([P - 1]).int().cuda()
    ta.kv_pages_copy_q4(pages, last, last - 1)
    assert torch.equal(pages[P - 2], small[-1]) and torch.equal(pages[P - 1], small[-1])
    assert torch.equal(pages[P - c.P:P - 2], small[:-2]) and ta.device_status() == 0


@pytest.mark.parametrize("one", [False, True])
def test_rotated_rows_in_pages_beyond_32_bit_offsets(ta, one):
    """kv_append_paged_rope into pages more than 2^32 elements from the pool's start."""
    Hkv, S, D, P = 8, 128, 128, 33000
    assert (P - 20) * Hkv * S * D > 2 ** 32
    g = torch.Generator().manual_seed(9)
    news = [1, 1, 1] if one else [200, 1, 40]
    c = Cache([300, 40, 127], news, S, 10)
    q, kn, vn, cu = new_rows(g, news, 2, Hkv, D, "bf16")
    small = [randn(g, c.P, Hkv, S, D).bfloat16().cuda() for _ in "kv"]
    big = [torch.empty(P, Hkv, S, D, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    first = [x.clone() for x in small]
    for x, y in zip(big, small):
        x[P - c.P:] = y
    far = torch.where(c.dev >= 0, c.dev + (P - c.P), c.dev)
    f, lens = ta.rope_frequencies(D), c.sl.clone()
    cu = None if one else cu
    a = ta.kv_append_paged_rope(*small, kn, vn, c.dev, c.sl, f, cu_new=cu, q=q)
    b = ta.kv_append_paged_rope(*big, kn, vn, far, lens, f, cu_new=cu, q=q)
    assert torch.equal(a, b) and torch.equal(c.sl, lens) and ta.device_status() == 0
    for x, y, z in zip(big, small, first):
        assert torch.equal(x[P - c.P:], y)
        changed = (y != z).flatten(2).any(-1).any(-1).cpu()
        for i, (n, m) in enumerate(zip(c.lens, news)):
            assert changed[c.rows(i, n, n + m)[0]].all()

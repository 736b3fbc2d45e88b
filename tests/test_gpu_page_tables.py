"""Page tables that are part of something larger."""
import pytest
import torch

from tests.cache_helpers import Paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("news", [1, 30])
def test_output_right_behind_a_column_slice(news):
    """The last columns of a wide table, with the output in the same buffer right behind it."""
    import w4a16_weight_only_dequant_amd as w4
    c = Paged([200, 130, 256], [news] * 3, 4, 2, 64, "bf16", 16, seed=71)
    columns, wide = c.page_table.shape[1], 48
    values = c.q.numel()
    buf = torch.full((3 * wide + values // 2,), -7, dtype=torch.int32, device="cuda")
    table = buf[:3 * wide].view(3, wide)[:, wide - columns:]
    table.copy_(c.page_table)
    out = buf[3 * wide:].view(torch.bfloat16).view(c.q.shape)
    assert out.data_ptr() == table.data_ptr() + 4 * (2 * wide + columns)
    lse = c.lse_buffer()
    got = w4.attention(c.q_dev, c.k_cache, c.v_cache, table, c.kv_lens, q_starts=c.q_starts, max_q_len=news, out=out, lse=lse)
    assert got is out
    c.check(out, lse)
    assert torch.equal(table, c.page_table) and bool((buf[:wide - columns] == -7).all())


@pytest.mark.parametrize("news", [1, 30])
def test_no_pages_at_all(news):
    """Sequences without a key and a page table without a column: every row sees nothing."""
    import w4a16_weight_only_dequant_amd as w4
    c = Paged([5, 9], [news] * 2, 4, 2, 64, "f16", 16, seed=72)
    lse = c.lse_buffer()
    out = w4.attention(c.q_dev, c.k_cache, c.v_cache, c.page_table[:, :0], torch.zeros_like(c.kv_lens), q_starts=c.q_starts,
                       max_q_len=news, lse=lse)
    assert bool((out == 0).all()) and bool((lse == -float("inf")).all())
    out = w4.attention(c.q_dev, c.k_cache, c.v_cache, torch.zeros(2, 0, dtype=torch.int32, device="cuda"), torch.zeros_like(c.kv_lens),
                       q_starts=c.q_starts, max_q_len=news)
    assert bool((out == 0).all())
    # a length that the page table has no room for is held to none, and reported
    out = w4.attention(c.q_dev, c.k_cache, c.v_cache, torch.zeros(2, 0, dtype=torch.int32, device="cuda"), c.kv_lens,
                       q_starts=c.q_starts, max_q_len=news)
    torch.cuda.synchronize()
    assert bool((out == 0).all())
    with pytest.raises(w4.W4A16Error) as e:
        w4.attention(c.q_dev, c.k_cache, c.v_cache, c.page_table, c.kv_lens, q_starts=c.q_starts, max_q_len=news)
    assert e.value.status == 3


@pytest.mark.parametrize("news", [1, 30])
def test_strides_of_dimensions_of_one(news):
    """A cache of one KV head kept as [pages][page_size][1][dim], a page table of one column kept as a row: the same memory,
    with other strides where there is one of something."""
    import w4a16_weight_only_dequant_amd as w4
    c = Paged([14, 9, 16], [min(news, 9)] * 3, 4 if news == 1 else 8, 1, 64, "f16", 16, seed=73)
    lse = c.lse_buffer()
    kc, vc = (torch.empty(len(x), 16, 1, 64, dtype=x.dtype, device="cuda").transpose(1, 2).copy_(x) for x in (c.k_cache, c.v_cache))
    table = c.page_table[:, 0].contiguous()
    assert kc.stride(1) != c.k_cache.stride(1) and kc.data_ptr() != c.k_cache.data_ptr()
    table = table.as_strided((3, 1), (1, 3))
    for k, v in ((kc, vc), (kc, c.v_cache), (c.k_cache, vc)):
        out = w4.attention(c.q_dev, k, v, table, c.kv_lens, q_starts=c.q_starts, max_q_len=max(c.news), lse=lse)
        c.check(out, lse)
    # appending through such a view writes the cache itself
    new = torch.randn(2, 1, 64, device="cuda").to(torch.float16)
    w4.kv_append(None, new, new, kc, vc, torch.tensor([15, 5], device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(kc[0, 0, [15, 5]], new[:, 0]) and torch.equal(vc[0, 0, [15, 5]], new[:, 0])

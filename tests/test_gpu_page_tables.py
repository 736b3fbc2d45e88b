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

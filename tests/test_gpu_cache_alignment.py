"""Token rows that do not start on 16 bytes: read through a copy, refused where they are written."""
import pytest
import torch

from tests.cache_helpers import Paged

pytestmark = pytest.mark.gpu


def _shifted(x, by):
    """x's values `by` elements into a buffer, with the strides that x has."""
    buf = torch.empty(x.numel() + 8, dtype=x.dtype, device="cuda")
    return buf[by:by + x.numel()].view(x.shape).copy_(x)


@pytest.mark.parametrize("by", [1, 4, 7])
@pytest.mark.parametrize("news", [1, 30])
def test_attention(by, news):
    import w4a16_weight_only_dequant_amd as w4
    c = Paged([90, 70], [news] * 2, 6, 3, 64, "f16", 16, seed=95)
    lse = c.lse_buffer()
    q = _shifted(c.q_dev, by)
    assert q.data_ptr() % 16 and q.is_contiguous()
    args = dict(q_starts=c.q_starts, max_q_len=news, lse=lse)
    out = w4.attention(q, c.k_cache, c.v_cache, c.page_table, c.kv_lens, **args)
    c.check(out, lse)
    with pytest.raises(ValueError, match="16 bytes"):
        w4.attention(c.q_dev, c.k_cache, c.v_cache, c.page_table, c.kv_lens, out=_shifted(out, by), **args)


@pytest.mark.parametrize("by", [1, 4])
def test_append(by):
    import w4a16_weight_only_dequant_amd as w4
    gen = torch.Generator().manual_seed(96)
    q, k, v = (torch.randn(5, h, 64, generator=gen).to(torch.bfloat16).cuda() for h in (4, 2, 2))
    angles = torch.rand(9, 64, generator=gen).cuda()
    slots, positions = torch.tensor([3, 20, 7, 31, 0], device="cuda"), torch.tensor([0, 8, 3, 1, 2], dtype=torch.int32, device="cuda")
    caches = [[torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(2)]
    want = w4.kv_append(q, k, v, *caches[0], slots, positions, angles)
    shifted = [_shifted(x, by) for x in (q, k, v)]
    got = w4.kv_append(*shifted, *caches[1], slots, positions, angles)
    assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(*caches))
    with pytest.raises(ValueError, match="16 bytes"):
        w4.kv_append(shifted[0], k, v, *caches[1], slots, positions, angles, q_out=shifted[0])

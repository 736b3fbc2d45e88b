"""Rows with a score of NaN: NaN in the output and in lse, and in no other row's."""
import math

import pytest
import torch

from tests.cache_helpers import Paged

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens", [[40, 7, 33], [2900, 40, 1500]])
@pytest.mark.parametrize("news", [[1, 1, 1], [3, 4, 2], [20, 5, 30]])
def test_nan_queries_and_keys(dtype, dim, lens, news):
    """A query of NaN (every score is), a key of NaN that all rows of a sequence see and one that the last row alone
    sees; keys divided over workgroups and not."""
    import w4a16_weight_only_dequant_amd as w4
    c = Paged(lens, news, 4, 2, dim, dtype, 16, seed=61)
    lse, ref_lse = c.lse_buffer(), c.lse_buffer()

    def call(lse):
        return w4.attention(c.q_dev, c.k_cache, c.v_cache, c.page_table, c.kv_lens, q_starts=c.q_starts, max_q_len=max(news), lse=lse)
    ref = call(ref_lse)
    c.check(ref, ref_lse)
    bad = torch.zeros(c.q.shape[:2], dtype=torch.bool)
    c.q_dev[c.starts[0], 1] = math.nan                       # one head of sequence 0's first new token
    bad[c.starts[0], 1] = True
    for b, j, h in ((1, 1, 0), (2, lens[2] - 1, 1)):         # sequence 1: all rows, if they see key 1; sequence 2: the last row
        c.k_cache[int(c.page_table[b, j // 16]), h, j % 16, 3] = math.nan
        for i in range(news[b]):
            if j <= lens[b] - news[b] + i:
                bad[c.starts[b] + i, 2 * h:2 * h + 2] = True
    out = call(lse)
    torch.cuda.synchronize()
    bad = bad.cuda()
    assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all())
    out[bad], lse[bad] = ref[bad], ref_lse[bad]
    c.check(out, lse)

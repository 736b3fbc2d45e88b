"""The workspace's checks where one is needed with a single compute unit too, as the plan counts them without a device."""
import pytest

G = 1 << 32   # regions this far apart; no pointer here is ever read


def test_missing_short_and_overlapping_workspaces():
    import torch
    import w4a16_weight_only_dequant_amd as w4
    need = w4.attention_workspace_bytes(1, 32, 1, 64, 1, 64000)
    assert need > 0

    def call(**change):
        a = dict(q=1 * G, q_stride=2048, dtype=0, k_cache=2 * G, v_cache=3 * G, pages=4000, page_size=16, page_stride=16 * 64,
                 page_table=4 * G, table_stride=4000, kv_lens=5 * G, q_starts=None, tokens=1, batch=1, heads=32, kv_heads=1, dim=64,
                 max_q_len=1, max_kv_len=64000, scale=0.125, window=0, sinks=0, out=7 * G, out_stride=2048, lse=8 * G,
                 workspace=9 * G, workspace_bytes=need, stream=None)
        assert set(change) <= set(a)
        a.update(change)
        return w4.raw().w4a16_attention(*a.values())
    assert call(workspace=None) == 4
    assert call(workspace_bytes=need - 1) == 4
    assert call(workspace_bytes=0) == 4
    assert call(workspace=9 * G + 4) == 1
    for at in (G, 2 * G, 3 * G, 4 * G, 5 * G, 7 * G, 8 * G, 7 * G - 16, 8 * G + 112, 2 * G - need + 16):
        assert call(workspace=at) == 1, at
    if not torch.cuda.is_available():       # (with a device the call would go on to its launch)
        for at in (9 * G, 8 * G + 128, 7 * G + 4096, 2 * G - need - need % 16):
            assert call(workspace=at) not in (1, 4), at


@pytest.mark.parametrize("window", [0, 4000])
def test_workspace_grows_with_the_lengths(window):
    import w4a16_weight_only_dequant_amd as w4
    sizes = [w4.attention_workspace_bytes(1, 32, 1, 64, 1, n, window) for n in (0, 16, 320, 64000)]
    assert sizes[:2] == [0, 0] and sizes[-1] > 0 and sizes == sorted(sizes)

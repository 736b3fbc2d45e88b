"""What may lie right behind the page table: nothing that is not read counts as an overlap."""
import pytest


@pytest.fixture(scope="module")
def attend():
    import w4a16_weight_only_dequant_amd as w4
    G = 1 << 32

    def call(**change):
        a = dict(q=1 * G, q_stride=1024, dtype=1, k_cache=2 * G, v_cache=3 * G, pages=100, page_size=16, page_stride=2 * 16 * 128,
                 page_table=4 * G, table_stride=40, kv_lens=5 * G, q_starts=6 * G, tokens=12, batch=3, heads=8, kv_heads=2, dim=128,
                 max_q_len=4, max_kv_len=320, scale=0.1, window=0, sinks=0, out=7 * G, out_stride=1024, lse=None,
                 workspace=9 * G, workspace_bytes=1 << 31, stream=None)
        assert set(change) <= set(a)
        a.update(change)
        return w4.raw().w4a16_attention(*a.values())
    return call


def _refused(status):
    """Argument error; any other status is of what comes after the checks (no kernel runs without a device)."""
    return status == 1


def test_a_page_table_that_is_a_column_slice(attend):
    """[3][40] entries, columns 20 .. 39: the last entry read is the buffer's last, and `out` or lse may follow it."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("addresses here are not memory: with a device the call would go on to its launch")
    G = 1 << 32
    begin, end = 4 * G, 4 * G + 3 * 40 * 4        # 480 bytes
    table = begin + 20 * 4
    assert not _refused(attend(page_table=table, out=end))
    assert not _refused(attend(page_table=table, lse=end))
    for bad in (dict(out=end - 16), dict(lse=end - 4), dict(out=table + 8), dict(lse=table)):
        assert _refused(attend(page_table=table, **bad)), bad
    assert _refused(attend(page_table=table, table_stride=19))


def test_no_page_table_where_there_are_no_keys(attend):
    import torch
    if torch.cuda.is_available():
        pytest.skip("addresses here are not memory: with a device the call would go on to its launch")
    assert not _refused(attend(page_table=None, max_kv_len=0, table_stride=0))
    assert _refused(attend(page_table=None, max_kv_len=1))

"""What the cache operators' binding refuses before the library is called, and their workspaces."""
import pytest
import torch

from tests.cache_helpers import Paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import w4a16_weight_only_dequant_amd as w4
    return w4


@pytest.fixture(scope="module")
def c():
    return Paged([90, 70, 33], [2, 3, 1], 6, 3, 64, "f16", 16, seed=91)


def _i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_attention_arguments(w4, c):
    good = dict(q=c.q_dev, k_cache=c.k_cache, v_cache=c.v_cache, page_table=c.page_table, kv_lens=c.kv_lens, q_starts=c.q_starts,
                max_q_len=3)
    room = torch.zeros(6, 6 * 64 + 4, dtype=torch.float16, device="cuda")
    bads = {
        "more than the page table": [dict(max_kv_len=c.page_table.shape[1] * 16 + 1)],
        "needs max_q_len": [dict(max_q_len=None)],
        "every sequence has one token": [dict(q_starts=None, max_q_len=None), dict(q_starts=None, q=c.q_dev[:3], max_q_len=2)],
        "q must be": [dict(q=c.q_dev.bfloat16()), dict(q=c.q_dev.cpu()), dict(q=c.q_dev.flatten(1)), dict(q=c.q_dev[..., :32])],
        "k_cache must be": [dict(k_cache=c.k_cache.float()), dict(k_cache=c.k_cache[0]), dict(k_cache=c.k_cache.cpu())],
        "v_cache must have": [dict(v_cache=c.v_cache.bfloat16()), dict(v_cache=c.v_cache[1:]), dict(v_cache=c.v_cache[:, :, :8])],
        "pages must be contiguous": [dict(k_cache=c.k_cache.transpose(1, 2).contiguous().transpose(1, 2)),
                                     dict(v_cache=torch.stack([c.v_cache, c.v_cache], 1)[:, 0])],
        "page_table must be": [dict(page_table=c.page_table.long()), dict(page_table=c.page_table.cpu()), dict(page_table=c.page_table[0]),
                               dict(page_table=c.page_table.t().contiguous().t())],
        "kv_lens must be": [dict(kv_lens=c.kv_lens.long()), dict(kv_lens=c.kv_lens[:2]), dict(kv_lens=c.kv_lens.cpu())],
        "q_starts must be": [dict(q_starts=c.q_starts.long()), dict(q_starts=c.q_starts[:3])],
        "out must be": [dict(out=c.q_dev[:5]), dict(out=c.q_dev.float())],
        "out's heads must be": [dict(out=room[:, :384].unflatten(1, (6, 64))), dict(out=torch.zeros_like(c.q_dev)[:1].expand(6, 6, 64)),
                                dict(out=torch.zeros(6, 6, 128, dtype=torch.float16, device="cuda")[..., :64])],
        "lse must be": [dict(lse=torch.zeros(6, 6, dtype=torch.float16, device="cuda")), dict(lse=torch.zeros(6, 5, device="cuda")),
                        dict(lse=torch.zeros(6, 12, device="cuda")[:, ::2]), dict(lse=torch.zeros(6, 6))],
    }
    for match, changes in bads.items():
        for change in changes:
            with pytest.raises(ValueError, match=match):
                w4.attention(**{**good, **change})
    for bad in (dict(scale=0.0), dict(scale=float("nan")), dict(window=-1), dict(sinks=-1), dict(max_q_len=0), dict(max_kv_len=-1),
                dict(q=c.q_dev[:, :4]), dict(out=c.q_dev)):
        with pytest.raises(w4.W4A16Error) as e:
            w4.attention(**{**good, **bad})
        assert e.value.status == 1, bad
    lse = c.lse_buffer()
    c.check(w4.attention(**good, lse=lse), lse)       # none of them left anything behind


def test_append_arguments(w4):
    q, k = (torch.randn(5, h, 64, device="cuda").to(torch.float16) for h in (6, 3))
    cache = torch.zeros(4, 3, 16, 64, dtype=torch.float16, device="cuda")
    angles = torch.zeros(50, 32, device="cuda")
    good = dict(q=q, k=k, v=k.clone(), k_cache=cache, v_cache=cache.clone(), slots=torch.arange(5, device="cuda"), positions=_i32(0, 1, 2, 3, 4),
                cos_sin=angles)
    norm = torch.ones(64, dtype=torch.float16, device="cuda")
    bads = {
        "slots must be": [dict(slots=good["slots"].int()), dict(slots=good["slots"][:4]), dict(slots=good["slots"].cpu())],
        "positions must be": [dict(positions=good["positions"].long()), dict(positions=good["positions"][:3])],
        "a rotation takes": [dict(positions=None), dict(cos_sin=angles[0])],
        "cos_sin must be": [dict(cos_sin=angles.half()), dict(cos_sin=angles[:, ::2])],
        "q_norm must be": [dict(q_norm=norm.float()), dict(q_norm=norm[:32])],
        "k_norm must be": [dict(k_norm=norm[None])],
        "k and v must be": [dict(k=k[:, :2], v=k[:, :2]), dict(v=k[:4])],
        "same tokens": [dict(q=q[:4])],
        "k must be": [dict(k=k.bfloat16()), dict(k=k.flatten(1))],
        "q_out must be": [dict(q_out=q[:4]), dict(q_out=q.bfloat16())],
        "q_out's heads must be": [dict(q_out=q.transpose(0, 1).contiguous().transpose(0, 1))],
        "v_cache must have": [dict(v_cache=cache[:3])],
    }
    for match, changes in bads.items():
        for change in changes:
            with pytest.raises(ValueError, match=match):
                w4.kv_append(**{**good, **change})
    for bad in (dict(eps=-1.0), dict(cos_sin=angles[:, :24].contiguous()), dict(v_cache=cache)):
        with pytest.raises(w4.W4A16Error) as e:
            w4.kv_append(**{**good, **bad})
        assert e.value.status == 1, bad


@pytest.mark.parametrize("heads,new,lens", [(4, 1, 70000), (32, 20, 20000)])
def test_workspaces(w4, heads, new, lens):
    """Missing, short, misaligned or overlapping: refused, whichever kernel the rows take."""
    lib = w4.raw()
    need = w4.attention_workspace_bytes(1, heads, 2, 64, new, lens)
    assert need > 0
    q, out = (torch.zeros(new, heads, 64, dtype=torch.float16, device="cuda") for _ in range(2))
    cache = torch.zeros(2, 1, 2, 64, 64, dtype=torch.float16, device="cuda")
    table = torch.zeros(1, -(-lens // 64), dtype=torch.int32, device="cuda")
    kv_lens, starts = _i32(0), _i32(0, new)
    ws = torch.zeros(need + 64, dtype=torch.uint8, device="cuda")

    def call(at, size):
        return lib.w4a16_attention(q.data_ptr(), heads * 64, 0, cache[0].data_ptr(), cache[1].data_ptr(), 1, 64, 2 * 64 * 64, table.data_ptr(),
                                   table.shape[1], kv_lens.data_ptr(), starts.data_ptr(), new, 1, heads, 2, 64, new, lens, 0.125, 0, 0,
                                   out.data_ptr(), heads * 64, None, at, size, torch.cuda.current_stream().cuda_stream)
    assert call(None, need) == 4 and call(ws.data_ptr(), need - 1) == 4
    assert call(ws.data_ptr() + 4, need) == 1
    for t in (q, out, cache[0], cache[1], table):
        assert call(t.data_ptr(), need) == 1
    out.fill_(3.0)
    assert call(ws.data_ptr(), need) == 0
    torch.cuda.synchronize()
    assert bool((out == 0).all())       # (no key: every row sees nothing)

"""Infinities and NaN among the values: they reach the rows that see them, and those alone, at a bounded cost."""
import math

import pytest
import torch

from tests.cache_helpers import Paged, attention_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import w4a16_weight_only_dequant_amd as w4
    return w4


def _spoil(c, where):
    """Puts value `x` into element `d` of KV head `h` of sequence b's key j, in the case's plain copy and in the cache."""
    for b, j, h, d, x in where:
        c.values[b][j, h, d] = x
        page = c.v_cache.shape[2]
        c.v_cache[int(c.page_table[b, j // page]), h, j % page, d] = x


def _check(c, out, lse, window, sinks):
    """Against the formula in 64 bits: what a row sees of infinities and NaN decides its value, the rest holds to the bound."""
    share = c.q.shape[1] // c.k_cache.shape[1]
    out, lse = out.cpu().double(), lse.cpu().double()
    for b in range(len(c.lens)):
        n, kv = c.news[b], c.lens[b]
        rows = slice(c.starts[b], c.starts[b] + n)
        v = c.values[b].double()
        clean = torch.where(torch.isfinite(c.values[b]), c.values[b], torch.zeros_like(c.values[b]))
        ref, ref_lse, bound, lse_bound = attention_ref(c.q[rows], c.keys[b], clean, kv, c.dim ** -0.5, window, sinks)
        p, j = torch.arange(kv - n, kv)[:, None], torch.arange(kv)[None]
        seen = j <= p
        if window:
            seen &= (j > p - window) | (j < sinks)
        count = [(seen.double() @ m.double().flatten(1)).unflatten(1, v.shape[1:]).repeat_interleave(share, 1) > 0
                 for m in (v == math.inf, v == -math.inf, v.isnan())]
        up, down, nan = count[0], count[1], count[2] | (count[0] & count[1])
        got = out[rows]
        assert bool(got[nan].isnan().all())
        assert bool((got[up & ~nan] == math.inf).all()) and bool((got[down & ~nan] == -math.inf).all())
        rest = ~(up | down | nan)
        assert bool(((got - ref).abs()[rest] <= bound[rest]).all()), f"sequence {b}"
        some = ~torch.isinf(ref_lse)
        assert bool(((lse[rows] - ref_lse).abs()[some] <= lse_bound[some]).all())


def _attend(w4, c, lse, window, sinks, **kw):
    return w4.attention(c.q_dev, c.k_cache, c.v_cache, c.page_table, c.kv_lens, q_starts=c.q_starts, max_q_len=max(c.news),
                        window=window, sinks=sinks, lse=lse, **kw)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("news", [[1, 1, 1], [5, 3, 4], [40, 9, 150]])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 70), (130, 3)])
def test_values_that_some_rows_see(w4, dtype, dim, news, window, sinks):
    """All three kinds at the new tokens, at the window's edges, among and behind the first tokens, many in one key
    and in one tile; keys split over workgroups and not."""
    kinds = [math.inf, -math.inf, math.nan]
    for lens, kv_heads in (([1300, 420, 333], 2), ([300, 260, 310], 2)):
        c = Paged(lens, news, 4, kv_heads, dim, dtype, 16, seed=51)
        where, n = [], 0
        for b in range(3):
            first = lens[b] - news[b]
            at = {lens[b] - 1, lens[b] - 1 - news[b] // 2, first, max(0, first - 1), max(0, first - window), max(0, lens[b] - window),
                  max(0, first - window // 2), sinks, max(0, sinks - 1), 0, 40, 100, lens[b] - 2}
            for j in sorted(x for x in at if x < lens[b]):
                where.append((b, j, n % kv_heads, (7 * n) % dim, kinds[n % 3]))
                where.append((b, j, (n + 1) % kv_heads, (7 * n + dim // 2) % dim, kinds[(n + 1) % 3]))
                n += 1
        where += [(1, lens[1] - 1, 1, d, math.inf) for d in range(dim // 2, dim)]
        _spoil(c, where)
        lse = c.lse_buffer()
        out = _attend(w4, c, lse, window, sinks)
        torch.cuda.synchronize()
        _check(c, out, lse, window, sinks)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_missing_page_beside_them(w4, dim):
    """A page number behind the cache in a tile that all rows see otherwise, whose other half holds a NaN and an infinity."""
    c = Paged([700], [40], 4, 2, dim, "bf16", 16, seed=52)
    _spoil(c, [(0, 200, 0, 3, math.nan), (0, 201, 1, 4, math.inf)])       # tile of keys 192 .. 223
    table = c.page_table.clone()
    table[0, 13] = c.k_cache.shape[0]                                      # keys 208 .. 223
    out = w4.attention(c.q_dev, c.k_cache, c.v_cache, table, c.kv_lens, q_starts=c.q_starts, max_q_len=40)
    torch.cuda.synchronize()
    with pytest.raises(w4.W4A16Error) as e:
        w4.attention(c.q_dev, c.k_cache, c.v_cache, table, c.kv_lens, q_starts=c.q_starts, max_q_len=40)
    assert e.value.status == 3
    out = out.cpu()
    assert bool(out[:, :2, 3].isnan().all()) and bool((out[:, 2:, 4] == math.inf).all())
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[:, :2, 3] = keep[:, 2:, 4] = False
    assert bool(torch.isfinite(out[keep]).all())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("what", ["one", "all"])
def test_their_cost_is_bounded(w4, dim, what):
    """Row tiles whose own tokens' values hold one NaN, or hundreds of infinities, behind 6000 keys: some
    times the call without them (1.05 and 7 at most), not hundreds as where all keys of a row tile are gone through."""
    c = Paged([6020], [20], 8, 2, dim, "bf16", 64, seed=53)
    batch = 260                      # of the same pages: enough row tiles that no one's keys are divided
    q, table = c.q_dev.repeat(batch, 1, 1), c.page_table.repeat(batch, 1)
    lens = c.kv_lens.repeat(batch)
    starts = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * 20

    def timed():
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        for n in range(8):
            if n == 3:
                a.record()
            w4.attention(q, c.k_cache, c.v_cache, table, lens, q_starts=starts, max_q_len=20, max_kv_len=6020)
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b) / 5
    clean = timed()
    _spoil(c, [(0, j, h, d, math.inf) for j in range(6000, 6020) for h in range(2) for d in range(0, dim, 4)] if what == "all"
           else [(0, 6010, h, 5, math.nan) for h in range(2)])
    spoilt = timed()
    print(f"{clean * 1e3:.0f} us, {spoilt * 1e3:.0f} us with them")
    assert spoilt < 30 * clean

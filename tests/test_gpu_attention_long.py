"""Keys beyond the first 32 tiles that a wave or workgroup takes, whose page numbers come in a second and third
look at the page table. The bounds are cache_helpers', on the device in 64 bits."""
import pytest
import torch

from tests.cache_helpers import EPS32, TYPES, UNIT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import w4a16_weight_only_dequant_amd as w4
    return w4


class Long:
    """One sequence of n keys in shuffled pages. Queries look at element 0 alone: there the `marked` keys hold 24 and all others
    0, so that a row is the marked keys' values and little else, and one key too few or a wrong one shows."""

    def __init__(self, n, new, heads, kv_heads, dim, dtype, page, marked, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        dt = TYPES[dtype]
        pages = -(-n // page)
        self.n, self.new, self.page, self.dim, self.share = n, new, page, dim, heads // kv_heads
        self.k = torch.randn(pages + 2, kv_heads, page, dim, generator=gen, device="cuda", dtype=dt)
        self.v = torch.randn(pages + 2, kv_heads, page, dim, generator=gen, device="cuda", dtype=dt)
        self.k[..., 0] = 0.0
        self.table = torch.randperm(pages + 2, generator=gen, device="cuda")[:pages].int()[None]
        marked = torch.tensor(sorted({j for j in marked if 0 <= j < n}), device="cuda")
        self.k[self.table[0].long()[marked // page], :, marked % page, 0] = 24.0
        self.q = torch.zeros(new, heads, dim, dtype=dt, device="cuda")
        self.q[..., 0] = 4.0
        self.lens = torch.tensor([n], dtype=torch.int32, device="cuda")
        self.starts = torch.tensor([0, new], dtype=torch.int32, device="cuda")

    def attend(self, w4, table=None, window=0, sinks=0):
        lse = torch.zeros(self.q.shape[:2], device="cuda")
        out = w4.attention(self.q, self.k, self.v, self.table if table is None else table, self.lens, q_starts=self.starts,
                           max_q_len=self.new, max_kv_len=self.n, scale=0.125, window=window, sinks=sinks, lse=lse)
        return out, lse

    def check(self, out, lse, samples, window=0, sinks=0, hidden=None):
        u = UNIT[out.dtype]
        j = torch.arange(self.n, device="cuda")
        for i, h in samples:
            p = self.n - self.new + i
            seen = j <= p
            if window:
                seen &= (j > p - window) | (j < sinks)
            if hidden is not None:
                seen &= (j // self.page) != hidden
            rows = self.table[0].long()
            k = self.k[rows, h // self.share].flatten(0, 1)[:self.n][seen].double()
            v = self.v[rows, h // self.share].flatten(0, 1)[:self.n][seen].double()
            x = self.q[i, h].double()
            s = (k @ x) * 0.125
            want_lse = torch.logsumexp(s, 0)
            w = torch.exp(s - want_lse)
            want, size, n = w @ v, w @ v.abs(), int(seen.sum())
            d = float((k.abs() @ x.abs()).max()) * 0.125 * self.dim * EPS32
            bound = u * want.abs() + size * (u + 2 * d + 2.0 ** -21 + n * EPS32) + 2.0 ** -24
            off = (out[i, h].double() - want).abs()
            assert bool((off <= bound).all()), (i, h, float((off / bound).max()))
            assert abs(float(lse[i, h]) - float(want_lse)) <= 2 * d + n * EPS32 + 2.0 ** -21 + 4 * EPS32 * abs(float(want_lse)), (i, h)


def _reported(w4, c, table):
    torch.cuda.synchronize()
    with pytest.raises(w4.W4A16Error) as e:
        c.attend(w4, table)
    assert e.value.status == 3


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("new", [1, 8])
def test_few_rows(w4, dtype, dim, new):
    """140000 keys of 16 heads: 16 parts of each, some 273 tiles, 68 a wave. Marked: keys of each wave's tiles around the
    second and third look, in the first, a middle and the last part."""
    n, page, parts = 140000, 64, torch.cuda.get_device_properties(0).multi_processor_count // 16
    tiles = -(-n // 32)
    marked = [32 * (tiles * g // parts + w + 4 * t) + 11 for g in (0, parts // 2, parts - 1) for w in range(4)
              for t in (0, 31, 32, 33, 63, 64)]
    c = Long(n, new, 16, 16, dim, dtype, page, marked, 81)
    samples = [(0, 0), (new - 1, 7), (new // 2, 15)]
    c.check(*c.attend(w4), samples)
    table = c.table.clone()
    hidden = 32 * (4 * 33 + 2) // page             # of the third wave's 34th tile
    table[0, hidden] = c.k.shape[0] + 5
    got = c.attend(w4, table)
    _reported(w4, c, table)
    c.check(*got, samples, hidden=hidden)
    with pytest.raises(AssertionError):   # (one page shows)
        c.check(*got, samples)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (3000, 70)])
def test_many_rows(w4, dtype, dim, window, sinks):
    """6000 keys, the last 1500 of them new, 32 heads on 8: up to 94 tiles a workgroup and more. Marked: keys of the tiles
    around its second and third look, from the first key, from a split's and from the window's on."""
    n, new, page = 6000, 1500, 16
    tiles = -(-n // 32)
    marked = [32 * (start + t) + 5 for start in (0, tiles // 2, (n - new - window) // 32, (n - 700 - window) // 32) for t in (0, 31, 32, 33, 63, 64, 65)]
    c = Long(n, new, 32, 8, dim, dtype, page, marked + [3, 69, 4990, 5990], 82)
    samples = [(0, 0), (1, 9), (127, 31), (700, 16), (1234, 5), (1499, 30)]
    c.check(*c.attend(w4, window=window, sinks=sinks), samples, window, sinks)
    if window == 0:
        table = c.table.clone()
        hidden = 32 * 33 // page                   # the first half of tile 33, with a marked key
        table[0, hidden] = -3
        got = c.attend(w4, table)
        _reported(w4, c, table)
        c.check(*got, samples, hidden=hidden)
        with pytest.raises(AssertionError):   # (one page shows)
            c.check(*got, samples)

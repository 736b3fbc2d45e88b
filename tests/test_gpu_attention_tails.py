"""Weights far below the largest: many of them together still count, in fp16 too."""
import math

import pytest
import torch

from tests.cache_helpers import EPS32, TYPES, UNIT

pytestmark = pytest.mark.gpu


def _few_large(news, below, n, dim, dtype, scale):
    """Keys 0, 32, 64 and 96 score `below` over all others, whose scores are equal. Their values are zero in the first half of
    the dimension and one in the second, the others' the other way round."""
    dt = TYPES[dtype]
    heads, page = 2, 256
    pages = -(-n // page) + 1
    k = torch.zeros(pages * page, dim, dtype=dt)
    v = torch.zeros(pages * page, dim, dtype=dt)
    large = [0, 32, 64, 96]
    k[large, 0] = below / scale / 4
    v[:, :dim // 2] = 1.0
    v[large, :dim // 2] = 0.0
    v[large, dim // 2:] = 1.0
    q = torch.zeros(news, heads, dim, dtype=dt)
    q[:, 0, 0], q[:, 1, 0] = 4.0, 2.0       # (the second head: half as far below)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(1))
    kc, vc = torch.empty(pages, 1, page, dim, dtype=dt), torch.empty(pages, 1, page, dim, dtype=dt)
    kc[order], vc[order] = k.view(pages, 1, page, dim), v.view(pages, 1, page, dim)
    return q, float(k[0, 0]) * scale, kc, vc, order.int()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("news", [1, 8, 20])
@pytest.mark.parametrize("below", [13.0, 16.25, 17.5])
def test_many_small_weights_beside_a_few_large(dtype, dim, news, below):
    """exp(-13) .. exp(-17.5) of the largest weight, 131068 times, in sequences enough (of the same pages) that no
    sequence's keys are divided over workgroups, each part with a maximum of its own. Bound: a weight is rounded to the
    type (u), its exponent is off by some 2^-19 (scores of up to 18 in fp32), n sums of fp32 add n e at most; the output is
    rounded once. In fp16 a weight under 2^-14 of 2^15 (few rows) or of 2^7 at least (many), its range, has an absolute
    error of 2^-25: 2^-32 of the largest, n of them beside a sum of weights of four at least."""
    import w4a16_weight_only_dequant_amd as w4
    n, scale = 131072, 0.125
    batch = torch.cuda.get_device_properties(0).multi_processor_count * (1 if news <= 8 else 4)
    q, unit, kc, vc, table = _few_large(news, below, n, dim, dtype, scale)
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    starts = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * news
    lse = torch.full((batch * news, 2), 7.0, device="cuda")
    out = w4.attention(q.cuda().repeat(batch, 1, 1), kc.cuda(), vc.cuda(), table.cuda().repeat(batch, 1), lens, q_starts=starts,
                       max_q_len=news, max_kv_len=n, scale=scale, lse=lse)
    out, lse = out.unflatten(0, (batch, news)), lse.unflatten(0, (batch, news))
    u = UNIT[TYPES[dtype]]
    for b in (0, 1, batch // 2, batch - 1):
        for i in range(news):
            many = n - news + i + 1 - 4
            for h in (0, 1):
                s = float(q[i, h, 0]) * unit       # the large keys' score; the others' is 0
                total = 4.0 + many * math.exp(-s)
                low, high = many * math.exp(-s) / total, 4.0 / total
                rel = 2 * u + 2.0 ** -18 + n * EPS32
                tail = n * 2.0 ** -34 if dtype == "f16" else 0.0
                got = out[b, i, h].cpu().double()
                assert bool(((got[:dim // 2] - low).abs() <= low * rel + tail + 2.0 ** -25).all()), (i, h, float(got[0]), low)
                assert bool(((got[dim // 2:] - high).abs() <= high * rel).all()), (i, h, float(got[-1]), high)
                assert abs(float(lse[b, i, h]) - (s + math.log(total))) <= n * EPS32 + 2.0 ** -18


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("news", [1, 8, 20])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_scores_of_millions(dtype, news, dim):
    """Scores whose steps in fp32 are larger than one: one key takes all, the weights stay in the type's range, and
    the output is that key's value. Bounds: its weight and the output are rounded to the type (2 u); lse has some six
    roundings to fp32 of a number of its size."""
    import w4a16_weight_only_dequant_amd as w4
    gen = torch.Generator().manual_seed(5)
    dt, n, page = TYPES[dtype], 700, 64
    pages = -(-n // page)
    k = torch.zeros(pages * page, dim, dtype=dt)
    best = 311
    # distinct multiples of 2^-4 under the best, far apart beside the scores' rounding
    k[:, 0] = (torch.randint(0, 128, (pages * page,), generator=gen) * 8.0).to(dt)
    k[best, 0] = 2048.0
    v = torch.randn(pages * page, dim, generator=gen).to(dt)
    q = torch.zeros(news, 2, dim, dtype=dt)
    q[:, 0, 0], q[:, 1, 0] = 16384.0, 4096.0     # scores of 2^25 and 2^23 times the scale
    scale = 0.75
    lse = torch.zeros(news, 2, device="cuda")
    out = w4.attention(q.cuda(), k.view(pages, 1, page, dim).cuda(), v.view(pages, 1, page, dim).cuda(),
                       torch.arange(pages, dtype=torch.int32, device="cuda")[None], torch.tensor([n], dtype=torch.int32).cuda(),
                       q_starts=torch.tensor([0, news], dtype=torch.int32).cuda(), max_q_len=news, scale=scale, lse=lse)
    want = v[best].double().expand(news, 2, dim)
    assert bool(((out.cpu().double() - want).abs() <= 2 * UNIT[dt] * want.abs() + 2.0 ** -24).all())
    want = q[:, :, 0].double() * 2048.0 * scale
    assert bool(((lse.cpu().double() - want).abs() <= want * 2.0 ** -21).all())

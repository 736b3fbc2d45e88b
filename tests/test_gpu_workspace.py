"""The workspaces of captured calls: larger calls, other tensors and other
graphs in between change nothing."""
import pytest
import torch

from tests.cache_helpers import Paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w4():
    import w4a16_weight_only_dequant_amd as w4
    return w4


def _attend(w4, c, **kw):
    return w4.attention(c.q_dev, c.k_cache, c.v_cache, c.page_table, c.kv_lens, q_starts=c.q_starts, max_q_len=max(c.news), **kw)


def _graph(stream, fn):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        out = fn()
    return g, out


def _warm(stream, fn):
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        out = fn()
    stream.synchronize()
    return out


@pytest.mark.parametrize("news", [1, 40])
@pytest.mark.parametrize("own", [False, True])
def test_captured_attention_survives_growth(w4, news, own):
    """Capture on a stream, then a call on it that needs far more: replays use no memory that others have got since."""
    c = Paged([3000, 1500], [news] * 2, 8, 2, 128, "bf16", 16, seed=31)
    big = Paged([3000], [200], 32, 2, 128, "bf16", 16, seed=32)
    small_bytes = w4.attention_workspace_bytes(2, 8, 2, 128, news, c.page_table.shape[1] * 16)
    big_bytes = w4.attention_workspace_bytes(1, 32, 2, 128, 200, big.page_table.shape[1] * 16)
    assert small_bytes > 0 and big_bytes > max(small_bytes, 1 << 20)
    ws = w4.Workspace("cuda") if own else None
    s = torch.cuda.Stream()
    want = _warm(s, lambda: _attend(w4, c, workspace=ws))
    g, out = _graph(s, lambda: _attend(w4, c, workspace=ws))
    _warm(s, lambda: _attend(w4, big, workspace=ws))
    others = []
    with torch.cuda.stream(s):
        for size in [small_bytes] * 20 + [1 << 20] * 20 + [4 << 20] * 20:
            others.append(torch.full((size,), 165, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    for _ in range(4):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert all(bool((t == 165).all()) for t in others)
        _warm(s, lambda: _attend(w4, big, workspace=ws))


def test_captured_linear_survives_growth(w4):
    """The same of the linear layer's workspace, whose partial tiles grow with M."""
    gen = torch.Generator(device="cuda").manual_seed(33)
    N, K, group = 4096, 4096, 128
    w = torch.randn(N, K, generator=gen, device="cuda") * 0.02
    pw = w4.pack(w, group)
    sizes = sorted(((w4.workspace_bytes(m, N, K, group), m) for m in range(1, 2048, 37)))
    need, m = next(x for x in sizes if x[0] > 0)
    most, big = sizes[-1]
    assert most > need
    x = torch.randn(m, K, generator=gen, device="cuda").to(torch.float16)
    xb = torch.randn(big, K, generator=gen, device="cuda").to(torch.float16)
    s = torch.cuda.Stream()
    want = _warm(s, lambda: w4.linear(x, pw))
    g, out = _graph(s, lambda: w4.linear(x, pw))
    _warm(s, lambda: w4.linear(xb, pw))
    others = [torch.full((n,), 165, dtype=torch.uint8, device="cuda") for n in [need, 1 << 20] * 20]
    torch.cuda.synchronize()
    for _ in range(4):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and all(bool((t == 165).all()) for t in others)
        _warm(s, lambda: w4.linear(xb, pw))


@pytest.mark.parametrize("news", [1, 40])
def test_graphs_replay_side_by_side(w4, news):
    """Two graphs of split calls, captured one after the other on one stream, replayed on two streams at once."""
    cases = [Paged([6000, 3000], [news] * 2, 8, 2, 128, "f16", 16, seed=s) for s in (34, 35)]
    wants = [_attend(w4, c) for c in cases]
    s = torch.cuda.Stream()
    for c in cases:
        _warm(s, lambda: _attend(w4, c))
    graphs = [_graph(s, lambda: _attend(w4, c)) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for (g, out), t in zip(graphs, streams):
            with torch.cuda.stream(t):
                g.replay()
    torch.cuda.synchronize()
    for (g, out), want in zip(graphs, wants):
        assert torch.equal(out, want)

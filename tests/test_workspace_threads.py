"""Threads that share a workspace: what one call queues stays together, and its
buffer stays until then."""
import contextlib
import threading
import time
import weakref

import pytest
import torch


class Stream:
    cuda_stream = 0
    device_index = 0


def _run(jobs):
    errors = []

    def guarded(job):
        try:
            job()
        except BaseException as e:   # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=guarded, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("default", [True, False])
def test_calls_on_one_workspace_take_turns(monkeypatch, default):
    """A call queues two launches; none of another thread's comes between, and growth frees no buffer before them."""
    from w4a16_weight_only_dequant_amd import _lib
    stream = Stream()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(_lib, "_workspaces", {})
    own = None if default else _lib.Workspace("cpu")
    queued, alive = [], {}

    def job(name, nbytes):
        def call(address, size):
            ws = own or _lib._workspaces[(None, 0)]
            assert address == ws.buf.data_ptr() and size >= nbytes
            held = weakref.ref(ws.buf)
            queued.append(name)
            time.sleep(0.01)
            queued.append(name)
            alive[name] = held() is not None
            return 0
        assert _lib._queue(own, torch.device("cpu"), stream, nbytes, call) == 0
    _run([lambda i=i: job(i, (1 + i) << 20) for i in range(8)])
    assert len(queued) == 16 and queued[::2] == queued[1::2] and all(alive.values())


def test_no_workspace_no_turns():
    """A call that needs none waits for nobody."""
    from w4a16_weight_only_dequant_amd import _lib
    ws = _lib.Workspace("cpu")
    with ws.lock:
        assert _lib._queue(ws, torch.device("cpu"), None, 0, lambda a, n: (a, n)) == (None, 0)


@pytest.mark.gpu
@pytest.mark.parametrize("news", [1, 40])
def test_threads_on_one_stream(news):
    """Calls whose keys are split, from several threads on the default stream, which grow its workspace as they come."""
    import w4a16_weight_only_dequant_amd as w4
    from tests.cache_helpers import Paged
    cases = [Paged([n, n // 2], [news] * 2, 8, 2, 128, "f16", 16, seed=40 + i) for i, n in enumerate((700, 2000, 4000, 6000))]

    def attend(c):
        return w4.attention(c.q_dev, c.k_cache, c.v_cache, c.page_table, c.kv_lens, q_starts=c.q_starts, max_q_len=news)
    wants = [attend(c) for c in cases]
    torch.cuda.synchronize()
    outs = [[] for _ in cases]
    _run([lambda c=c, o=o: o.extend(attend(c) for _ in range(50)) for c, o in zip(cases, outs)])
    torch.cuda.synchronize()
    for got, want in zip(outs, wants):
        assert len(got) == 50 and all(torch.equal(x, want) for x in got)


@pytest.mark.gpu
def test_threads_on_one_stream_awq():
    """The linear layer's call of two launches, which passes scaled activations on in its workspace."""
    import w4a16_weight_only_dequant_amd as w4
    gen = torch.Generator(device="cuda").manual_seed(45)
    N, K = 1024, 2048
    pw = w4.pack(torch.randn(N, K, generator=gen, device="cuda") * 0.02, 128)
    mul = torch.rand(K, generator=gen, device="cuda") + 0.5
    xs = [torch.randn(m, K, generator=gen, device="cuda").to(torch.float16) for m in (33, 200, 500)]
    wants = [w4.linear_awq(x, mul, pw) for x in xs]
    torch.cuda.synchronize()
    outs = [[] for _ in xs]
    _run([lambda x=x, o=o: o.extend(w4.linear_awq(x, mul, pw) for _ in range(50)) for x, o in zip(xs, outs)])
    torch.cuda.synchronize()
    for got, want in zip(outs, wants):
        assert len(got) == 50 and all(torch.equal(y, want) for y in got)

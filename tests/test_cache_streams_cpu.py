"""A stream of another device than the caches' is refused."""
import pytest
import torch


class Stream:
    device = torch.device("cuda", 1)
    cuda_stream = 0


@pytest.mark.parametrize("call", ["attention", "kv_append"])
def test_streams_of_another_device(call):
    import w4a16_weight_only_dequant_amd as w4
    x = torch.zeros(1, 8, 128, dtype=torch.float16)
    cache = torch.zeros(4, 2, 16, 128, dtype=torch.float16)
    args = {"attention": (x, cache, cache, torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)),
            "kv_append": (x, x, x, cache, cache, torch.zeros(1, dtype=torch.int64))}[call]
    with pytest.raises(ValueError, match="the stream is one of cuda:1"):
        getattr(w4, call)(*args, stream=Stream())

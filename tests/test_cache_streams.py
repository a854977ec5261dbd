"""A stream of another device than the cache's is refused by every call of the cache (no GPU: the check comes first)."""
import pytest
import torch


class On:
    """What has a device (a cache, a stream) and nothing else."""

    def __init__(self, device):
        self.device = torch.device(device)


@pytest.fixture
def calls(monkeypatch):
    """The compiled module's stand-in."""
    from gather_radix_select_gb300 import _native

    class Module:
        made = []

        def __getattr__(self, name):
            return lambda *args: self.made.append(name)

    module = Module()
    Module.made = []
    monkeypatch.setattr(_native, "binding", lambda: module)
    return Module.made


@pytest.mark.parametrize("cache,stream", [("cuda:0", "cuda:1"), ("cuda:1", "cuda:0")])
def test_a_stream_of_another_device_is_refused(calls, cache, stream):
    import gather_radix_select_gb300 as sel
    from gather_radix_select_gb300 import cache as module
    for call in (lambda: sel.cache_append(None, On(cache), None, None, None, stream=On(stream)),
                 lambda: sel.cache_attention(None, On(cache), None, window=4, stream=On(stream)),
                 lambda: sel.cache_attention(None, On(cache), None, shared=4, stream=On(stream)),
                 lambda: module._launch(torch.device(cache), On(stream), calls.append)):  # (the other calls' way)
        with pytest.raises(ValueError, match="stream"):
            call()
    assert calls == []


@pytest.mark.gpu
def test_streams_of_the_caches_device_are_taken():
    import gather_radix_select_gb300 as sel
    cache = torch.randn((4, 8, 64), device="cuda").to(torch.bfloat16)
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    q = torch.randn((1, 2, 64), device="cuda").to(torch.bfloat16)
    torch.cuda.synchronize()
    want, _ = sel.cache_attention(q, cache, table, window=9)
    for stream in (torch.cuda.Stream(), torch.cuda.default_stream(), torch.cuda.ExternalStream(torch.cuda.Stream().cuda_stream)):
        got, _ = sel.cache_attention(q, cache, table, window=9, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want)

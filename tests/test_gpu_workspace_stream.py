"""The workspace that a call allocates belongs to the stream its kernels run on,
however the stream is given: memory of another stream could be handed out
again while they use it."""
import pytest

from gpu_util import torch_cuda

pytestmark = pytest.mark.gpu


class Handle:
    """A stream of another library: an object with its handle."""

    def __init__(self, raw):
        self.cuda_stream = raw


@pytest.mark.parametrize("kind", ["none", "default", "zero", "stream", "integer", "object", "default_object"])
def test_workspace_of_the_calls_stream(monkeypatch, kind):
    torch = torch_cuda()
    from stochastic_rounding_gb300 import _lib
    own = torch.cuda.Stream()
    given, raw = {"none": (None, own.cuda_stream), "default": (torch.cuda.default_stream(), 0), "zero": (0, 0),
                  "stream": (own, own.cuda_stream), "integer": (own.cuda_stream, own.cuda_stream),
                  "object": (Handle(own.cuda_stream), own.cuda_stream), "default_object": (Handle(0), 0)}[kind]
    seen, empty = [], torch.empty

    def record(*a, **kw):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return empty(*a, **kw)
    device = torch.device("cuda", torch.cuda.current_device())
    monkeypatch.setattr(torch, "empty", record)
    with torch.cuda.stream(own if kind == "none" else torch.cuda.Stream()):
        buf, pointer, size = _lib._workspace(None, 512, device, given)
        assert (_lib._stream_handle(device, given).value or 0) == raw
    assert seen == [raw] and size == 512 and pointer == buf.data_ptr()


@pytest.mark.parametrize("kind", ["zero", "integer", "object"])
def test_calls_take_a_stream_by_its_handle(kind):
    torch = torch_cuda()
    import stochastic_rounding_gb300 as asr
    torch.manual_seed(0)
    g = torch.randn(200, 300, device="cuda")
    want, out = (torch.empty(200, 300, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    asr.asr_newton_schulz([(g, want)])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    given = {"zero": 0, "integer": s.cuda_stream, "object": Handle(s.cuda_stream)}[kind]
    asr.asr_newton_schulz([(g, out)], stream=given)
    torch.cuda.synchronize()
    assert torch.equal(out, want)

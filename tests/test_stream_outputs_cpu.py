"""Outputs that a helper allocates itself come from the memory of the stream the
call runs on.  Tensors, streams and the library are stand-ins: what is looked at
is which stream was current at each allocation."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

import int8_dequant_gemm_b200 as rtq  # noqa: E402


CURRENT = 5                                      # handle of the current stream


class OnDevice(torch.Tensor):
    """A host tensor that says it is on cuda:0."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


def on_device(*shape, dtype=torch.float32):
    return torch.Tensor._make_subclass(OnDevice, torch.zeros(*shape, dtype=dtype))


class Stream:
    """torch.cuda.Stream with no CUDA behind it."""
    def __init__(self, handle=77):
        self.cuda_stream = handle
        self.device = torch.device("cuda", 0)


class OtherStream:
    """A stream of another library: a handle and a device."""
    cuda_stream = 78
    device = torch.device("cuda", 0)


class Library:
    """Every call succeeds; the last argument of each is the stream's handle."""
    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        def call(*args):
            self.streams.append(getattr(args[-1], "value", args[-1]))
            return 0
        return call


@pytest.fixture
def world(monkeypatch):
    """(library, handles of the streams current at each allocation)."""
    current, seen, library, plain = [None], [], Library(), torch.empty

    @contextlib.contextmanager
    def as_current(stream):
        before, current[0] = current[0], stream.cuda_stream
        yield
        current[0] = before

    def empty(shape, dtype=None, device=None):
        seen.append(current[0])
        return torch.Tensor._make_subclass(OnDevice, plain(shape, dtype=dtype))

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "stream", as_current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: Stream(CURRENT))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: Stream(handle))
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(rtq, "_lib", library)
    monkeypatch.setattr(rtq, "_a8_state", (
        {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}, {8: torch.int8, 3: torch.uint8},
        torch.float32, lambda index: None, lambda: 0, library))
    return library, seen


def calls():
    x, c, s = on_device(8, 64), on_device(8, 64, dtype=torch.int8), on_device(8)
    e, u16 = on_device(8, 64, dtype=torch.uint8), on_device(8, 4, 2, dtype=torch.uint16)
    x2 = on_device(8, 128)
    return {
        "quantize_a8": (2, lambda **k: rtq.quantize_a8(x, **k)),
        "addnorm_a8": (3, lambda **k: rtq.addnorm_a8(x, residual=x, **k)),
        "gate_a8": (2, lambda **k: rtq.gate_a8(x2, **k)),
        "dequant_a8": (1, lambda **k: rtq.dequant_a8(8, c, s, **k)),
        "qgemm_a8": (1, lambda **k: rtq.qgemm_a8(8, c, s, c, s, **k)),
        "qgemm_q4": (1, lambda **k: rtq.qgemm_q4(x2, e, u16, **k)),
        "qgemm_q8": (1, lambda **k: rtq.qgemm_q8(x, c, s, **k)),
        "qgemm": (1, lambda **k: rtq.qgemm(8, x, c, s, **k)),
        "gemm_e4m3": (1, lambda **k: rtq.gemm_e4m3(x, e, **k)),
        "dequant_e4m3_f32": (1, lambda **k: rtq.dequant_e4m3_f32(e, **k)),
        "dequant_e4m3_f16": (1, lambda **k: rtq.dequant_e4m3_f16(e, **k)),
        "dequant_q4_f32": (1, lambda **k: rtq.dequant_q4_f32(e, u16, **k)),
        "dequant_q4_f16": (1, lambda **k: rtq.dequant_q4_f16(e, u16, **k)),
        "dequant_q8_f32": (1, lambda **k: rtq.dequant_q8_f32(c, s, **k)),
    }


@pytest.mark.parametrize("name", list(calls()))
@pytest.mark.parametrize("stream", [Stream(), OtherStream()])
def test_outputs_belong_to_the_stream_of_the_call(world, name, stream):
    library, seen = world
    outputs, call = calls()[name]
    call(stream=stream)
    assert library.streams == [stream.cuda_stream]
    assert seen == [stream.cuda_stream] * outputs


@pytest.mark.parametrize("arguments", [{}, {"stream": Stream(CURRENT)}])
def test_on_the_current_stream_they_come_from_it_as_it_is(world, arguments):
    for name in ("quantize_a8", "addnorm_a8", "gate_a8", "dequant_a8", "qgemm_a8"):
        calls()[name][1](**arguments)
    assert world[1] == [None] * 9

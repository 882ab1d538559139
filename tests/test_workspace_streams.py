"""A workspace's memory is taken and cleared on one stream of one device: the
given stream, or the device's current one.  With a torch that only keeps
account, on the CPU; and on the device, with work pending on the other stream.
"""
import contextlib

import pytest

import hyena_long_convolution_b200 as hy


class Stream:
    def __init__(self, device, handle):
        self.device, self.cuda_stream = device, handle


class Cuda:
    """The current device and the current stream of each of two devices."""
    Stream = Stream

    def __init__(self):
        self.dev, self.streams = 0, [Stream(0, 100), Stream(1, 200)]

    def current_device(self):
        return self.dev

    def ExternalStream(self, handle):
        return Stream(self.dev, handle)

    def default_stream(self):
        return Stream(self.dev, 0)

    @contextlib.contextmanager
    def device(self, dev):
        old, self.dev = self.dev, self.dev if dev in (None, "cuda") else int(str(dev).split(":")[-1])
        yield
        self.dev = old

    @contextlib.contextmanager
    def stream(self, s):
        if s is None:
            yield
            return
        dev, old = self.dev, self.streams[s.device]
        self.dev, self.streams[s.device] = s.device, s
        yield
        self.dev, self.streams[s.device] = dev, old


class Torch:
    uint8 = "uint8"

    def __init__(self):
        self.cuda = Cuda()
        self._C = self

    def _cuda_getCurrentRawStream(self, dev):
        return self.cuda.streams[dev].cuda_stream

    def empty(self, n, dtype, device):
        with self.cuda.device(device):
            return Buffer(self.cuda.dev, self.cuda.streams[self.cuda.dev].cuda_stream)


class Buffer:
    def __init__(self, dev, stream):
        self.dev, self.stream = dev, stream

    def data_ptr(self):
        return 0x1000


class Lib:
    def __init__(self, torch):
        self.torch, self.cleared = torch, None

    def hyena_modal_workspace_init(self, ptr, n, stream):
        self.cleared = (self.torch.cuda.dev, stream)
        return 0

    def __getattr__(self, name):  # the size functions
        return lambda *a: 256


SIDE = Stream(0, 7)


@pytest.mark.parametrize("make", [lambda **k: hy.ModalWorkspace(1, 64, 8, **k),
                                  lambda **k: hy.HostWorkspace(1, 64, 8, **k),
                                  lambda **k: hy.RecurrenceWorkspace(1, 64, 64, **k)])
@pytest.mark.parametrize("kw,where", [
    (dict(), (0, 100)), (dict(device="cuda"), (0, 100)), (dict(device="cuda:1"), (1, 200)), (dict(device=1), (1, 200)),
    (dict(stream=SIDE), (0, 7)), (dict(stream=9), (0, 9)), (dict(stream=0), (0, 0)),
    (dict(stream=SIDE, device="cuda:0"), (0, 7)), (dict(stream=9, device="cuda:1"), (1, 9)),
    (dict(stream=9, device="cuda"), (0, 9)), (dict(stream=Stream(1, 8)), (1, 8))])
def test_taken_and_cleared_in_one_place(make, kw, where, monkeypatch):
    torch = Torch()
    lib = Lib(torch)
    monkeypatch.setattr(hy, "_torch", lambda: torch)
    monkeypatch.setattr(hy, "lib", lambda: lib)
    ws = make(**kw)
    assert (ws.buf.dev, ws.buf.stream) == where
    assert lib.cleared == where
    assert torch.cuda.dev == 0 and [s.cuda_stream for s in torch.cuda.streams] == [100, 200]


def test_refuses_a_stream_of_another_device(monkeypatch):
    torch = Torch()
    monkeypatch.setattr(hy, "_torch", lambda: torch)
    monkeypatch.setattr(hy, "lib", lambda: Lib(torch))
    with pytest.raises(ValueError, match="another device"):
        hy.RecurrenceWorkspace(1, 64, 64, device="cuda:1", stream=SIDE)


@pytest.mark.gpu
def test_work_pending_on_the_current_stream_does_not_reach_it():
    import torch
    n = hy.lib().hyena_gated_recurrence_workspace_size(2, 20000, 1024)
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        old = torch.empty(n, dtype=torch.uint8, device="cuda")
        a = torch.randn(8192, 8192, device="cuda")
        for _ in range(3):
            a = a @ a
        old.fill_(255)  # still to come when the workspace is made
        del old
        ws = hy.RecurrenceWorkspace(2, 20000, 1024, stream=stream)
        torch.cuda.synchronize()
        assert ws.nbytes == n and not ws.buf.any()

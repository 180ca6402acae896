"""The binding's calls on host tensors: what the library would be given, and nothing run."""
import torch


def host_calls(monkeypatch, fp8, on_run=None):
    """Lets the package's calls take host tensors until the test ends.  Returns the
    list of (library function, arguments) that they would have run; on_run(fn, args)
    is called in the place of the library."""
    calls = []

    class HostCall(fp8._Call):
        __slots__ = ()

        def __init__(self, first, stream):
            self.dev, self.index, self.stream, self.alloc = first.device, first.get_device(), 0, None

        def run(self, fn, *args):
            calls.append((fn, args))
            if on_run is not None:
                on_run(fn, args)

    monkeypatch.setattr(fp8, "_Call", HostCall)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # a host tensor's get_device
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return calls

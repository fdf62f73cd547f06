"""The paged calls of the binding on the CPU: which device and stream a call runs on, where it allocates,
and what it refuses. Tensors and the library are stand-ins that record."""
import contextlib

import pytest
import torch

from local_linear_attention_gb300 import binding


class Fake:
    """What the binding asks of a tensor."""

    def __init__(self, *shape, dtype=torch.bfloat16, index=1, contiguous=True, log=None):
        self.shape, self.dtype, self.index, self.contiguous, self.log = torch.Size(shape), dtype, index, contiguous, log
        self.device = torch.device("cuda", index) if index >= 0 else torch.device("cpu")

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return 4096

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def new_empty(self, shape, dtype=None):
        self.log.append(("new", Machine.stream))
        return Fake(*shape, dtype=dtype or self.dtype, index=self.index)


class Machine:
    """Two devices; 0 is current."""
    current, stream = 0, "current"

    @staticmethod
    @contextlib.contextmanager
    def device(index):
        before, Machine.current = Machine.current, index
        yield
        Machine.current = before

    @staticmethod
    @contextlib.contextmanager
    def on(stream):
        before, Machine.stream = Machine.stream, stream
        yield
        Machine.stream = before


@pytest.fixture
def calls(monkeypatch):
    """The library's calls as (name, current device, stream)."""
    log = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: log.append((name, Machine.current, args[-1])) or 0
    monkeypatch.setattr(binding, "_load", Library)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: Machine.current, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Machine.device)
    monkeypatch.setattr(torch.cuda, "stream", Machine.on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda raw, device: ("external", raw, device.index))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: ("default", device.index))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index, raising=False)
    return log


def problem(index, log=None):
    i32 = dict(dtype=torch.int32, index=index)
    cache = lambda: binding.PagedCache(  # noqa: E731
        Fake(4, 2, 16, 64, index=index), Fake(4, 2, 16, 64, index=index), Fake(3, 2, **i32), Fake(3, **i32),
        Fake(4, 2, 16, dtype=torch.float32, index=index))
    rows = Fake(5, 2, 64, index=index, log=log)
    return cache(), cache(), rows, Fake(4, **i32), Fake(5, 2, 64, index=index), Fake(5, 2, dtype=torch.float32, index=index)


@pytest.mark.parametrize("index", [0, 1])
def test_calls_run_on_the_device_of_the_cache(calls, index):
    cache, to, rows, starts, out, lse = problem(index)
    kept = Fake(3, 2, 8, dtype=torch.int32, index=index)
    binding.lla_paged_append(rows, rows, cache, starts)
    binding.lla_paged_attention(rows, cache, starts, 8.0, out=out, lse=lse)
    binding.lla_paged_evict(cache, to, 8, kept=kept)
    assert calls == [(f"lla_paged_{x}", index, 100 + index) for x in ("append", "attention", "evict")]
    assert Machine.current == 0


def test_a_stream_of_another_device_is_refused(calls):
    cache, to, rows, starts, out, lse = problem(1)

    class Stream:
        cuda_stream, device_index = 7, 0
    with pytest.raises(ValueError):
        binding.lla_paged_append(rows, rows, cache, starts, stream=Stream)
    with pytest.raises(ValueError):
        binding.lla_paged_attention(rows, cache, starts, 8.0, out=out, lse=lse, stream=Stream)
    with pytest.raises(ValueError):
        binding.lla_paged_evict(cache, to, 8, kept=Fake(3, 2, 8, dtype=torch.int32), stream=Stream)
    assert not calls


@pytest.mark.parametrize("raw,where", [(7, ("external", 7, 1)), (0, ("default", 1))])
def test_outputs_of_a_call_on_a_raw_stream_belong_to_it(calls, raw, where):
    log = []
    cache, to, rows, starts, _, _ = problem(1, log)
    binding.lla_paged_attention(rows, cache, starts, 8.0, stream=raw)
    assert log == [("new", where)] * 2 and calls == [("lla_paged_attention", 1, raw)]


@pytest.mark.parametrize("bad", [dict(index=0), dict(index=-1), dict(contiguous=False)])
def test_a_workspace_elsewhere_is_refused(calls, bad):
    cache, to, rows, starts, out, lse = problem(1)
    with pytest.raises(ValueError):
        binding.lla_paged_attention(rows, cache, starts, 8.0, out=out, lse=lse,
                                    workspace=Fake(4096, dtype=torch.uint8, **{"index": 1, **bad}))
    assert not calls

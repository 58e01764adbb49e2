"""Calls that go by their tensors' device do so prepared as well, whatever device is current when they are launched.  Without
a GPU: tensors, a library and a current device that stand in for them."""

import types

import pytest
import torch

import fp8_blockwise_quantized_amd as fq
from fp8_blockwise_quantized_amd import _marshal


class OnTwo(torch.Tensor):
    is_cuda = True

    def get_device(self):
        return 2


def on_two(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnTwo)


@pytest.fixture
def place(monkeypatch):
    """The current device, and those that launches were made on."""
    p = types.SimpleNamespace(current=0, launches=[])

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, p.current = p.current, self.index

        def __exit__(self, *_):
            p.current = self.before

    def launched(*_):
        p.launches.append(p.current)
        return 0

    monkeypatch.setattr(fq, "lib", lambda: types.SimpleNamespace(fp8bq_gather_rows=launched, fp8bq_quantize_int8=launched))
    monkeypatch.setattr(_marshal, "_current_device", lambda: p.current)
    monkeypatch.setattr(_marshal, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "device", Device)
    return p


CALLS = [(fq.fp8bq_gather_rows, (on_two(4, 16), on_two(8, dtype=torch.int32), 2, on_two(8, 16))),
         (fq.fp8bq_quantize_int8, (on_two(4, 16), on_two(4, 16, dtype=torch.int8), on_two(4)))]


@pytest.mark.parametrize("fn,args", CALLS, ids=lambda v: getattr(v, "__name__", ""))
def test_direct_and_prepared(place, fn, args):
    for place.current in (0, 2, 1):
        fn(*args)
        launch = fq.prepare(fn, *args)
        for place.current in (1, 2, 0):
            launch()
    assert place.launches == [2] * 12

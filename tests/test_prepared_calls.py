"""Prepared calls and the memory they hold, on the CPU: streams and tensors are
stand-ins that write down what is asked of them."""

import contextlib
from types import SimpleNamespace

import pytest

import channel_token_sparse_b200 as ds

DEV = SimpleNamespace(index=0)


class Stream:
    def __init__(self, handle, capturing=False):
        self.cuda_stream, self.capturing = handle, capturing


class Tensor:
    def __init__(self):
        self.recorded = []

    def record_stream(self, s):
        self.recorded.append(s.cuda_stream)


@pytest.fixture
def cuda(monkeypatch):
    state = SimpleNamespace(current=Stream(7), launched=[])

    @contextlib.contextmanager
    def stream(s):
        before, state.current = state.current, s
        yield
        state.current = before

    fake = SimpleNamespace(current_stream=lambda dev=None: state.current, current_device=lambda: 0, stream=stream,
                           is_current_stream_capturing=lambda: state.current.capturing)
    monkeypatch.setattr(ds, "_torch", lambda: SimpleNamespace(cuda=fake))
    return state


def handle(cuda, stream=None):
    kept, ws, out = Tensor(), Tensor(), Tensor()
    h = ds._Prepared()

    def fn(*args):
        # memory that this launch uses is promised to its stream by now
        cuda.launched.append((args[-1], list(ws.recorded)))
        return ds.DS_OK

    h._bind(fn, [1, 2], DEV, stream, (kept, None, ws), (out, None))
    return h, kept, ws, out


def test_calls_on_the_stream_of_the_memory_record_nothing(cuda):
    h, *tensors = handle(cuda)
    assert h()[0] is tensors[2] and h()[1] is None
    assert [t.recorded for t in tensors] == [[], [], []] and cuda.launched == [(7, []), (7, [])]


def test_calls_on_other_streams_keep_the_memory(cuda):
    """Made on one stream, called on others and then dropped: the workspace,
    the inputs and the output must wait for each of them, from before the launch."""
    h, *tensors = handle(cuda)
    for s in (8, 8, 9, 7, 8):
        cuda.current = Stream(s)
        h()
    assert [t.recorded for t in tensors] == [[8, 9]] * 3
    assert cuda.launched == [(8, [8]), (8, [8]), (9, [8, 9]), (7, [8, 9]), (8, [8, 9])]


def test_a_bound_stream_is_recorded(cuda):
    """Inputs of the current stream, used on the stream that was given."""
    h, *tensors = handle(cuda, Stream(11))
    h()
    h()
    assert [t.recorded for t in tensors] == [[11]] * 3 and cuda.launched == [(11, [11])] * 2


def test_captured_calls_record_at_the_first_real_one(cuda):
    h, *tensors = handle(cuda)
    cuda.current = Stream(8, capturing=True)
    h()
    assert [t.recorded for t in tensors] == [[]] * 3
    cuda.current = Stream(8)
    h()
    assert [t.recorded for t in tensors] == [[8]] * 3


def test_a_call_made_at_once_takes_the_stream_of_its_call(cuda):
    kept, out = Tensor(), Tensor()
    for stream, recorded in ((None, []), (Stream(12), [12])):
        h = ds._Prepared()
        h._bind(lambda *a: ds.DS_OK, [], DEV, stream, (kept,), out, True)
        assert h() is out and kept.recorded == recorded and out.recorded == recorded

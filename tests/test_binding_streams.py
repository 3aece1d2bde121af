"""CPU checks of where the binding takes its own workspaces from: the pool of the stream that
will use them (a fake of torch's streams and allocator records it; no call reaches a GPU)."""
import contextlib
from types import SimpleNamespace

import pytest
import torch


@pytest.fixture(scope="module")
def Y():
    import gated_retention_shared_gb300 as Y
    return Y


class Stream:
    def __init__(self, cuda_stream):
        self.cuda_stream = cuda_stream


class Memory:
    """What torch.empty gives here: memory of the stream that is current."""

    def __init__(self, nbytes, pool):
        self.nbytes, self.pool = nbytes, pool

    def data_ptr(self):
        return 0x10000

    def record_stream(self, stream):
        pass


@pytest.fixture
def current(Y, monkeypatch):
    """The stack of current streams' handles; stream 1 is current outside any context."""
    stack = [1]

    @contextlib.contextmanager
    def stream(s):
        stack.append(s.cuda_stream)
        yield
        stack.pop()

    cuda = SimpleNamespace(stream=stream, Stream=Stream, ExternalStream=lambda handle, device=None: Stream(handle))
    empty = lambda n, dtype=None, device=None: Memory(n, stack[-1])  # noqa: E731
    monkeypatch.setattr(Y, "torch", SimpleNamespace(cuda=cuda, empty=empty, uint8=torch.uint8))
    return stack


CACHE = SimpleNamespace(k=SimpleNamespace(device="cuda:0"), _dev=0)


@pytest.mark.parametrize("stream,pool", [(None, 1), (Stream(7), 7), (SimpleNamespace(cuda_stream=9), 9)])
@pytest.mark.parametrize("nbytes", [512, lambda: 512])
def test_paged_workspace_belongs_to_the_stream_that_uses_it(Y, current, stream, pool, nbytes):
    ws, ptr, n = Y._paged_workspace(nbytes, CACHE, None, stream)
    assert (ws.pool, n) == (pool, 512) and current == [1]


@pytest.mark.parametrize("stream,pool", [(None, 1), (Stream(7), 7), (SimpleNamespace(cuda_stream=9), 9)])
def test_workspace_belongs_to_the_stream_that_uses_it(Y, current, stream, pool):
    assert Y._workspace(512, "cuda:0", None, stream).pool == pool and current == [1]
    assert Y._workspace(0, "cuda:0", None, stream) is None  # a call that needs none
    assert Y._workspace(512, "cuda:0", "mine", stream) == "mine"


def test_every_call_says_which_stream_its_workspace_is_for(Y):
    """Each call's workspace is made for the stream that the call is given."""
    import inspect
    import re
    source = inspect.getsource(Y)
    made = re.findall(r"ws(?:, wp, wn)? = _(?:paged_)?workspace\(.*", source)
    assert made and all(m.endswith("workspace, stream)") for m in made)

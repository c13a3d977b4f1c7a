"""Which workspace a call without one of its own gets (CPU; the stream, its
capture state and the device allocation are stand-ins)."""
import types

import pytest
import torch

from int4_output_head_amd import binding

DEV = torch.device("cuda:0")


class Made:
    def __init__(self, nbytes, device):
        self.nbytes, self.device = nbytes, device


@pytest.fixture
def state(monkeypatch):
    s = types.SimpleNamespace(stream=7, capturing=False)
    monkeypatch.setattr(binding, "Workspace", Made)
    monkeypatch.setattr(binding, "_ws_cache", {})
    monkeypatch.setattr(binding, "_current_device", lambda: 0)
    monkeypatch.setattr(binding, "_raw_stream", lambda index: s.stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: s.capturing)
    return s


def test_eager_calls_of_a_stream_share_one_and_grow_it(state):
    a = binding._default_workspace(DEV, 100)
    assert binding._default_workspace(DEV, 80) is a
    b = binding._default_workspace(DEV, 200)
    assert b is not a and b.nbytes == 200 and binding._default_workspace(DEV, 100) is b
    state.stream = 8
    assert binding._default_workspace(DEV, 100) is not b


def test_a_capture_never_holds_the_shared_one(state):
    """A graph keeps the addresses that it was captured with, and a larger
    eager call frees the shared workspace: what a capture uses must be its own."""
    a = binding._default_workspace(DEV, 100)
    state.capturing = True
    g1, g2 = binding._default_workspace(DEV, 100), binding._default_workspace(DEV, 300)
    assert len({id(w) for w in (a, g1, g2)}) == 3 and g2.nbytes == 300
    state.capturing = False
    assert binding._default_workspace(DEV, 100) is a


def test_a_capture_leaves_nothing_for_eager_calls(state):
    """Its initialisation is only recorded: an eager call would find a workspace
    that nothing has initialised yet."""
    state.capturing = True
    g = binding._default_workspace(DEV, 100)
    state.capturing = False
    assert binding._default_workspace(DEV, 100) is not g


def test_a_failed_launch_drops_the_shared_ones(state):
    """A call of several kernels that fails between them leaves its control
    words set: the next call has to get an initialised workspace."""
    a = binding._default_workspace(DEV, 100)
    with pytest.raises(RuntimeError):
        binding._raise(binding.EINVAL, "call")
    assert binding._default_workspace(DEV, 100) is a
    with pytest.raises(RuntimeError):
        binding._raise(binding.EHIP, "call")
    assert binding._default_workspace(DEV, 100) is not a

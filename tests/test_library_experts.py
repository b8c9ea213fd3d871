"""The plans of a compressed expert layer without a GPU: which are kept, which streams use their memory, on which device they run."""
import contextlib
import gc
import types
import weakref

import pytest
import torch

import lossless_entropy_coded_ecf8_amd as E
from lossless_entropy_coded_ecf8_amd import binding
from lossless_entropy_coded_ecf8_amd import experts as X


class Plan:
    made = 0

    def __init__(self, encs, out, offsets, stream):
        Plan.made += 1
        self.encs, self.offsets, self.runs = encs, offsets, 0

    def run(self, stream):
        self.runs += 1


@pytest.fixture
def layer(monkeypatch):
    """A layer of five experts whose plans are stand-ins, on the CPU; layer.state.capturing: whether the launch stream is captured."""
    state = types.SimpleNamespace(capturing=False, launches=[])

    @contextlib.contextmanager
    def launch(device, stream):
        state.launches.append((device, stream))
        yield 0

    monkeypatch.setattr(X.binding, "DecodePlan", Plan)
    monkeypatch.setattr(X, "_capturing", lambda stream: state.capturing)
    monkeypatch.setattr(X, "_empty", lambda n, dtype, device, stream: torch.empty(n, dtype=dtype))
    monkeypatch.setattr(X, "_Launch", launch)
    g = torch.Generator().manual_seed(1)
    stack = [torch.randint(0, 100, (16, 16), generator=g, dtype=torch.uint8) for _ in range(5)]
    made = E.ECF8Experts(stack, stack, stack, torch.ones(3, 5), device="cpu")
    made.state = state
    Plan.made = 0
    return made


def test_a_plan_that_a_capture_used_lives_as_long_as_the_layer(layer):
    """The graph's replays read the plan's workspace, whichever experts are named in the meantime."""
    layer.decode([0, 3])
    ref = weakref.ref(layer._plan((0, 3), None))
    layer.state.capturing = True
    layer.decode([3, 0])
    layer.state.capturing = False
    for other in ([1], [2], [1, 4]):
        layer.decode(other)
    gc.collect()
    assert ref() is not None
    made = Plan.made
    layer.decode([0, 3])                                          # its plan again
    assert Plan.made == made and ref().runs == 3
    layer.state.capturing = True
    layer.decode([0, 3])                                          # another graph
    layer.state.capturing = False
    layer.decode([2])
    gc.collect()
    assert ref() is not None and ref().runs == 4


def test_a_plan_that_no_capture_used_goes_when_others_are_named(layer):
    layer.decode([0, 3])
    ref = weakref.ref(layer._plan((0, 3), None))
    layer.decode()
    layer.decode([1])
    gc.collect()
    assert ref() is None
    layer.state.capturing = True
    layer.decode()                                                # the whole layer's plan stays anyway
    with pytest.raises(RuntimeError):
        layer.decode([0, 3])


def test_decoding_runs_on_the_layers_device(layer):
    """Whichever device is current: the launch is made as the products are."""
    side = object()
    layer.decode([1], stream=side)
    layer.decode()
    assert layer.state.launches == [(layer.device, side), (layer.device, None)] and layer.device == layer.scales.device


class Memory:
    def __init__(self):
        self.users = []

    def record_stream(self, stream):
        self.users.append(stream)


class Stream:
    def __init__(self, handle):
        self.cuda_stream, self.waits = handle, []

    def wait_event(self, event):
        self.waits.append(event)


@pytest.mark.parametrize("kind", [binding.DecodePlan, binding.DecodePlanV])
def test_a_plans_memory_is_known_to_be_used_on_the_streams_that_run_it(kind):
    """Freed while such a stream still runs it, the memory goes to no other work of the stream that prepared it before that run ends."""
    plan = object.__new__(kind)
    maker, side = Stream(5), Stream(6)
    plan.workspace, plan.out, plan._ready, plan._synced = Memory(), Memory(), "event", {maker.cuda_stream}
    for _ in range(2):
        assert plan._launch_stream(maker).value == 5 and plan._launch_stream(side).value == 6
    assert plan.workspace.users == [side] and plan.out.users == [side] and side.waits == ["event"] and maker.waits == []

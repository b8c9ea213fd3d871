"""How the operators of include/ecf8a.h order streams, without a GPU: stand-ins for torch's streams and events, and for
the library."""
import contextlib
import os
import subprocess
import sys
import types

import pytest
import torch

from lossless_entropy_coded_ecf8_amd import adapters as A

DEV = torch.device("cuda", 0)


class Stream:
    def __init__(self, handle, name, device=DEV):
        self.cuda_stream, self.name, self.device, self.waits, self.capturing = handle, name, device, [], False

    def wait_event(self, event):
        self.waits.append(event)


class Event:
    made = 0

    def __init__(self):
        self.on = None
        Event.made += 1

    def record(self, stream):
        self.on = stream


class Memory:
    """A device buffer: who else uses it."""

    def __init__(self):
        self.users = []

    def record_stream(self, stream):
        self.users.append(stream)

    def data_ptr(self):
        return 1 << 40

    def numel(self):
        return 1 << 30


class Operand:
    """A tensor on the GPU, as far as the argument checks look at one."""

    def __init__(self, n, dtype):
        self.n, self.dtype, self.device, self.is_cuda = n, dtype, DEV, True

    def dim(self):
        return 1

    def is_contiguous(self):
        return True

    def numel(self):
        return self.n

    def data_ptr(self):
        return 1 << 41

    def record_stream(self, stream):
        pass


@pytest.fixture
def gpu(monkeypatch):
    """The default stream (handle 0) current on one device; a stream made from handle 0 is a new one, as torch's is."""
    g = types.SimpleNamespace(default=Stream(0, "default"), calls=[])
    g.current = g.default

    @contextlib.contextmanager
    def stream(s):
        before, g.current = g.current, s
        yield
        g.current = before

    def call(name):
        return lambda *a: g.calls.append(name) or 0

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: g.current)
    known = {}                                                    # torch's identity of a stream: id, device, type
    monkeypatch.setattr(torch._C, "_cuda_getCurrentStream", lambda i: known.setdefault(id(g.current), g.current) and (id(g.current), i, 1), raising=False)
    monkeypatch.setattr(torch.cuda, "Stream", lambda stream_id, device_index, device_type: known[stream_id])
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: g.current.capturing)
    monkeypatch.setattr(torch.cuda, "Event", Event)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle or 999, "from a handle"))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: g.current.cuda_stream, raising=False)
    monkeypatch.setattr(A, "_empty", lambda *a: Memory())
    lib = types.SimpleNamespace(ecf8a_plan_bytes=lambda *a: 256, ecf8a_plan_prepare=call("plan"),
                                ecf8a_clip_bytes=lambda *a: 256, ecf8a_clip_prepare=call("clip_prepare"), ecf8a_clip_run=call("clip_run"))
    monkeypatch.setattr(A, "_lib", lambda: lib)
    return g


def use(plan, gpu, stream=None):
    """What a call does that uses the plan on `stream`."""
    plan._order((stream or gpu.current).cuda_stream, stream)


def test_a_plan_of_the_default_stream_is_waited_for(gpu):
    """The event lies on the stream that groups, also where that is the default one, whose handle is 0."""
    plan = A.AdapterPlan(Operand(10, torch.int32), 2)
    use(plan, gpu)
    side = Stream(5, "side")
    use(plan, gpu, side)
    assert gpu.default.waits == [] and [e.on for e in side.waits] == [gpu.default] and plan.workspace.users == [side]


def test_a_plan_of_the_current_side_stream_is_waited_for(gpu):
    maker, side = Stream(5, "maker"), Stream(6, "side")
    with torch.cuda.stream(maker):
        plan = A.AdapterPlan(Operand(10, torch.int32), 2)
        use(plan, gpu)
    use(plan, gpu)
    use(plan, gpu, side)
    assert maker.waits == [] and [e.on for e in gpu.default.waits + side.waits] == [maker, maker]


def test_another_thread_sees_the_event_only_once_it_is_recorded(gpu, monkeypatch):
    plan = A.AdapterPlan(Operand(10, torch.int32), 2)
    other = Stream(6, "other thread's")

    def record(event, stream):
        monkeypatch.setattr(Event, "record", lambda e, s: setattr(e, "on", s))
        use(plan, gpu, other)                                     # in the middle of this thread's record
        event.on = stream

    monkeypatch.setattr(Event, "record", record)
    use(plan, gpu, Stream(5, "side"))
    assert [e.on for e in other.waits] == [gpu.default]


def test_captured_calls_and_captured_plans(gpu):
    """What counts is whether the launch stream is captured, not whether the current one is."""
    plan = A.AdapterPlan(Operand(10, torch.int32), 2)
    side, eager = Stream(5, "side"), Stream(6, "eager")
    side.capturing = True
    use(plan, gpu, side)                                          # captured: no wait
    with torch.cuda.stream(side):
        captured = A.AdapterPlan(Operand(10, torch.int32), 2)
        use(plan, gpu, eager)                                     # not captured, beside a capture
    use(captured, gpu, eager)                                     # filled by the replay, which the caller orders
    assert side.waits == [] and [e.on for e in eager.waits] == [gpu.default]
    with torch.cuda.stream(Stream(7, "maker")) as _:
        maker, plan = gpu.current, A.AdapterPlan(Operand(10, torch.int32), 2)
    maker.capturing = True                                        # an event of it would be the capture's
    with pytest.raises(RuntimeError):
        use(plan, gpu, eager)


@pytest.mark.parametrize("given", [True, False])
def test_a_clip_is_not_made_in_a_capture(gpu, given):
    """Its list comes from host memory that is gone when a replay would copy it."""
    side = Stream(5, "side")
    side.capturing = True
    grads = [Operand(10, torch.float32)]
    with contextlib.nullcontext() if given else torch.cuda.stream(side):
        for make in (A.GradClip, lambda g, stream: A.clip_grad_norm(g, 1.0, stream=stream)):
            with pytest.raises(RuntimeError):
                make(grads, stream=side if given else None)
    assert gpu.calls == []


STAND_IN = r"""
extern "C" int status, copies;
int status = 0, copies = 0;
extern "C" int hipStreamIsCapturing(void*, int* s) { *s = status; return 0; }
extern "C" int hipMemcpyAsync(void*, const void*, unsigned long, int, void*) { ++copies; return 0; }
"""

PREPARE = r"""
import ctypes, sys
hip = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)           # before the library, so that it finds these functions
from lossless_entropy_coded_ecf8_amd import adapters as A
L, P = A._lib(), 1 << 40
status, copies = (ctypes.c_int.in_dll(hip, n) for n in ("status", "copies"))
got = []
for status.value in (0, 1, 2):                                    # none, active, invalidated
    arr, c = (A.GradA * 1)(A.GradA(P, P, 8)), A.ClipPlanA()
    got += [L.ecf8a_clip_prepare(arr, 1, 3, P, 1 << 30, None, ctypes.byref(c)), copies.value, int(c.pieces)]
print(got)
"""


def test_the_library_refuses_a_captured_stream(tmp_path):
    """ecf8a_clip_prepare on a stream whose capture status the stand-in gives: no copy is asked for in a capture."""
    src, so = tmp_path / "hip.cpp", tmp_path / "hip.so"
    src.write_text(STAND_IN)
    subprocess.run(["g++", "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    p = subprocess.run([sys.executable, "-c", PREPARE, str(so)], cwd=root, capture_output=True, text=True, timeout=300)
    assert p.stdout.strip() == str([0, 1, 1, -1, 1, 0, -1, 1, 0]), (p.stdout, p.stderr[-2000:])


def test_runs_of_one_clip_wait_for_each_other(gpu):
    """They share the partial sums: a run waits for the last one's stream, whichever that was."""
    plan = A.GradClip([Operand(10, torch.float32)])
    one, two = Stream(5, "one"), Stream(6, "two")
    plan.run(1.0)
    assert gpu.default.waits == []
    plan.run(1.0, stream=one)
    plan.run(1.0, stream=one)
    assert [e.on for e in one.waits] == [gpu.default]
    plan.run(1.0, stream=two)
    assert [e.on for e in two.waits] == [one]
    plan.run(1.0)
    assert [e.on for e in gpu.default.waits] == [two] and plan.workspace.users == [one, two, gpu.default]
    assert gpu.calls == ["clip_prepare"] + ["clip_run"] * 5


def test_captured_runs_of_a_clip(gpu):
    """A captured run does not wait and is not waited for; the stream that counts is the launch stream."""
    plan = A.GradClip([Operand(10, torch.float32)])
    captured, eager = Stream(5, "captured"), Stream(6, "eager")
    captured.capturing = True
    plan.run(1.0, stream=captured)
    with torch.cuda.stream(captured):
        plan.run(1.0)
        plan.run(1.0, stream=eager)                               # not captured, beside a capture
    assert captured.waits == [] and [e.on for e in eager.waits] == [gpu.default]
    eager.capturing = True                                        # an event of it would be the capture's
    with pytest.raises(RuntimeError):
        plan.run(1.0)

"""CPU checks of how the binding (retnet_scale_retention_amd/msr.py) uses torch's
memory, streams and devices: host tensors that say they lie on the device, a
library that records its calls, and streams that are names.  Nothing is
launched."""
import contextlib

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from retnet_scale_retention_amd import msr as m  # noqa: E402


class OnDevice(torch.Tensor):
    """A host tensor that passes for a tensor on device `index` and knows the stream whose pool it came from."""
    index, pool = 0, "the caller's"
    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.index))

    def get_device(self):
        return self.index

    def record_stream(self, stream):
        self.recorded = [*getattr(self, "recorded", []), stream]


class Stream:
    def __init__(self, name, index=0):
        self.name, self.device_index, self.device, self.cuda_stream = name, index, torch.device("cuda", index), 0x5000 + 16 * index


class Library:
    """Every entry point records its arguments and the device that is current, and succeeds."""

    def __init__(self, world):
        self.world, self.calls = world, []

    def __getattr__(self, name):
        def call(*args):
            if name in ("msr_workspace_size", "msr_add_rmsnorm_backward_workspace"):
                if name == "msr_workspace_size":
                    args[3]._obj.value = 4096
                    return 0
                return 4096
            self.calls.append((name, args, self.world.device))
            return 0
        return call


class World:
    """The current device and stream, and every tensor that the binding allocated."""

    def __init__(self, monkeypatch):
        self.device, self.stream, self.made = 0, Stream("current"), []
        real = torch.empty

        def empty(*shape, dtype=None, device=None, **kw):
            t = real(*shape, dtype=dtype, **kw).as_subclass(OnDevice)
            t.index, t.pool = torch.device(device).index or 0, self.stream
            self.made.append(t)
            return t

        @contextlib.contextmanager
        def on_stream(stream):
            old = self.device, self.stream
            self.device, self.stream = stream.device_index, stream
            yield
            self.device, self.stream = old

        @contextlib.contextmanager
        def on_device(index):
            old, self.device = self.device, torch.device("cuda", index).index if isinstance(index, int) else index.index
            yield
            self.device = old

        monkeypatch.setattr(torch, "empty", empty)
        monkeypatch.setattr(torch, "empty_like", lambda t, **kw: empty(t.shape, dtype=t.dtype, device=t.device))
        monkeypatch.setattr(torch.cuda, "stream", on_stream)
        monkeypatch.setattr(torch.cuda, "device", on_device)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.stream)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.device)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: self.device, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
        monkeypatch.setattr(m, "_tc", None)
        self.lib = Library(self)
        monkeypatch.setattr(m, "_lib", self.lib)
        monkeypatch.setattr(m, "load", lambda: self.lib)


@pytest.fixture
def world(monkeypatch):
    return World(monkeypatch)


def on_device(*shape, dtype=torch.bfloat16, index=0):
    t = torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)
    t.index = index
    return t


F8 = torch.float8_e4m3fn
GAMMA = np.full(2, 0.9, np.float32)


def calls(index=0):
    """name -> a call of every entry point that takes a stream, on tensors of device `index`."""
    t = lambda *s, dtype=torch.bfloat16: on_device(*s, dtype=dtype, index=index)
    x, f32 = t(64, 256), torch.float32
    q, k, v = t(1, 8, 2, 16), t(1, 8, 2, 16), t(1, 8, 2, 32)
    xs, wq, wk, wv = t(1, 8, 64), t(32, 64), t(32, 64), t(64, 64)
    return {
        "add_rmsnorm": lambda **kw: m.msr_add_rmsnorm(x, t(256), t(64, 256), want_q=True, **kw),
        "add_rmsnorm_backward": lambda **kw: m.msr_add_rmsnorm_backward(x, t(256), t(64, 256), **kw),
        "quantize": lambda **kw: m.msr_quantize(x, want_transposed=True, **kw),
        "scaled_matmul": lambda **kw: m.msr_scaled_matmul(t(4, 128, dtype=F8), t(4, 1, dtype=f32), t(9, 128, dtype=F8),
                                                          t(9, 1, dtype=f32), **kw),
        "parallel": lambda **kw: m.msr_parallel(q, k, v, GAMMA, **kw),
        "chunkwise": lambda **kw: m.msr_chunkwise(q, k, v, GAMMA, 8, **kw),
        "chunkwise_backward": lambda **kw: m.msr_chunkwise_backward(q, k, v, GAMMA, 8, t(1, 8, 2, 32), **kw),
        "qkv_projection": lambda **kw: m.msr_qkv_projection(xs, wq, wk, wv, 2, **kw),
        "qkv_chunkwise": lambda **kw: m.msr_qkv_chunkwise(xs, wq, wk, wv, GAMMA, 8, **kw),
        "recurrent_step": lambda **kw: m.msr_recurrent_step(t(1, 2, 16), t(1, 2, 16), t(1, 2, 32),
                                                            t(1, 2, 16, 32, dtype=f32), GAMMA, 3, **kw),
    }


NAMES = sorted(calls())


def flat(r):
    return [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_on_a_stream_comes_from_that_stream(world, name):
    here, there = world.stream, Stream("another")
    results = flat(calls()[name](stream=there))
    assert world.made and world.stream is here
    for t in world.made:
        # the pool of the stream that writes it, so that nothing else is under way in it, and nothing else gets it early
        assert t.pool is there
        kept = any(t is r for r in results)
        # what the caller gets may be dropped while the caller's stream still reads it
        assert getattr(t, "recorded", []) == ([here] if kept else [])


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_on_the_current_stream(world, name):
    calls()[name]()
    assert world.made and all(t.pool is world.stream and not hasattr(t, "recorded") for t in world.made)


WITH_WORKSPACE = ["add_rmsnorm_backward", "parallel", "chunkwise", "chunkwise_backward", "qkv_chunkwise"]


@pytest.mark.parametrize("name", WITH_WORKSPACE)
def test_workspace_that_the_kernels_cannot_write_is_refused(world, name):
    bad = {"host": torch.zeros(8192, dtype=torch.uint8),
           "another device": on_device(8192, dtype=torch.uint8, index=1),
           "expanded": on_device(1, dtype=torch.uint8).expand(8192),
           "strided": on_device(8192, 2, dtype=torch.uint8)[:, 0]}
    for what, ws in bad.items():
        with pytest.raises(ValueError, match="workspace"):
            calls()[name](workspace=ws)
        assert not world.lib.calls, what


@pytest.mark.parametrize("name", WITH_WORKSPACE)
def test_workspace_is_taken_by_its_bytes(world, name):
    def passed(ws):
        world.lib.calls.clear()
        calls()[name](workspace=ws)
        values = [getattr(a, "value", a) for a in world.lib.calls[0][1]]
        return ws.data_ptr() in values, values
    used, values = passed(on_device(1024, dtype=torch.float32))  # 4096 bytes: as many as are needed
    assert used and 4096 in values
    used, values = passed(on_device(9000, dtype=torch.uint8))    # the whole size is passed on
    assert used and 9000 in values
    used, values = passed(on_device(1023, dtype=torch.float32))  # too small: the call brings its own
    assert not used and 4096 in values


NOALLOC = {"chunkwise_noalloc": lambda index: lambda **kw: m.msr_chunkwise_noalloc(
    *(on_device(1, 8, 2, w, index=index) for w in (16, 16, 32)), GAMMA, 8, out=on_device(1, 8, 2, 32, index=index), **kw)}


@pytest.mark.parametrize("name", NAMES + sorted(NOALLOC))
def test_launches_go_to_the_tensors_device(world, name):
    for index in (0, 1):
        world.lib.calls.clear()
        (NOALLOC[name](index) if name in NOALLOC else calls(index)[name])()
        assert [c[2] for c in world.lib.calls] == [index] and world.device == 0


@pytest.mark.parametrize("name", NAMES + sorted(NOALLOC))
def test_a_stream_of_another_device_is_refused(world, name):
    call = NOALLOC[name](0) if name in NOALLOC else calls(0)[name]
    with pytest.raises(ValueError, match="stream is of device 1"):
        call(stream=Stream("elsewhere", 1))
    assert not world.lib.calls and world.device == 0

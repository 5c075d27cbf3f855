"""CPU checks of how the binding of the operators next to retention uses torch's
memory, streams and devices, with the stand-ins of test_binding_cpu.py: host
tensors that say they lie on the device, and a library that records its calls.
Nothing is launched."""
import pytest

torch = pytest.importorskip("torch")

from retnet_scale_retention_amd import msr as m  # noqa: E402
from tests import test_binding_cpu as base  # noqa: E402
from tests.test_binding_cpu import OnDevice, Stream, flat, on_device  # noqa: E402


class Library(base.Library):
    def __getattr__(self, name):
        return (lambda *a: 4096) if name.endswith("_workspace") else super().__getattr__(name)


@pytest.fixture
def world(monkeypatch):
    w = base.World(monkeypatch)
    w.lib = Library(w)
    monkeypatch.setattr(m, "_lib", w.lib)
    monkeypatch.setattr(m, "load", lambda: w.lib)
    m._setup()
    monkeypatch.setattr(m._tc, "tensor", OnDevice)
    return w


F32 = torch.float32


def calls(index=0):
    t = lambda *s, dtype=torch.bfloat16: on_device(*s, dtype=dtype, index=index)
    q, k, x, rate = t(2, 8, 4, 16), t(2, 8, 2, 16), t(2, 100, 24), t(24, dtype=F32)
    return {
        "qk_norm_rotate": lambda **kw: m.msr_qk_norm_rotate(q, k, t(16), t(16), **kw),
        "qk_norm_rotate q": lambda **kw: m.msr_qk_norm_rotate(q, **kw),
        "qk_norm_rotate_backward": lambda **kw: m.msr_qk_norm_rotate_backward(q, k, t(16), None, t(2, 8, 4, 16), t(2, 8, 2, 16), **kw),
        "gated_recurrence": lambda **kw: m.msr_gated_recurrence(x, t(2, 100, 24), rate, state_in=t(2, 24, dtype=F32), want_carry=True, **kw),
        "gated_recurrence_step": lambda **kw: m.msr_gated_recurrence_step(t(2, 24), t(2, 24), t(2, 24, dtype=F32), rate, **kw),
        "gated_recurrence_backward": lambda **kw: m.msr_gated_recurrence_backward(x, t(2, 100, 24), rate, t(2, 100, 24), **kw),
        "gradient_norm": lambda **kw: m.msr_gradient_norm([t(5, 7), t(3, dtype=F32)], **kw),
        "clip_gradients": lambda **kw: m.msr_clip_gradients([t(5, 7), t(3, dtype=F32)], 1.0, **kw)[1],
    }


NAMES = sorted(calls())
WITH_WORKSPACE = ["qk_norm_rotate_backward", "gated_recurrence", "gated_recurrence_backward", "gradient_norm", "clip_gradients"]


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_on_a_stream_comes_from_that_stream(world, name):
    here, there = world.stream, Stream("another")
    results = flat(calls()[name](stream=there))
    assert world.made and world.stream is here
    for t in world.made:
        assert t.pool is there
        assert getattr(t, "recorded", []) == ([here] if any(t is r for r in results) else [])


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_on_the_current_stream(world, name):
    calls()[name]()
    assert world.made and all(t.pool is world.stream and not hasattr(t, "recorded") for t in world.made)


@pytest.mark.parametrize("name", WITH_WORKSPACE)
def test_workspace_is_checked_and_taken_by_its_bytes(world, name):
    for ws in (torch.zeros(8192, dtype=torch.uint8), on_device(8192, dtype=torch.uint8, index=1),
               on_device(1, dtype=torch.uint8).expand(8192), on_device(8192, 2, dtype=torch.uint8)[:, 0]):
        with pytest.raises(ValueError, match="workspace"):
            calls()[name](workspace=ws)
        assert not world.lib.calls

    def passed(ws):
        world.lib.calls.clear()
        calls()[name](workspace=ws)
        values = [getattr(a, "value", a) for a in world.lib.calls[0][1]]
        return ws.data_ptr() in values, values
    used, values = passed(on_device(1024, dtype=F32))
    assert used and 4096 in values
    used, values = passed(on_device(9000, dtype=torch.uint8))
    assert used and 9000 in values
    used, values = passed(on_device(1023, dtype=F32))
    assert not used and 4096 in values


@pytest.mark.parametrize("name", NAMES)
def test_launches_go_to_the_tensors_device(world, name):
    for index in (0, 1):
        world.lib.calls.clear()
        calls(index)[name]()
        assert [c[2] for c in world.lib.calls] == [index] and world.device == 0


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(world, name):
    with pytest.raises(ValueError, match="stream is of device 1"):
        calls()[name](stream=Stream("elsewhere", 1))
    assert not world.lib.calls and world.device == 0


def test_tensors_that_do_not_fit_are_refused(world):
    t = lambda *s, dtype=torch.bfloat16, index=0: on_device(*s, dtype=dtype, index=index)
    q, k, x, rate = t(2, 8, 4, 16), t(2, 8, 2, 16), t(2, 100, 24), t(24, dtype=F32)
    bad = [lambda: m.msr_qk_norm_rotate(q, t(2, 8, 2, 16, index=1)), lambda: m.msr_qk_norm_rotate(q, t(2, 8, 2, 16, dtype=F32)),
           lambda: m.msr_qk_norm_rotate(q, t(2, 7, 2, 16)), lambda: m.msr_qk_norm_rotate(q, t(2, 8, 2, 18)),
           lambda: m.msr_qk_norm_rotate(q, k, t(15)), lambda: m.msr_qk_norm_rotate(q, k, t(16), t(16, dtype=F32)),
           lambda: m.msr_qk_norm_rotate(q, k, theta=[1.0]), lambda: m.msr_qk_norm_rotate(q, k, pos_rows=t(2, dtype=torch.int32)),
           lambda: m.msr_qk_norm_rotate(q, k, pos_rows=t(3, dtype=torch.int64)), lambda: m.msr_qk_norm_rotate(t(2, 8, 4, 16, dtype=torch.float16)),
           lambda: m.msr_qk_norm_rotate(q, k, out=(t(2, 8, 4, 32)[..., :16], None)),
           lambda: m.msr_qk_norm_rotate_backward(q, k, None, None, t(2, 8, 4, 15), k),
           lambda: m.msr_qk_norm_rotate_backward(q, k, None, None, q, k, out=(t(2, 8, 3, 16), None, None, None)),
           lambda: m.msr_gated_recurrence(x, t(2, 99, 24), rate), lambda: m.msr_gated_recurrence(x, x, t(24)),
           lambda: m.msr_gated_recurrence(x, x, t(23, dtype=F32)), lambda: m.msr_gated_recurrence(x[0], x[0], rate),
           lambda: m.msr_gated_recurrence(x.transpose(0, 1), x.transpose(0, 1), rate),
           lambda: m.msr_gated_recurrence(x, x, rate, state_in=t(2, 24)), lambda: m.msr_gated_recurrence(x, x, rate, out=(t(2, 100, 25), None, None)),
           lambda: m.msr_gated_recurrence_step(x, x, x, rate), lambda: m.msr_gated_recurrence_step(x[0], x[0], t(100, 24), rate),
           lambda: m.msr_gated_recurrence_backward(x, x, rate, x, carry=t(2, 1, 24, dtype=F32)),
           lambda: m.msr_gated_recurrence_backward(x, x, rate, t(2, 100, 24, dtype=F32)),
           lambda: m.msr_gradient_norm([t(4), t(4, index=1)]), lambda: m.msr_gradient_norm([t(4, 4).t()]),
           lambda: m.msr_gradient_norm([t(4, dtype=torch.float16)]), lambda: m.msr_clip_gradients([t(4)], 1.0, out=[]),
           lambda: m.msr_clip_gradients([t(4)], 1.0, out=[t(5)]), lambda: m.msr_clip_gradients([t(4)], 1.0, out=[t(4, dtype=F32)]),
           lambda: m.msr_clip_gradients([t(4)], 1.0, norm=t(1, dtype=F32)), lambda: m.msr_clip_gradients([t(4)], 1.0, norm_out=t(dtype=torch.bfloat16))]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
        assert not world.lib.calls, i


def test_a_norm_is_given_or_written(world):
    g, scalar = on_device(4, dtype=F32), lambda: on_device(dtype=F32)
    with pytest.raises(ValueError, match="norm_out"):
        m.msr_clip_gradients([g], 1.0, norm=scalar(), norm_out=scalar())
    assert not world.lib.calls
    for kw in (dict(norm=scalar()), dict(norm_out=scalar())):
        assert m.msr_clip_gradients([g], 1.0, **kw)[1] is list(kw.values())[0]

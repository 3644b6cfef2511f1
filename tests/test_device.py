"""Tensors of another GPU than the current one, without a GPU: stand-ins that
say where they are, and a library that notes what was current when it was called."""
import contextlib
import types

import pytest
import torch

import selective_state_space_64_amd as ssm


class Placed(torch.Tensor):
    """A CPU tensor that says it is on GPU `at`."""
    @staticmethod
    def of(t, at):
        t = t.as_subclass(Placed)
        t.at = at
        return t
    is_cuda = property(lambda self: True)
    get_device = lambda self: self.at  # noqa: E731


@pytest.fixture
def machine(monkeypatch):
    """Two GPUs, the first one current; `calls` gets (function, current device, stream)."""
    now, calls = [0], []

    @contextlib.contextmanager
    def device(d):
        now.append(d)
        yield
        now.pop()

    @contextlib.contextmanager
    def on_stream(s):
        now.append(s.device_index)
        yield
        now.pop()

    def function(name):
        def call(*args):
            calls.append((name, now[-1], args[-1]))
            return 0
        return call
    library = types.SimpleNamespace(**{n: function(n) for n in ssm.EXPORTS})
    monkeypatch.setattr(ssm, "lib", lambda: library)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[-1])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", on_stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: types.SimpleNamespace(cuda_stream=("current", now[-1])))
    return calls


def update(at, **other):
    shapes = dict(state=(2, 4, 16, 8), x=(2, 4, 8), dt=(2, 4), A=(4,), Bm=(2, 2, 16), Cm=(2, 2, 16), y=(2, 4, 8))
    t = {n: Placed.of(torch.zeros(s), other.get(n, at)) for n, s in shapes.items()}
    return lambda **kw: ssm.ssm_head_scan_update(**t, **kw)


def norm(at, **other):
    t = {n: Placed.of(torch.zeros(3, 8), other.get(n, at)) for n in ("x", "residual", "residual_out", "y")}
    return lambda **kw: ssm.ssm_rms_norm_fwd(t.pop("x"), **t, **kw)


def group(at, **other):
    t = {n: Placed.of(torch.zeros(2, 3, 8), other.get(n, at)) for n in ("x", "y")}
    return lambda **kw: ssm.ssm_group_norm_fwd(t["x"], 2, y=t["y"], **kw)


@pytest.mark.parametrize("call", [update, norm, group], ids=lambda f: f.__name__)
def test_the_tensors_device_is_current(machine, call):
    for at in (0, 1):
        call(at)()
        assert machine.pop()[1:] == (at, ("current", at)) and not machine


@pytest.mark.parametrize("call", [update, norm, group], ids=lambda f: f.__name__)
def test_a_stream_of_the_tensors_device(machine, call):
    stream = types.SimpleNamespace(device_index=1, cuda_stream="one")
    call(1)(stream=stream)
    assert machine.pop()[1:] == (1, "one")
    with pytest.raises(ValueError, match="device"):
        call(0)(stream=stream)
    assert not machine


@pytest.mark.parametrize("call,other", [(update, "A"), (update, "Cm"), (update, "y"), (norm, "residual"), (norm, "y"),
                                        (group, "y")], ids=str)
def test_tensors_of_two_devices(machine, call, other):
    for at in (0, 1):
        with pytest.raises(ValueError, match="device"):
            call(at, **{other: 1 - at})()
    assert not machine


def test_tensors_of_no_gpu(machine):
    with pytest.raises(TypeError):
        update(-1)()
    assert not machine

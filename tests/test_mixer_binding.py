"""What the binding of the sequence-mixing operators does around a launch, on
the CPU: the library and torch's device and stream switches are replaced by
stand-ins that record, and nothing is launched."""
import contextlib

import pytest
import torch

from convolution_lowering_amd import mixer


class _Stand:
    """What the binding asks of a device tensor."""

    def __init__(self, shape, dtype=torch.bfloat16, device=torch.device("cuda", 1)):
        self.shape, self.dtype, self.device, self.is_cuda = torch.Size(shape), dtype, device, True

    def stride(self):
        out, one = [], 1
        for n in reversed(self.shape):
            out.append(one)
            one *= n
        return tuple(reversed(out))

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x1000


class _World:
    """The current device, the entered streams and what was seen at each
    allocation and launch."""

    def __init__(self, monkeypatch):
        self.device, self.stream, self.seen = 0, None, []

        @contextlib.contextmanager
        def on_device(device):
            old, self.device = self.device, torch.device(device).index
            yield
            self.device = old

        @contextlib.contextmanager
        def on_stream(stream):
            old, self.stream, self.device = (self.stream, self.device), stream, stream.device.index
            yield
            self.stream, self.device = old

        def empty(shape, *more, dtype=None, device=None):
            self.seen.append(("empty", self.device, self.stream))
            return _Stand(shape if not isinstance(shape, int) else (shape,), dtype, device)

        def launch(name):
            def call(*args):
                if name.endswith("_size"):
                    args[-1]._obj.value = 64
                else:
                    self.seen.append((name, self.device, self.stream))
                return 0
            return call

        class Lib:
            def __getattr__(self, name):
                return launch(name)

        monkeypatch.setattr(torch.cuda, "device", on_device)
        monkeypatch.setattr(torch.cuda, "stream", on_stream)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.device)
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: self.device, raising=False)
        monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0, raising=False)
        monkeypatch.setattr(torch, "empty", empty)
        lib = Lib()
        monkeypatch.setattr(mixer, "_mixer_lib", lambda: lib)


class _Stream:
    def __init__(self, index):
        self.device, self.cuda_stream = torch.device("cuda", index), 0x77


def _calls(dev):
    f32, i32 = torch.float32, torch.int32
    t = lambda *shape, dtype=torch.bfloat16: _Stand(shape, dtype, dev)
    x, w, b = t(8, 64), t(64, 4), t(64)
    q, v, g, beta = t(8, 2, 64), t(8, 4, 64), t(8, 4, dtype=f32), t(8, 4)
    saved, gate = t(4096, dtype=torch.uint8), t(8, 64)
    return {
        "conv1d_causal_fwd": lambda s: mixer.conv1d_causal_fwd(x, w, b, want_state=True, stream=s),
        "conv1d_causal_bwd": lambda s: mixer.conv1d_causal_bwd(x, x, w, b, stream=s),
        "conv1d_causal_step": lambda s: mixer.conv1d_causal_step(x, w, b, t(9, 3, 64), t(8, dtype=i32), stream=s),
        "delta_rule_fwd": lambda s: mixer.delta_rule_fwd(q, q, v, g, beta, save=True, stream=s),
        "delta_rule_bwd": lambda s: mixer.delta_rule_bwd(v, q, q, v, g, beta, saved, stream=s),
        "delta_rule_step": lambda s: mixer.delta_rule_step(q, q, v, g, beta, t(9, 4, 64, 64, dtype=f32),
                                                           t(8, dtype=i32), stream=s),
        "branch_norm_fwd": lambda s: mixer.branch_norm_fwd(x, x, b, gate, b, save=True, stream=s),
        "branch_norm_bwd": lambda s: mixer.branch_norm_bwd(x, x, x, x, b, gate, b, t(2, 8, dtype=f32), stream=s),
    }


NAMES = sorted(_calls(None))


@pytest.mark.parametrize("name", NAMES)
def test_a_call_runs_on_its_tensors_device(name, monkeypatch):
    """Tensors on the second GPU while the first is torch's current one."""
    world = _World(monkeypatch)
    _calls(torch.device("cuda", 1))[name](None)
    assert (name, 1, None) in world.seen
    assert all(device == 1 for _, device, _ in world.seen) and world.device == 0
    world.seen.clear()
    _calls(torch.device("cuda", 0))[name](None)
    assert (name, 0, None) in world.seen and world.device == 0


@pytest.mark.parametrize("name", NAMES)
def test_a_call_launches_inside_its_stream(name, monkeypatch):
    world = _World(monkeypatch)
    stream = _Stream(1)
    _calls(torch.device("cuda", 1))[name](stream)
    assert (name, 1, stream) in world.seen
    assert all(entered is stream for _, _, entered in world.seen) and world.stream is None

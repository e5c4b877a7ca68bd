"""The binding of the operators around an AllReduce on a machine of several
GPUs, and with tensors that torch differentiates.  Stand-ins take the place of
device tensors and of the library's launching entry points.  No GPU needed."""
import contextlib
import types

import pytest
import torch

import ring_all_reduce_channelmask_amd as rar
from ring_all_reduce_channelmask_amd import _lib, model_ops


class Tensor:
    """What the binding asks of a device tensor."""
    device = "cpu"  # of what the binding allocates beside it

    def __init__(self, *shape, dtype=torch.float32, dev=1, requires_grad=False):
        self.shape, self.dtype, self.dev, self.requires_grad = shape, dtype, dev, requires_grad

    def get_device(self):
        return self.dev

    def size(self, i):
        return self.shape[i]

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for k in self.shape:
            n *= k
        return n

    def stride(self):
        return tuple(Tensor(*self.shape[i + 1:]).numel() for i in range(len(self.shape)))

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 40


def _int64(*shape):
    return Tensor(*shape, dtype=torch.int64)


@pytest.fixture
def machine(monkeypatch):
    """A machine whose current device is 0; .launches has each launch's entry
    point, the device that was current and the stream."""
    m = types.SimpleNamespace(current=0, launches=[])

    @contextlib.contextmanager
    def device(index):
        before, m.current = m.current, index
        try:
            yield
        finally:
            m.current = before

    class Library:
        def __getattr__(self, name):
            if name.endswith("_workspace"):
                return getattr(real, name)
            return lambda *args: m.launches.append((name, m.current, args[-1])) or _lib.SUCCESS
    real, library = _lib.load(), Library()
    monkeypatch.setattr(_lib, "load", lambda: library)
    monkeypatch.setattr(torch.cuda, "device", device)
    with contextlib.suppress(ValueError):  # the binding looks torch up on its first call
        rar.dropout_allreduce([torch.zeros(1)], [], 0.0, None)
    monkeypatch.setattr(model_ops, "_raw_stream", lambda dev: 1000 + dev)
    monkeypatch.setattr(model_ops, "_current_device", lambda: m.current, raising=False)
    return m


def _calls(dev=1, stream=None, grad=None):
    """Every operator with tensors on a device; argument `grad` = (operator,
    argument) requires a gradient."""
    def t(key, *shape):
        return Tensor(*shape, dev=dev, requires_grad=key == grad)

    def whole(*shape):
        return Tensor(*shape, dtype=torch.int64, dev=dev)
    yield "dropout", lambda: rar.dropout_allreduce([t(("dropout", "sends"), 8)], [t(("dropout", "recvs"), 8)], 0.1, whole(2),
                                                   residual=t(("dropout", "residual"), 8), stream=stream)
    yield "dropout_backward", lambda: rar.dropout_allreduce_backward(
        [t(("dropout_backward", "grads"), 8)], [t(("dropout_backward", "dsends"), 8)], 0.1, whole(2),
        dresidual=t(("dropout_backward", "dresidual"), 8), stream=stream)
    yield "logprobs", lambda: rar.logprobs([t(("logprobs", "shards"), 2, 5)], whole(2),
                                           out=rar.LogProbs(*[t(("logprobs", "out"), 2) for _ in range(3)],
                                                            Tensor(2, 0, dtype=torch.int32, dev=dev), Tensor(2, 0, dev=dev)), stream=stream)
    yield "logprobs_backward", lambda: rar.logprobs_backward(
        [t(("logprobs_backward", "shards"), 2, 5)], whole(2), t(("logprobs_backward", "lse"), 2), t(("logprobs_backward", "entropy"), 2),
        t(("logprobs_backward", "grad_logprob"), 2), t(("logprobs_backward", "grad_entropy"), 2),
        t(("logprobs_backward", "grad_lse"), 2), grads=[t(("logprobs_backward", "grads"), 2, 5)], stream=stream)
    yield "adapter", lambda: rar.adapter_allreduce(
        [t(("adapter", "xs"), 2, 5)], [t(("adapter", "partials"), 2, 7)], [t(("adapter", "recvs"), 2, 7)], [t(("adapter", "downs"), 3, 4, 5)],
        t(("adapter", "up"), 3, 7, 4), whole(2), t(("adapter", "scales"), 3), stream=stream)


def test_calls_run_on_the_tensors_device(machine):
    for dev in (1, 0, 3):
        for name, call in _calls(dev):
            call()
            assert machine.launches.pop()[1:] == (dev, 1000 + dev), name
            assert machine.current == 0 and not machine.launches


def test_a_given_stream_is_of_the_tensors_device(machine, monkeypatch):
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    there, elsewhere = (types.SimpleNamespace(cuda_stream=77, device_index=d) for d in (1, 0))
    for name, call in _calls(stream=there):
        call()
        assert machine.launches.pop()[1:] == (1, 77), name
    for name, call in _calls(stream=elsewhere):
        with pytest.raises(ValueError, match="stream"):
            call()
        assert not machine.launches, name


INPUTS = {
    "dropout": ("sends", "residual"),
    "dropout_backward": ("grads",),
    "logprobs": ("shards",),
    "logprobs_backward": ("shards", "lse", "entropy", "grad_logprob", "grad_entropy", "grad_lse"),
    "adapter": ("xs", "partials", "downs", "up", "scales"),
}


@pytest.mark.parametrize("operator,argument", [(k, v) for k, vs in INPUTS.items() for v in vs])
def test_a_gradient_that_nothing_would_record_is_refused(machine, operator, argument):
    """As torch does of functions that write into given tensors; where no
    gradients are recorded, the call goes through."""
    call = dict(_calls(grad=(operator, argument)))[operator]
    with pytest.raises(RuntimeError, match="no_grad"):
        call()
    assert not machine.launches
    for off in (torch.no_grad(), torch.inference_mode()):
        with off:
            call()
        assert machine.launches.pop()[1] == 1

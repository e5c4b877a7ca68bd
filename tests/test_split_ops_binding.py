"""The binding of embeddings, norms and 8-bit projections on a machine of
several GPUs, and with tensors that torch differentiates.  Stand-ins take the
place of device tensors and of the library's launching entry points.  No GPU
needed."""
import contextlib
import types

import pytest
import torch

import ring_all_reduce_channelmask_amd as rar

from .test_model_ops_binding import Tensor, machine  # noqa: F401


def _calls(dev=1, stream=None, grad=None):
    """Every operator with tensors on a device; argument `grad` = (operator,
    argument) requires a gradient."""
    def t(key, *shape, dtype=torch.float32):
        return Tensor(*shape, dtype=dtype, dev=dev, requires_grad=key == grad)

    def whole(*shape):
        return Tensor(*shape, dtype=torch.int64, dev=dev)
    k = "embedding"
    yield k, lambda: rar.embedding_allreduce([t(("embedding", "tables"), 3, 5)], whole(2), [t(("embedding", "recvs"), 2, 5)], stream=stream)
    yield "embedding_backward", lambda: rar.embedding_allreduce_backward(
        [t(("embedding_backward", "grads"), 2, 5)], whole(2), [t(("embedding_backward", "dtables"), 3, 5)], stream=stream)

    def n(key, *shape):
        return t(("norm", key), *shape)
    yield "norm", lambda: rar.norm_allreduce([n("partials", 2, 5)], [n("hidden", 2, 5)], [n("outs", 2, 5)], residual=n("residual", 2, 5), post_weight=n("post_weight", 5),
                                             gate=n("gate", 2, 5), pre_weight=n("pre_weight", 5), total=n("total", 2, 5), stream=stream)

    def b(key, *shape):
        return t(("norm_backward", key), *shape)
    yield "norm_backward", lambda: rar.norm_allreduce_backward(
        [b("grad_hidden", 2, 5)], [b("grad_outs", 2, 5)], [b("dpartials", 2, 5)], total=b("total", 2, 5), hidden=b("hidden", 2, 5), post_weight=b("post_weight", 5),
        gate=b("gate", 5), pre_weight=b("pre_weight", 5), dresidual=b("dresidual", 2, 5), dpost_weight=b("dpost_weight", 5), dgate=b("dgate", 5),
        dpre_weight=b("dpre_weight", 5), stream=stream)
    i8 = torch.int8
    yield "quantize", lambda: rar.quantize_rows([t(("quantize", "xs"), 2, 5)], quantized=[t(None, 2, 5, dtype=i8)], scales=t(("quantize", "scales"), 2), stream=stream)
    yield "projection", lambda: rar.int8_projection_allreduce(
        [t(None, 2, 5, dtype=i8)], t(("projection", "x_scales"), 2), [t(None, 7, 5, dtype=i8)], t(("projection", "weight_scales"), 7),
        [t(("projection", "recvs"), 2, 7)], residual=t(("projection", "residual"), 2, 7), stream=stream)


@pytest.fixture(autouse=True)
def workspaces(monkeypatch):
    """What the binding allocates beside the stand-ins is on the host."""
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())


def test_calls_run_on_the_tensors_device(machine):  # noqa: F811
    for dev in (1, 0, 3):
        for name, call in _calls(dev):
            call()
            assert machine.launches.pop()[1:] == (dev, 1000 + dev), name
            assert machine.current == 0 and not machine.launches


def test_a_given_stream_is_of_the_tensors_device(machine):  # noqa: F811
    there, elsewhere = (types.SimpleNamespace(cuda_stream=77, device_index=d) for d in (1, 0))
    for name, call in _calls(stream=there):
        call()
        assert machine.launches.pop()[1:] == (1, 77), name
    for name, call in _calls(stream=elsewhere):
        with pytest.raises(ValueError, match="stream"):
            call()
        assert not machine.launches, name


INPUTS = {
    "embedding": ("tables",),
    "embedding_backward": ("grads",),
    "norm": ("partials", "residual", "post_weight", "gate", "pre_weight"),
    "norm_backward": ("grad_hidden", "grad_outs", "total", "hidden", "post_weight", "gate", "pre_weight"),
    "quantize": ("xs",),
    "projection": ("x_scales", "weight_scales", "residual"),
}


@pytest.mark.parametrize("operator,argument", [(k, v) for k, vs in INPUTS.items() for v in vs])
def test_a_gradient_that_nothing_would_record_is_refused(machine, operator, argument):  # noqa: F811
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

"""Gates of the norms around a block where there are no rows, and gates of no
groups.  Stand-ins take the place of device tensors and of the library's
launching entry points.  No GPU needed."""
import contextlib
import types

import pytest
import torch

import ring_all_reduce_channelmask_amd as rar
from ring_all_reduce_channelmask_amd import _lib

from .test_model_ops_binding import Tensor, machine  # noqa: F401


class Written(Tensor):
    """Counts how often it is zeroed and notes on which stream."""

    def __init__(self, *shape, log, **kw):
        super().__init__(*shape, **kw)
        self.log = log

    def zero_(self):
        self.log.append(tuple(self.streams))


@pytest.fixture
def log(monkeypatch):
    """Each zeroing: the streams that were made current around it."""
    current, zeroed = [], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        try:
            yield
        finally:
            current.pop()
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(Written, "streams", current, raising=False)
    return zeroed


def _no_rows(log, stream=None, dgate=None, gate=None, **kw):
    e, w = Tensor(0, 5), Tensor(5)
    args = dict(total=e, hidden=e, post_weight=w, pre_weight=w, gate=Tensor(3, 5) if gate is None else gate,
                dgate=Written(3, 5, log=log) if dgate is None else dgate, stream=stream)
    args.update(kw)
    rar.norm_allreduce_backward([e], [e], [e], **args)


def test_a_gates_gradient_of_no_rows_is_zeroed_on_the_calls_stream(machine, log):  # noqa: F811
    _no_rows(log)
    assert log == [()]
    side = types.SimpleNamespace(cuda_stream=77, device_index=1)
    _no_rows(log, side)
    assert log == [(), (side,)]
    assert [m[2] for m in machine.launches] == [1001, 77]


def test_a_refused_call_of_no_rows_changes_no_gradient(machine, log, monkeypatch):  # noqa: F811
    elsewhere = types.SimpleNamespace(cuda_stream=77, device_index=0)
    bad = [dict(stream=elsewhere), dict(dgate=Written(3, 5, log=log, dtype=torch.bfloat16)), dict(dgate=Written(3, 5, log=log, dev=0)),
           dict(gate=Tensor(3, 5, dtype=torch.bfloat16)), dict(gate=Tensor(3, 5, dev=0)), dict(dgate=Written(2, 5, log=log)),
           dict(gate=Tensor(3, 4), dgate=Written(3, 4, log=log)), dict(total=Tensor(1, 5)), dict(dpre_weight=Tensor(4)), dict(dresidual=Tensor(2, 5))]
    for kw in bad:
        with pytest.raises(ValueError):
            _no_rows(log, **kw)
    assert not log and not machine.launches
    with monkeypatch.context() as m:  # the library refuses
        real = _lib.load()
        m.setattr(type(real), "rar_norm_allreduce_backward", lambda *a: _lib.INVALID_ARGUMENT, raising=False)
        for name in ("rar_get_last_error", "rar_get_error_string"):
            m.setattr(type(real), name, lambda *a: b"no", raising=False)
        with pytest.raises(rar.RarError):
            _no_rows(log)
    assert not log


def test_a_gate_of_no_groups_is_refused(machine, log):  # noqa: F811
    """An empty tensor has no address, which would mean: no gate."""
    class Empty(Tensor):
        def data_ptr(self):
            return 0
    x, w, gate = Tensor(4, 5), Tensor(5), Empty(0, 5)
    with pytest.raises(ValueError, match="groups"):
        rar.norm_allreduce([x], [x], [], gate=gate)
    with pytest.raises(ValueError, match="groups"):
        rar.norm_allreduce_backward([x], [], [x], total=x, gate=gate)
    with pytest.raises(ValueError, match="groups"):
        rar.norm_allreduce_backward([x], [], [x], total=x, gate=gate, dgate=Empty(0, 5))
    assert not machine.launches
    e = Tensor(0, 5)  # without rows there is nothing to gate
    rar.norm_allreduce([e], [e], [], gate=gate)
    rar.norm_allreduce_backward([e], [], [e], total=e, gate=gate, dgate=Written(0, 5, log=log))
    assert len(machine.launches) == 2 and len(log) == 1
    assert rar.norm_allreduce([x], [x], [], gate=Tensor(2, 5), post_weight=w) is None

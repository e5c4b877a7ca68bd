"""What the operators around an AllReduce refuse beyond malformed arguments:
buffers that workgroups would race on, row strides beyond any memory.  Every
call below fails on the host, before any HIP call; the addresses are made up
and never dereferenced.  No GPU needed."""
import pytest

from ring_all_reduce_channelmask_amd import _lib

from .test_model_ops_args import A, BAD, BF16, F32, _adapters, _backward, _dropout, _logprobs

LOGITS = (A, A + (1 << 20))


def _message():
    return _lib.load().rar_get_last_error().decode()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [1, 4])
def test_a_gradient_over_another_ranks_logits_of_the_same_shape(dtype, rows):
    """Other workgroups still read those logits: only a rank's own may be
    written in place."""
    for grads in ((LOGITS[1], LOGITS[0]), (LOGITS[1], A + (7 << 20)), (A + (7 << 20), LOGITS[0])):
        assert _backward(logits=LOGITS, widths=(100, 100), rows=rows, dtype=dtype, grads=grads) == BAD, grads
        assert "logits" in _message()
    # three ranks, turned by one; the middle one without columns
    three = (A, A + (1 << 20), A + (9 << 20))
    for widths in ((64, 64, 64), (64, 0, 64)):
        assert _backward(logits=three, widths=widths, rows=rows, dtype=dtype, grads=three[1:] + three[:1]) == BAD, widths
    # two ranks that read the same logits: the gradient of either would be over the other's
    assert _backward(logits=(A, A), widths=(100, 100), rows=rows, dtype=dtype, grads=(A, A + (7 << 20))) == BAD


def test_a_gradient_over_what_every_workgroup_reads():
    """One row, where the vectors are as large as a rank's gradients."""
    at = dict(ids=A + (2 << 20), lse=A + (3 << 20), ent=A + (4 << 20), g=A + (5 << 20), h=A + (8 << 20), l=A + (9 << 20))
    for what, p in at.items():
        width = 2 if what == "ids" else 1
        assert _backward(widths=(width, 100), rows=1, grads=(p, A + (7 << 20)), h=at["h"], l=at["l"]) == BAD, what


@pytest.mark.parametrize("back", [False, True])
def test_the_generators_state_as_an_output(back):
    for dtype, count in ((F32, 4), (BF16, 8)):
        assert _dropout(count=count, dtype=dtype, recv=(A + 65536,), back=back) == BAD
        assert "rng" in _message()
    if back:
        assert _dropout(count=4, res=A + 65536, back=True) == BAD


@pytest.mark.parametrize("stride", [1 << 62, 1 << 61, (1 << 63) - 1, 1 << 57])
def test_row_strides_beyond_any_memory(stride):
    """Rows so far apart that their offsets in bytes leave 64 bits: refused,
    whichever operand has them (a multiple of 2^64 bytes divided by zero).  One
    row has no use for its stride."""
    far = (stride, stride)
    one = dict(strides=far, gstrides=far, grads=(A + 64, A + (7 << 20)))  # in part over the logits
    assert _backward(rows=1, **one) == BAD and "overlaps" in _message()
    for kw in (dict(strides=far), dict(gstrides=far), one):
        assert _backward(**kw) == BAD and "stride" in _message(), kw
    assert _logprobs(strides=far, lp=A + 64) == BAD and "stride" in _message()
    for kw in (dict(xstrides=far), dict(pstrides=far), dict(ostrides=far[:1])):
        assert _adapters(**kw) == BAD and "stride" in _message(), kw
        assert _adapters(tokens=1, outs=(A,), **kw) == BAD and "overlaps" in _message(), kw

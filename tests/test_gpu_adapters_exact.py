"""Adapters: a token's result does not depend on how many others are in the
call, in its last bits as with infinities.  Few tokens go one by one, more 16
at a time."""
import pytest

pytestmark = pytest.mark.gpu

DTYPES = ["float32", "bfloat16"]
FEW, MANY = 5, 600  # tokens


def _call(dtype, tokens, x, down, up, partials):
    """One token's adapters, the token repeated: adapter 1 of 3, rank 32."""
    import torch
    import ring_all_reduce_channelmask_amd as rar
    t = getattr(torch, dtype)

    def make(rows):
        return torch.tensor(rows, dtype=torch.float64).to(t).cuda()
    downs, ups = (torch.ones(shape, dtype=t, device="cuda") for shape in ((3, 32, len(x)), (3, len(up), 32)))
    downs[1], ups[1] = make(down), make(up)
    xs = make([x] * tokens)
    ps = [make([p] * tokens) for p in partials]
    ids = torch.arange(tokens, device="cuda") % 4 - 1
    out = torch.empty((tokens, len(up)), dtype=t, device="cuda")
    none = torch.empty((tokens, 0), dtype=t, device="cuda")
    zero = torch.empty((3, 32, 0), dtype=t, device="cuda")
    rar.adapter_allreduce([xs] + [none] * (len(ps) - 1), ps, [out], [downs] + [zero] * (len(ps) - 1), ups, ids)
    rows = out[2::4].double().cpu()
    assert all(torch.allclose(r, rows[0], rtol=0, atol=0, equal_nan=True) for r in rows)
    return rows[0]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [FEW, MANY])
def test_all_bits_of_the_inner_sum_arrive(dtype, tokens):
    """h = 1 + 2^-10 + 2^-20 exactly; the partials take its upper parts away,
    and the lowest is the result."""
    low = [2.0 ** -20, 2.0 ** -23]
    for least in low:
        down = [[1.0, 1.0, 1.0]] + [[0.0] * 3] * 31
        up = [[1.0] + [0.0] * 31] * 70
        y = _call(dtype, tokens, [1.0, 2.0 ** -10, least], down, up, [[-1.0] * 70, [-2.0 ** -10] * 70])
        assert (y == least).all(), y


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [FEW, MANY])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_an_infinite_inner_sum(dtype, tokens, sign):
    """Every place of h is infinite; each output is infinite with the sign of
    its weights, and NaN where a weight is 0."""
    inf = float("inf")
    up = [[(1.0 if c % 2 else -1.0) * (1 + k) for k in range(32)] for c in range(70)]
    up[5] = [0.0] * 32
    up[6] = [1.0, -1.0] * 16
    y = _call(dtype, tokens, [sign * inf, 1.0], [[1.0, 1.0]] * 32, up, [[1.0] * 70])
    for c in range(70):
        if c in (5, 6):
            assert y[c].isnan()
        else:
            assert y[c] == (inf if (c % 2 == 1) == (sign > 0) else -inf), c


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [FEW, MANY])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_an_inner_sum_between_the_largest_numbers(dtype, tokens, sign):
    """h = 1.9990234375 * 2^127, finite in fp32 and above bfloat16's largest
    number (1.9921875 * 2^127): the result is finite."""
    big = 1.9921875 * 2.0 ** 127
    down = [[1.0, 1.0]] + [[0.0, 0.0]] * 31
    up = [[2.0 ** -10] + [0.0] * 31] * 70
    y = _call(dtype, tokens, [sign * big, sign * 0.0068359375 * 2.0 ** 127], down, up, [[0.0] * 70])
    want = 1.9990234375 * 2.0 ** 117
    if dtype == "bfloat16":
        want = 2.0 ** 118  # rounded to 8 bits
    assert (y == sign * want).all(), y


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [FEW, MANY])
@pytest.mark.parametrize("h", [1.0, 1.0 - 2.0 ** -12, -3.0 - 2.0 ** -9, 0.0])
def test_infinite_weights_of_the_second_matrix(dtype, tokens, h):
    """An output with an infinite weight is infinite with the sign of its
    product; NaN where the inner sum is 0 or where two such products differ."""
    inf = float("inf")
    up = [[1.0] * 32 for _ in range(70)]
    up[3][0], up[4][31], up[69][9] = inf, -inf, inf
    up[64][2], up[64][3] = inf, -inf
    up[65][2] = float("nan")
    first = round(h)
    down = [[float(first), h - first]] * 32
    y = _call(dtype, tokens, [1.0, 1.0], down, up, [[1.0] * 70])
    for c, sign in ((3, 1), (4, -1), (69, 1)):
        assert y[c].isnan() if h == 0 else y[c] == sign * (inf if h > 0 else -inf), c
    assert y[64].isnan() and y[65].isnan()
    rest = [c for c in range(70) if c not in (3, 4, 64, 65, 69)]
    assert (y[rest] - (1 + 32 * h)).abs().max() <= abs(1 + 32 * h) * 2.0 ** -8

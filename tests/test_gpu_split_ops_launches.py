"""Calls of embeddings, norms and 8-bit projections whose workgroups take more
than one launch (a grid holds less than 2^32 threads): what the second launch
computes is right, and what the first one did is left as it was."""
import pytest

pytestmark = pytest.mark.gpu

ALL = 1 << 24


@pytest.fixture(autouse=True)
def room():
    """Up to 60 GB of device memory, given back behind each test."""
    import torch
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 70e9:
        pytest.skip("needs 70 GB of device memory")
    yield
    torch.cuda.empty_cache()


def test_embedding_of_2_24_tokens():
    """A workgroup a token: the last one is alone in the second launch."""
    import torch
    import ring_all_reduce_channelmask_amd as rar
    ids = torch.arange(ALL, device="cuda").flip(0) % 1003 - 1
    table = torch.randn(1000, 513, device="cuda").bfloat16()
    out = torch.empty(ALL, 513, dtype=torch.bfloat16, device="cuda")
    rar.embedding_allreduce([table[:400], table[400:]], ids, [out])
    whole = torch.zeros(1003, 513, dtype=torch.bfloat16, device="cuda")  # ids -1, 1000 and 1001: zeros
    whole[1:1001] = table
    for at in range(0, ALL, 1 << 22):
        part = slice(at, at + (1 << 22))
        assert torch.equal(out[part], whole[ids[part] + 1])


@pytest.mark.parametrize("tokens", [0, 700, 5000, 9000])
def test_gradient_of_2_30_table_rows(tokens):
    """2^24 workgroups zero the table, behind those that sum; the sorts' keys
    have 31 bits (four passes)."""
    import torch
    import ring_all_reduce_channelmask_amd as rar
    vocab = 1 << 30
    # distinct tokens at both ends of the table and between, then some of them again
    at = torch.cat([torch.arange(tokens // 3), vocab - 1 - torch.arange(tokens // 3), torch.arange(tokens - 2 * (tokens // 3)) * 100003 + 12345])
    ids = at[torch.randint(0, max(tokens, 1), (tokens,), generator=torch.Generator().manual_seed(1))] if tokens else at
    ids[tokens // 2:tokens // 2 + 3] = -1
    ids = ids.cuda()
    grad = torch.randint(-4, 5, (tokens, 1), device="cuda").bfloat16()
    table = torch.full((vocab, 1), float("nan"), dtype=torch.bfloat16, device="cuda")
    rar.embedding_allreduce_backward([grad], ids, [table[:vocab // 2 + 1], table[vocab // 2 + 1:]])
    used, place = torch.unique(ids[ids >= 0], return_inverse=True)
    want = torch.zeros(used.numel(), device="cuda").index_add_(0, place, grad[ids >= 0, 0].float())  # whole numbers, exact
    assert torch.equal(table[used, 0].float(), want)
    table[used] = 0
    for part in table.view(16, -1):
        assert torch.count_nonzero(part) == 0  # NaN counts


def test_gradient_of_few_tokens_of_2_24_columns():
    """520 tokens of 32768 workgroups each: tokens 512 to 519 are in the second launch."""
    import torch
    import ring_all_reduce_channelmask_amd as rar
    tokens = 520
    ids = torch.zeros(tokens, dtype=torch.int64, device="cuda")
    ids[511:] = torch.tensor([1, 2, 1, 3, 4, -1, 5, 4, 5], device="cuda")
    row = torch.randint(-3, 4, (ALL,), device="cuda").bfloat16()
    grad = torch.empty(tokens, ALL, dtype=torch.bfloat16, device="cuda")
    grad.copy_(row)
    grad[515:].mul_(2)
    table = torch.ones(6, ALL, dtype=torch.bfloat16, device="cuda")
    rar.embedding_allreduce_backward([grad], ids, [table], scale=0.5, accumulate=True)
    # sums of whole numbers times a half: exact in fp32, rounded once
    weight = torch.ones(tokens, device="cuda")
    weight[515:] = 2
    for v in range(6):
        want = (1 + 0.5 * (weight * (ids == v)).sum() * row.float()).bfloat16()
        assert torch.equal(table[v], want), v


def test_norms_of_2_24_rows():
    """A workgroup of 256 threads a row: the last row is alone in the second
    launch.  In place; the rows are some hundred, over and over."""
    import torch
    import ring_all_reduce_channelmask_amd as rar
    width = 1544
    some = torch.randn(255, width, device="cuda").bfloat16()
    x = torch.empty(ALL, width, dtype=torch.bfloat16, device="cuda")
    ids = torch.arange(ALL, device="cuda") % 255
    for at in range(0, ALL, 1 << 21):
        x[at:at + (1 << 21)] = some[ids[at:at + (1 << 21)]]
    weight, gate = torch.randn(width, device="cuda").bfloat16(), torch.randn(2, width, device="cuda").bfloat16()
    wants = []
    for k in range(2):
        want = torch.empty_like(some)
        rar.norm_allreduce([some], [], [want], gate=gate[k], pre_weight=weight)
        wants.append(want)
    rar.norm_allreduce([x], [], [x], gate=gate, pre_weight=weight)
    for at in range(0, ALL, 1 << 21):
        assert torch.equal(x[at:at + (1 << 21)], wants[at // (ALL // 2)][ids[at:at + (1 << 21)]])


def test_quantisation_of_2_24_rows():
    """64 ranks of a column each, 16 waves a row: five launches."""
    import torch
    import ring_all_reduce_channelmask_amd as rar
    x = torch.randint(-4, 5, (64, ALL, 1), device="cuda").bfloat16()
    q = torch.full((64, ALL, 1), 99, dtype=torch.int8, device="cuda")
    _, scales = rar.quantize_rows(list(x), quantized=list(q))
    most = x.abs().amax((0, 2)).float()
    assert torch.equal(scales, most / 127)
    for k in range(0, 64, 16):  # whole numbers up to 4: no quotient but 127/2 is near a tie, and 127 x is exact
        want = (x[k:k + 16, :, 0].float() * 127 / most.clamp(min=1)).round().to(torch.int8)
        assert torch.equal(q[k:k + 16, :, 0], want)


def test_projection_of_2_24_unaligned_tokens():
    """Rows of 4112 bytes, a byte off: 257 pieces of 16 for each token are laid
    out, 2^24 + 2^16 workgroups."""
    import torch
    import ring_all_reduce_channelmask_amd as rar
    if torch.cuda.mem_get_info()[0] < 150e9:
        pytest.skip("needs 150 GB of device memory")
    width = 4112
    # enough rows for the second launch to lay out the last ones
    some = torch.randint(-127, 128, (255, width), dtype=torch.int8, device="cuda")
    held = torch.empty(ALL * width + 1, dtype=torch.int8, device="cuda")
    x = held[1:].view(ALL, width)
    ids = torch.arange(ALL, device="cuda") % 255
    for at in range(0, ALL, 1 << 20):
        x[at:at + (1 << 20)] = some[ids[at:at + (1 << 20)]]
    w = torch.randint(-127, 128, (3, width), dtype=torch.int8, device="cuda")
    scale = 0.5 + torch.rand(ALL, device="cuda")
    y = torch.empty(ALL, 3, device="cuda")
    rar.int8_projection_allreduce([x], scale, [w], torch.ones(3, device="cuda"), [y])
    sums = (some.double() @ w.double().T).float()  # below 2^53: exact, rounded once
    assert torch.equal(y, sums[ids] * scale[:, None])

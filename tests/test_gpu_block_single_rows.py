"""A dimension of one row, request or head has no neighbour, so its stride says
nothing about alignment: such calls work whatever the stride is, and give the
bits of the same call with dense tensors."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _restrided(t, dim, stride):
    """`t` (one element along `dim`) with another stride there."""
    strides = list(t.stride())
    strides[dim] = stride
    return t.as_strided(t.shape, strides)


@pytest.mark.parametrize("stride", [0, 1, 67, 2 ** 40])
def test_one_token_of_an_adapter(gpu_lib, stride):
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(1, 64, generator=g, device="cuda").bfloat16()
    y = torch.randn(1, 40, generator=g, device="cuda")
    A = torch.randn(2, 8, 64, generator=g, device="cuda").bfloat16()
    B = torch.randn(2, 40, 8, generator=g, device="cuda").bfloat16()
    ids = torch.ones(1, dtype=torch.int32, device="cuda")
    want = gpu_lib.adapter_add(y, x, A, B, ids)
    assert torch.equal(gpu_lib.adapter_add(y, _restrided(x, 0, stride), A, B, ids), want)
    assert torch.equal(gpu_lib.adapter_add(_restrided(y, 0, stride), x, A, B, ids), want)


@pytest.mark.parametrize("stride", [0, 1, 67, 2 ** 40])
def test_one_request_or_head_of_the_attention(gpu_lib, stride):
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = (torch.randn(4, 1, 16, 64, generator=g, device="cuda").bfloat16() for _ in "kv")
    for batch, heads, dim in ((1, 3, 0), (3, 1, 1), (1, 1, 0), (1, 1, 1)):
        q = torch.randn(batch, heads, 64, generator=g, device="cuda").bfloat16()
        table = torch.arange(4, dtype=torch.int32, device="cuda").repeat(batch, 1)
        n = torch.full((batch,), 50, dtype=torch.int32, device="cuda")
        want = gpu_lib.paged_attention(q, k, v, table, n)
        assert torch.equal(gpu_lib.paged_attention(_restrided(q, dim, stride), k, v, table, n), want)
        if batch == 1:
            assert torch.equal(gpu_lib.paged_attention(q, k, v, _restrided(table, 0, stride), n), want)


def test_rows_that_are_not_aligned_are_still_refused(gpu_lib):
    x = torch.zeros(2, 67, dtype=torch.bfloat16, device="cuda")
    A, B = torch.zeros(1, 8, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 40, 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(gpu_lib.OrbitError):
        gpu_lib.adapter_add(torch.zeros(2, 40, device="cuda"), x[:, :64], A, B, torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(gpu_lib.OrbitError):  # one row, and its first element is not aligned
        gpu_lib.adapter_add(torch.zeros(1, 40, device="cuda"), x[:1, 1:65], A, B, torch.zeros(1, dtype=torch.int32, device="cuda"))

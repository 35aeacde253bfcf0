"""Flags that have no truth value: the error is the caller's own, raised before
anything is computed."""
import pytest
import torch

pytestmark = pytest.mark.gpu


class NoTruth:
    def __bool__(self):
        raise ValueError("neither")


@pytest.mark.parametrize("flag", ["interleaved", "hadamard"])
def test_append(gpu_lib, flag):
    k = torch.ones(1, 1, 64, device="cuda").bfloat16()
    cache = torch.zeros(2, 1, 4, 64, device="cuda").bfloat16()
    with pytest.raises(ValueError, match="neither"):
        gpu_lib.kv_append(k, k, cache, cache.clone(), torch.zeros(1, dtype=torch.int64, device="cuda"), **{flag: NoTruth()})
    assert not cache.any()


def test_attention(gpu_lib):
    q = torch.ones(1, 1, 64, device="cuda").bfloat16()
    cache = torch.ones(2, 1, 4, 64, device="cuda").bfloat16()
    out = torch.zeros_like(q)
    with pytest.raises(ValueError, match="neither"):
        gpu_lib.paged_attention(q, cache, cache, torch.zeros(1, 2, dtype=torch.int32, device="cuda"),
                                torch.ones(1, dtype=torch.int32, device="cuda"), out=out, return_lse=NoTruth())
    assert not out.any()

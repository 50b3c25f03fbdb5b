"""Checks of the serving operators' binding on host tensors (CPU only: nothing is launched)."""
import pytest
import torch

import speculative_decoding_draft_05_gb300 as dspark


class Named(dspark.PagedCache):
    """A user's cache with more to it."""


class Named4(dspark.PagedCacheFp4):
    pass


def z(*shape, dt=torch.int32):
    return torch.zeros(*shape, dtype=dt)


@pytest.mark.parametrize("cls", [dspark.PagedCache, Named])
@pytest.mark.parametrize("dtype, other", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
def test_rows_of_another_type_than_the_cache(monkeypatch, cls, dtype, other):
    # (The library takes the rows' type from the cache: rows of fewer bytes would be read and written past their end.)
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    c = cls(z(1, 4, 16, 2, 64, dt=dtype), z(1, 4, 16, 2, 64, dt=dtype))
    tables = (z(3), z(2), z(2, 4))
    rows = z(5, 2, 64, dt=other)
    with pytest.raises(TypeError, match="q must be"):
        dspark.dspark_paged_attention(z(5, 4, 64, dt=other), c, 0, *tables, 0.1)
    with pytest.raises(TypeError, match="k_new must be"):
        dspark.dspark_cache_append(c, 0, rows, rows, *tables)
    with pytest.raises(TypeError, match="k_new must be"):
        dspark.dspark_cache_append_rotary(c, 0, rows, rows, *tables)
    with pytest.raises(TypeError, match="dtype must be"):
        dspark.dspark_cache_read(c, 0, *tables, 5, dtype=other)


@pytest.mark.parametrize("cls", [dspark.PagedCacheFp4, Named4])
def test_rows_of_a_4_bit_cache(monkeypatch, cls):
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    c = cls(z(1, 4, 2, 1, 576, dt=torch.uint8), z(1, 4, 2, 1, 576, dt=torch.uint8))
    tables = (z(3), z(2), z(2, 4))
    for t in (torch.float16, torch.float64, torch.int32):
        with pytest.raises(TypeError, match="q must be"):
            dspark.dspark_paged_attention(z(5, 4, 64, dt=t), c, 0, *tables, 0.1)
        with pytest.raises(TypeError, match="k_new must be"):
            dspark.dspark_cache_append(c, 0, z(5, 2, 64, dt=t), z(5, 2, 64, dt=t), *tables)

"""Numbers of experts out of range are refused, not allocated for (CPU only: without a GPU every call ends in a refusal)."""
import pytest
import torch

from tests.test_block_args_cpu import L   # noqa: F401  (the fixture)


@pytest.mark.parametrize("E", [2 ** 31 - 1, 2 ** 31 - 2, 2049, 0, -1, -2 ** 31])
def test_sort_rows_of_so_many_experts(L, E):   # noqa: F811
    x, ids = torch.zeros(8, 4), torch.zeros(8, 2, dtype=torch.int32)
    with pytest.raises(L.MoeError):
        L.moe_sort_rows(x, ids, E)


def test_sort_rows_of_more_experts_than_its_offsets_count(L):   # noqa: F811
    x, ids = torch.zeros(8, 4), torch.zeros(8, 2, dtype=torch.int32)
    for E in (2 ** 31 - 1, 9, 7):
        with pytest.raises(ValueError, match="offsets"):
            L.moe_sort_rows(x, ids, E, offsets=torch.zeros(9, dtype=torch.int32))

"""The sizes that GPU tests take for kernels and branches of their own still take them."""
import pytest

import attention_cases as cases


@pytest.mark.parametrize("itemsize", [2, 4])
def test_many_rows_on_few_keys(itemsize):
    for size, heads in cases.THIN.items():
        assert cases.thin_heads(size, itemsize) == heads[itemsize == 4], size
    assert cases.thin_heads((1, 5000, 70, 2, 1, 32), itemsize) == 0  # too few rows
    assert cases.thin_heads((1, 1_000_000, 2000, 4, 4, 32), itemsize) == 0  # too many keys


@pytest.mark.parametrize("itemsize", [2, 4])
def test_few_rows_on_very_many_keys(itemsize):
    for size, heads in cases.FEW_HEADS.items():
        assert cases.few_heads(size, itemsize) == heads[itemsize == 4], size
    assert cases.few_heads((1, 8, 60_000, 4, 4, 32), itemsize) == 1
    assert cases.few_heads((1, 33, 70_001, 4, 4, 32), itemsize) == 0

"""Cross attention at sizes that take kernels and branches of their own (attention_cases.py), against the definition in
64 bits with the bounds of test_gpu_attention.py."""
import pytest
import torch

import attention_cases as cases
import test_gpu_attention as attention

pytestmark = pytest.mark.gpu
TYPES = attention.TYPES


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["all", "both", "empty"])
@pytest.mark.parametrize("size", cases.THIN)
def test_many_rows_on_few_keys(size, kind, dtype):
    """With lse, and without, which whole tiles of rows are then stored apart for; gradients."""
    from differentiable_gaussian_splatting_dgs_amd import network
    q, k, v, dout = attention.inputs(size, dtype)
    valid = attention.valid_of(kind, size)
    got = attention.compare(q, k, v, dout, valid)
    print("without lse", flush=True)
    with torch.no_grad():
        assert torch.equal(network.cross_attention(q, k, v, *valid), got[0])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["mask", "lengths", "both"])
@pytest.mark.parametrize("size", cases.FEW_HEADS)
def test_few_rows_on_very_many_keys(size, kind, dtype):
    attention.compare(*attention.inputs(size, dtype), attention.valid_of(kind, size))


# few rows forward and back; blocks of rows, forward and back; few keys back; many rows on few keys
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", [(2, 3, 900, 2, 1, 64), (2, 20, 150, 1, 1, 40), (2, 70, 300, 2, 1, 48),
                                  (2, 70, 300, 2, 1, 128), (64, 700, 70, 9, 9, 40)])
def test_negative_scales(size, dtype):
    attention.compare(*attention.inputs(size, dtype), attention.valid_of("both", size), -0.2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,lead", [(0, 1), (1, 0), (8, 3), (5, 5)])
@pytest.mark.parametrize("order", [(0, 1, 2), (0, 2, 1), (2, 0, 1), (1, 0, 2)])
def test_strides_of_many_keys(order, pad, lead, dtype):
    """Rows at any element through loads that write LDS by themselves, in every kernel that has them."""
    for size in ((2, 70, 300, 4, 2, 24), (1, 70, 300, 2, 2, 64), (1, 70, 300, 1, 1, 128)):
        attention.compare(*attention.inputs(size, dtype, order=order, pad=pad, lead=lead),
                          attention.valid_of("both", size))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", [(1, 20, 3000, 2, 2, 3), (1, 9, 3000, 2, 1, 3), (1, 100, 3000, 1, 1, 3),
                                  (16, 700, 64, 32, 32, 3), (2, 20, 70_001, 2, 2, 2)])
def test_rows_shorter_than_a_chunk(size, dtype):
    """Which every rule sends to kernels with one tile of rows a wave, with the splits of the kernel that it names."""
    attention.compare(*attention.inputs(size, dtype), attention.valid_of("both", size))

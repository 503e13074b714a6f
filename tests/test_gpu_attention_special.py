"""Cross attention where something that counts is infinite or NaN, and where kernels meet: results against the
definition in 64 bits with the bounds of test_gpu_attention.py, and bits where they are known exactly."""
import pytest
import torch

import test_gpu_attention as attention

pytestmark = pytest.mark.gpu
TYPES = attention.TYPES


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


# batch, nq, nk, heads, kv_heads, d: rows by one and by two tiles, shared heads, odd heads, two and four heads a block
FEW = [(2, 3, 900, 2, 1, 64), (1, 20, 333, 2, 2, 40), (2, 2, 200, 6, 2, 61), (1, 3, 140, 4, 4, 256),
       (1, 8, 70_001, 4, 4, 32)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [0.125, -0.125])
@pytest.mark.parametrize("size", FEW)
def test_keys_past_the_length_have_zero_gradients_beside_infinite_rows(size, scale, dtype):
    """The tile that the length ends in is written by one wave alone: zeros past the length, bit for bit, however often
    it runs, where a query or a gradient that counts is infinite."""
    batch, _, nk = size[:3]
    q, k, v, dout = attention.inputs(size, dtype)
    q[:, 0, 0, 0] = float("inf")
    dout[:, 1, 0, 1] = -float("inf")
    k_lengths = torch.tensor([nk - 9, 70][:batch], dtype=torch.int32, device="cuda")
    first = None
    for _ in range(3):
        got = attention.run(q, k, v, dout, (None, None, k_lengths), scale)
        for b in range(batch):
            for grad in got[3:]:
                assert not bits(grad[b, int(k_lengths[b]):]).any()
        first = first or got
        assert all(torch.equal(bits(x), bits(y)) for x, y in zip(first, got))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [0.125, -0.125])
@pytest.mark.parametrize("size", FEW + [(2, 70, 100, 4, 2, 40), (2, 70, 300, 4, 2, 40), (1, 70, 200, 2, 1, 256)])
def test_masked_keys_have_zero_gradients_beside_infinite_rows(size, scale, dtype):
    """A key that its mask takes out has gradients of 0 whatever the rows hold that count: no 0 times infinity or NaN."""
    batch, nq, nk = size[:3]
    gen = torch.Generator(device="cuda").manual_seed(nk)
    mask = torch.rand(batch, nk, generator=gen, device="cuda") < 0.6
    for bad in (float("inf"), float("nan")):
        for which in (0, 3):
            ins = attention.inputs(size, dtype)
            ins[which][:, nq - 1, 0, 1] = bad
            got = attention.run(*ins, (mask, None, None), scale)
            for grad in got[3:]:
                assert not bits(grad[~mask]).any(), (bad, which)

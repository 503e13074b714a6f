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


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("size", [(1, 7, 200, 96, 1, 32), (2, 1, 300, 64, 1, 40), (1, 30, 200, 10, 2, 64),
                                  (2, 1, 2000, 14, 2, 128), (1, 3, 90, 120, 1, 48), (2, 40, 700, 21, 3, 33)])
def test_many_heads_share_their_keys(size, dtype):
    """Groups of 5, 7 and more heads than a tile has rows."""
    attention.compare(*attention.inputs(size, dtype), attention.valid_of("both", size))


@pytest.mark.parametrize("need", [(True, False, False), (False, True, False), (False, False, True), (True, True, False)])
@pytest.mark.parametrize("size", [(1, 70, 300, 2, 1, 32), (1, 500, 2000, 1, 1, 64), (2, 3, 90, 2, 1, 64),
                                  (1, 8, 70_001, 4, 4, 32), (1, 5000, 100, 1, 1, 32)])
def test_gradients_one_at_a_time(size, need):
    """By every backward kernel, with and without splits."""
    from differentiable_gaussian_splatting_dgs_amd import network
    for dtype in TYPES:
        q, k, v, dout = attention.inputs(size, dtype)
        valid = attention.valid_of("mask", size)
        out, lse, *want = attention.run(q, k, v, dout, valid)
        got = network.cross_attention_backward(dout, q, k, v, out, lse, *valid, need=need)
        for g, w, n in zip(got, want, need):
            assert (g is None) if not n else torch.equal(g, w), need


@pytest.mark.parametrize("size", [(1, 70, 200, 1, 1, 64), (1, 3, 200, 1, 1, 64), (1, 200, 70, 1, 1, 64)])
def test_rows_as_far_apart_as_32_bit_offsets_reach(size):
    """64 keys of float16, or 66 rows, nearly 2^31 bytes apart: the widest that loads take from a tile's first row."""
    q0, k0, v0, dout0 = attention.inputs(size, torch.float16)
    of_keys, of_rows = (1 << 24) - 64, (1 << 30) // 66 - 64
    print("far rows", size, flush=True)

    def far(a, b, stride):
        buf = torch.empty(a.shape[1] * stride, dtype=torch.float16, device="cuda")
        return [torch.as_strided(buf, t.shape, (0, stride, 64, 1), at).copy_(t) for t, at in ((a, 0), (b, 128))]

    (q, dout), (k, v) = far(q0, dout0, of_rows), far(k0, v0, of_keys)
    want = attention.run(q0, k0, v0, dout0, (None, None, None))
    got = attention.run(q, k, v, dout, (None, None, None))
    assert all(torch.equal(a, b) for a, b in zip(got, want))

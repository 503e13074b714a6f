"""The bias gradient of 16-bit layers is summed from dz before its rounding, whatever kernels a size takes."""
import pytest
import torch

from test_gpu_linear import TINY, U32, inputs

pytestmark = pytest.mark.gpu

# few rows; one pass; in parts; dz by few tiles, by the streaming kernel at several depths and widths (those whose
# weights fill most of LDS among them), by the wide kernel; no inputs at all
SIZES = [(16, 40, 300), (2000, 100, 90), (65_601, 20, 300), (301, 300, 40), (1500, 40, 200), (3001, 513, 100),
         (20_011, 33, 700), (20_000, 60, 257), (20_011, 120, 180), (16_400, 128, 520), (20_003, 128, 600),
         (12_345, 150, 310), (20_002, 250, 190), (9_007, 256, 300), (9_001, 700, 130), (40_000, 300, 513), (3_000, 0, 50)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("size", SIZES)
def test_db_of_terms_that_cancel(size, act, dtype):
    """All rows have one x, and dy runs q, q, q, -3 q down them: db is 0, while three times the rounded dz of q is not
    the rounded dz of 3 q, and sums of those grow with the rows.

    Bound: z has the same bits in every row, so the terms are s q and -3 s q in float32, off by u32 each.  A kernel adds
    rows of one residue modulo 16 for at most 16 tiles before it adds residues: no partial sum passes 16 times the
    largest term, and each of at most 2 additions a row rounds by u32 of that."""
    from differentiable_gaussian_splatting_dgs_amd import network
    rows, n_in, n_out = size
    x, w, b, _, dy = inputs(*size, dtype)
    x.copy_(x[:1].clone().expand_as(x))
    q = (torch.arange(n_out, device="cuda") * 7 % 40 + 1).float() / 64
    run = torch.tensor([1.0, 1.0, 1.0, -3.0], device="cuda").repeat(rows // 4 + 1)[:rows]
    run[rows // 4 * 4:] = 0
    dy.copy_((run[:, None] * q).to(dtype))
    assert torch.equal(dy.float(), run[:, None] * q)
    print(size, act, dtype, flush=True)
    db = network.linear_backward(dy, x, w, b, act=act)[2].double()
    tol = (2 * 16 + 1) * rows * U32 * 3 * 1.13 * q.double() + TINY[dtype]
    bad = ~(db.abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float((db.abs() / tol).max()))

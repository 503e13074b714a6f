"""Sizes of cross attention that take kernels and branches which small sizes do not, and the rules by which they do,
written again from csrc/attention.h (its constants are read there): batch, nq, nk, heads, kv_heads, d."""
import os
import re

_HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       "differentiable_gaussian_splatting_dgs_amd", "csrc", "attention.h")

# many rows on few keys, and the heads that a block takes: of 16 bits, of float32
THIN = {(16, 700, 64, 32, 32, 32): (4, 4), (64, 700, 70, 9, 9, 40): (1, 1), (32, 700, 40, 12, 6, 100): (2, 1),
        (16, 700, 64, 32, 32, 33): (4, 2)}
# gradients of few rows on very many keys, and the heads that a block takes
FEW_HEADS = {(1, 8, 70_001, 4, 4, 32): (4, 4), (1, 5, 70_001, 6, 6, 32): (2, 2), (2, 20, 70_001, 2, 2, 61): (2, 1)}


def constants():
    with open(_HEADER) as f:
        text = f.read()
    found = dict(re.findall(r"constexpr int (k\w+) = ([\d *]+);", text))
    return {k: eval(v) for k, v in found.items()}  # digits and products alone


def pitch_of(d):
    return next(p for p in (32, 64, 128, 256) if d <= p)


def columns(d, itemsize):
    """That products take."""
    return next(c for c in (32, 48, 64, 96, 128, 192, 256) if d <= c and (c != 48 or itemsize == 4))


def split(n, blocks, want, least):
    return max(1, min(want // blocks if blocks else 1, n // least, 512))


def thin_heads(size, itemsize):
    """Heads of keys that a block of k_attn_thin takes, or 0 where another kernel runs."""
    batch, nq, nk, heads, kv_heads, d = size
    c, wide, half = constants(), columns(d, itemsize), itemsize == 2
    group, problems = heads // kv_heads, batch * kv_heads
    rows = nq * group
    pitch = pitch_of(wide)
    tile_rows = min(16384 // (pitch * itemsize), 64)
    tile_bytes, tiles = tile_rows * pitch * itemsize, -(-nk // tile_rows)
    forward = (4 if wide <= 64 else 2 if wide <= 128 else 1) if half else 2 if wide <= 96 else 1
    if 2 * rows <= 64 * forward:
        forward = 1
    if rows <= 32 or d < 16 // itemsize or split(nk, problems * -(-rows // (64 * forward)), 512, 512) > 1:
        return 0
    if tiles > c["kThinTiles"] or tiles * 2 * tile_bytes > c["kThinBytes"]:
        return 0
    together = 0
    while together < 2 and kv_heads % (2 << together) == 0 and tiles * 4 * tile_bytes << together <= c["kThinBytes"]:
        together += 1
    each = -(-c["kThinBlocks"] // (problems >> together))
    tiles_a_wave = (4 if half else 2) if wide <= 32 else (2 if half else 1) if wide <= 128 else 1
    return 1 << together if -(-rows // (64 * tiles_a_wave >> together)) >= 2 * each else 0


def few_heads(size, itemsize):
    """Heads of keys that a block of k_attn_few_bwd takes, or 0 where another kernel runs."""
    _, nq, nk, heads, kv_heads, d = size
    rows, wide = nq * heads // kv_heads, columns(d, itemsize)
    if rows > 32 or (rows > 16 and itemsize == 4 and wide > 128):
        return 0
    together = 0
    if wide * itemsize <= 128 and nk >= constants()["kHeadsApart"]:
        while together < 2 and kv_heads % (2 << together) == 0:
            together += 1
    return 1 << together

"""Plain 64-bit forms of the 4-bit formats, their layout, the product and the
routing, written from the definitions, for the tests to compare with.

Tolerance of the product.  The operands are exact in the reference, so what
separates a result from it is (1) fp32 accumulation: taking the hardware to
truncate once per product and once per partial sum at fp32 precision, at most
2 K_pad errors of 2^-23 of the largest partial sum, which S = sum |a b| bounds,
K_pad being K rounded up to 64 (one instruction's depth); (2) alpha, 2^-24;
(3) the last rounding, half a unit: 2^-11 (fp16) or 2^-8 (bf16) of the result, or
half the smallest subnormal in fp16.
"""
import numpy as np
import torch

BLOCK = {"nvfp4": 16, "mxfp4": 32}
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def round_half_even(a, bits, least):
    """a >= 0 to the nearest number of `bits` significant bits and exponent >= least."""
    _, e = np.frexp(a)
    unit = np.ldexp(1.0, np.maximum(e - 1, least) - (bits - 1))
    return np.rint(a / unit) * unit


def quantise(x, form, exponent=0):
    """(signed elements of the grid, scales) of a float64 matrix; a block with a NaN or an
    infinity has scale NaN and elements 0."""
    rows, cols = x.shape
    size = BLOCK[form]
    blocks = -(-cols // size)
    wide = np.zeros((rows, blocks * size))
    wide[:, :cols] = x / 2.0 ** exponent
    b = wide.reshape(rows, blocks, size)
    top = np.abs(b).max(axis=2) if cols else np.zeros((rows, 0))
    finite = np.isfinite(top)
    safe = np.where(finite, top, 0.0)
    if form == "nvfp4":
        scale = np.minimum(round_half_even(safe / 6, 4, -6), 448.0)
    else:
        _, e = np.frexp(safe)
        scale = np.where(safe > 0, np.ldexp(1.0, np.maximum(e - 3, -127)), 2.0 ** -127)
    step = np.where(scale > 0, scale, 1.0)[..., None]
    with np.errstate(invalid="ignore"):
        q = np.where((scale > 0)[..., None] & finite[..., None], np.nan_to_num(b) / step, 0.0)
    el = np.minimum(round_half_even(np.abs(q), 2, 0), 6.0)
    el = np.copysign(el, q)
    return el.reshape(rows, -1)[:, :cols], np.where(finite, scale, np.nan)


def values(x, form, exponent=0):
    el, scale = quantise(x, form, exponent)
    return el * np.repeat(scale, BLOCK[form], axis=1)[:, :x.shape[1]] * 2.0 ** exponent


def tile_of(row, first, tile0):
    """(tile, row within it) of a row of a group that begins at row `first` and tile `tile0`."""
    return tile0 + (row - first) // 128, (row - first) % 128


def stored(q, groups=None):
    """(elements, scales) that an Fp4Matrix holds, read by the layout's definition.  Rows of no
    group come back as NaN scales."""
    codes = q.codes.cpu().numpy()
    both = np.stack((codes & 15, codes >> 4), axis=2).reshape(codes.shape[0], -1)
    assert not both[:, q.cols:].any() or q.routing is not None
    el = np.copysign(GRID[both & 7], np.where(both >= 8, -1.0, 1.0))[:, :q.cols]
    scales = q.scales.cpu().numpy().reshape(-1)
    size = BLOCK[q.format]
    blocks = -(-q.cols // size)
    tile_bytes = -(-q.cols // 256) * (256 // size // 4) * 512
    out = np.full((q.rows, blocks), np.nan)
    if q.routing is not None:
        off = q.routing.offsets.cpu().numpy()
        where = [(e, off[e], off[e + 1], off[e] // 128 + e) for e in range(len(off) - 1)]
    else:
        g = q.group_rows
        where = [(i, i * g, (i + 1) * g, i * -(-g // 128)) for i in range(q.groups)]
    b = np.arange(blocks)
    for _, first, end, tile0 in where:
        for r in range(first, end):
            t, in_tile = tile_of(r, first, tile0)
            at = t * tile_bytes + b // 4 * 512 + 16 * (in_tile % 32) + 4 * (in_tile // 32) + b % 4
            out[r] = decode_scales(scales[at], q.format)
    return el, out


def decode_scales(byte, form):
    byte = byte.astype(np.int64)
    if form == "mxfp4":
        return np.where(byte == 255, np.nan, np.ldexp(1.0, byte - 127))
    e, f = byte >> 3, byte & 7
    v = np.where(e > 0, np.ldexp(8.0 + f, e - 10), np.ldexp(1.0 * f, -9))
    return np.where(byte == 127, np.nan, v)


def sort(ids, experts):
    """(offsets, rows, pairs) of an int array tokens x top_k."""
    key = np.where((ids < 0) | (ids >= experts), experts, ids).reshape(-1)
    pairs = np.argsort(key, kind="stable")
    rows = np.empty_like(pairs)
    rows[pairs] = np.arange(pairs.size)
    offsets = np.searchsorted(key[pairs], np.arange(experts + 1))
    return offsets, rows.reshape(ids.shape), pairs


def half_unit(ref, dtype):
    """Half the spacing of `dtype` at |ref|, rounded up to a power of two."""
    a = np.abs(ref)
    if dtype == torch.float16:
        return np.maximum(a * 2.0 ** -11, 2.0 ** -25)
    return a * 2.0 ** -8


def product_tolerance(ref, magnitude, k, dtype):
    pad = max(-(-k // 64) * 64, 64)
    acc = 2 * pad * 2.0 ** -23 * magnitude
    return acc + half_unit(np.abs(ref) + acc, dtype) + 2.0 ** -24 * np.abs(ref)


def to_numpy(t):
    return t.detach().double().cpu().numpy()

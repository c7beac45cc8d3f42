"""Plain 64-bit forms of the F8 operators (numpy, on the host): the codec by search in the table
of element values, and products block by block."""
import numpy as np
import torch

BLOCK = 128
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
HALF_STEP = {"f32": 2.0**-24, "f16": 2.0**-11, "bf16": 2.0**-8}
TINY = {"f32": 2.0**-126, "f16": 2.0**-25, "bf16": 2.0**-126}


def element_values(fmt):
    """Values of the non-negative finite codes, in code order."""
    bits, bias, n = (3, 7, 127) if fmt == "e4m3" else (2, 15, 124)
    c = np.arange(n)
    ex, fr = c >> bits, (c & ((1 << bits) - 1)) / (1 << bits)
    return np.where(ex == 0, 2.0 ** (1 - bias) * fr, 2.0 ** (ex.astype(float) - bias) * (1 + fr))


def padded(n):
    return -(-n // BLOCK) * BLOCK


def spread(s, rows, cols, blocks):
    """Scales in their order of memory -> one for each element."""
    if blocks == "tiles":
        return np.repeat(np.repeat(s, BLOCK, 0)[:rows], BLOCK, 1)[:, :cols]
    return np.repeat(s.T, BLOCK, 1)[:, :cols]


def factors(x, fmt, blocks):
    """(r, scale) of the blocks, in the scales' order of memory; r is NaN for a block with an
    infinity or a NaN."""
    rows, cols = x.shape
    high = BLOCK if blocks == "tiles" else 1
    full = np.zeros((-(-rows // high) * high, padded(cols)))
    full[:rows, :cols] = np.abs(x)
    amax = full.reshape(full.shape[0] // high, high, -1, BLOCK).max((1, 3))
    top = TOP[fmt]
    with np.errstate(invalid="ignore"):
        r = np.float32(1) / np.maximum(amax, top * 2.0**-126).astype(np.float32) * np.float32(top)    # both in fp32
    r = (r.view(np.uint32) & np.uint32(~0x7ff & 0xffffffff)).view(np.float32).astype(float)
    r = np.where(np.isfinite(amax), r, np.nan)
    with np.errstate(invalid="ignore"):
        s = (1 / r).astype(np.float32)
    return (r, s) if blocks == "tiles" else (r.T.copy(), s.T.copy())


def quantize(x, fmt, blocks="rows"):
    """(codes, scales) in their order of memory, from values in fp64."""
    rows, cols = x.shape
    r, s = factors(x, fmt, blocks)
    r = spread(r, rows, cols, blocks)
    bad = np.isnan(r)
    grid = element_values(fmt)
    a = np.abs(np.where(bad, 0.0, x)) * np.where(bad, 0.0, r)       # 24 and 13 bits: exact
    hi = np.minimum(np.searchsorted(grid, a), len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    down, up = a - grid[lo], grid[hi] - a
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    codes = np.zeros((rows, padded(cols)), np.uint8)
    codes[:, :cols] = code + 128 * (np.signbit(x) & ~bad)
    return codes, s


def dequantize(codes, scales, cols, fmt, blocks="rows"):
    """Values in fp64, codes of infinities and NaN included."""
    grid = element_values(fmt)
    more = [np.nan] if fmt == "e4m3" else [np.inf, np.nan, np.nan, np.nan]
    g = np.concatenate((grid, more))
    v = np.concatenate((g, -g))[codes[:, :cols]]
    return v * spread(scales.astype(float), codes.shape[0], cols, blocks)


def product_bound(a, b, exact, out, fast):
    """How far a product of F8 values a b^T (fp64 tensors of torch) may be from `exact`, absolutely.

    Sums in fp32: a block's 128 products, then one multiplication by the scales' product (rounded
    itself) and one addition for each block: below (128 + 3 + blocks) roundings of 2^-24 of partial
    sums, each at most S = sum |a| |b|; on the way of few rows at most 16 more, one for each wave.
    The 8-bit instruction (`fast`) keeps of a block's products what is not below 2^-17 of the
    largest, which is at most the product of the largest elements: 128 times 2^-17 of that, and once
    more for the sum's own cut.  Then half a step of the output."""
    k = a.shape[1]
    acc = (128 + 3 + 16 + -(-k // BLOCK)) * 2.0**-24 * (a.abs() @ b.abs().t())
    if fast:
        a, b = (torch.nn.functional.pad(t.abs(), (0, -k % BLOCK)).unflatten(1, (-1, BLOCK)).amax(2) for t in (a, b))
        acc = acc + 129 * 2.0**-17 * (a @ b.t())
    return acc + HALF_STEP[out] * (exact.abs() + acc) + TINY[out]

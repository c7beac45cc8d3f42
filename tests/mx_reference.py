"""Plain 64-bit forms of the MX operators (numpy, on the host): the block codec by search
in the table of element values, products and gradients as fp64 matrix products, and the
error bounds the GPU tests hold the kernels to."""
import numpy as np

BLOCK, PAD = 32, 128
# output roundings: half a step relative to the value, and half the smallest step
HALF_STEP = {"f32": 2.0**-24, "f16": 2.0**-11, "bf16": 2.0**-8}
TINY = {"f32": 2.0**-126, "f16": 2.0**-25, "bf16": 2.0**-126}


def element_values(fmt):
    """Values of the non-negative codes, in code order."""
    bits, bias, n = (1, 1, 8) if fmt == "e2m1" else (3, 7, 127)
    c = np.arange(n)
    ex, fr = c >> bits, (c & ((1 << bits) - 1)) / (1 << bits)
    return np.where(ex == 0, 2.0 ** (1 - bias) * fr, 2.0 ** (ex.astype(float) - bias) * (1 + fr))


def padded(cols):
    return -(-cols // PAD) * PAD


def quantize(x, fmt):
    """(codes, scales) as bytes in the padded layout, from values in fp64."""
    rows, cols = x.shape
    kp = padded(cols)
    full = np.zeros((rows, kp))
    full[:, :cols] = x
    blocks = full.reshape(rows, kp // BLOCK, BLOCK)
    grid = element_values(fmt)
    amax = np.abs(blocks).max(2)                       # NaN if the block holds one
    bad = ~np.isfinite(amax)
    safe = np.where(bad | (amax == 0), 1.0, amax)
    m, ex = np.frexp(safe / grid[-1])                  # smallest e with amax <= top 2^e
    # safe / top may round to a power of two from above: decide on the products instead
    e = ex - 1
    e = np.where(np.ldexp(grid[-1], e) < safe, e + 1, e)
    e = np.where(np.ldexp(grid[-1], e - 1) >= safe, e - 1, e)
    e = np.maximum(np.where(amax == 0, -127, e), -127)
    a = np.abs(np.where(bad[:, :, None], 0.0, blocks)) * np.ldexp(1.0, -e)[:, :, None]
    hi = np.minimum(np.searchsorted(grid, a), len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    down, up = a - grid[lo], grid[hi] - a
    code = np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    sign = np.signbit(blocks) & ~bad[:, :, None]
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    if fmt == "e4m3":
        return (code + 128 * sign).astype(np.uint8).reshape(rows, kp), scales
    c = (code + 8 * sign).astype(np.uint8).reshape(rows, kp)
    return c[:, 0::2] | (c[:, 1::2] << 4), scales


def dequantize(codes, scales, cols, fmt):
    """Values in fp64 (NaN where the scale byte is 255 or the code is NaN)."""
    grid = element_values(fmt)
    rows = codes.shape[0]
    if fmt == "e2m1":
        c = np.stack((codes & 15, codes >> 4), 2).reshape(rows, -1)
        v = np.concatenate((grid, -grid))[c]
    else:
        g = np.concatenate((grid, [np.nan]))
        v = np.concatenate((g, -g))[codes]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    return (v * np.repeat(s, BLOCK, 1))[:, :cols]


def product_bound(a, b, exact, out):
    """How far an fp32-summed product a b^T, rounded once into `out`, may be from `exact`: one
    rounding of 2^-24 of the partial sum for each of the k additions and the products are
    exact, so k 2^-24 sum |a| |b|; then half a step of the output."""
    k = a.shape[1]
    s = np.abs(a) @ np.abs(b).T
    acc = (k + 8) * 2.0**-24 * s
    return acc + HALF_STEP[out] * (np.abs(exact) + acc) + TINY[out]


def sigmoid(g):
    return np.where(g >= 0, 1 / (1 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))


def swiglu(g, u):
    return g * sigmoid(g) * u


def swiglu_grads(g, u, dy):
    s = sigmoid(g)
    return dy * u * s * (1 + g * sigmoid(-g)), dy * g * s

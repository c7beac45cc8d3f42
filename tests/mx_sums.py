"""Sums that show a wrong kernel: operands whose fp32 sums are exact in any order, so results are
compared bit for bit, and a bound for random operands that follows the sums' order instead of
the contraction's length."""
import numpy as np

from mx_reference import HALF_STEP, TINY


def whole_numbers(seed, rows, cols, bits):
    """Whole numbers -3 .. 3 in blocks of 32, one block in eight of them times 2^bits; the last
    column holds no zero.  Every element is exact in E2M1, E4M3, fp16 and bf16, and a product of
    two such matrices with bits 5 and 4 has a sum |a| |b| of about 41 k, below 2^24 by a factor
    of three at k = 2^17, so its fp32 sums are exact in any order."""
    rng = np.random.default_rng(seed)
    x = rng.integers(-3, 4, (rows, cols)).astype(np.float64)
    x[:, -1] = rng.choice([-3, -1, 1, 3], rows)
    big = rng.random((rows, -(-cols // 32))) < 0.125
    return x * np.where(np.repeat(big, 32, 1)[:, :cols], 2.0**bits, 1.0)


def sums_bound(a2b2, k, exact, out):
    """How far a product summed in fp32 may be from `exact`, from the sums of the squared products.
    a2b2 = sum a^2 b^2; the elements of both operands have random signs.

    One matrix instruction adds at least 32 products to its sum: a result is made of a chain of
    k / 32 sums of that kind, each of 32 and the one before, then of at most 16 sums of waves.
    That is at most k / 32 + 48 roundings in a row on any way from a product to the result, each
    of at most one unit, 2^-23 of the partial sum it rounds (half a unit where an instruction
    rounds to nearest, a whole one where it drops bits).  A partial sum of products with random
    signs exceeds eight times the root of the sum of all squares with a chance below 1e-14."""
    acc = (k / 32 + 48) * 2.0**-23 * 8 * np.sqrt(a2b2)
    return acc + HALF_STEP[out] * (np.abs(exact) + acc) + TINY[out]

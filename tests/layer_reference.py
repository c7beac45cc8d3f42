"""Plain forms of dropout and of the embedding with its gradient (numpy, on the host)."""
import numpy as np

HALF_STEP = {"f32": 2.0**-24, "f16": 2.0**-11, "bf16": 2.0**-8}
TINY = {"f32": 2.0**-126, "f16": 2.0**-25, "bf16": 2.0**-126}


def philox(counter, key, rounds=10):
    """One block of Philox4x32 from Python's whole numbers: the paper's round, and its key schedule."""
    c, k = list(counter), list(key)
    for _ in range(rounds):
        p, q = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(q >> 32) ^ c[1] ^ k[0], q % 2**32, (p >> 32) ^ c[3] ^ k[1], p % 2**32]
        k = [(k[0] + 0x9E3779B9) % 2**32, (k[1] + 0xBB67AE85) % 2**32]
    return c


def bits(rows, cols, seed, call):
    """The 16 random bits of every element; the same rounds on whole arrays."""
    groups = -(-cols // 8)
    lo, sh = np.uint64(2**32 - 1), np.uint64(32)
    c = [np.broadcast_to(np.arange(groups, dtype=np.uint64), (rows, groups)),
         np.broadcast_to(np.arange(rows, dtype=np.uint64)[:, None], (rows, groups)),
         np.full((rows, groups), call % 2**32, np.uint64), np.full((rows, groups), call >> 32, np.uint64)]
    k = [seed % 2**32, seed >> 32]
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> sh) ^ c[1] ^ np.uint64(k[0]), q & lo, (p >> sh) ^ c[3] ^ np.uint64(k[1]), p & lo]
        k = [(k[0] + 0x9E3779B9) % 2**32, (k[1] + 0xBB67AE85) % 2**32]
    half = [h for w in c for h in (w & np.uint64(0xffff), w >> np.uint64(16))]
    return np.stack(half, 2).reshape(rows, -1)[:, :cols].astype(np.int64)


def dropout(x, p, seed, call, residual=None):
    """In fp32, before the rounding into the result's type: x and residual are fp32 arrays."""
    t = int(round(p * 65536))
    kept = bits(*x.shape, seed, call) >= t
    grow = np.float32(65536 / (65536 - t)) if t < 65536 else np.float32(0)
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.where(kept, x * grow, np.float32(0))
        return y if residual is None else y + residual


def embedding_grad(dy, tokens, vocab, scale):
    """(gradient, bound): the sum in fp64, and how far one in fp32 may be off -- a rounding of 2^-24
    for each row added, for the parts' joining (no more of them than rows) and for the scale."""
    out, mag, n = np.zeros((vocab, dy.shape[1])), np.zeros((vocab, dy.shape[1])), np.zeros((vocab, 1))
    inside = (tokens >= 0) & (tokens < vocab)
    np.add.at(out, tokens[inside], dy[inside])
    np.add.at(mag, tokens[inside], np.abs(dy[inside]))
    np.add.at(n, tokens[inside], 1)
    return out * scale, (2 * n + 2) * 2.0**-24 * mag * abs(scale)

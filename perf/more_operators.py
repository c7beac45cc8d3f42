"""Cases that measure the operators around a linear layer of a training or decoding step:
products in 8-bit floating point with a scale for each block of 128, dropout whose mask
is never stored, and the embedding lookup with its gradient.

F8 matrices: a block is 128 consecutive elements of a row ("rows") or a tile of 128 x 128
("tiles").  With top the largest element value (E4M3: 448, E5M2: 57344) and amax the
block's largest |x|, at least top 2^-126: r = top / amax in fp32, cut to 13 significant
bits; elements x r rounded to nearest, ties to the even code; scale 1 / r in fp32.  Rows
of codes are padded to 128 with zeros.  Scales of row blocks lie block by block (block,
row), those of tiles as the tiles do.

Dropout: T = round(65536 p); an element is kept when its 16 random bits are not below T, and
grows by 65536 / (65536 - T).  Row r, column c take half c % 2 of word c % 8 / 2 of
Philox4x32-10 (Salmon, Moraes, Dror, Shaw 2011) with the seed as key and the counter
(c / 8, r, call, call >> 32).

Embedding: rows of a table times a factor; a token outside the table (padding) gives zeros
and takes no gradient.

Sizes: a hidden width of 2048, a feed-forward width of 8192 and a vocabulary of 50257 are
those of the 1.3B-parameter tensor set of this repository's benchmark; the others are odd
or ragged on purpose.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 128
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
FRACTION = {"e4m3": 3, "e5m2": 2}
LOWEST = {"e4m3": -6, "e5m2": -14}        # exponent of the smallest normal element
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


# ------------------------------------------------------------------------- cases

def listed():
    return [
        # feed-forward up projection over a long prompt or training batch
        dict(name="f8_linear_prompt", op="linear", tokens=8192, k=2048, n=8192, dtype="bf16"),
        # the down projection of a middle-sized batch
        dict(name="f8_linear_down", op="linear", tokens=1024, k=8192, n=2048, dtype="bf16"),
        # one token through the vocabulary head
        dict(name="f8_linear_token_head", op="linear", tokens=1, k=2048, n=50257, dtype="bf16"),
        # a small decoding batch, ragged in every size
        dict(name="f8_linear_batch_odd", op="linear", tokens=17, k=1999, n=4093, dtype="f16"),
        # backward of the up projection: input saved in 8 bits, gradient of the weights in fp32
        dict(name="f8_grads_up", op="grads", dy_fmt="e5m2", tokens=8192, k=2048, n=8192, dtype="bf16", dw="f32"),
        # the same for a short ragged batch, gradient of the weights in 16 bits
        dict(name="f8_grads_odd", op="grads", dy_fmt="e4m3", tokens=777, k=513, n=1001, dtype="f16", dw="f16"),
        # weights after an optimizer step, for the forward and the backward product
        dict(name="f8_codec_weight", op="codec", fmt="e4m3", blocks="tiles", rows=8192, cols=2048, dtype="f32"),
        # activations of a ragged batch, for the forward product and the gradient of the weights
        dict(name="f8_codec_tokens_odd", op="codec", fmt="e4m3", blocks="rows", rows=1001, cols=1333, dtype="bf16"),
        # output of a sublayer onto the residual stream in a training step, and its backward pass
        dict(name="dropout_step", op="dropout", rows=32768, cols=2048, dtype="bf16", p=0.1, residual=True),
        # a few ragged rows without a residual
        dict(name="dropout_rows_odd", op="dropout", rows=5, cols=1365, dtype="f32", p=0.25, residual=False),
        # a training step's tokens through an fp32 table, and the table's whole gradient
        dict(name="embedding_step", op="embedding", tokens=8192, vocab=50257, width=2048, table="f32", dtype="bf16",
             grad="f32", accumulate=False),
        # a ragged batch from a 4-bit table tied to the head, its gradient added to the head's
        dict(name="embedding_tied_odd", op="embedding", tokens=1001, vocab=4093, width=1365, table="e2m1", dtype="f16",
             grad="f32", accumulate=True),
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi]; half of those above 256 are whole tiles."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v > 256 and rng.random() < 0.5:
        v = v // 128 * 128
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["linear", "linear", "grads", "codec", "dropout", "embedding"])
    if op == "codec":
        return dict(op=op, fmt=rng.choice(["e4m3", "e5m2"]), blocks=rng.choice(["rows", "tiles"]),
                    rows=_size(rng, 16, 8192), cols=_size(rng, 32, 2048), dtype=rng.choice(list(DTYPES)))
    if op == "dropout":
        return dict(op=op, rows=_size(rng, 4, 32768), cols=_size(rng, 64, 2048), dtype=rng.choice(list(DTYPES)),
                    p=round(rng.uniform(0.02, 0.6), 3), residual=rng.random() < 0.5)
    if op == "embedding":
        while True:
            tokens, vocab, width = _size(rng, 1, 65536), _size(rng, 256, 50257), _size(rng, 64, 4096)
            if tokens * width <= 8192 * 4096 and vocab * width <= 50257 * 2048:
                break
        return dict(op=op, tokens=tokens, vocab=vocab, width=width,
                    table=rng.choice(["f32", "f16", "bf16", "e2m1", "e4m3"]), dtype=rng.choice(["f16", "bf16"]),
                    grad=rng.choice(["f32", "bf16"]), accumulate=rng.random() < 0.5)
    while True:
        few = op == "linear" and rng.random() < 0.5
        tokens = _size(rng, 1, 64) if few else _size(rng, 64, 8192)
        k, n = _size(rng, 128, 8192), _size(rng, 128, 50257 if few else 8192)
        if tokens * k * n <= 8192 * 2048 * 8192 and k * n <= 50257 * 2048:
            break
    if op == "linear":
        return dict(op=op, tokens=tokens, k=k, n=n, dtype=rng.choice(["f16", "bf16"]))
    return dict(op=op, dy_fmt=rng.choice(["e4m3", "e5m2"]), tokens=tokens, k=k, n=n, dtype=rng.choice(["f16", "bf16"]),
                dw=rng.choice(["f32", "bf16"]))


# ------------------------------------------------------- F8 in elementary operations

def _pow2(e):
    """2^e in fp32 for whole e in [-126, 127], from its bits (a power function may round)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _grown(s, dim, n):
    """A scale for each block along `dim` -> one for each of n elements."""
    return s.repeat_interleave(BLOCK, dim).narrow(dim, 0, n)


def _plain_rounded(x, fmt, tiles):
    """(elements, scales) in fp32: the rounded elements, and scales as (row, block) or by tiles."""
    rows, cols = x.shape
    v = x.float()
    full = torch.nn.functional.pad(v.abs(), (0, -cols % BLOCK, 0, -rows % BLOCK if tiles else 0))
    if tiles:
        amax = full.unflatten(1, (-1, BLOCK)).amax(2).unflatten(0, (-1, BLOCK)).amax(1)
    else:
        amax = full.unflatten(1, (-1, BLOCK)).amax(2)
    r = (TOP[fmt] / amax.clamp(min=TOP[fmt] * 2.0**-126)).view(torch.int32).bitwise_and(~0x7ff).view(torch.float32)
    whole = _grown(r, 1, cols)
    if tiles:
        whole = _grown(whole, 0, rows)
    # fp64: an fp32 product of 24 and 13 bits may be rounded onto the border of two elements
    q = v.double() * whole.double()
    _, e = torch.frexp(q.abs().float())
    step = _pow2((e - 1).clamp(min=LOWEST[fmt]) - FRACTION[fmt]).double()
    # a value that fp32 rounds up to a power of two gets that one's wider step: the same element
    return (torch.round(q / step) * step).float(), 1 / r


def _pack(q, s, fmt, tiles):
    """Codes in padded rows and scales in their order of memory."""
    rows, cols = q.shape
    codes = torch.zeros(rows, -(-cols // BLOCK) * BLOCK, dtype=torch.uint8, device=q.device)
    codes[:, :cols] = q.to(F8[fmt]).view(torch.uint8)
    return codes, s if tiles else s.t().contiguous()


def _encode(x, fmt, tiles):
    return _pack(*_plain_rounded(x, fmt, tiles), fmt, tiles)


def _plain_decode(codes, scales, cols, fmt, tiles):
    s = _grown(scales if tiles else scales.t(), 1, cols)
    if tiles:
        s = _grown(s, 0, codes.shape[0])
    return codes.view(F8[fmt])[:, :cols].float() * s


def _plain_coded(x, fmt, tiles=False):
    """The values that x's elements and scales stand for."""
    q, s = _plain_rounded(x, fmt, tiles)
    s = _grown(s, 1, x.shape[1])
    return q * (_grown(s, 0, x.shape[0]) if tiles else s)


# ---------------------------------------------------------------- dropout's random bits

def _multiply(a, m):
    """High and low 32 bits of a m for int64 tensors of 32-bit values and a 32-bit constant."""
    low, high = a * (m & 0xffff), a * (m >> 16)
    total = low + ((high & 0xffff) << 16)
    return (high >> 16) + (total >> 32), total & 0xffffffff


def _plain_bits(rows, cols, seed, call, device):
    groups = -(-cols // 8)
    a = torch.arange(groups, device=device).expand(rows, groups)
    b = torch.arange(rows, device=device).unsqueeze(1).expand(rows, groups)
    c, d = torch.full_like(a, call & 0xffffffff), torch.full_like(a, call >> 32)
    k0, k1 = seed & 0xffffffff, seed >> 32
    for _ in range(10):
        h0, l0 = _multiply(a, 0xD2511F53)
        h1, l1 = _multiply(c, 0xCD9E8D57)
        a, b, c, d = h1 ^ b ^ k0, l1, h0 ^ d ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xffffffff, (k1 + 0xBB67AE85) & 0xffffffff
    w = torch.stack((a, b, c, d), 2)
    return torch.stack((w & 0xffff, w >> 16), 3).reshape(rows, -1)[:, :cols]


def _threshold(p):
    return int(round(p * 65536))


# ------------------------------------------------------------------- the MX tables

MX_TOP = {"e2m1": (1.5, 2), "e4m3": (1.75, 8)}


def _mx_encode(x, fmt):
    """Codes and scale bytes of a table in MX form: blocks of 32, the smallest power of two as scale
    with which no element is above the largest, rows padded to 128."""
    rows, cols = x.shape
    m, top = MX_TOP[fmt]
    v = torch.nn.functional.pad(x.float(), (0, -cols % 128)).view(rows, -1, 32)
    amax = v.abs().amax(2)
    frac, ex = torch.frexp(amax)
    e = torch.where(amax == 0, torch.full_like(ex, -126), (ex - 1 - top + (2 * frac > m).int()).clamp(min=-126))
    s = v * _pow2(-e).unsqueeze(2)
    scales = torch.where(amax == 0, torch.zeros_like(e), e + 127).to(torch.uint8)
    if fmt == "e4m3":
        return s.to(F8[fmt]).view(torch.uint8).view(rows, -1), scales
    a = s.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.round(a / step) * step
    c = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    c = (c | torch.signbit(s).to(torch.uint8) << 3).view(rows, -1)
    return c[:, 0::2] | c[:, 1::2] << 4, scales


def _mx_rows(codes, scales, cols, fmt):
    rows = codes.shape[0]
    if fmt == "e2m1":
        table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
        v = table[torch.stack((codes & 15, codes >> 4), 2).view(rows, -1).int()]
    else:
        v = codes.view(F8[fmt]).float()
    s = torch.where(scales > 0, scales.int() - 127, -126)
    return (v.view(rows, -1, 32) * _pow2(s).unsqueeze(2)).view(rows, -1)[:, :cols]


# ------------------------------------------------------------------------- inputs

def _normal(gen, rows, cols, scale, dtype, outliers=False, heavy=False, empty=0.0):
    """Normal values; `outliers` widens one channel in 64 (activations), `heavy` gives rows
    magnitudes over two decades (gradients), `empty` is the share of rows of padding, all zero."""
    x = torch.randn(rows, cols, device="cuda", generator=gen) * scale
    if outliers:
        x *= 1 + 19 * (torch.rand(cols, device="cuda", generator=gen) < 1 / 64).float()
    if heavy:
        x *= 10 ** (2 * torch.rand(rows, 1, device="cuda", generator=gen) - 1)
    if empty and rows > 8:
        x *= (torch.rand(rows, 1, device="cuda", generator=gen) >= empty).float()
    return x.to(DTYPES[dtype])


def _tokens(gen, count, vocab):
    """Token numbers: the k-th most frequent one about 1 / k as often as the first, whose number is
    anywhere in the table; one in fifty is padding."""
    rank = (vocab ** torch.rand(count, device="cuda", generator=gen, dtype=torch.float64)).long() - 1
    t = torch.randperm(vocab, device="cuda", generator=gen)[rank.clamp(0, vocab - 1)]
    padding = torch.rand(count, device="cuda", generator=gen) < 0.02
    return torch.where(padding & (count > 8), torch.full_like(t, -1), t)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c, dt = case, case["dtype"]
    st = dict(case=case)
    if c["op"] == "codec":
        st["x"] = _normal(gen, c["rows"], c["cols"], 0.02 if c["blocks"] == "tiles" else 1.0, dt,
                          outliers=c["blocks"] == "rows", empty=0.02)
    elif c["op"] == "linear":
        st["x"] = _normal(gen, c["tokens"], c["k"], 1.0, dt, outliers=True, empty=0.02)
        st["w"] = _encode(_normal(gen, c["n"], c["k"], 0.02, "f32"), "e4m3", True)
    elif c["op"] == "grads":
        st["dy"] = _normal(gen, c["tokens"], c["n"], 1e-2, dt, heavy=True, empty=0.02)
        w = _normal(gen, c["n"], c["k"], 0.02, "f32")
        st["wt"] = _encode(w.t(), "e4m3", True)         # tiles: the transposed codes of the forward product's
        st["xt"] = _encode(_normal(gen, c["tokens"], c["k"], 1.0, dt, outliers=True).t(), "e4m3", False)
    elif c["op"] == "dropout":
        st["x"] = _normal(gen, c["rows"], c["cols"], 1.0, dt, outliers=True)
        st["residual"] = _normal(gen, c["rows"], c["cols"], 2.0, dt) if c["residual"] else None
        st["dy"] = _normal(gen, c["rows"], c["cols"], 1e-2, dt, heavy=True)
        st["seed"], st["call"] = 0x9E3779B97F4A7C15 * (seed + 1) % 2**63, 2**33 + 7 * seed
    else:
        st["tokens"] = _tokens(gen, c["tokens"], c["vocab"])
        if c["table"] in DTYPES:
            st["table"] = _normal(gen, c["vocab"], c["width"], 0.02, c["table"])
        else:
            st["table"] = _mx_encode(_normal(gen, c["vocab"], c["width"], 0.02, "f32"), c["table"])
        st["dy"] = _normal(gen, c["tokens"], c["width"], 1e-2, dt, heavy=True)
        st["scale"] = math.sqrt(c["width"])
        if c["accumulate"]:
            st["head"] = _normal(gen, c["vocab"], c["width"], 1e-2, c["grad"])
    return st


# --------------------------------------------------------------------------- runs

def _run_own(st):
    from bit_optimizers_block_amd import bitopt
    c = st["case"]
    if c["op"] == "codec":
        codes, scales, codes_t, scales_t = bitopt.f8_quantize(st["x"], c["fmt"], c["blocks"], give="both")
        dt = st["x"].dtype
        return (bitopt.f8_dequantize(codes, scales, c["cols"], c["fmt"], c["blocks"], dtype=dt),
                bitopt.f8_dequantize(codes_t, scales_t, c["rows"], c["fmt"], c["blocks"], dtype=dt))
    if c["op"] == "linear":
        codes, scales = bitopt.f8_quantize(st["x"], "e4m3")
        return bitopt.f8_matmul(codes, scales, *st["w"], c["k"], b_blocks="tiles", dtype=st["x"].dtype)
    if c["op"] == "grads":
        fmt = c["dy_fmt"]
        codes, scales, codes_t, scales_t = bitopt.f8_quantize(st["dy"], fmt, give="both")
        dx = bitopt.f8_matmul(codes, scales, *st["wt"], c["n"], a_fmt=fmt, b_blocks="tiles", dtype=st["dy"].dtype)
        dw = bitopt.f8_matmul(codes_t, scales_t, *st["xt"], c["tokens"], a_fmt=fmt, dtype=DTYPES[c["dw"]])
        return dx, dw
    if c["op"] == "dropout":
        y = bitopt.dropout(st["x"], c["p"], st["seed"], st["call"], residual=st["residual"])
        return y, bitopt.dropout_backward(st["dy"], c["p"], st["seed"], st["call"])
    dt = DTYPES[c["dtype"]]
    if c["table"] in DTYPES:
        y = bitopt.embedding(st["tokens"], st["table"], st["scale"], dtype=dt)
    else:
        y = bitopt.mx_embedding(st["tokens"], *st["table"], c["width"], c["table"], st["scale"], dtype=dt)
    if c["accumulate"]:
        return y, bitopt.embedding_backward(st["dy"], st["tokens"], c["vocab"], st["scale"], out=st["head"].clone(),
                                            accumulate=True)
    return y, bitopt.embedding_backward(st["dy"], st["tokens"], c["vocab"], st["scale"], dtype=DTYPES[c["grad"]])


def run(state):
    if own:
        return _run_own(state)
    c, dt = state["case"], DTYPES[state["case"]["dtype"]]
    if c["op"] == "codec":
        x, tiles = state["x"], c["blocks"] == "tiles"
        return (_plain_coded(x, c["fmt"], tiles).to(dt), _plain_coded(x.t(), c["fmt"], tiles).to(dt))
    if c["op"] == "linear":
        return (_plain_coded(state["x"], "e4m3") @ _plain_decode(*state["w"], c["k"], "e4m3", True).t()).to(dt)
    if c["op"] == "grads":
        dy = state["dy"]
        wt = _plain_decode(*state["wt"], c["n"], "e4m3", True)
        xt = _plain_decode(*state["xt"], c["tokens"], "e4m3", False)
        dw = _plain_coded(dy.t(), c["dy_fmt"]) @ xt.t()
        return (_plain_coded(dy, c["dy_fmt"]) @ wt.t()).to(dt), dw.to(DTYPES[c["dw"]])
    if c["op"] == "dropout":
        t = _threshold(c["p"])
        kept = _plain_bits(c["rows"], c["cols"], state["seed"], state["call"], state["x"].device) >= t
        grow = 65536 / (65536 - t)
        y = torch.where(kept, state["x"].float() * grow, 0.0)
        if state["residual"] is not None:
            y = state["residual"].float() + y
        return y.to(dt), torch.where(kept, state["dy"].float() * grow, 0.0).to(dt)
    tokens, table = state["tokens"], state["table"]
    inside = (tokens >= 0).unsqueeze(1)
    at = tokens.clamp(min=0)
    rows = table[at].float() if c["table"] in DTYPES else _mx_rows(table[0][at], table[1][at], c["width"], c["table"])
    y = torch.where(inside, rows * state["scale"], 0.0).to(dt)
    dtable = torch.zeros(c["vocab"], c["width"], device=tokens.device)
    dtable.index_add_(0, at, torch.where(inside, state["dy"].float(), 0.0))
    dtable *= state["scale"]
    if c["accumulate"]:
        dtable += state["head"].float()
    return y, dtable.to(DTYPES[c["grad"]])


# --------------------------------------------------------------------------- work

def _f8_bytes(rows, cols, tiles):
    blocks = -(-cols // BLOCK)
    return rows * cols + 4 * blocks * (-(-rows // BLOCK) if tiles else rows)


def work(case):
    c, es = case, SIZES[case["dtype"]]
    if c["op"] == "codec":
        n = c["rows"] * c["cols"]
        return dict(bytes=3 * es * n, flops=4 * n)
    if c["op"] == "dropout":
        n = c["rows"] * c["cols"]
        return dict(bytes=(4 + c["residual"]) * es * n, flops=4 * n)
    if c["op"] == "embedding":
        n, ts = c["tokens"] * c["width"], c["vocab"] * c["width"]
        per = SIZES[c["table"]] if c["table"] in DTYPES else (0.53 if c["table"] == "e2m1" else 1.03)
        gs = SIZES[c["grad"]]
        # the whole gradient is written; where it is added to the head's, that one is read
        return dict(bytes=8 * c["tokens"] + (per + 2 * es) * n + gs * (2 * ts if c["accumulate"] else ts), flops=2 * n)
    t, k, n = c["tokens"], c["k"], c["n"]
    if c["op"] == "linear":
        return dict(bytes=es * t * k + _f8_bytes(n, k, True) + es * t * n, flops=2 * t * k * n)
    return dict(bytes=es * t * n + _f8_bytes(k, n, True) + _f8_bytes(k, t, False) + es * t * k + SIZES[c["dw"]] * n * k,
                flops=4 * t * k * n)


# -------------------------------------------------------------------------- exact

def _grid(fmt):
    """Non-negative element values in code order, from the formats' definitions."""
    bits, bias, n = {"e2m1": (1, 1, 8), "e4m3": (3, 7, 127), "e5m2": (2, 15, 124)}[fmt]
    out = []
    for c in range(n):
        ex, fr = c >> bits, c & ((1 << bits) - 1)
        out.append(2.0 ** (1 - bias) * fr / (1 << bits) if ex == 0 else 2.0 ** (ex - bias) * (1 + fr / (1 << bits)))
    return out


def _nearest(x, fmt):
    """x in fp64 -> the nearest element value, of two equally near ones that of the even code."""
    grid = torch.tensor(_grid(fmt), dtype=torch.float64, device=x.device)
    a = x.abs().contiguous()
    hi = torch.searchsorted(grid, a).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    below, above = a - grid[lo], grid[hi] - a
    return torch.copysign(torch.where((below < above) | ((below == above) & (lo % 2 == 0)), grid[lo], grid[hi]), x)


def _cut(v):
    """An fp64 value rounded to fp32, then cut to 13 significant bits."""
    m, e = torch.frexp(v.float().double())
    return torch.ldexp(torch.floor(m * 2.0**13) * 2.0**-13, e)


def _exact_coded(x, fmt, tiles=False):
    """x in fp64 -> the values of its F8 form in fp64, block by block of a padded copy."""
    rows, cols = x.shape
    high = BLOCK if tiles else 1
    full = torch.zeros(-(-rows // high) * high, -(-cols // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    full[:rows, :cols] = x
    b = full.reshape(full.shape[0] // high, high, -1, BLOCK)
    top = max(_grid(fmt))
    amax = b.abs().amax((1, 3), keepdim=True).clamp(min=math.ldexp(top, -126))
    r = _cut(top / amax)
    return (_nearest(b * r, fmt) * (1 / r).float().double()).reshape(full.shape)[:rows, :cols]


def _exact_decode(codes, scales, cols, fmt, tiles):
    grid = torch.tensor(_grid(fmt), dtype=torch.float64, device=codes.device)
    c = codes.long()[:, :cols]
    row = torch.arange(c.shape[0], device=c.device).unsqueeze(1)
    block = torch.arange(cols, device=c.device).unsqueeze(0) // BLOCK
    s = scales[row // BLOCK, block] if tiles else scales[block, row]
    return grid[(c % 128).clamp(max=len(grid) - 1)] * (1 - 2 * (c // 128)) * s.double()


def _exact_bits(rows, cols, seed, call):
    """The random bits on the host, with whole numbers of numpy."""
    import numpy as np
    lo = np.uint64(0xffffffff)
    x = [np.broadcast_to(np.arange(-(-cols // 8), dtype=np.uint64), (rows, -(-cols // 8))),
         np.broadcast_to(np.arange(rows, dtype=np.uint64)[:, None], (rows, -(-cols // 8))),
         np.uint64(call % 2**32), np.uint64(call // 2**32)]
    key = [seed % 2**32, seed // 2**32]
    for _ in range(10):
        p, q = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(q >> np.uint64(32)) ^ x[1] ^ np.uint64(key[0]), q & lo,
             (p >> np.uint64(32)) ^ x[3] ^ np.uint64(key[1]), p & lo]
        key = [(key[0] + 0x9E3779B9) % 2**32, (key[1] + 0xBB67AE85) % 2**32]
    halves = [h for w in x for h in (w % np.uint64(65536), w // np.uint64(65536))]
    return np.stack(halves, 2).reshape(rows, -1)[:, :cols].astype(np.int32)


def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] == "codec":
        x, tiles = st["x"].double(), c["blocks"] == "tiles"
        return _exact_coded(x, c["fmt"], tiles), _exact_coded(x.t(), c["fmt"], tiles)
    if c["op"] == "linear":
        return _exact_coded(st["x"].double(), "e4m3") @ _exact_decode(*st["w"], c["k"], "e4m3", True).t()
    if c["op"] == "grads":
        dy = st["dy"].double()
        dx = _exact_coded(dy, c["dy_fmt"]) @ _exact_decode(*st["wt"], c["n"], "e4m3", True).t()
        return dx, _exact_coded(dy.t(), c["dy_fmt"]) @ _exact_decode(*st["xt"], c["tokens"], "e4m3", False).t()
    if c["op"] == "dropout":
        t = round(c["p"] * 2**16)
        kept = (torch.from_numpy(_exact_bits(c["rows"], c["cols"], st["seed"], st["call"])).to("cuda") >= t).double()
        grow = 2**16 / (2**16 - t)
        y = st["x"].double() * kept * grow
        return y if st["residual"] is None else y + st["residual"].double(), st["dy"].double() * kept * grow
    tokens, scale = st["tokens"].cpu(), st["scale"]
    table = st["table"]
    if c["table"] in DTYPES:
        table = table.double()
    else:
        codes, s = table[0].long(), table[1].double()
        if c["table"] == "e2m1":
            codes = torch.cat((codes.unsqueeze(2) % 16, codes.unsqueeze(2) // 16), 2).flatten(1)
        grid = torch.tensor(_grid(c["table"]), dtype=torch.float64, device="cuda")
        half = 8 if c["table"] == "e2m1" else 128
        v = grid[(codes % half).clamp(max=len(grid) - 1)] * (1 - 2 * (codes // half))
        table = (v * torch.exp2(s - 127).repeat_interleave(32, 1))[:, :c["width"]]
    # one zero row behind the table for padding
    at = torch.where(tokens < 0, c["vocab"], tokens).cuda()
    y = torch.cat((table, torch.zeros_like(table[:1])))[at] * scale
    order = torch.argsort(at, stable=True)
    count = torch.bincount(at, minlength=c["vocab"] + 1)
    total = torch.cumsum(st["dy"].double()[order] * scale, 0)
    total = torch.cat((torch.zeros_like(total[:1]), total))
    end = torch.cumsum(count, 0)
    grad = (total[end] - total[end - count])[:-1]
    return y, grad + st["head"].double() if c["accumulate"] else grad

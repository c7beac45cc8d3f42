"""Cases that measure the microscaled (MX) operators: the block codec in 4 and 8 bits,
the products of its codes, a linear layer's three products against them, and SwiGLU
with its inputs kept in 8 bits for the backward pass.

A matrix in MX form has blocks of 32 consecutive elements of a row.  Block scale: the
smallest power of two 2^e (e >= -127, stored as the byte e + 127) whose largest
element value is not below the block's absolute maximum.  Elements: x / 2^e rounded to
nearest, ties to the even code, in E2M1 (4 bits, largest value 6) or E4M3 (8 bits,
largest value 448).  Rows are padded to 128 elements with zero codes and zero scale
bytes; E2M1 codes lie two to a byte, the even column in the low half.

Sizes: a hidden width of 2048, a feed-forward width of 8192 and a vocabulary of 50257
are those of the 1.3B-parameter tensor set of this repository's benchmark, 4096 x 4096
its single-tensor workload; the others are odd or ragged on purpose.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK, PAD = 32, 128
# largest element: significand in [1, 2) and exponent
TOP = {"e2m1": (1.5, 2), "e4m3": (1.75, 8)}


# ------------------------------------------------------------------------- cases

def listed():
    return [
        # a weight matrix brought to 4 bits and back (fake quantisation, export check)
        dict(name="codec_weight_e2m1", op="codec", fmt="e2m1", rows=8192, cols=2048, dtype="bf16"),
        # activations of a ragged batch to 8 bits and back
        dict(name="codec_tokens_e4m3_odd", op="codec", fmt="e4m3", rows=1001, cols=1333, dtype="f32"),
        # feed-forward up projection over a long prompt, both sides in 4 bits
        dict(name="product_prompt_e2m1", op="product", a_fmt="e2m1", b_fmt="e2m1", tokens=8192, k=2048, n=8192,
             dtype="bf16", out="bf16"),
        # 8-bit activations against 4-bit weights, fp32 result
        dict(name="product_square_e4m3_e2m1", op="product", a_fmt="e4m3", b_fmt="e2m1", tokens=4096, k=4096, n=4096,
             dtype="bf16", out="f32"),
        # one token through the 4-bit product
        dict(name="product_token_e2m1", op="product", a_fmt="e2m1", b_fmt="e2m1", tokens=1, k=2048, n=8192,
             dtype="bf16", out="bf16"),
        # one token through the vocabulary head with 4-bit weights
        dict(name="linear_token_head", op="linear", fmt="e2m1", tokens=1, k=2048, n=50257, dtype="bf16"),
        # a small decoding batch, ragged in every size
        dict(name="linear_batch_odd", op="linear", fmt="e2m1", tokens=17, k=1999, n=4093, dtype="f16"),
        # a prompt through the down projection with 8-bit weights
        dict(name="linear_prompt_e4m3", op="linear", fmt="e4m3", tokens=4096, k=8192, n=2048, dtype="bf16"),
        # backward of the up projection: 4-bit weights, input saved in 8 bits
        dict(name="grads_up_projection", op="grads", w_fmt="e2m1", x_fmt="e4m3", tokens=8192, k=2048, n=8192,
             dtype="bf16"),
        # the same for a short ragged batch
        dict(name="grads_short_odd", op="grads", w_fmt="e2m1", x_fmt="e4m3", tokens=777, k=513, n=1001, dtype="f16"),
        # the feed-forward activation of a training step
        dict(name="swiglu_step", op="swiglu", rows=8192, cols=8192, dtype="bf16"),
        # a few ragged rows
        dict(name="swiglu_rows_odd", op="swiglu", rows=5, cols=1365, dtype="f32"),
    ]


def _size(rng, lo, hi):
    """A size spread over the logarithm of [lo, hi]; half of those above 256 are whole tiles."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v > 256 and rng.random() < 0.5:
        v = v // 128 * 128
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["codec", "product", "linear", "grads", "swiglu"])
    if op == "codec":
        return dict(op=op, fmt=rng.choice(["e2m1", "e4m3"]), rows=_size(rng, 16, 8192), cols=_size(rng, 32, 2048),
                    dtype=rng.choice(list(DTYPES)))
    if op == "swiglu":
        return dict(op=op, rows=_size(rng, 4, 8192), cols=_size(rng, 64, 8192), dtype=rng.choice(["f32", "f16", "bf16"]))
    while True:
        few = op != "grads" and rng.random() < 0.5
        tokens = _size(rng, 1, 64) if few else _size(rng, 64, 8192)
        k, n = _size(rng, 128, 8192), _size(rng, 128, 50257 if few else 8192)
        if tokens * k * n <= 8192 * 2048 * 8192 and k * n <= 50257 * 2048:
            break
    if op == "product":
        return dict(op=op, a_fmt=rng.choice(["e2m1", "e4m3"]), b_fmt=rng.choice(["e2m1", "e4m3"]), tokens=tokens, k=k,
                    n=n, dtype=rng.choice(list(DTYPES)), out=rng.choice(["f32", "bf16"]))
    if op == "linear":
        return dict(op=op, fmt=rng.choice(["e2m1", "e4m3"]), tokens=tokens, k=k, n=n,
                    dtype=rng.choice(["f16", "bf16"]))
    return dict(op=op, w_fmt=rng.choice(["e2m1", "e4m3"]), x_fmt=rng.choice(["e2m1", "e4m3"]), tokens=tokens, k=k, n=n,
                dtype=rng.choice(["f16", "bf16"]))


# ------------------------------------------------- the codec in elementary operations

def _pow2(e):
    """2^e in fp32 for whole e in [-127, 127], from its bits (a power function may round)."""
    e = e.int()
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _plain_values(x, fmt):
    """(values, e) in fp32: the rounded elements over their scales, and the blocks' exponents,
    both over whole blocks (cols padded to 32)."""
    rows, cols = x.shape
    m, top = TOP[fmt]
    pad = -cols % BLOCK
    v = torch.nn.functional.pad(x.float(), (0, pad)).view(rows, -1, BLOCK)
    amax = v.abs().amax(2)
    frac, ex = torch.frexp(amax)                       # amax = (2 frac) * 2^(ex - 1)
    e = ex - 1 - top + (2 * frac > m).int()
    e = torch.where(amax == 0, torch.full_like(e, -127), e.clamp(min=-127))
    s = v * _pow2(-e).unsqueeze(2)
    a = s.abs()
    if fmt == "e2m1":
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        q = torch.round(a / step) * step
    else:
        _, ae = torch.frexp(a)
        sh = (ae - 1).clamp(min=-6) - 3
        q = torch.round(a * _pow2(-sh)) * _pow2(sh)
    return torch.copysign(q, s), e


def _plain_decoded(x, fmt):
    q, e = _plain_values(x, fmt)
    return (q * _pow2(e).unsqueeze(2)).reshape(x.shape[0], -1)[:, :x.shape[1]]


def _encode(x, fmt):
    """Codes and scale bytes in the padded layout."""
    q, e = _plain_values(x, fmt)
    rows, blocks = e.shape
    kp = -(-x.shape[1] // PAD) * PAD
    scales = torch.zeros(rows, kp // BLOCK, dtype=torch.uint8, device=x.device)
    scales[:, :blocks] = (e + 127).to(torch.uint8)
    q = q.reshape(rows, -1)
    if fmt == "e4m3":
        codes = torch.zeros(rows, kp, dtype=torch.uint8, device=x.device)
        codes[:, :q.shape[1]] = q.to(torch.float8_e4m3fn).view(torch.uint8)
        return codes, scales
    a = q.abs()
    c = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    c = c | (torch.signbit(q).to(torch.uint8) << 3)
    full = torch.zeros(rows, kp, dtype=torch.uint8, device=x.device)
    full[:, :c.shape[1]] = c
    return full[:, 0::2] | (full[:, 1::2] << 4), scales


def _plain_decode(codes, scales, cols, fmt):
    rows = codes.shape[0]
    if fmt == "e2m1":
        table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
        c = torch.stack((codes & 15, codes >> 4), 2).view(rows, -1)
        v = table[c.int()]
    else:
        v = codes.view(torch.float8_e4m3fn).float()
    e = scales.int() - 127
    return (v.view(rows, -1, BLOCK) * _pow2(e).unsqueeze(2)).reshape(rows, -1)[:, :cols]


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c, dt = case, case["dtype"]
    st = dict(case=case)
    if c["op"] == "codec":
        st["x"] = _normal(gen, c["rows"], c["cols"], 0.02 if c["fmt"] == "e2m1" else 1.0, dt,
                          outliers=c["fmt"] == "e4m3", empty=0.02)
    elif c["op"] == "swiglu":
        st["gate"] = _normal(gen, c["rows"], c["cols"], 1.5, dt, outliers=True, empty=0.02)
        st["up"] = _normal(gen, c["rows"], c["cols"], 1.0, dt, empty=0.02)
        st["dy"] = _normal(gen, c["rows"], c["cols"], 1e-2, dt, heavy=True)
    elif c["op"] in ("product", "linear"):
        st["x"] = _normal(gen, c["tokens"], c["k"], 1.0, dt, outliers=True, empty=0.02)
        fmt = c["b_fmt"] if c["op"] == "product" else c["fmt"]
        st["w"] = _encode(_normal(gen, c["n"], c["k"], 0.02, "f32"), fmt)
    else:
        st["dy"] = _normal(gen, c["tokens"], c["n"], 1e-2, dt, heavy=True, empty=0.02)
        st["w"] = _encode(_normal(gen, c["n"], c["k"], 0.02, "f32"), c["w_fmt"])
        st["x"] = _encode(_normal(gen, c["tokens"], c["k"], 1.0, "f32", outliers=True), c["x_fmt"])
    return st


# --------------------------------------------------------------------------- runs

def _run_own(st):
    from bit_optimizers_block_amd import bitopt
    c = st["case"]
    if c["op"] == "codec":
        codes, scales = bitopt.mx_quantize(st["x"], c["fmt"])
        return bitopt.mx_dequantize(codes, scales, c["cols"], c["fmt"], dtype=st["x"].dtype)
    if c["op"] == "swiglu":
        y, saved = bitopt.swiglu_save8(st["gate"], st["up"])
        dgate, dup = bitopt.swiglu_backward8(st["dy"], saved)
        return y, dgate, dup
    if c["op"] == "product":
        codes, scales = bitopt.mx_quantize(st["x"], c["a_fmt"])
        return bitopt.mx_matmul(codes, scales, *st["w"], c["k"], c["a_fmt"], c["b_fmt"], dtype=DTYPES[c["out"]])
    if c["op"] == "linear":
        return bitopt.mx_linear(st["x"], *st["w"], c["fmt"])
    dx = bitopt.mx_linear_grad_input(st["dy"], *st["w"], c["k"], c["w_fmt"])
    dw = bitopt.mx_linear_grad_weight(st["dy"], *st["x"], c["k"], c["x_fmt"])
    return dx, dw


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    if c["op"] == "codec":
        return _plain_decoded(state["x"], c["fmt"]).to(state["x"].dtype)
    if c["op"] == "swiglu":
        dt = state["gate"].dtype
        g, u, dy = state["gate"].float(), state["up"].float(), state["dy"].float()
        y = g * u / (1 + torch.exp(-g))
        g, u = _plain_decoded(g, "e4m3"), _plain_decoded(u, "e4m3")
        s = 1 / (1 + torch.exp(-g))
        return y.to(dt), (dy * u * s * (1 + g * (1 - s))).to(dt), (dy * g * s).to(dt)
    if c["op"] == "product":
        a = _plain_decoded(state["x"], c["a_fmt"])
        return (a @ _plain_decode(*state["w"], c["k"], c["b_fmt"]).t()).to(DTYPES[c["out"]])
    dt = DTYPES[c["dtype"]]
    if c["op"] == "linear":
        w = _plain_decode(*state["w"], c["k"], c["fmt"]).to(dt).float()
        return (state["x"].float() @ w.t()).to(dt)
    dy = state["dy"].float()
    w = _plain_decode(*state["w"], c["k"], c["w_fmt"]).to(dt).float()
    x = _plain_decode(*state["x"], c["k"], c["x_fmt"]).to(dt).float()
    return (dy @ w).to(dt), dy.t() @ x


# --------------------------------------------------------------------------- work

def _mx_bytes(rows, cols, fmt):
    return rows * cols * (0.5 if fmt == "e2m1" else 1) + rows * -(-cols // BLOCK)


def work(case):
    c, es = case, SIZES[case["dtype"]]
    if c["op"] == "codec":
        n = c["rows"] * c["cols"]
        return dict(bytes=2 * es * n, flops=4 * n)
    if c["op"] == "swiglu":
        n = c["rows"] * c["cols"]
        return dict(bytes=6 * es * n, flops=24 * n)
    t, k, n = c["tokens"], c["k"], c["n"]
    if c["op"] == "product":
        return dict(bytes=es * t * k + _mx_bytes(n, k, c["b_fmt"]) + SIZES[c["out"]] * t * n, flops=2 * t * k * n)
    if c["op"] == "linear":
        return dict(bytes=es * t * k + _mx_bytes(n, k, c["fmt"]) + es * t * n, flops=2 * t * k * n)
    return dict(bytes=es * t * n + _mx_bytes(n, k, c["w_fmt"]) + _mx_bytes(t, k, c["x_fmt"]) + es * t * k + 4 * n * k,
                flops=4 * t * k * n)


# -------------------------------------------------------------------------- exact

def _power(e):
    """2^e in fp64 for whole e in [-1022, 1023], from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _grid(fmt):
    """Non-negative element values in code order, from the formats' definitions."""
    bits, bias, n = (1, 1, 8) if fmt == "e2m1" else (3, 7, 127)
    out = []
    for c in range(n):
        ex, fr = c >> bits, c & ((1 << bits) - 1)
        out.append(2.0 ** (1 - bias) * fr / (1 << bits) if ex == 0 else 2.0 ** (ex - bias) * (1 + fr / (1 << bits)))
    return out


def _exact_rounded(x, fmt):
    """x in fp64 -> its MX value in fp64, by search in the table of element values."""
    grid = torch.tensor(_grid(fmt), dtype=torch.float64, device=x.device)
    blocks = torch.nn.functional.pad(x, (0, -x.shape[1] % BLOCK)).unflatten(1, (-1, BLOCK))
    amax = blocks.abs().amax(2, keepdim=True)
    e = torch.ceil(torch.log2(amax / grid[-1])).clamp(min=-127)
    e = torch.where(_power(e - 1) * grid[-1] >= amax, e - 1, e)          # log2's own rounding
    e = torch.where(_power(e) * grid[-1] < amax, e + 1, e).clamp(min=-127)
    scale = _power(e)
    a = (blocks / scale).abs().contiguous()
    hi = torch.searchsorted(grid, a).clamp(max=len(grid) - 1)            # first value not below a
    lo = (hi - 1).clamp(min=0)
    below, above = a - grid[lo], grid[hi] - a
    take_lo = (below < above) | ((below == above) & (lo % 2 == 0))
    v = torch.where(take_lo, grid[lo], grid[hi])
    return (torch.where(blocks < 0, -v, v) * scale).flatten(1)[:, :x.shape[1]]


def _exact_decode(codes, scales, cols, fmt):
    grid = torch.tensor(_grid(fmt), dtype=torch.float64, device=codes.device)
    c = codes.long()
    if fmt == "e2m1":
        c = torch.cat((c.unsqueeze(2) % 16, c.unsqueeze(2) // 16), 2).flatten(1)
        v = grid[c % 8] * (1 - 2 * (c // 8))
    else:
        v = grid[(c % 128).clamp(max=126)] * (1 - 2 * (c // 128))
    return (v * _power(scales.long() - 127).repeat_interleave(BLOCK, 1))[:, :cols]


def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] == "codec":
        return _exact_rounded(st["x"].double(), c["fmt"])
    if c["op"] == "swiglu":
        g, u, dy = st["gate"].double(), st["up"].double(), st["dy"].double()
        y = torch.sigmoid(g) * g * u
        g, u = _exact_rounded(g, "e4m3"), _exact_rounded(u, "e4m3")
        s = torch.sigmoid(g)
        return y, dy * u * (s + g * s * torch.sigmoid(-g)), dy * (g * s)
    if c["op"] == "product":
        return _exact_rounded(st["x"].double(), c["a_fmt"]) @ _exact_decode(*st["w"], c["k"], c["b_fmt"]).t()
    # a 16-bit product takes the decoded values in its own type
    dt = DTYPES[c["dtype"]]
    if c["op"] == "linear":
        return st["x"].double() @ _exact_decode(*st["w"], c["k"], c["fmt"]).to(dt).double().t()
    dy = st["dy"].double()
    return (dy @ _exact_decode(*st["w"], c["k"], c["w_fmt"]).to(dt).double(),
            dy.t() @ _exact_decode(*st["x"], c["k"], c["x_fmt"]).to(dt).double())

"""GPU: the F8 operators against the plain 64-bit forms of f8_reference -- codes and scales bit for
bit, products within the bound derived there -- at ragged sizes, strided and unaligned rows, every
form of the product, extreme and non-finite values; and on other streams and captured."""
import numpy as np
import pytest
import torch

import f8_reference as R
from bit_optimizers_block_amd import bitopt
from test_gpu_mx import DT, host, padded_rows, values

pytestmark = pytest.mark.gpu
FMT = ["e4m3", "e5m2"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    bitopt.lib()


# --------------------------------------------------------------------------- codec

SHAPES = [(1, 1), (1, 127), (3, 128), (5, 129), (128, 128), (127, 257), (129, 60), (300, 1000), (1200, 513)]


def same_codes(x, fmt, blocks, give="both", **kw):
    got = bitopt.f8_quantize(x, fmt, blocks, give, **kw)
    v = host(x)
    want = () if give == "columns" else R.quantize(v, fmt, blocks)
    if give != "rows":
        want += R.quantize(v.T, fmt, blocks)
    assert len(got) == len(want)
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g.cpu().numpy(), w)
    return got


@pytest.mark.parametrize("blocks", ["rows", "tiles"])
@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize(rows, cols, dtype, fmt, blocks):
    x = values(rows + cols, rows, cols, dtype, spread=2)
    codes, scales, codes_t, scales_t = same_codes(x, fmt, blocks)
    for give, want in (("rows", (codes, scales)), ("columns", (codes_t, scales_t))):
        assert all(torch.equal(a, b) for a, b in zip(bitopt.f8_quantize(x, fmt, blocks, give), want))
    for out in DT:
        # in fp32, then rounded into the type
        v = torch.from_numpy(R.dequantize(codes.cpu().numpy(), scales.cpu().numpy(), cols, fmt, blocks))
        assert torch.equal(bitopt.f8_dequantize(codes, scales, cols, fmt, blocks, dtype=DT[out]).cpu(), v.float().to(DT[out]))
        t = bitopt.f8_dequantize(codes_t, scales_t, rows, fmt, blocks, dtype=DT[out])
        if blocks == "tiles":
            assert torch.equal(t.t().cpu(), v.float().to(DT[out]))


@pytest.mark.parametrize("blocks", ["rows", "tiles"])
@pytest.mark.parametrize("dtype", list(DT))
def test_quantize_strided_rows_and_guards(dtype, blocks):
    rows, cols = 141, 211
    x = padded_rows(values(5, rows, cols, dtype), 13, 1)
    buffers, out = [], []
    for r, c in ((rows, cols), (cols, rows)):
        kb, shape = bitopt.f8_code_bytes(c), bitopt.f8_scale_shape(r, c, blocks)
        n = shape[0] * shape[1]
        cbuf = torch.full((r + 2, kb), 0xA5, dtype=torch.uint8, device="cuda")
        sbuf = torch.full((4 + n + 4,), 77.0, device="cuda")
        buffers += [cbuf, sbuf]
        out += [cbuf[1:-1], sbuf[4:4 + n].view(shape)]
    same_codes(x, "e4m3", blocks, out=out)
    for cbuf, sbuf in (buffers[:2], buffers[2:]):
        assert (cbuf[0] == 0xA5).all() and (cbuf[-1] == 0xA5).all()
        assert (sbuf[:4] == 77).all() and (sbuf[-4:] == 77).all()
    y = padded_rows(torch.zeros(rows, cols, dtype=DT[dtype], device="cuda"), 7, 3, fill=99.0)
    bitopt.f8_dequantize(out[0], out[1], cols, "e4m3", blocks, out=y)
    assert torch.equal(y, bitopt.f8_dequantize(out[0], out[1], cols, "e4m3", blocks, dtype=DT[dtype]))
    assert (y._base[:3] == 99).all() and (y._base[3 + rows * (cols + 7):] == 99).all()
    assert (y._base[3:3 + rows * (cols + 7)].view(rows, -1)[:, cols:] == 99).all()


@pytest.mark.parametrize("fmt", FMT)
def test_quantize_borders(fmt):
    """Maxima over fp32's whole range, and in each block elements on and next to every border of two
    codes: x r one rounding off a border is where a product rounded to fp32 would err."""
    grid = R.element_values(fmt)
    ties = (grid[:-1] + grid[1:]) / 2
    rows = []
    for amax in [2.0**-149, 2.0**-140, 2.0**-126, 2.0**-119 * 1.7, 2.0**-110, 1e-20, 0.7, 1.0, 3.3, 448.0, 1e4, 1e30, 3.4e38]:
        probe = np.zeros((1, 128), np.float32)
        probe[0, 0] = amax
        r = R.factors(probe.astype(float), fmt, "rows")[0][0, 0]
        x = (ties / r).astype(np.float32)
        near = np.concatenate([x, np.nextafter(x, np.float32(0)), np.nextafter(x, np.float32(3e38))])
        near = near[near < probe[0, 0]]
        near = np.resize(near, -(-max(1, len(near)) // 127) * 127).reshape(-1, 127) if len(near) else np.zeros((1, 127), np.float32)
        sign = np.where(np.arange(127) % 2, -1, 1).astype(np.float32)
        rows.append(np.concatenate((np.full((len(near), 1), probe[0, 0]), near * sign), 1).astype(np.float32))
    x = torch.from_numpy(np.concatenate(rows)).cuda()
    same_codes(x, fmt, "rows")
    same_codes(x.t().contiguous(), fmt, "rows")


@pytest.mark.parametrize("blocks", ["rows", "tiles"])
@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("dtype", list(DT))
def test_quantize_non_finite(dtype, fmt, blocks):
    x = values(3, 200, 300, dtype)
    x[0, 5], x[3, 200], x[190, 140], x[140, 299] = float("inf"), float("nan"), float("-inf"), float("nan")
    same_codes(x, fmt, blocks)


def test_quantize_large_offsets():
    """Rows beyond 2^31 bytes of input and codes: the last ones against the same rows alone."""
    rows, cols = 131200, 16500
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").uniform_(-1, 1)
    codes, scales, codes_t, scales_t = bitopt.f8_quantize(x, give="both")
    tail = bitopt.f8_quantize(x[-128:].contiguous(), give="both")      # rows is a whole number of blocks
    assert torch.equal(codes[-128:], tail[0]) and torch.equal(scales[:, -128:], tail[1])
    assert torch.equal(codes_t[:, -128:], tail[2]) and torch.equal(scales_t[-1:], tail[3])
    y = bitopt.f8_dequantize(codes, scales, cols, dtype=torch.bfloat16)
    assert torch.equal(y[-128:], bitopt.f8_dequantize(*tail[:2], cols, dtype=torch.bfloat16))


# ------------------------------------------------------------------------- products

def matrix(seed, rows, cols, fmt, blocks="rows", scale=1.0):
    """A random F8 matrix on the device: codes, scales, values in fp64."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(rows, cols, device="cuda", generator=g) * scale
    x *= 10 ** (2 * torch.rand(rows, 1, device="cuda", generator=g) - 1)
    codes, scales = bitopt.f8_quantize(x, fmt, blocks)
    return codes, scales, decoded(codes, scales, cols, fmt, blocks)


def decoded(codes, scales, cols, fmt, blocks):
    grid = R.element_values(fmt)
    more = [np.nan] if fmt == "e4m3" else [np.inf, np.nan, np.nan, np.nan]
    g = np.concatenate((grid, more))
    table = torch.from_numpy(np.concatenate((g, -g))).cuda()
    s = scales.double()
    if blocks == "tiles":
        s = s.repeat_interleave(128, 0)[:codes.shape[0]].repeat_interleave(128, 1)[:, :cols]
    else:
        s = s.t().repeat_interleave(128, 1)[:, :cols]
    return table[codes[:, :cols].int()] * s


def check(got, exact, bound, what=""):
    off = (got.double() - exact).abs()
    bad = ~(off <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}, worst {float((off / bound).max())}"


# few rows; every form of tiles, also split over the contraction with 1 to 4 blocks in the last stage;
# one row, one column, less than a block, whole and ragged sizes
PRODUCTS = [(1, 1, 1), (1, 300, 128), (3, 17, 129), (16, 129, 640), (17, 64, 2048), (32, 128, 1100), (2, 40, 5000),
            (20, 33, 4500), (33, 400, 300), (64, 128, 1100), (65, 1, 1), (65, 65, 127), (128, 128, 128), (200, 333, 515),
            (65, 700, 1024), (1700, 1500, 256), (1664, 1664, 384), (3584, 3584, 128), (3700, 3500, 300), (1100, 1500, 300),
            (300, 500, 1025), (257, 100, 1290), (70, 900, 1500), (512, 512, 2000)]


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("af,bf,blocks", [("e4m3", "e4m3", "tiles"), ("e5m2", "e4m3", "rows"), ("e4m3", "e5m2", "tiles"),
                                          ("e5m2", "e5m2", "tiles"), ("e4m3", "e4m3", "rows"), ("e5m2", "e4m3", "tiles"),
                                          ("e4m3", "e5m2", "rows"), ("e5m2", "e5m2", "rows")])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(m, n, k, af, bf, blocks, out):
    a = matrix(m + k, m, k, af)
    b = matrix(n + 1, n, k, bf, blocks, 0.1)
    y = bitopt.f8_matmul(*a[:2], *b[:2], k, af, bf, blocks, dtype=DT[out])
    exact = a[2] @ b[2].t()
    check(y, exact, R.product_bound(a[2], b[2], exact, out, m > 32 and out != "f32"))


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("k", [300, 1100])
@pytest.mark.parametrize("m", [5, 20, 130])
def test_product_accumulates_into_strided_rows(m, k, out):
    n = 77
    a, b = matrix(1, m, k, "e5m2"), matrix(2, n, k, "e4m3")
    old = values(3, m, n, out)
    y = padded_rows(old, 5, 1, fill=99.0)
    bitopt.f8_matmul(*a[:2], *b[:2], k, "e5m2", out=y, accumulate=True)
    exact = a[2] @ b[2].t()
    # the addition itself is one more fp32 rounding of the sum
    bound = R.product_bound(a[2], b[2], exact, out, m > 32 and out != "f32")
    bound = bound + (2.0**-24 + R.HALF_STEP[out]) * (exact.abs() + old.double().abs() + bound)
    check(y, exact + old.double(), bound)
    assert (y._base[:1] == 99).all() and (y._base[1 + m * (n + 5):] == 99).all()
    assert (y._base[1:1 + m * (n + 5)].view(m, -1)[:, n:] == 99).all()
    bitopt.f8_matmul(*a[:2], *b[:2], k, "e5m2", out=y)
    check(y, exact, R.product_bound(a[2], b[2], exact, out, m > 32 and out != "f32"))


@pytest.mark.parametrize("k", [400, 1300])
@pytest.mark.parametrize("m", [5, 130])
@pytest.mark.parametrize("blocks", ["rows", "tiles"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_non_finite_blocks_stay_in_their_rows(m, k, blocks, out):
    n = 300
    a, b = matrix(1, m, k, "e4m3"), matrix(2, n, k, "e4m3", blocks)
    a[1][1, 3] = float("nan")
    b[1][0, 140 if blocks == "rows" else 1] = float("nan")
    y = bitopt.f8_matmul(*a[:2], *b[:2], k, b_blocks=blocks, dtype=DT[out])
    nan = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    nan[3] = True
    if blocks == "rows":
        nan[:, 140] = True
    elif blocks == "tiles":
        nan[:, :128] = True         # tile row 0, tile column 1
    assert torch.equal(y.isnan(), nan)


def test_codes_of_infinity_and_nan():
    """Codes that no quantization here writes, but another's may."""
    for m in (4, 70):
        for fmt, code, want in (("e4m3", 0x7f, "nan"), ("e5m2", 0x7c, "inf"), ("e5m2", 0xfc, "-inf"), ("e5m2", 0x7e, "nan")):
            for out in ("f32", "bf16"):
                a, b = torch.zeros(m, 128, dtype=torch.uint8, device="cuda"), torch.zeros(80, 128, dtype=torch.uint8, device="cuda")
                sa, sb = torch.ones(1, m, device="cuda"), torch.ones(1, 80, device="cuda")
                b[:, 7] = 0x38 if fmt == "e4m3" else 0x3c      # one
                a[2, 7] = code
                y = bitopt.f8_matmul(a, sa, b, sb, 128, fmt, fmt, dtype=DT[out]).double()
                assert (y[[0, 1, 3]] == 0).all()
                assert y[2].isnan().all() if want == "nan" else (y[2] == float(want)).all()


@pytest.mark.parametrize("m", [3, 100])
def test_products_without_a_contraction(m):
    e8 = torch.empty(m, 0, dtype=torch.uint8, device="cuda"), torch.empty(0, m, device="cuda")
    w8 = torch.empty(50, 0, dtype=torch.uint8, device="cuda"), torch.empty(0, 50, device="cuda")
    for out in DT:
        assert (bitopt.f8_matmul(*e8, *w8, 0, dtype=DT[out]) == 0).all()
        y = torch.ones(m, 50, dtype=DT[out], device="cuda")
        bitopt.f8_matmul(*e8, *w8, 0, out=y, accumulate=True)
        assert (y == 1).all()


@pytest.mark.parametrize("m,n,k", [(70, 260, 2**23), (3, 140, 2**24)])
def test_product_with_large_offsets(m, n, k):
    """Rows of codes beyond 2^31 bytes: only elements near the ends of the last rows are not zero."""
    a, b = torch.zeros(m, k, dtype=torch.uint8, device="cuda"), torch.zeros(n, k, dtype=torch.uint8, device="cuda")
    sa, sb = torch.ones(k // 128, m, device="cuda"), torch.ones(k // 128, n, device="cuda")
    sa[-1], sb[-2] = 2.0, 0.25
    a[:, [5, k - 130, k - 1]], b[:, [5, k - 130, k - 1]] = 0x38, 0x40        # one, two
    b[-1] = 0
    b[-1, k - 1] = 0x30                                                       # a half
    for out in ("f32", "bf16"):
        y = bitopt.f8_matmul(a, sa, b, sb, k, dtype=DT[out])
        # 2 + 2 / 4 + 2 * 2, and 2 / 2 in the last column
        assert (y[:, :-1] == 6.5).all() and (y[:, -1] == 1.0).all()


def test_scales_of_other_makers():
    """Any finite scale may stand in a block: no power of two, none that this codec would choose."""
    m, n, k = 90, 260, 700
    a, b = matrix(1, m, k, "e4m3"), matrix(2, n, k, "e4m3", "tiles")
    sa, sb = a[1] * 3.7e-3, -b[1] * 1.3e2
    sa[2, :7] = 0.0
    for rows in (m, 20):
        ca, s = a[0][:rows].contiguous(), sa[:, :rows].contiguous()
        va, vb = decoded(ca, s, k, "e4m3", "rows"), decoded(b[0], sb, k, "e4m3", "tiles")
        exact = va @ vb.t()
        for out in DT:
            y = bitopt.f8_matmul(ca, s, b[0], sb, k, b_blocks="tiles", dtype=DT[out])
            check(y, exact, R.product_bound(va, vb, exact, out, rows > 32 and out != "f32"))


def test_same_bits_on_other_streams_and_in_graphs():
    x, dy = values(1, 300, 500, "bf16"), values(2, 300, 260, "bf16")
    w = bitopt.f8_quantize(values(3, 260, 500, "f32", 0.02), blocks="tiles", give="both")

    def step():
        xq, dq = bitopt.f8_quantize(x, give="both"), bitopt.f8_quantize(dy, "e5m2", give="both")
        return (bitopt.f8_matmul(*xq[:2], *w[:2], 500, b_blocks="tiles"),
                bitopt.f8_matmul(*dq[:2], *w[2:], 260, "e5m2", b_blocks="tiles"),
                bitopt.f8_matmul(*dq[2:], *xq[2:], 300, "e5m2", dtype=torch.float32),
                bitopt.f8_matmul(*(t[..., :8].contiguous() if t is xq[1] else t[:8].contiguous() for t in xq[:2]), *w[:2], 500,
                                 b_blocks="tiles"))
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = step()
    torch.cuda.synchronize()
    graphs, results = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            results.append(step())
    assert all(torch.equal(a, b) for a, b in zip(again, want))
    for seed in (11, 12, 13):
        x.copy_(values(seed, 300, 500, "bf16"))
        dy.copy_(values(seed + 50, 300, 260, "bf16"))
        want = step()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for r in results:
            assert all(torch.equal(a, b) for a, b in zip(r, want))

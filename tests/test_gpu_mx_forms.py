"""GPU: the forms of the MX products, each on both sides of the size at which it is taken,
against the 64-bit forms of mx_reference."""
import pytest
import torch

import mx_reference as R
from bit_optimizers_block_amd import bitopt
from test_gpu_mx import DT, check, host, mx, padded_rows, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    bitopt.lib()


# ------------------------------------------------------------- whole tiles and ragged ones

# (M, N, K) of the result and the contraction, per tile of 64, 128 and 256 rows: all whole,
# then one of them a little off.  Rows of codes are padded to 128, so 192 columns end inside
# a padded row.
WHOLE = [(64, 128, 128), (64, 128, 129), (64, 128, 127), (64, 192, 64), (64, 129, 64), (72, 128, 64), (63, 128, 64),
         (71, 128, 128), (64, 127, 65), (68, 100, 70),
         (1536, 2048, 128), (1536, 2048, 130), (1500, 2048, 128), (1536, 1990, 128), (1529, 2050, 190),
         (3328, 3840, 64), (3328, 3840, 72), (3320, 3840, 64), (3328, 3848, 64), (3325, 3850, 100)]


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("m,n,k", WHOLE)
def test_whole_and_ragged_tiles(m, n, k, fmt):
    """The three products of a linear layer whose result is m x n over k, from rows with NaN
    between them."""
    dtype = "bf16" if m % 2 else "f16"
    def operand(seed, rows, cols):
        return padded_rows(values(seed, rows, cols, dtype, 0.5), 8 if cols % 8 == 0 else 3, 0)
    def codes(seed, rows, cols):
        c, s, v = mx(seed, rows, cols, fmt, 0.1)
        return c, s, host(torch.from_numpy(v).to(DT[dtype]))
    if m > 64:
        x, (c, s, w) = operand(1, m, k), codes(2, n, k)
        exact = host(x) @ w.T
        check(bitopt.mx_linear(x, c, s, fmt), exact, R.product_bound(host(x), w, exact, dtype), "forward")
    dy, (c, s, w) = operand(3, m, k), codes(4, k, n)
    exact = host(dy) @ w
    check(bitopt.mx_linear_grad_input(dy, c, s, n, fmt), exact, R.product_bound(host(dy), w.T, exact, dtype), "dx")
    dy, (c, s, x) = operand(5, k, m), codes(6, k, n)
    exact = host(dy).T @ x
    check(bitopt.mx_linear_grad_weight(dy, c, s, n, fmt), exact, R.product_bound(host(dy).T, x.T, exact, "f32"), "dw")


@pytest.mark.parametrize("t", [3, 70])
def test_rows_of_two_to_the_22_elements(t):
    """Rows of 2^22 elements and bytes, from which a tile's offsets no longer fit 32 bits: few
    rows and tiles, 16-bit operands a long way apart, codes of rows that long."""
    far, n, k = 2**22, 37, 150
    c, s, w = mx(1, n, k, "e2m1", 0.1)
    buf = torch.full((max(t, 70) * far,), float("nan"), dtype=torch.bfloat16, device="cuda")

    def spread(x):
        v = buf.view(-1, far)[:x.shape[0], 3:3 + x.shape[1]]
        v.copy_(x)
        return v
    x = spread(values(2, t, k, "bf16"))
    exact = host(x) @ w.T
    check(bitopt.mx_linear(x, c, s, dtype=torch.float32), exact, R.product_bound(host(x), w, exact, "f32"), "forward")
    dy = spread(values(3, t, n, "bf16"))
    exact = host(dy) @ w
    check(bitopt.mx_linear_grad_input(dy, c, s, k, dtype=torch.float32), exact, R.product_bound(host(dy), w.T, exact, "f32"), "dx")
    c, s, v = mx(4, t, k, "e4m3")
    exact = host(dy).T @ v
    check(bitopt.mx_linear_grad_weight(dy, c, s, k), exact, R.product_bound(host(dy).T, v.T, exact, "f32"), "dw")
    # codes: 130 columns far behind a row's begin and 130 at its end, the rest zero
    cols, pick = far + 72, torch.cat((torch.arange(130) + far // 2, torch.arange(130) + far - 58))

    def long_rows(seed, rows):
        z = torch.zeros(rows, cols, device="cuda")
        z[:, pick] = values(seed, rows, 260, "f32")
        q = bitopt.mx_quantize(z, "e4m3")
        del z
        v = bitopt.mx_dequantize(*q, cols, "e4m3", dtype=torch.bfloat16)
        return q, host(v[:, pick])
    qa, a = long_rows(5, t)
    qb, b = long_rows(6, 5)
    exact = a @ b.T
    check(bitopt.mx_matmul(*qa, *qb, cols, "e4m3", "e4m3", dtype=torch.float32), exact, R.product_bound(a, b, exact, "f32"),
          "product")
    dy = values(7, t, 5, "bf16")
    exact = host(dy) @ b
    got = bitopt.mx_linear_grad_input(dy, *qb, cols, "e4m3", dtype=torch.float32)
    check(got[:, pick], exact, R.product_bound(host(dy), b.T, exact, "f32"), "dx of long rows")
    assert int(got.count_nonzero()) == int(got[:, pick].count_nonzero())
    exact = host(dy).T @ a
    got = bitopt.mx_linear_grad_weight(dy, *qa, cols, "e4m3")
    check(got[:, pick], exact, R.product_bound(host(dy).T, a.T, exact, "f32"), "dw of long rows")

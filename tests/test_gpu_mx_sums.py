"""GPU: the sums of the MX products in every form -- operands whose sums are exact, compared bit
for bit, and random ones within the bound of mx_sums -- with contractions on both sides of the
lengths at which the forms change."""
import pytest
import torch

import mx_sums as S
from bit_optimizers_block_amd import bitopt

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    bitopt.lib()


# (M, N, K).  Up to 16 rows: A in registers for contractions to 2048 (four waves), 4096 (eight) and,
# two E2M1 operands, 8192 (sixteen); beyond those and for more rows, by 1, 2 or 4 tiles of 16 rows
# of A and of B (B: from 6144 and 32768 rows).  Then tiles of 64, 128 and 256.
FORMS = [(1, 50, 1), (1, 40, 127), (16, 37, 2048), (7, 37, 2049), (16, 21, 4096), (9, 37, 4097), (16, 40, 8192),
         (3, 37, 8193), (16, 16, 12000),
         (10, 6200, 4097), (9, 6177, 8321), (5, 33000, 4100), (2, 32769, 8200),
         (17, 70, 2100), (32, 50, 4100), (20, 6200, 260), (31, 6150, 1200), (20, 33000, 130), (32, 32800, 600),
         (33, 70, 2100), (64, 40, 8200), (64, 6200, 1300), (50, 32800, 600),
         (65, 70, 2100), (90, 130, 8200), (200, 64, 64), (1300, 2000, 1100), (1290, 2048, 2112), (2100, 6000, 1100),
         (3328, 4096, 640)]


def whole(seed, rows, cols, bits):
    return torch.from_numpy(S.whole_numbers(seed, rows, cols, bits)).cuda()


def random(seed, rows, cols, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.float64) * scale


def mx(x, fmt):
    """The MX form of x and its values in fp64."""
    q = bitopt.mx_quantize(x.float(), fmt)
    return q, bitopt.mx_dequantize(*q, x.shape[1], fmt).double()


def same(got, exact):
    assert got.shape == exact.shape
    assert torch.equal(got.double(), exact), f"{int((got.double() != exact).sum())} of {exact.numel()} differ"


def near(got, a, b, k):
    """got against a b^T in fp64."""
    exact = a @ b.T
    limit = torch.from_numpy(S.sums_bound(((a * a) @ (b * b).T).cpu().numpy(), k, exact.cpu().numpy(), "f32"))
    off = (got.double() - exact).abs().cpu()
    assert (off <= limit).all(), f"worst {float((off / limit).max())}"


@pytest.mark.parametrize("fmts", ["e2m1 e2m1", "e2m1 e4m3", "e4m3 e2m1", "e4m3 e4m3"])
@pytest.mark.parametrize("m,n,k", FORMS)
def test_product(m, n, k, fmts):
    fa, fb = fmts.split()
    a, b = whole(1, m, k, 5), whole(2, n, k, 4)
    (qa, va), (qb, vb) = mx(a, fa), mx(b, fb)
    assert torch.equal(va, a) and torch.equal(vb, b) and float((a.abs() @ b.abs().T).max()) < 2**24
    same(bitopt.mx_matmul(*qa, *qb, k, fa, fb, dtype=torch.float32), a @ b.T)
    (qa, va), (qb, vb) = mx(random(3, m, k), fa), mx(random(4, n, k, 0.02), fb)
    near(bitopt.mx_matmul(*qa, *qb, k, fa, fb, dtype=torch.float32), va, vb, k)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k", FORMS)
def test_linear(m, n, k, dtype, fmt):
    a, b = whole(1, m, k, 5), whole(2, n, k, 4)
    assert float((a.abs() @ b.abs().T).max()) < 2**24
    same(bitopt.mx_linear(a.to(DT[dtype]), *mx(b, fmt)[0], fmt, dtype=torch.float32), a @ b.T)
    x, (q, v) = random(3, m, k).to(DT[dtype]), mx(random(4, n, k, 0.02), fmt)
    near(bitopt.mx_linear(x, *q, fmt, dtype=torch.float32), x.double(), v.to(DT[dtype]).double(), k)


# (M, N, K): K runs over n for the input gradient and over the tokens for the weight gradient
GRADS = [(1, 50, 1), (1, 40, 8200), (64, 64, 2100), (70, 200, 8193), (1300, 2000, 1100), (1280, 2048, 2112),
         (2100, 6000, 1100), (3328, 4096, 640)]


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k", GRADS)
def test_gradients(m, n, k, dtype, fmt):
    d, b = whole(1, m, k, 5), whole(3, k, n, 4)
    b[-1] = whole(6, n, 1, 0)[:, 0]                     # no zero in the last row of the contraction
    assert float((d.abs() @ b.abs()).max()) < 2**24
    q, v = mx(b, fmt)
    assert torch.equal(v, b)
    same(bitopt.mx_linear_grad_input(d.to(DT[dtype]), *q, n, fmt, dtype=torch.float32), d @ b)
    dt = d.t().contiguous().to(DT[dtype])
    got = bitopt.mx_linear_grad_weight(dt, *q, n, fmt)
    same(got, d @ b)
    bitopt.mx_linear_grad_weight(dt, *q, n, fmt, out=got, accumulate=True)
    same(got, 2 * (d @ b))                              # below 2^25 and even
    d, (q, v) = random(4, m, k).to(DT[dtype]), mx(random(5, k, n, 0.02), fmt)
    v = v.to(DT[dtype]).double()
    near(bitopt.mx_linear_grad_input(d, *q, n, fmt, dtype=torch.float32), d.double(), v.T, k)
    near(bitopt.mx_linear_grad_weight(d.t().contiguous(), *q, n, fmt), d.double(), v.T, k)

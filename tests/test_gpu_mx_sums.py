"""GPU: the sums of the MX products in every form -- operands whose sums are exact, compared bit
for bit, and random ones within the bound of mx_sums -- with contractions on both sides of the
lengths at which the forms change."""
import pytest
import torch

import mx_reference as R
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


# ------------------------------------------- elements below the normal numbers of 16 bits

def small(seed, rows, cols, fmt, dtype):
    """Random codes under scales that put most elements below `dtype`'s normal numbers, many below
    its smallest step or half way between two; as an MX matrix, and as values rounded to
    `dtype`.  In units of the smallest step (2^-133, 2^-24) an element is at most 448 2^7 < 2^16,
    so sums of up to 2^8 of them times one power of two are exact in fp32."""
    g = torch.Generator()
    g.manual_seed(seed)
    kp = (cols + 127) // 128 * 128
    codes = torch.randint(0, 256, (rows, kp // (2 if fmt == "e2m1" else 1)), generator=g, dtype=torch.uint8)
    if fmt == "e4m3":
        codes[(codes & 127) == 127] = 1                 # no NaN
        codes[:, cols:] = 0
    else:
        full = torch.stack((codes & 15, codes >> 4), 2).view(rows, -1)
        full[:, cols:] = 0
        codes = full[:, 0::2] | full[:, 1::2] << 4
    low = {"f16": 127 - 24, "bf16": 0}[dtype]
    scales = low + torch.randint(0, 2, (rows, kp // 32), generator=g, dtype=torch.uint8)
    scales[:, (cols + 31) // 32:] = 0
    v = torch.from_numpy(R.dequantize(codes.numpy(), scales.numpy(), cols, fmt))
    r = v.float().to(DT[dtype])                         # exact in fp32, then rounded to nearest even
    below = r.float().abs() < torch.finfo(DT[dtype]).tiny
    assert below.float().mean() > 0.2 and (r[below] != 0).any()
    # E2M1's least element is 2^-128, above bf16's smallest step: nothing is rounded there
    assert rows == 1 or (r.double() != v).any() == ((fmt, dtype) != ("e2m1", "bf16"))
    return (codes.cuda(), scales.cuda()), r.double().cuda()


def signs(seed, rows, cols, dtype):
    """One power of two with random signs, large enough that products are normal in fp32."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = (torch.randint(0, 2, (rows, cols), generator=g, device="cuda").double() * 2 - 1)
    return x * {"f16": 2.0**12, "bf16": 2.0**100}[dtype]


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("t", [1, 24, 60, 70, 200])
def test_elements_below_the_normal_numbers(t, dtype, fmt):
    n, k = 90, 130
    q, w = small(1, n, k, fmt, dtype)
    x, dy = signs(2, t, k, dtype), signs(3, t, n, dtype)
    same(bitopt.mx_linear(x.to(DT[dtype]), *q, fmt, dtype=torch.float32), x @ w.T)
    same(bitopt.mx_linear_grad_input(dy.to(DT[dtype]), *q, k, fmt, dtype=torch.float32), dy @ w)
    q, v = small(4, t, k, fmt, dtype)
    same(bitopt.mx_linear_grad_weight(dy.to(DT[dtype]), *q, k, fmt), dy.T @ v)
    if dtype == "bf16":                                 # products of two MX matrices decode to bf16
        q, w = small(5, n, k, fmt, dtype)
        for fa in ("e2m1", "e4m3"):
            qa, a = mx(x, fa)
            assert torch.equal(a, x)
            if fa == fmt == "e2m1":                     # multiplied as codes: nothing is rounded
                w = torch.from_numpy(R.dequantize(q[0].cpu().numpy(), q[1].cpu().numpy(), k, fmt)).cuda()
            same(bitopt.mx_matmul(*qa, *q, k, fa, fmt, dtype=torch.float32), x @ w.T)

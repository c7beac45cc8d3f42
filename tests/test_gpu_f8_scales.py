"""GPU: F8 products of scales whose product leaves fp32's range, or its normal numbers, where the results do not, in
every form: few rows, each size of tiles, split over the contraction.  Against 64 bits, which hold any such product,
within f8_reference.product_bound: taking a scale apart into a power of two and the rest rounds nothing."""
import numpy as np
import pytest
import torch

import f8_reference as R
from bit_optimizers_block_amd import bitopt
from test_gpu_f8 import decoded, matrix
from test_gpu_mx import DT

pytestmark = pytest.mark.gpu

# m, n, k of few rows (four and eight waves), of the tiles with 16-bit and with fp32 results, and split
FORMS = [(1, 40, 700), (17, 50, 5000), (65, 700, 300), (70, 900, 1500), (520, 500, 600), (1100, 1500, 300), (2300, 2100, 300),
         (4200, 4100, 128), (130, 200, 1300)]
LARGEST = {"f32": 2.0**128 * (1 - 2.0**-24), "f16": 65504.0, "bf16": 2.0**128 * (1 - 2.0**-8)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    bitopt.lib()


def fast(m, out):
    return m > 32 and out == "bf16"


def check(y, va, vb, out, m, old=None, what=""):
    exact = va @ vb.t()
    bound = R.product_bound(va, vb, exact, out, fast(m, out))
    if old is not None:
        bound = bound + (2.0**-24 + R.HALF_STEP[out]) * (exact.abs() + old.abs() + bound)
        exact = exact + old
    over = exact.abs() > LARGEST[out] + bound
    near = ~over & (exact.abs() > LARGEST[out] - bound)
    y = y.double()
    bad = torch.where(over, y != torch.copysign(torch.full_like(y, float("inf")), exact), ~((y - exact).abs() <= bound)) & ~near
    # sums are taken in fp32, and one of the terms up to any of them is at most the sum of their magnitudes: where
    # that is beyond fp32, so may be a sum on the way, and then the result is infinite or NaN
    bad &= (va.abs() @ vb.abs().t() < LARGEST["f32"] / 2) | (y.abs() < float("inf")) & over
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist(), y[bad][0].item(), exact[bad][0].item(),
                           bound[bad][0].item())


def operands(m, n, k, af, bf, blocks):
    a, b = matrix(m + k, m, k, af), matrix(n + 1, n, k, bf, blocks)
    return a[0], torch.ones_like(a[1]), b[0], torch.ones_like(b[1])


def spread(s, seed, low, high):
    """Scales of random significands and signs with exponents from `low` up to `high`."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    e = torch.randint(low, high, s.shape, device="cuda", generator=g).double()
    v = (1 + torch.rand(s.shape, device="cuda", generator=g, dtype=torch.float64)) * torch.exp2(e)
    return torch.where(torch.rand(s.shape, device="cuda", generator=g) < 0.3, -v, v).float()


# exponents of A's scales and of B's, from and up to: results of ordinary size, of fp32's smallest and largest
# normal ones, with subnormal scales, and each with ordinary scales between
RANGES = [((-90, -80), (60, 70)), ((70, 80), (-95, -85)), ((-130, -120), (105, 115)), ((-149, -140), (118, 127)),
          ((118, 127), (-149, -140)), ((-75, -70), (-60, -50)), ((-70, -64), (-70, -64)), ((-64, -62), (-55, -50)),
          ((40, 60), (30, 50)), ((60, 70), (60, 70)), ((63, 65), (-80, -60)), ((-120, 120), (-120, 120)), ((-149, 128), (-149, 128))]


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("af,bf,blocks", [("e4m3", "e4m3", "tiles"), ("e5m2", "e4m3", "rows"), ("e5m2", "e5m2", "tiles"),
                                          ("e4m3", "e5m2", "rows")])
@pytest.mark.parametrize("m,n,k", FORMS)
def test_scales_of_any_size(m, n, k, af, bf, blocks, out):
    a, sa, b, sb = operands(m, n, k, af, bf, blocks)
    for i, (ea, eb) in enumerate(RANGES):
        ta, tb = spread(sa, i, *ea), spread(sb, i + 50, *eb)
        y = bitopt.f8_matmul(a, ta, b, tb, k, af, bf, blocks, dtype=DT[out])
        va, vb = decoded(a, ta, k, af, "rows"), decoded(b, tb, k, bf, blocks)
        if i + 2 >= len(RANGES):            # sums over blocks with products of any size: the largest have to fit
            big = va.abs() @ vb.abs().t() >= 2.0**127
            exact = va @ vb.t()
            bound = R.product_bound(va, vb, exact, out, fast(m, out))
            over = exact.abs() > LARGEST[out] - bound
            assert (((y.double() - exact).abs() <= bound) | big | over).all(), (ea, eb)
        else:
            check(y, va, vb, out, m, what=(ea, eb))


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("blocks", ["rows", "tiles"])
@pytest.mark.parametrize("m,n,k", FORMS)
def test_blocks_that_add_nothing(m, n, k, blocks, out):
    """A block whose products are all zero adds nothing, whatever its scales."""
    a, sa, _ = matrix(1, m, k, "e4m3")
    b, sb, _ = matrix(2, n, k, "e4m3", blocks)
    a[:, 0:128:2], b[:, 1:128:2] = 0, 0
    sa[0] = spread(sa[0], 5, 118, 127)
    tb = sb.clone()
    if blocks == "rows":
        tb[0] = spread(sb[0], 6, 20, 127)
    else:
        tb[:, 0] = spread(sb[:, 0], 6, 20, 127)
    va, vb = decoded(a, sa, k, "e4m3", "rows"), decoded(b, tb, k, "e4m3", blocks)
    check(bitopt.f8_matmul(a, sa, b, tb, k, b_blocks=blocks, dtype=DT[out]), va, vb, out, m)
    # products of one block that cancel, the scales' product beyond fp32
    a[:, :128], b[:, :128] = 0, 0
    a[:, [3, 77]], b[:, 3], b[:, 77] = 0x30, 0x08, 0x88               # a half times +-2^-6
    sa[0], tb = 2.0**90, sb.clone()
    if blocks == "rows":
        tb[0] = 2.0**44
    else:
        tb[:, 0] = 2.0**44
    y = bitopt.f8_matmul(a, sa, b, tb, k, b_blocks=blocks, dtype=DT[out])
    if k == 128:
        assert (y == 0).all()
        return
    va = decoded(a[:, 128:], sa[1:], k - 128, "e4m3", "rows")
    vb = decoded(b[:, 128:], tb[1:] if blocks == "rows" else tb[:, 1:], k - 128, "e4m3", blocks)
    check(y, va, vb, out, m)


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("blocks", ["rows", "tiles"])
@pytest.mark.parametrize("m,n,k", FORMS)
def test_other_results_keep_their_bits(m, n, k, blocks, out):
    """Rows of zeros, rows and columns of extreme scales among ordinary ones: the ordinary results are the
    same, rows of zeros give zeros, and accumulation adds once."""
    a, sa, _ = matrix(1, m, k, "e5m2")
    b, sb, _ = matrix(2, n, k, "e4m3", blocks, 0.02)
    call = lambda a, sa, sb, **kw: bitopt.f8_matmul(a, sa, b, sb, k, "e5m2", b_blocks=blocks, **kw)
    want = call(a, sa, sb, dtype=DT[out])
    ta, ca = sa.clone(), a.clone()
    zero, small, large = 0, m // 2, m - 1
    ta[:, small] = spread(sa[:, small], 1, -120, -115)
    ta[:, large] = spread(sa[:, large], 2, 110, 115)
    ca[zero], ta[:, zero] = 0, 2.0**-126
    y = call(ca, ta, sb, dtype=DT[out])
    keep = torch.ones(m, dtype=torch.bool, device="cuda")
    keep[[zero, small, large]] = False
    assert torch.equal(y[keep], want[keep])
    assert not y[zero].any()
    va, vb = decoded(ca, ta, k, "e5m2", "rows"), decoded(b, sb, k, "e4m3", blocks)
    check(y, va, vb, out, m)
    old = torch.randn(m, n, device="cuda").to(DT[out])
    z = old.clone()
    call(ca, ta, sb, out=z, accumulate=True)
    check(z, va, vb, out, m, old.double())


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("blocks", ["rows", "tiles"])
@pytest.mark.parametrize("m,n,k", [(3, 40, 700), (70, 900, 1500), (130, 200, 300)])
def test_results_beyond_the_type_are_infinite(m, n, k, blocks, out):
    a, sa, _ = matrix(1, m, k, "e4m3")
    b, sb, _ = matrix(2, n, k, "e4m3", blocks)
    ta, tb = sa.abs() * 2.0**100, sb.abs() * 2.0**100
    y = bitopt.f8_matmul(a, ta, b, tb, k, b_blocks=blocks, dtype=DT[out])
    exact = decoded(a, ta, k, "e4m3", "rows") @ decoded(b, tb, k, "e4m3", blocks).t()
    sure = exact.abs() > 2.0**190               # far beyond: NaN where blocks of both signs are
    assert sure.any() and not (y[sure].abs() < float("inf")).any()
    # of one sign
    a, b = a & 0x7f, b & 0x7f
    y = bitopt.f8_matmul(a, ta, b, tb, k, b_blocks=blocks, dtype=DT[out])
    exact = decoded(a, ta, k, "e4m3", "rows") @ decoded(b, tb, k, "e4m3", blocks).t()
    assert (y[exact > 2.0**130] == float("inf")).all()


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("blocks", ["rows", "tiles"])
@pytest.mark.parametrize("m,n,k", FORMS)
def test_zeros(m, n, k, blocks, out):
    """Results of zero: rows of 0 and of -0, columns of zeros, and rows and columns that share no element."""
    x, w = torch.randn(m, k, device="cuda"), torch.randn(n, k, device="cuda")
    x[::3] = 0.0
    x[1::3] = -0.0
    w[n // 2:n // 2 + 3] = 0.0
    for sparse in (False, True):
        if sparse:
            x[2::3, k // 2:] = 0
            w[::2, :k // 2] = 0
        a, b = bitopt.f8_quantize(x), bitopt.f8_quantize(w, blocks=blocks)
        va, vb = decoded(*a, k, "e4m3", "rows"), decoded(*b, k, "e4m3", blocks)
        y = bitopt.f8_matmul(*a, *b, k, b_blocks=blocks, dtype=DT[out])
        check(y, va, vb, out, m)
        assert (y[va.abs() @ vb.abs().t() == 0] == 0).all()        # other sums may cancel in one precision alone


def test_values_whose_blocks_are_tiny():
    """The codec's own scales: activations of 2^-110 by weights of 2^-10 and of 2^100."""
    k = 640
    for m in (1, 20, 70, 300):
        for af in ("e4m3", "e5m2"):
            x = torch.randn(m, k, device="cuda") * 2.0**-110
            for w in (2.0**-10, 2.0**100):
                a, b = bitopt.f8_quantize(x, af), bitopt.f8_quantize(torch.randn(200, k, device="cuda") * w, blocks="tiles")
                va, vb = decoded(*a, k, af, "rows"), decoded(*b, k, "e4m3", "tiles")
                for out in ("f32", "bf16"):
                    y = bitopt.f8_matmul(*a, *b, k, af, b_blocks="tiles", dtype=DT[out])
                    check(y, va, vb, out, m, what=(m, af, w))

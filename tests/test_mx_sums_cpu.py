"""What the checks of the MX products reject, on the host: sums kept in too few bits, and a lost
last element of the contraction."""
import numpy as np
import pytest
import torch

import mx_reference as R
import mx_sums as S

SHAPES = [(16, 40, 5000), (3, 70, 8300), (9, 14, 4300), (5, 33, 2049), (8, 20, 200)]


def operands(m, n, k, fmt="e4m3"):
    rng = np.random.default_rng(m + k)
    a, b = rng.standard_normal((m, k)), rng.standard_normal((n, k)) * 0.02
    a, b = (R.dequantize(*R.quantize(x, f), k, f) for x, f in ((a, fmt), (b, "e2m1")))
    return a, b, a @ b.T


def kept(a, b, dtype, chunk=32):
    """a b^T in steps of `chunk`, the running sum kept in `dtype`."""
    s = np.zeros((a.shape[0], b.shape[0]))
    for i in range(0, a.shape[1], chunk):
        s = torch.from_numpy(s + a[:, i:i + chunk] @ b[:, i:i + chunk].T).to(dtype).double().numpy()
    return s


def bound(a, b, exact):
    return S.sums_bound((a * a) @ (b * b).T, a.shape[1], exact, "f32")


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_bound_takes_fp32_sums_only(m, n, k):
    a, b, exact = operands(m, n, k)
    limit = bound(a, b, exact)
    assert (np.abs(kept(a, b, torch.float32) - exact) <= limit).all()
    assert (np.abs(kept(a, b, torch.float32, 1) - exact) <= k / 32 * limit).all()
    rounded = torch.from_numpy(exact).bfloat16().double().numpy()       # joined in bf16 once
    assert (np.abs(rounded - exact) > limit).mean() > 0.5
    assert (np.abs(kept(a, b, torch.bfloat16) - exact) > limit).mean() > 0.9
    assert (np.abs(kept(a, b, torch.float16) - exact) > limit).mean() > 0.5
    short = a[:, :-1] @ b[:, :-1].T
    assert (np.abs(short - exact) > limit).mean() > 0.5


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_exact_sums_show_every_fault(m, n, k):
    a, b = S.whole_numbers(1, m, k, 5), S.whole_numbers(2, n, k, 4)
    for x, fmt in ((a, "e2m1"), (a, "e4m3"), (b, "e2m1"), (b, "e4m3")):
        np.testing.assert_array_equal(R.dequantize(*R.quantize(x, fmt), k, fmt), x)
    for x in (a, b):
        for t in (torch.float16, torch.bfloat16):
            np.testing.assert_array_equal(torch.from_numpy(x).to(t).double().numpy(), x)
    exact = a @ b.T
    assert (np.abs(a) @ np.abs(b).T < 2**24).all()
    np.testing.assert_array_equal(kept(a, b, torch.float32), exact)
    np.testing.assert_array_equal(kept(a, b, torch.float32, 1), exact)
    assert (kept(a, b, torch.bfloat16) != exact).mean() > 0.5
    assert (torch.from_numpy(exact).bfloat16().double().numpy() != exact).mean() > 0.5
    assert (a[:, :-1] @ b[:, :-1].T != exact).all()


def test_sums_stay_exact_up_to_the_longest_contraction():
    """Mean |a| of the whole numbers is 12/7 (7/8 + 2^bits / 8)."""
    mean = [12 / 7 * (7 / 8 + 2.0**bits / 8) for bits in (5, 4)]
    assert mean[0] * mean[1] * 2**17 < 2**23


@pytest.mark.parametrize("m,n,k", SHAPES[:2])
def test_bound_of_the_contraction_length_takes_bf16_sums(m, n, k):
    """Why these checks stand beside product_bound: its k roundings of the sum of magnitudes cover
    a result that was rounded to bf16."""
    a, b, exact = operands(m, n, k)
    rounded = torch.from_numpy(exact).bfloat16().double().numpy()
    assert (np.abs(rounded - exact) <= R.product_bound(a, b, exact, "f32")).all()

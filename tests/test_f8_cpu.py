"""F8 operators on the host, without a GPU: the reference codec the GPU tests use, sizes, and every
refusal of the C ABI and of the binding.  No call reaches a launch."""
import numpy as np
import pytest
import torch

import f8_reference as R


@pytest.fixture(scope="module")
def B():
    import os
    from bit_optimizers_block_amd import bitopt
    if not os.path.exists(bitopt.LIB_PATH):
        from bit_optimizers_block_amd import build
        build.build()
    bitopt.lib()
    return bitopt


# --------------------------------------------------------------- the reference itself

@pytest.mark.parametrize("fmt,dtype", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
def test_element_values(fmt, dtype):
    v = R.element_values(fmt)
    want = torch.arange(len(v), dtype=torch.uint8).view(dtype).double().numpy()
    np.testing.assert_array_equal(v, want)
    assert v[-1] == R.TOP[fmt]


@pytest.mark.parametrize("blocks", ["rows", "tiles"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_reference_round_trip(fmt, blocks):
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((150, 300)) * 10.0 ** rng.integers(-6, 6, (150, 1))).astype(np.float32).astype(float)
    codes, scales = R.quantize(x, fmt, blocks)
    y = R.dequantize(codes, scales, 300, fmt, blocks)
    s = R.spread(scales.astype(float), 150, 300, blocks)
    # half a step of the element, or half the smallest one; a cut of r costs nothing more
    step = 2.0**-4 if fmt == "e4m3" else 2.0**-3
    assert (np.abs(x - y) <= np.maximum(np.abs(x) * step, s * (2.0**-10 if fmt == "e4m3" else 2.0**-17)) * (1 + 1e-6)).all()
    assert (np.abs(y) <= R.TOP[fmt] * s).all()
    # the largest element of a block is not below half of the format's range of exponents
    r, _ = R.factors(x, fmt, blocks)
    assert (r * scales > 1 - 2.0**-23).all() and (r * scales < 1 + 2.0**-23).all()


def test_reference_extremes():
    for v in (0.0, 2.0**-149, 2.0**-126, 448 * 2.0**-126, 3.4e38):
        x = np.zeros((1, 128))
        x[0, 3] = np.float32(v)
        codes, scales = R.quantize(x, "e4m3")
        assert np.isfinite(scales).all() and scales.min() >= 2.0**-126 and not codes[0, :3].any()
    x[0, 3] = np.inf
    codes, scales = R.quantize(x, "e4m3")
    assert np.isnan(scales).all() and not codes.any()


# ------------------------------------------------------------------------ sizes

def test_sizes(B):
    L = B.lib()
    for cols in (0, 1, 127, 128, 129, 2048, 50257):
        assert L.bitopt_f8_code_bytes(cols) == R.padded(cols) == B.f8_code_bytes(cols)
        for rows in (0, 1, 128, 300):
            for blocks, n in (("rows", 0), ("tiles", 1)):
                shape = B.f8_scale_shape(rows, cols, blocks)
                assert L.bitopt_f8_scale_count(rows, cols, n) == shape[0] * shape[1]
    assert L.bitopt_f8_code_bytes(-1) == L.bitopt_f8_code_bytes(2**30 + 1) == -1
    assert L.bitopt_f8_scale_count(-1, 1, 0) == L.bitopt_f8_scale_count(1, -1, 0) == L.bitopt_f8_scale_count(1, 1, 2) == -1


# ------------------------------------------------------------------------- refusals

P = [(1 << 20) + (i << 16) for i in range(8)]


def quantize(L, x=P[0], dtype=0, rows=4, cols=40, ldx=40, fmt=0, blocks=0, codes=P[1], scales=P[2], ct=P[3], st=P[4]):
    return L.bitopt_f8_quantize(x, dtype, rows, cols, ldx, fmt, blocks, codes, scales, ct, st, None)


def dequantize(L, codes=P[0], scales=P[1], fmt=0, blocks=0, rows=4, cols=40, out=P[2], dtype=0, ldo=40):
    return L.bitopt_f8_dequantize(codes, scales, fmt, blocks, rows, cols, out, dtype, ldo, None)


def matmul(L, a=P[0], sa=P[1], fa=0, b=P[2], sb=P[3], fb=0, blocks=0, m=4, n=5, k=40, out=P[4], dtype=0, ldo=5, acc=0):
    return L.bitopt_f8_matmul(a, sa, fa, b, sb, fb, blocks, m, n, k, out, dtype, ldo, acc, None)


REFUSED = [
    (quantize, dict(x=None), "NULL"), (quantize, dict(codes=None), "NULL"), (quantize, dict(st=None), "NULL"),
    (quantize, dict(codes=None, scales=None, ct=None, st=None), "NULL"), (quantize, dict(scales=None), "NULL"),
    (quantize, dict(ct=None), "NULL"), (quantize, dict(dtype=3), "dtype"), (quantize, dict(fmt=2), "format"),
    (quantize, dict(blocks=2), "blocks"), (quantize, dict(rows=-1), "rows"), (quantize, dict(cols=-1), "cols"),
    (quantize, dict(ldx=39), "apart"), (quantize, dict(x=P[0] + 2), "aligned"), (quantize, dict(codes=P[1] + 8), "aligned"),
    (quantize, dict(st=P[4] + 4), "aligned"), (quantize, dict(codes=P[0]), "overlaps x"),
    (quantize, dict(scales=P[1]), "overlaps"), (quantize, dict(ct=P[1] + 384), "overlaps"),
    (quantize, dict(st=P[3] + 128 * 39), "overlaps"),
    (dequantize, dict(codes=None), "NULL"), (dequantize, dict(out=None), "NULL"), (dequantize, dict(fmt=-1), "format"),
    (dequantize, dict(blocks=-1), "blocks"), (dequantize, dict(ldo=1), "apart"), (dequantize, dict(dtype=9), "dtype"),
    (dequantize, dict(out=P[0] + 128), "overlaps codes"), (dequantize, dict(out=P[1]), "overlaps scales"),
    (matmul, dict(a=None), "NULL"), (matmul, dict(sb=None), "NULL"), (matmul, dict(out=None), "NULL"),
    (matmul, dict(fa=7), "format"), (matmul, dict(fb=7), "format"), (matmul, dict(blocks=3), "blocks"),
    (matmul, dict(m=-1), "m < 0"), (matmul, dict(n=-1), "n < 0"), (matmul, dict(k=-1), "k < 0"),
    (matmul, dict(ldo=4), "apart"), (matmul, dict(b=P[2] + 4), "aligned"), (matmul, dict(dtype=-1), "dtype"),
    (matmul, dict(out=P[0] + 64), "overlaps a"), (matmul, dict(out=P[3]), "overlaps b's scales"),
]


@pytest.mark.parametrize("call,args,text", REFUSED, ids=[f"{c.__name__}-{i}" for i, (c, _, _) in enumerate(REFUSED)])
def test_refused(B, call, args, text):
    assert call(B.lib(), **args) == B.ERR_INVALID_ARG
    assert text in B.last_error() and call.__name__ in B.last_error()


@pytest.mark.parametrize("call,args", [
    (quantize, dict(rows=2**30 + 1)), (dequantize, dict(cols=2**31)), (matmul, dict(k=2**24 + 1)),
    (matmul, dict(m=2**29, n=2**29, ldo=2**29)), (matmul, dict(m=32, n=2**27, ldo=2**27)),
    (matmul, dict(m=2**20, n=2**19, ldo=2**19)), (matmul, dict(m=2**31)),
])
def test_unsupported(B, call, args):
    assert call(B.lib(), **args) == B.ERR_UNSUPPORTED and B.last_error()


@pytest.mark.parametrize("call,args", [
    (quantize, dict(rows=0, x=None, codes=None)), (quantize, dict(cols=0, x=None)), (dequantize, dict(rows=0, out=None)),
    (matmul, dict(m=0, a=None)), (matmul, dict(n=0, b=None)),
])
def test_nothing_to_do(B, call, args):
    assert call(B.lib(), **args) == B.OK and B.last_error() == ""


def test_binding_refuses(B):
    """The binding checks before it allocates or launches: host tensors stop every call, and shapes
    and names are checked first where they are wrong too."""
    x = torch.zeros(4, 40, dtype=torch.bfloat16)
    c, s = torch.zeros(5, 128, dtype=torch.uint8), torch.zeros(1, 5)
    for call in (lambda: B.f8_quantize(x), lambda: B.f8_dequantize(c, s, 40), lambda: B.f8_matmul(c, s, c, s, 40)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(ValueError, match="format"):
        B.f8_dequantize(c, s, 40, "e2m1")
    with pytest.raises(ValueError, match="blocks"):
        B.f8_dequantize(c, s, 40, blocks="columns")
    with pytest.raises(ValueError, match="bytes a row"):
        B.f8_dequantize(c, s, 140)
    with pytest.raises(ValueError, match="scales"):
        B.f8_dequantize(c, s, 40, blocks="tiles")
    with pytest.raises(TypeError, match="uint8"):
        B.f8_dequantize(c.to(torch.int32), s, 40)
    with pytest.raises(TypeError, match="float32"):
        B.f8_matmul(c, s.double(), c, s, 40)


def test_calls_are_declared(B):
    """Every argument list of the binding has the length of the header's declaration."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "bitopt.h")).read(), flags=re.S)
    names = re.findall(r"\b(bitopt_f8_\w+)\s*\(", src)
    assert len(names) == 5
    for name in names:
        decl = re.search(name + r"\s*\(([^)]*)\)", src).group(1)
        assert len(getattr(B.lib(), name).argtypes) == len(decl.split(",")), name

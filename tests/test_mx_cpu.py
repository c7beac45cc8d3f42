"""MX operators on the host, without a GPU: the reference codec the GPU tests use, row
sizes, and every refusal of the C ABI and of the binding.  No call reaches a launch."""
import ctypes

import numpy as np
import pytest
import torch

import mx_reference as R


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

def test_element_values():
    assert R.element_values("e2m1").tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    v = R.element_values("e4m3")
    assert v[-1] == 448 and v[1] == 2.0**-9 and v[8] == 2.0**-6 and len(v) == 127
    want = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(v, want)


@pytest.mark.parametrize("fmt,top", [("e2m1", 6.0), ("e4m3", 448.0)])
def test_reference_scale_rule(fmt, top):
    for amax in (top, np.nextafter(top, 1e9), np.nextafter(top, 0), 1.0, 1e-3, 1e30, 3.5 * 2.0**-140, 0.0):
        x = np.zeros((1, 32))
        x[0, 7] = amax
        codes, scales = R.quantize(x, fmt)
        e = int(scales[0, 0]) - 127
        assert amax <= top * 2.0**e and (e == -127 or amax > top * 2.0 ** (e - 1))
        assert not codes[:, (16 if fmt == "e2m1" else 32):].any()


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_reference_round_trip_and_error(fmt):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((9, 100)) * 10.0 ** rng.integers(-6, 6, (9, 1))
    codes, scales = R.quantize(x, fmt)
    y = R.dequantize(codes, scales, 100, fmt)
    # half a step: 2^-2 of the value in E2M1's upper range, 2^-4 in E4M3's, else the step at 0
    top = 6.0 if fmt == "e2m1" else 448.0
    s = np.repeat(np.ldexp(1.0, scales.astype(int) - 127), 32, 1)[:, :100]
    assert (np.abs(x - y) <= np.maximum(np.abs(x) * (0.25 if fmt == "e2m1" else 2.0**-4),
                                        s * (0.25 if fmt == "e2m1" else 2.0**-10))).all()
    assert (np.abs(y) <= top * s).all()
    again, same = R.quantize(y, fmt)
    np.testing.assert_array_equal(R.dequantize(again, same, 100, fmt), y)


# ------------------------------------------------------------------------ row sizes

def test_row_sizes(B):
    L = B.lib()
    for cols in (0, 1, 31, 127, 128, 129, 2048, 50257):
        kp = R.padded(cols)
        assert L.bitopt_mx_code_bytes(cols, 0) == kp // 2 == B.mx_code_bytes(cols, "e2m1")
        assert L.bitopt_mx_code_bytes(cols, 1) == kp == B.mx_code_bytes(cols, "e4m3")
        assert L.bitopt_mx_scale_bytes(cols) == kp // 32 == B.mx_scale_bytes(cols)
    assert L.bitopt_mx_code_bytes(-1, 0) == L.bitopt_mx_code_bytes(8, 2) == -1
    assert L.bitopt_mx_scale_bytes(-1) == L.bitopt_mx_scale_bytes(2**30 + 1) == -1


# ------------------------------------------------------------------------- refusals

P16, ODD = 1 << 20, (1 << 20) + 8


def quantize(L, x=P16, dtype=0, rows=4, cols=40, ldx=40, fmt=0, codes=P16, scales=P16):
    return L.bitopt_mx_quantize(x, dtype, rows, cols, ldx, fmt, codes, scales, None)


def dequantize(L, codes=P16, scales=P16, fmt=0, rows=4, cols=40, out=P16, dtype=0, ldo=40):
    return L.bitopt_mx_dequantize(codes, scales, fmt, rows, cols, out, dtype, ldo, None)


def matmul(L, a=P16, sa=P16, fa=0, b=P16, sb=P16, fb=1, m=4, n=5, k=40, out=P16, dtype=0, ldo=5):
    return L.bitopt_mx_matmul(a, sa, fa, b, sb, fb, m, n, k, out, dtype, ldo, None)


def linear(L, x=P16, dtype=2, ldx=40, w=P16, sw=P16, fmt=0, tokens=4, n=5, k=40, out=P16, od=0, ldo=5):
    return L.bitopt_mx_linear(x, dtype, ldx, w, sw, fmt, tokens, n, k, out, od, ldo, None)


def grad_input(L, dy=P16, dtype=2, lddy=5, w=P16, sw=P16, fmt=0, tokens=4, n=5, k=40, out=P16, od=0, ldo=40):
    return L.bitopt_mx_linear_grad_input(dy, dtype, lddy, w, sw, fmt, tokens, n, k, out, od, ldo, None)


def grad_weight(L, dy=P16, dtype=2, lddy=5, x=P16, sx=P16, fmt=1, tokens=4, n=5, k=40, out=P16, od=0, ldo=40):
    return L.bitopt_mx_linear_grad_weight(dy, dtype, lddy, x, sx, fmt, tokens, n, k, out, od, ldo, 0, None)


def swiglu_forward(L, gate=P16, up=P16, dtype=0, rows=4, cols=40, ldg=40, ldu=40, y=P16, ldy=40, gc=P16, gs=P16, uc=P16,
                   us=P16):
    return L.bitopt_swiglu_forward_mx8(gate, up, dtype, rows, cols, ldg, ldu, y, ldy, gc, gs, uc, us, None)


def swiglu_backward(L, dy=P16, dtype=0, rows=4, cols=40, lddy=40, gc=P16, gs=P16, uc=P16, us=P16, dg=P16, lddg=40,
                    du=P16, lddu=40):
    return L.bitopt_swiglu_backward_mx8(dy, dtype, rows, cols, lddy, gc, gs, uc, us, dg, lddg, du, lddu, None)


REFUSED = [
    (quantize, dict(x=None), "NULL"), (quantize, dict(codes=None), "NULL"), (quantize, dict(scales=None), "NULL"),
    (quantize, dict(dtype=3), "dtype"), (quantize, dict(fmt=2), "format"), (quantize, dict(fmt=-1), "format"),
    (quantize, dict(rows=-1), "rows"), (quantize, dict(cols=-1), "cols"), (quantize, dict(ldx=39), "apart"),
    (quantize, dict(ldx=-40), "apart"), (quantize, dict(x=P16 + 2), "aligned"), (quantize, dict(codes=ODD), "aligned"),
    (quantize, dict(scales=ODD), "aligned"), (quantize, dict(dtype=1, x=P16 + 1), "aligned"),
    (dequantize, dict(codes=None), "NULL"), (dequantize, dict(out=None), "NULL"), (dequantize, dict(fmt=5), "format"),
    (dequantize, dict(ldo=1), "apart"), (dequantize, dict(dtype=-1), "dtype"), (dequantize, dict(rows=-5), "rows"),
    (matmul, dict(a=None), "NULL"), (matmul, dict(sb=None), "NULL"), (matmul, dict(out=None), "NULL"),
    (matmul, dict(fa=7), "format"), (matmul, dict(fb=7), "format"), (matmul, dict(m=-1), "m < 0"),
    (matmul, dict(n=-1), "n < 0"), (matmul, dict(k=-1), "k < 0"), (matmul, dict(ldo=4), "apart"),
    (matmul, dict(b=ODD), "aligned"), (matmul, dict(dtype=9), "dtype"),
    (linear, dict(x=None), "NULL"), (linear, dict(w=None), "NULL"), (linear, dict(ldx=8), "apart"),
    (linear, dict(x=P16 + 1), "aligned"), (linear, dict(od=4), "dtype"), (linear, dict(tokens=-2), "tokens"),
    (grad_input, dict(dy=None), "NULL"), (grad_input, dict(lddy=4), "apart"), (grad_input, dict(ldo=39), "apart"),
    (grad_input, dict(sw=ODD), "aligned"), (grad_input, dict(n=-1), "n < 0"),
    (grad_weight, dict(x=None), "NULL"), (grad_weight, dict(out=None), "NULL"), (grad_weight, dict(fmt=3), "format"),
    (grad_weight, dict(out=P16 + 2), "aligned"), (grad_weight, dict(k=-1), "k < 0"),
    (swiglu_forward, dict(gate=None), "NULL"), (swiglu_forward, dict(y=None), "NULL"),
    (swiglu_forward, dict(us=None), "NULL"), (swiglu_forward, dict(ldu=8), "apart"),
    (swiglu_forward, dict(gc=ODD), "aligned"), (swiglu_forward, dict(dtype=8), "dtype"),
    (swiglu_backward, dict(dy=None), "NULL"), (swiglu_backward, dict(dg=None), "NULL"),
    (swiglu_backward, dict(du=None), "NULL"), (swiglu_backward, dict(gs=None), "NULL"),
    (swiglu_backward, dict(lddu=39), "apart"), (swiglu_backward, dict(cols=-1), "cols"),
]


@pytest.mark.parametrize("call,args,text", REFUSED, ids=[f"{c.__name__}-{i}" for i, (c, _, _) in enumerate(REFUSED)])
def test_refused(B, call, args, text):
    assert call(B.lib(), **args) == B.ERR_INVALID_ARG
    assert text in B.last_error() and call.__name__.split("_")[0] in B.last_error()


@pytest.mark.parametrize("call,args", [
    (quantize, dict(rows=2**30 + 1)), (dequantize, dict(cols=2**31)), (matmul, dict(k=2**40)),
    (matmul, dict(m=2**29, n=2**29, ldo=2**29)), (linear, dict(dtype=0)), (grad_input, dict(dtype=0)),
    (grad_weight, dict(dtype=0)), (grad_weight, dict(tokens=2**30 + 1)), (swiglu_forward, dict(rows=2**33)),
    (linear, dict(tokens=2**30, n=2**30, ldo=2**30)), (grad_input, dict(tokens=2**30, k=2**30, ldo=2**30)),
    (grad_weight, dict(n=2**30, k=2**30, ldo=2**30)),
    # 2^32 threads and more in one launch: few rows, and the smallest such grid of large tiles
    (matmul, dict(m=17, n=2**30, ldo=2**30)), (linear, dict(tokens=64, n=2**30 - 63, ldo=2**30)),
    (linear, dict(tokens=2**20, n=2**19, ldo=2**19)), (grad_input, dict(tokens=2**21 - 256, k=2**18, ldo=2**18)),
    (grad_weight, dict(n=2**19, k=2**20, ldo=2**20)),
])
def test_unsupported(B, call, args):
    assert call(B.lib(), **args) == B.ERR_UNSUPPORTED and B.last_error()


@pytest.mark.parametrize("call,args", [
    (quantize, dict(rows=0, x=None, codes=None)), (quantize, dict(cols=0, x=None)), (dequantize, dict(rows=0, out=None)),
    (matmul, dict(m=0, a=None)), (matmul, dict(n=0, b=None)), (linear, dict(tokens=0, x=None)), (linear, dict(n=0, w=None)),
    (grad_input, dict(tokens=0)), (grad_input, dict(k=0)), (grad_weight, dict(n=0)), (grad_weight, dict(k=0)),
    (swiglu_forward, dict(rows=0, gate=None)), (swiglu_backward, dict(cols=0, dy=None)),
])
def test_nothing_to_do(B, call, args):
    assert call(B.lib(), **args) == B.OK and B.last_error() == ""


def test_binding_refuses(B):
    """The binding checks before it allocates or launches: host tensors stop every call, and
    shapes and formats are checked first where they are wrong too."""
    x = torch.zeros(4, 40, dtype=torch.bfloat16)
    c, s = torch.zeros(5, 64, dtype=torch.uint8), torch.zeros(5, 4, dtype=torch.uint8)
    for call in (lambda: B.mx_quantize(x), lambda: B.mx_dequantize(c, s, 40), lambda: B.mx_matmul(c, s, c, s, 40),
                 lambda: B.mx_linear(x, c, s), lambda: B.mx_linear_grad_input(x, c, s, 40),
                 lambda: B.mx_linear_grad_weight(x, c, s, 40, "e2m1"), lambda: B.swiglu_save8(x, x),
                 lambda: B.swiglu_backward8(x, (c, s, c, s))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError, match="two dimensions"):
        B.mx_quantize(torch.zeros(40))
    with pytest.raises(ValueError, match="format"):
        B.mx_dequantize(c, s, 40, "e5m2")
    with pytest.raises(ValueError, match="bytes a row"):
        B.mx_dequantize(c, s, 140)
    with pytest.raises(TypeError, match="uint8"):
        B.mx_dequantize(c.to(torch.int32), s, 40)


def test_results_are_declared(B):
    """Every argument list of the binding has the length of the header's declaration."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "bitopt.h")).read(), flags=re.S)
    for name in re.findall(r"\b(bitopt_(?:mx|swiglu)_\w+)\s*\(", src):
        decl = re.search(name + r"\s*\(([^)]*)\)", src).group(1)
        assert len(getattr(B.lib(), name).argtypes) == len(decl.split(",")), name
    assert ctypes.sizeof(ctypes.c_void_p) == 8

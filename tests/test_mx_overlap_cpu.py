"""Results of the MX calls that share memory with another matrix of the call, without a GPU: the
rows' arithmetic against a byte-by-byte form, and the refusals of the C ABI.  No call reaches a
launch."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from test_mx_cpu import (B, P16, dequantize, grad_input, grad_weight, linear, matmul, quantize,  # noqa: F401
                         swiglu_backward, swiglu_forward)

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_optimizers_block_amd", "csrc")


@pytest.fixture(scope="module")
def meet(tmp_path_factory):
    d = tmp_path_factory.mktemp("overlap")
    (d / "m.cpp").write_text('''#include "mx_overlap.h"
extern "C" int meet(uintptr_t p, int64_t r, int64_t w, int64_t s, uintptr_t q, int64_t t, int64_t v, int64_t u) {
    return bitopt::rows_meet({(const void*)p, r, w, s}, {(const void*)q, t, v, u});
}''')
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", f"-I{CSRC}", str(d / "m.cpp"), "-o", str(d / "m.so")],
                   check=True)
    f = ctypes.CDLL(str(d / "m.so")).meet
    f.argtypes = [ctypes.c_uint64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64] * 2
    return f


def touched(p, rows, width, stride):
    return {p + i * stride + j for i in range(rows) for j in range(width)}


def test_rows_meet(meet):
    rng = np.random.default_rng(0)
    both = 0
    for _ in range(20000):
        w, v = rng.integers(0, 7, 2)
        s = w + rng.integers(0, 6)
        u = max(s, v) if rng.random() < 0.5 else v + rng.integers(0, 6)
        a = (int(rng.integers(100, 160)), int(rng.integers(0, 6)), int(w), int(s))
        b = (int(rng.integers(100, 160)), int(rng.integers(0, 6)), int(v), int(u))
        want = bool(touched(*a) & touched(*b))
        assert meet(*a, *b) == meet(*b, *a) == want, (a, b)
        both += want
    assert 2000 < both < 18000


def test_rows_meet_far(meet):
    """Distances at and beyond 32 bits; a distance that no memory has."""
    p, far = 1 << 40, 1 << 33
    assert meet(p, 70000, 10, far, p + 69999 * far + 9, 1, 1, 1)
    assert not meet(p, 70000, 10, far, p + 69999 * far + 10, 1, 1, 1)
    assert not meet(p, 70000, 10, far, p + 10, 70000, 10, far)
    assert meet(p, 70000, 10, far, p + 9, 70000, 10, far)
    assert meet(p, 70000, 10, far, p + 10 + 5 * far, 30, far - 9, far)
    assert not meet(p, 2**30, 8, 2**62, p + 8, 2**30, 8, 2**62)
    assert meet(p, 2**30, 8, 2**62, p + 7, 2**30, 8, 2**62)


# quantize: 4 x 40 fp32 are 640 bytes, its codes 256, its scales 16
S = P16 + (1 << 12)
APART = dict(gc=P16 + 4096, gs=P16 + 8192, uc=P16 + 12288, us=P16 + 16384)
OVERLAPS = [
    (quantize, dict(codes=P16, scales=S), "codes overlaps x"), (quantize, dict(codes=S, scales=P16 + 624), "scales overlaps x"),
    (quantize, dict(x=S, codes=P16, scales=P16 + 240), "codes overlaps scales"),
    (dequantize, dict(scales=S), "out overlaps codes"), (dequantize, dict(codes=S, out=P16 + 12), "out overlaps scales"),
    (matmul, dict(a=S, sa=S, b=P16, sb=S), "out overlaps b"), (matmul, dict(a=P16 + 64, b=S, sa=S, sb=S), "out overlaps a"),
    (matmul, dict(a=S, b=S, sb=S), "out overlaps a's scales"), (matmul, dict(a=S, b=S, sa=S), "out overlaps b's scales"),
    (linear, dict(w=S, sw=S), "out overlaps x"), (linear, dict(x=S, sw=S), "out overlaps w"),
    (linear, dict(x=S, w=S), "out overlaps w's scales"), (linear, dict(w=S, sw=S, n=40, ldo=40, od=2), "out overlaps x"),
    (linear, dict(x=P16 + 2, w=S, sw=S, ldx=80, ldo=77), "out overlaps x"),
    (grad_input, dict(w=S, sw=S), "dx overlaps dy"), (grad_input, dict(dy=S, sw=S), "dx overlaps w"),
    (grad_weight, dict(x=S, sx=S), "dw overlaps dy"), (grad_weight, dict(dy=S, sx=S), "dw overlaps x"),
    (grad_weight, dict(dy=S, x=S), "dw overlaps x's scales"),
    (swiglu_forward, dict(gate=P16 + 4, up=S, **APART), "y overlaps gate"),
    (swiglu_forward, dict(up=P16 + 160, gate=S, **APART), "y overlaps up"),
    (swiglu_forward, dict(ldg=41, up=S, **APART), "y overlaps gate"),
    (swiglu_forward, dict(gate=S, up=S, **{**APART, "uc": P16 + 4096}), "gate's codes overlaps up's codes"),
    (swiglu_forward, dict(gate=S, up=S, **{**APART, "gs": P16}), "y overlaps gate's scales"),
    (swiglu_forward, dict(gate=P16 + 4096, y=P16 + (1 << 15), up=P16 + 20480, **APART), "gate's codes overlaps gate"),
    # 64 bf16 columns: codes of the same pointer, width and distance of rows
    (swiglu_forward, dict(dtype=2, cols=64, ldg=64, ldu=64, ldy=64, gate=P16 + 4096, up=S + 65536, **APART),
     "gate's codes overlaps gate"),
    (swiglu_backward, dict(dy=S, **APART), "dgate overlaps dup"),
    (swiglu_backward, dict(dg=P16 + 640, dy=P16 + 8, **APART), "dgate overlaps dy"),
    (swiglu_backward, dict(dg=P16 + 4096, dy=S + 65536, **APART), "dgate overlaps gate's codes"),
    (swiglu_backward, dict(dg=P16 + 65536, du=P16 + 4, **APART), "dup overlaps dy"),
    (swiglu_backward, dict(dg=P16 + 65536, lddu=48, **APART), "dup overlaps dy"),
]


@pytest.mark.parametrize("call,args,text", OVERLAPS, ids=[f"{c.__name__}-{i}" for i, (c, _, _) in enumerate(OVERLAPS)])
def test_overlap_refused(B, call, args, text):  # noqa: F811
    assert call(B.lib(), **args) == B.ERR_INVALID_ARG
    assert text in B.last_error()

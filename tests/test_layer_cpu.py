"""Dropout and the embedding on the host, without a GPU: the reference generator, and every refusal
of the C ABI and of the binding.  No call reaches a launch."""
import numpy as np
import pytest
import torch

import layer_reference as R


@pytest.fixture(scope="module")
def B():
    import os
    from bit_optimizers_block_amd import bitopt
    if not os.path.exists(bitopt.LIB_PATH):
        from bit_optimizers_block_amd import build
        build.build()
    bitopt.lib()
    return bitopt


def test_reference_bits():
    # the published answers for a counter and a key of zeros, and of ones
    assert R.philox([0] * 4, [0] * 2) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]
    assert R.philox([2**32 - 1] * 4, [2**32 - 1] * 2) == [0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd]
    seed, call = 0x0123456789abcdef, 0xfedcba9876543210
    got = R.bits(5, 21, seed, call)
    for r in range(5):
        for c in range(21):
            w = R.philox([c // 8, r, call % 2**32, call >> 32], [seed % 2**32, seed >> 32])
            assert got[r, c] == (w[c % 8 // 2] >> 16 * (c % 2)) % 2**16


def test_reference_bits_are_even():
    """Each bit is set in half of 2^20 draws: within 5 standard deviations of 2^9."""
    b = R.bits(512, 2048, 3, 5)
    for i in range(16):
        assert abs(int((b >> i & 1).sum()) - 2**19) < 5 * 2**9


# ------------------------------------------------------------------------- refusals

P = [(1 << 20) + (i << 16) for i in range(8)]


def dropout_forward(L, x=P[0], dtype=0, rows=4, cols=40, ldx=40, residual=P[1], ldr=40, p=0.5, seed=1, call=2, counter=P[2],
                    y=P[3], ldy=40):
    return L.bitopt_dropout_forward(x, dtype, rows, cols, ldx, residual, ldr, p, seed, call, counter, y, ldy, None)


def dropout_backward(L, dy=P[0], dtype=0, rows=4, cols=40, lddy=40, p=0.5, seed=1, call=2, counter=None, dx=P[3], lddx=40):
    return L.bitopt_dropout_backward(dy, dtype, rows, cols, lddy, p, seed, call, counter, dx, lddx, None)


def embedding_forward(L, tokens=P[0], kind=0, count=4, table=P[1], dtype=0, vocab=9, width=40, ldt=40, scale=1.0, out=P[2],
                      od=0, ldo=40):
    return L.bitopt_embedding_forward(tokens, kind, count, table, dtype, vocab, width, ldt, scale, out, od, ldo, None)


def mx_embedding_forward(L, tokens=P[0], kind=0, count=4, codes=P[1], scales=P[3], fmt=0, vocab=9, width=40, scale=1.0,
                         out=P[2], od=0, ldo=40):
    return L.bitopt_mx_embedding_forward(tokens, kind, count, codes, scales, fmt, vocab, width, scale, out, od, ldo, None)


def embedding_backward(L, dy=P[0], dtype=0, count=4, width=40, lddy=40, tokens=P[1], kind=1, vocab=9, scale=1.0, out=P[2],
                       od=0, ldd=40, acc=0, work=P[3], space=1 << 12):
    return L.bitopt_embedding_backward(dy, dtype, count, width, lddy, tokens, kind, vocab, scale, out, od, ldd, acc, work,
                                       space, None)


NAN = float("nan")
REFUSED = [
    (dropout_forward, dict(x=None), "x is NULL"), (dropout_forward, dict(y=None), "y is NULL"),
    (dropout_forward, dict(dtype=3), "dtype"), (dropout_forward, dict(rows=-1), "rows"), (dropout_forward, dict(ldx=39), "apart"),
    (dropout_forward, dict(ldr=39), "apart"), (dropout_forward, dict(residual=P[1] + 2), "aligned"),
    (dropout_forward, dict(p=-0.01), "p must"), (dropout_forward, dict(p=1.01), "p must"), (dropout_forward, dict(p=NAN), "p must"),
    (dropout_forward, dict(counter=P[2] + 4), "counter"), (dropout_forward, dict(y=P[0] + 4), "overlaps x"),
    (dropout_forward, dict(y=P[1], ldy=80), "overlaps residual"), (dropout_forward, dict(y=P[2] - 8), "overlaps counter"),
    (dropout_backward, dict(dy=None), "dy is NULL"), (dropout_backward, dict(dx=None), "dx is NULL"),
    (dropout_backward, dict(p=2.0), "p must"), (dropout_backward, dict(lddx=1), "apart"),
    (dropout_backward, dict(dx=P[0] + 160), "overlaps dy"),
    (embedding_forward, dict(tokens=None), "tokens is NULL"), (embedding_forward, dict(kind=2), "token type"),
    (embedding_forward, dict(tokens=P[0] + 2), "aligned"), (embedding_forward, dict(kind=1, tokens=P[0] + 4), "aligned"),
    (embedding_forward, dict(table=None), "NULL"), (embedding_forward, dict(out=None), "NULL"),
    (embedding_forward, dict(dtype=5), "dtype"), (embedding_forward, dict(od=5), "dtype"),
    (embedding_forward, dict(vocab=-1), "vocab"), (embedding_forward, dict(count=-1), "count"),
    (embedding_forward, dict(width=-1), "width"), (embedding_forward, dict(ldt=39), "apart"),
    (embedding_forward, dict(scale=NAN), "scale"), (embedding_forward, dict(scale=float("inf")), "scale"),
    (embedding_forward, dict(out=P[1] + 320), "overlaps table"),
    (embedding_forward, dict(out=P[0] + 8), "overlaps tokens"),
    (mx_embedding_forward, dict(codes=None), "NULL"), (mx_embedding_forward, dict(scales=P[3] + 4), "aligned"),
    (mx_embedding_forward, dict(fmt=2), "format"), (mx_embedding_forward, dict(out=P[1] + 64), "overlaps the table"),
    (mx_embedding_forward, dict(out=P[3]), "overlaps the table's scales"), (mx_embedding_forward, dict(scale=-NAN), "scale"),
    (embedding_backward, dict(dy=None), "NULL"), (embedding_backward, dict(tokens=None), "NULL"),
    (embedding_backward, dict(out=None), "NULL"), (embedding_backward, dict(work=None), "workspace"),
    (embedding_backward, dict(work=P[3] + 8), "workspace"), (embedding_backward, dict(space=31), "workspace"),
    (embedding_backward, dict(kind=-1), "token type"), (embedding_backward, dict(lddy=39), "apart"),
    (embedding_backward, dict(ldd=39), "apart"), (embedding_backward, dict(scale=NAN), "scale"),
    (embedding_backward, dict(out=P[0]), "overlaps dy"), (embedding_backward, dict(out=P[1]), "overlaps tokens"),
    (embedding_backward, dict(out=P[3] + 16), "overlaps the workspace"), (embedding_backward, dict(work=P[0] + 32), "overlaps dy"),
    (embedding_backward, dict(work=P[1] + 16), "overlaps tokens"), (embedding_backward, dict(vocab=-2), "vocab"),
]


@pytest.mark.parametrize("call,args,text", REFUSED, ids=[f"{c.__name__}-{i}" for i, (c, _, _) in enumerate(REFUSED)])
def test_refused(B, call, args, text):
    assert call(B.lib(), **args) == B.ERR_INVALID_ARG
    assert text in B.last_error() and call.__name__ in B.last_error()


@pytest.mark.parametrize("call,args", [
    (dropout_forward, dict(rows=2**30 + 1)), (dropout_backward, dict(cols=2**31)), (embedding_forward, dict(count=2**30 + 1)),
    (embedding_forward, dict(vocab=2**31)), (mx_embedding_forward, dict(width=2**40)), (embedding_backward, dict(count=2**33)),
    (embedding_backward, dict(vocab=2**30 + 1)),
])
def test_unsupported(B, call, args):
    assert call(B.lib(), **args) == B.ERR_UNSUPPORTED and B.last_error()


@pytest.mark.parametrize("call,args", [
    (dropout_forward, dict(rows=0, x=None)), (dropout_backward, dict(cols=0, dy=None)), (embedding_forward, dict(count=0, tokens=None)),
    (embedding_forward, dict(width=0, table=None)), (mx_embedding_forward, dict(count=0, codes=None)),
    (embedding_backward, dict(vocab=0, out=None)), (embedding_backward, dict(width=0)),
    (embedding_backward, dict(count=0, acc=1, dy=None, work=None)),
])
def test_nothing_to_do(B, call, args):
    assert call(B.lib(), **args) == B.OK and B.last_error() == ""


def test_workspace_bytes(B):
    L = B.lib().bitopt_embedding_workspace_bytes
    assert L(-1, 1, 1) == L(1, -1, 1) == L(1, 1, -1) == L(2**30 + 1, 1, 1) == -1
    assert L(0, 50257, 2048) == 0
    # a workspace for a count serves all smaller ones: also where parts get longer
    for vocab, width in ((50257, 2048), (2**25, 1), (3, 33)):
        last = 0
        for count in sorted(c + d for c in [2**i for i in range(1, 30)] for d in (-1, 0, 1)):
            n = L(count, vocab, width)
            assert n >= 8 * count and n >= last and n % 16 == 0
            last = n


def test_binding_refuses(B):
    x, t, w = torch.zeros(4, 40), torch.zeros(4, dtype=torch.int64), torch.zeros(9, 40)
    c, s = torch.zeros(9, 64, dtype=torch.uint8), torch.zeros(9, 4, dtype=torch.uint8)
    for call in (lambda: B.dropout(x, 0.5, 1), lambda: B.dropout_backward(x, 0.5, 1), lambda: B.embedding(t, w),
                 lambda: B.mx_embedding(t, c, s, 40), lambda: B.embedding_backward(x, t, 9)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(ValueError, match="two dimensions"):
        B.dropout(torch.zeros(40), 0.5, 1)
    with pytest.raises(ValueError, match="bytes a row"):
        B.mx_embedding(t, c, s, 140)


def test_calls_are_declared(B):
    """Every argument list of the binding has the length of the header's declaration."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "bitopt.h")).read(), flags=re.S)
    names = re.findall(r"\b(bitopt_(?:mx_)?(?:dropout|embedding)_\w+)\s*\(", src)
    assert len(names) == 6
    for name in names:
        decl = re.search(name + r"\s*\(([^)]*)\)", src).group(1)
        assert len(getattr(B.lib(), name).argtypes) == len(decl.split(",")), name

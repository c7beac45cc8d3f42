"""GPU: dropout bit for bit and the embedding with its gradient against the plain forms of
layer_reference -- ragged sizes, strided and unaligned rows, every type, tokens of every
distribution and outside the table -- and on other streams, captured, in place, and together as one
training step with the F8 products and the 8-bit optimizer."""
import numpy as np
import pytest
import torch

import f8_reference as F
import layer_reference as R
import mx_reference as M
from bit_optimizers_block_amd import bitopt
from test_gpu_f8 import decoded
from test_gpu_mx import DT, host, padded_rows, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    bitopt.lib()


def f32(t):
    return t.float().cpu().numpy()


def rounded(v, dtype):
    return torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(DT[dtype])


# ------------------------------------------------------------------------- dropout

SHAPES = [(1, 1), (1, 7), (3, 8), (5, 9), (33, 130), (2, 4099), (600, 1), (1200, 2100)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_dropout(rows, cols, dtype, residual):
    x, r = values(rows, rows, cols, dtype), values(cols, rows, cols, dtype, 2.0) if residual else None
    for p, seed, call in ((0.1, 7, 0), (0.5, 2**64 - 1, 2**64 - 2), (0.97, 2**40 + 3, 5 * 2**33)):
        want = rounded(R.dropout(f32(x), p, seed, call, f32(r) if residual else None), dtype)
        assert torch.equal(bitopt.dropout(x, p, seed, call, r).cpu(), want)
        if not residual:
            assert torch.equal(bitopt.dropout_backward(x, p, seed, call).cpu(), want)


@pytest.mark.parametrize("dtype", list(DT))
def test_dropout_probabilities(dtype):
    """Borders of what 16 bits can tell apart; none and all dropped; and the share that is kept."""
    x = values(1, 700, 1501, dtype)
    for p in (0.0, 2.0**-18, 2.0**-17, 1.5 * 2.0**-17, 2.0**-16, 1 / 3, 1 - 2.0**-16, 1 - 2.0**-17, 1.0):
        y = bitopt.dropout(x, p, 3)
        assert torch.equal(y.cpu(), rounded(R.dropout(f32(x), p, 3, 0), dtype)), p
        if p == 0.0:
            assert torch.equal(y, x)
        if p == 1.0:
            assert not y.any()
    ones = torch.ones(700, 1501, dtype=DT[dtype], device="cuda")
    for p in (0.1, 0.5, 0.9):
        n = ones.numel()
        kept = int((bitopt.dropout(ones, p, 11, 4) != 0).sum())
        assert abs(kept - n * (1 - p)) < 5 * (n * p * (1 - p)) ** 0.5 + n * 2.0**-17
    # other seeds, calls and rows draw other bits; the same ones the same
    a = bitopt.dropout(ones, 0.5, 1, 1)
    assert torch.equal(a, bitopt.dropout(ones, 0.5, 1, 1))
    for b in (bitopt.dropout(ones, 0.5, 2, 1), bitopt.dropout(ones, 0.5, 1, 2), bitopt.dropout(ones, 0.5, 1 + 2**32, 1),
              bitopt.dropout(ones, 0.5, 1, 1 + 2**32), a.roll(1, 0), a.roll(1, 1), a.roll(8, 1)):
        assert abs(float((a == b).float().mean()) - 0.5) < 0.01


@pytest.mark.parametrize("dtype", list(DT))
def test_dropout_of_non_finite_values(dtype):
    """What is dropped is zero, or the residual's value, whatever it held."""
    x = torch.full((40, 77), float("nan"), dtype=DT[dtype], device="cuda")
    x[1], x[2] = float("inf"), float("-inf")
    r = values(2, 40, 77, dtype)
    kept = torch.from_numpy(R.bits(40, 77, 9, 1) >= 2**15).cuda()
    y, z = bitopt.dropout(x, 0.5, 9, 1), bitopt.dropout(x, 0.5, 9, 1, residual=r)
    assert (y[~kept] == 0).all() and torch.equal(z[~kept], r[~kept])
    assert y[0][kept[0]].isnan().all() and (y[1][kept[1]] == float("inf")).all() and (z[2][kept[2]] == float("-inf")).all()


@pytest.mark.parametrize("dtype", list(DT))
def test_dropout_strided_and_in_place(dtype):
    rows, cols = 37, 213
    x, r = values(1, rows, cols, dtype), values(2, rows, cols, dtype)
    want, plain = bitopt.dropout(x, 0.3, 5, 6, r), bitopt.dropout(x, 0.3, 5, 6)
    a, b = padded_rows(x, 3, 1), padded_rows(r, 5, 3)
    y = padded_rows(torch.zeros_like(x), 7, 5, fill=99.0)
    bitopt.dropout(a, 0.3, 5, 6, b, out=y)
    assert torch.equal(y, want)
    assert (y._base[:5] == 99).all() and (y._base[5 + rows * (cols + 7):] == 99).all()
    assert (y._base[5:5 + rows * (cols + 7)].view(rows, -1)[:, cols:] == 99).all()
    bitopt.dropout(a, 0.3, 5, 6, b, out=b)
    assert torch.equal(b, want)
    bitopt.dropout(a, 0.3, 5, 6, r, out=a)
    assert torch.equal(a, want)
    d = padded_rows(x, 3, 1)
    bitopt.dropout_backward(d, 0.3, 5, 6, out=d)
    assert torch.equal(d, plain)
    same = x.clone()
    assert torch.equal(bitopt.dropout(same, 0.0, 1, residual=same, out=same), (2 * x.float()).to(DT[dtype]))
    with pytest.raises(bitopt.BitoptError, match="overlaps"):
        bitopt.dropout(x[:-1], 0.3, 5, 6, out=x[1:])


def test_dropout_counter_in_graphs():
    """Two captured graphs that share a counter: each replay draws what an eager call with the
    counter's value added to `call` draws."""
    x, r = values(1, 300, 515, "bf16"), values(2, 300, 515, "bf16")
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")
    bitopt.dropout(x, 0.2, 8, 3, r, counter=counter)
    torch.cuda.synchronize()
    graphs, out = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            y = bitopt.dropout(x, 0.2, 8, 3, r, counter=counter)
            out.append((y, bitopt.dropout_backward(y, 0.2, 8, 3, counter=counter)))
    for value in (0, 1, 2**32 - 1, 2**32, -3):          # -3: added modulo 2^64
        counter.fill_(value)
        x.copy_(values(value % 97, 300, 515, "bf16"))
        for g in graphs:
            g.replay()
        call = (3 + value) % 2**64
        y = bitopt.dropout(x, 0.2, 8, call, r)
        d = bitopt.dropout_backward(y, 0.2, 8, call)
        torch.cuda.synchronize()
        for a, b in out:
            assert torch.equal(a, y) and torch.equal(b, d)


def test_dropout_gradient_by_differences():
    """The sum of c * dropout(x) + c * residual is linear in x: its difference along a direction is
    the gradient's product with it.  In fp32, values of 12 bits: every product is exact but for the
    factor's rounding."""
    rng = np.random.default_rng(4)
    x, v, c = (torch.from_numpy(rng.integers(-2**11, 2**11, (65, 131)).astype(np.float32)).cuda() for _ in range(3))
    loss = lambda t: (bitopt.dropout(t, 0.5, 6, 7).double() * c.double()).sum()
    assert float(loss(x + v) - loss(x)) == float((bitopt.dropout_backward(c, 0.5, 6, 7).double() * v.double()).sum())


# ----------------------------------------------------------------------- embedding

def tokens_of(kind, count, vocab, seed=0):
    rng = np.random.default_rng(seed)
    t = {"any": lambda: rng.integers(0, vocab, count), "one": lambda: np.full(count, vocab - 1),
         "few": lambda: rng.integers(0, min(3, vocab), count),
         "often": lambda: np.minimum((vocab ** rng.uniform(size=count)).astype(np.int64), vocab) - 1,
         "outside": lambda: np.where(np.arange(count) % 2, -1, vocab + np.arange(count)),
         "padded": lambda: np.where(rng.uniform(size=count) < 0.3, rng.choice([-1, vocab, -2**31, 2**31 - 1], count),
                                    rng.integers(0, vocab, count))}[kind]()
    return t.astype(np.int64)


LOOKUPS = [(1, 1, 1), (1, 50, 9), (5, 7, 8), (130, 40, 77), (1000, 300, 1030), (3, 5000, 4100)]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dtype,out", [("f32", "bf16"), ("f32", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f16"),
                                       ("f32", "f16"), ("f16", "f16"), ("f16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("count,vocab,width", LOOKUPS)
def test_embedding(count, vocab, width, dtype, out, wide):
    table, t = values(1, vocab, width, dtype), tokens_of("padded", count, vocab)
    tokens = torch.from_numpy(t).to(torch.int64 if wide else torch.int32).cuda()
    inside = ((t >= 0) & (t < vocab))[:, None]
    for scale in (1.0, -3.7):
        want = np.where(inside, f32(table)[np.where(inside[:, 0], t, 0)] * np.float32(scale), np.float32(0))
        assert torch.equal(bitopt.embedding(tokens, table, scale, dtype=DT[out]).cpu(), rounded(want, out))
    a = padded_rows(table, 3, 1)
    y = padded_rows(torch.zeros(count, width, dtype=DT[out], device="cuda"), 5, 1, fill=99.0)
    bitopt.embedding(tokens, a, scale, out=y)
    assert torch.equal(y.cpu(), rounded(want, out))
    assert (y._base[:1] == 99).all() and (y._base[1 + count * (width + 5):] == 99).all()
    assert (y._base[1:1 + count * (width + 5)].view(count, -1)[:, width:] == 99).all()


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("count,vocab,width", LOOKUPS)
def test_mx_embedding(count, vocab, width, fmt, out):
    x = np.random.default_rng(3).standard_normal((vocab, width)) * 0.05
    codes, scales = (torch.from_numpy(v).cuda() for v in M.quantize(x, fmt))
    t = tokens_of("padded", count, vocab)
    inside = ((t >= 0) & (t < vocab))[:, None]
    table = M.dequantize(codes.cpu().numpy(), scales.cpu().numpy(), width, fmt).astype(np.float32)
    want = np.where(inside, table[np.where(inside[:, 0], t, 0)] * np.float32(11.3), np.float32(0))
    got = bitopt.mx_embedding(torch.from_numpy(t).cuda(), codes, scales, width, fmt, 11.3, dtype=DT[out])
    assert torch.equal(got.cpu(), rounded(want, out))


def test_embedding_shapes_of_tokens():
    table = values(1, 30, 40, "f32")
    tokens = torch.arange(24, dtype=torch.int32, device="cuda").view(2, 3, 4)
    assert torch.equal(bitopt.embedding(tokens, table), table[:24])
    assert bitopt.embedding(tokens[:0], table).shape == (0, 40)
    with pytest.raises(ValueError, match="contiguous"):
        bitopt.embedding(tokens.transpose(0, 1), table)
    with pytest.raises(TypeError, match="int32 or torch.int64"):
        bitopt.embedding(tokens.float(), table)
    empty = torch.empty(0, 40, device="cuda")
    assert not bitopt.embedding(tokens, empty).any()


def test_embedding_large_offsets():
    """A table and its gradient beyond 2^31 elements."""
    vocab, width = 70000, 32768
    table = torch.empty(vocab, width, dtype=torch.bfloat16, device="cuda")
    t = torch.tensor([69999, 3, 65536, 69999, 131072, 65535], device="cuda")
    for i in (3, 65535, 65536, 69999):
        table[i] = values(i, 1, width, "bf16")[0]
    y = bitopt.embedding(t, table)
    assert torch.equal(y[[0, 1, 2, 3, 5]], table[t[[0, 1, 2, 3, 5]]]) and not y[4].any()
    table.fill_(7.0)
    dy = values(5, 6, width, "bf16")
    bitopt.embedding_backward(dy, t, vocab, out=table)
    assert torch.equal(table[69999], (dy[0].float() + dy[3].float()).bfloat16()) and torch.equal(table[65536], dy[2])
    assert torch.equal(table[3], dy[1]) and torch.equal(table[65535], dy[5])
    assert int((table != 0).any(1).sum()) == 3         # dy's row 1, the only one of token 3, is all zero


# counts on both sides of one workgroup's sort at each of its sizes, and of a part's length
GRADS = [(1, 1, 1), (1, 50257, 9), (33, 7, 8), (700, 300, 130), (1024, 2**18, 33), (1025, 5000, 77), (4096, 4096, 40),
         (4097, 255, 256), (8193, 256, 16), (16384, 65535, 24), (16385, 65536, 24), (20000, 3, 513), (70000, 2**20, 5),
         (40, 2**27, 1)]


@pytest.mark.parametrize("kind", ["any", "one", "often", "padded", "outside", "few"])
@pytest.mark.parametrize("count,vocab,width", GRADS)
def test_embedding_backward(count, vocab, width, kind):
    t = tokens_of(kind, count, vocab, count)
    tokens = torch.from_numpy(t).cuda()
    # whole numbers whose sums are exact: the very result, in any order
    d = np.random.default_rng(1).integers(-100, 101, (count, width))
    dy = torch.from_numpy(d.astype(np.float32)).cuda()
    got = bitopt.embedding_backward(dy, tokens, vocab)
    want = torch.zeros(vocab, width, dtype=torch.float64, device="cuda")
    inside = (tokens >= 0) & (tokens < vocab)
    want.index_add_(0, tokens[inside], dy[inside].double())
    assert torch.equal(got.double(), want)
    # added to what is there, rows without a token untouched
    out = torch.full((vocab, width), 0.5, device="cuda")
    assert bitopt.embedding_backward(dy, tokens, vocab, 2.0, out=out, accumulate=True) is out
    assert torch.equal(out.double(), 2 * want + 0.5)


def test_embedding_backward_of_many_tokens():
    """More than a million, in one run that lies in every window and spread over a table."""
    count, vocab, width = 1100000, 70000, 9
    dy = torch.randint(-8, 9, (count, width), device="cuda").float()
    got = bitopt.embedding_backward(dy, torch.full((count,), 5, dtype=torch.int32, device="cuda"), 7)
    assert torch.equal(got[5].double(), dy.double().sum(0)) and not got[:5].any() and not got[6].any()
    tokens = torch.arange(count, device="cuda") * 7919 % vocab          # each in turn, as 7919 is prime
    got = bitopt.embedding_backward(dy, tokens, vocab)
    order = torch.argsort(tokens, stable=True)
    total = torch.cat((torch.zeros(1, width, dtype=torch.float64, device="cuda"), dy.double()[order].cumsum(0)))
    end = torch.bincount(tokens, minlength=vocab).cumsum(0)
    assert torch.equal(got.double(), total[end] - total[torch.cat((end.new_zeros(1), end[:-1]))])


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("count,vocab,width", [(5, 9, 7), (900, 40, 130), (5000, 1000, 64), (18000, 500, 40)])
def test_embedding_backward_bounds(count, vocab, width, dtype, out):
    t, scale = tokens_of("often", count, vocab, 3), 1.7
    tokens = torch.from_numpy(t).to(torch.int32).cuda()
    dy = values(4, count, width, dtype, 0.1, spread=1)
    scale = float(np.float32(scale))
    exact, acc = R.embedding_grad(host(dy), t, vocab, scale)

    def check(got, exact, acc):
        off = np.abs(host(got) - exact)
        bound = acc + R.HALF_STEP[out] * (np.abs(exact) + acc) + R.TINY[out]
        assert (off <= bound).all(), (off - bound).max()
    plain = bitopt.embedding_backward(dy, tokens, vocab, scale, dtype=DT[out])
    check(plain, exact, acc)
    # strided and unaligned rows, stale memory in the result and the workspace
    a = padded_rows(dy, 3, 1)
    y = padded_rows(values(5, vocab, width, out), 5, 1, fill=99.0)
    old = y.clone()
    work = torch.full((bitopt.embedding_workspace_bytes(count, vocab, width),), 0xA5, dtype=torch.uint8, device="cuda")
    bitopt.embedding_backward(a, tokens, vocab, scale, out=y, workspace=work)
    assert torch.equal(y, plain)
    y.copy_(old)
    bitopt.embedding_backward(a, tokens, vocab, scale, out=y, accumulate=True, workspace=work)
    # one more fp32 rounding, of the sum with the old value
    check(y, exact + host(old), acc + 2.0**-24 * (np.abs(exact) + acc + np.abs(host(old))))
    untouched = np.setdiff1d(np.arange(vocab), t)
    assert torch.equal(y[untouched], old[untouched])
    assert (y._base[:1] == 99).all() and (y._base[1 + vocab * (width + 5):] == 99).all()
    assert (y._base[1:1 + vocab * (width + 5)].view(vocab, -1)[:, width:] == 99).all()


def test_embedding_backward_without_tokens():
    y = torch.ones(50, 33, device="cuda")
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    bitopt.embedding_backward(torch.empty(0, 33, device="cuda"), t, 50, out=y, accumulate=True)
    assert (y == 1).all()
    bitopt.embedding_backward(torch.empty(0, 33, device="cuda"), t, 50, out=y)
    assert (y == 0).all()
    with pytest.raises(bitopt.BitoptError, match="workspace"):
        bitopt.embedding_backward(torch.ones(4, 33, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda"), 50,
                                  workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("count", [600, 17000])
def test_embedding_backward_on_streams_and_in_graphs(count):
    """The same bits from run to run, on another stream, and from two captured graphs with a
    workspace each, replayed with other tokens."""
    vocab, width = 90, 200
    dy, tokens = values(1, count, width, "bf16"), torch.from_numpy(tokens_of("often", count, vocab)).cuda()
    table = values(2, vocab, width, "f32")
    want = bitopt.embedding_backward(dy, tokens, vocab)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [bitopt.embedding_backward(dy, tokens, vocab) for _ in range(3)]
    on = bitopt.embedding_backward(dy, tokens, vocab, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) for a in again + [on])
    graphs, results = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            results.append((bitopt.embedding(tokens, table, 3.0), bitopt.embedding_backward(dy, tokens, vocab)))
    for seed in (5, 6, 7):
        tokens.copy_(torch.from_numpy(tokens_of("padded" if seed == 6 else "often", count, vocab, seed)))
        dy.copy_(values(seed, count, width, "bf16"))
        for g in graphs:
            g.replay()
        want = bitopt.embedding(tokens, table, 3.0), bitopt.embedding_backward(dy, tokens, vocab)
        torch.cuda.synchronize()
        for r in results:
            assert torch.equal(r[0], want[0]) and torch.equal(r[1], want[1])


def test_embedding_gradient_by_differences():
    """The sum of c * embedding(table) is linear in the table; whole numbers make it exact."""
    rng = np.random.default_rng(4)
    table, v = (torch.from_numpy(rng.integers(-100, 100, (60, 131)).astype(np.float32)).cuda() for _ in range(2))
    tokens = torch.from_numpy(tokens_of("padded", 500, 60)).cuda()
    c = torch.from_numpy(rng.integers(-100, 100, (500, 131)).astype(np.float32)).cuda()
    loss = lambda w: (bitopt.embedding(tokens, w, 2.0).double() * c.double()).sum()
    assert float(loss(table + v) - loss(table)) == float((bitopt.embedding_backward(c, tokens, 60, 2.0).double() * v.double()).sum())


# ------------------------------------------------------------- together, as in a step

def test_training_step():
    """Three steps of embedding, dropout, an F8 layer onto a residual through dropout, and the tied
    head's gradient in the table's: every result against its own inputs, then the fused 8-bit step on
    both weights."""
    tokens_n, vocab, d = 300, 500, 256
    table, w = values(1, vocab, d, "f32", 0.05), values(2, d, d, "f32", 0.05)
    q1, q2 = bitopt.create_dynamic_map(True).cuda(), bitopt.create_dynamic_map(False).cuda()
    hp = dict(optimizer="adamw", lr=1e-2, weight_decay=0.01, blocksize=256)
    state = {}
    for name, p in (("table", table), ("w", w)):
        n = p.numel()
        state[name] = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2)] + \
                      [torch.zeros((n + 255) // 256, device="cuda") for _ in range(2)]
    for step in (1, 2, 3):
        t = tokens_of("padded", tokens_n, vocab, step)
        tokens = torch.from_numpy(t).cuda()
        x = bitopt.embedding(tokens, table, 16.0, dtype=torch.bfloat16)
        h = bitopt.dropout(x, 0.1, 42, 2 * step)
        hq = bitopt.f8_quantize(h, give="both")
        wq = bitopt.f8_quantize(w, blocks="tiles", give="both")
        z = bitopt.f8_matmul(*hq[:2], *wq[:2], d, b_blocks="tiles")
        y = bitopt.dropout(z, 0.1, 42, 2 * step + 1, residual=h)
        dy = values(10 + step, tokens_n, d, "bf16", 0.01)
        dz = bitopt.dropout_backward(dy, 0.1, 42, 2 * step + 1)
        dq = bitopt.f8_quantize(dz, "e5m2", give="both")
        dw = bitopt.f8_matmul(*dq[2:], *hq[2:], tokens_n, "e5m2", dtype=torch.float32)
        dh = bitopt.f8_matmul(*dq[:2], *wq[2:], d, "e5m2", b_blocks="tiles", out=dy.clone(), accumulate=True)
        dx = bitopt.dropout_backward(dh, 0.1, 42, 2 * step)
        head = values(20 + step, vocab, d, "f32", 0.01)
        dtable = bitopt.embedding_backward(dx, tokens, vocab, 16.0, out=head.clone(), accumulate=True)

        inside = ((t >= 0) & (t < vocab))[:, None]
        assert torch.equal(x.cpu(), rounded(np.where(inside, f32(table)[np.where(inside[:, 0], t, 0)] * np.float32(16), 0), "bf16"))
        assert torch.equal(h.cpu(), rounded(R.dropout(f32(x), 0.1, 42, 2 * step), "bf16"))
        assert torch.equal(y.cpu(), rounded(R.dropout(f32(z), 0.1, 42, 2 * step + 1, f32(h)), "bf16"))
        assert torch.equal(dz.cpu(), rounded(R.dropout(f32(dy), 0.1, 42, 2 * step + 1), "bf16"))
        hv, wv = decoded(*hq[:2], d, "e4m3", "rows"), decoded(*wq[:2], d, "e4m3", "tiles")
        dv, dvt = decoded(*dq[:2], d, "e5m2", "rows"), decoded(*dq[2:], tokens_n, "e5m2", "rows")
        hvt, wvt = decoded(*hq[2:], tokens_n, "e4m3", "rows"), decoded(*wq[2:], d, "e4m3", "tiles")
        assert torch.equal(wvt, wv.t())
        for got, a, b, out, old in ((z, hv, wv, "bf16", None), (dw, dvt, hvt, "f32", None), (dh, dv, wvt, "bf16", dy.double())):
            exact = a @ b.t()
            bound = F.product_bound(a, b, exact, out, out != "f32")
            if old is not None:
                bound = bound + (2.0**-24 + F.HALF_STEP[out]) * (exact.abs() + old.abs() + bound)
                exact = exact + old
            assert ((got.double() - exact).abs() <= bound).all()
        exact, acc = R.embedding_grad(host(dx), t, vocab, 16.0)
        exact = exact + host(head)
        assert (np.abs(host(dtable) - exact) <= acc + 2.0**-23 * (np.abs(exact) + acc) + 2.0**-24 * np.abs(host(head))).all()

        for name, p, g in (("table", table, dtable), ("w", w, dw)):
            before = p.clone()
            s1, s2, a1, a2 = state[name]
            bitopt.step_8bit_blockwise_2state(hp, step, p.view(-1), g.contiguous().view(-1), s1, s2, a1, a2, q1, q2)
            moved = (p - before).abs().max()
            assert torch.isfinite(p).all() and 0 < float(moved) < 0.1


@pytest.mark.parametrize("given", ["own", "default"])
def test_streams_of_other_libraries(monkeypatch, given):
    """Any object with a stream's handle: the work of every call goes to that very stream."""
    x, table = values(1, 70, 130, "bf16"), values(2, 90, 130, "f32")
    tokens = torch.from_numpy(tokens_of("padded", 70, 90)).cuda()
    q = bitopt.f8_quantize(x, give="both")
    w, mx = bitopt.f8_quantize(table, blocks="tiles"), bitopt.mx_quantize(table)

    def calls(**stream):
        return [*bitopt.f8_quantize(x, give="both", **stream), bitopt.f8_dequantize(*q[:2], 130, **stream),
                bitopt.f8_matmul(*q[:2], *w, 130, b_blocks="tiles", **stream), bitopt.dropout(x, 0.3, 1, residual=x, **stream),
                bitopt.dropout_backward(x, 0.3, 1, **stream), bitopt.embedding(tokens, table, **stream),
                bitopt.mx_embedding(tokens, *mx, 130, **stream), bitopt.embedding_backward(x, tokens, 90, **stream)]
    want = calls()
    torch.cuda.synchronize()
    own = torch.cuda.Stream() if given == "own" else torch.cuda.default_stream()
    handle, seen, real = type("Handle", (), dict(cuda_stream=own.cuda_stream))(), [], bitopt.lib()

    class Library:
        def __getattr__(self, name):
            def call(*args):
                seen.append(args[-1])
                return getattr(real, name)(*args)
            return getattr(real, name) if name.endswith("bytes") or name == "bitopt_last_error" else call
    monkeypatch.setattr(bitopt, "lib", Library)
    with torch.cuda.stream(torch.cuda.Stream()):        # neither the given stream nor the default one
        got = calls(stream=handle)
    torch.cuda.synchronize()
    assert seen == [own.cuda_stream] * 8
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_results_have_no_history():
    """Arguments that require a gradient are taken, and their results require none; the gradient calls
    serve a torch.autograd.Function."""
    table = torch.nn.Parameter(values(1, 60, 40, "f32"))
    tokens = torch.from_numpy(tokens_of("padded", 100, 60)).cuda()

    class Embedding(torch.autograd.Function):
        @staticmethod
        def forward(ctx, table, call):
            ctx.call, ctx.vocab = call, table.shape[0]
            return bitopt.dropout(bitopt.embedding(tokens, table, 2.0), 0.25, 9, call)

        @staticmethod
        def backward(ctx, dy):
            return bitopt.embedding_backward(bitopt.dropout_backward(dy, 0.25, 9, ctx.call), tokens, ctx.vocab, 2.0), None
    y = bitopt.dropout(bitopt.embedding(tokens, table, 2.0), 0.25, 9, 3)
    assert not y.requires_grad and y.grad_fn is None
    got = Embedding.apply(table, 3)
    assert torch.equal(got, y)
    dy = values(2, 100, 40, "f32")
    got.backward(dy)
    assert torch.equal(table.grad, bitopt.embedding_backward(bitopt.dropout_backward(dy, 0.25, 9, 3), tokens, 60, 2.0))
    for t in bitopt.f8_quantize(table, give="both"):
        assert not t.requires_grad and t.grad_fn is None

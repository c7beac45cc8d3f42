"""GPU: how the MX operators are called -- results over and between other matrices, streams of any
kind -- through the binding."""
import pytest
import torch

from bit_optimizers_block_amd import bitopt
from test_gpu_mx import DT, padded_rows, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    bitopt.lib()


def raises(call, text):
    with pytest.raises(bitopt.BitoptError, match=text):
        call()


def test_results_over_other_matrices_are_refused():
    x = values(1, 70, 128, "bf16")
    q, q8 = bitopt.mx_quantize(x), bitopt.mx_quantize(x, "e4m3")
    w = bitopt.mx_quantize(values(2, 128, 128, "f32"))
    raises(lambda: bitopt.mx_linear(x, *w, out=x), "out overlaps x")
    raises(lambda: bitopt.mx_linear_grad_input(x, *w, 128, out=x), "dx overlaps dy")
    raises(lambda: bitopt.mx_linear_grad_input(x[:40], *w, 128, out=x[30:]), "dx overlaps dy")
    square = values(3, 128, 128, "bf16")
    raises(lambda: bitopt.mx_linear_grad_weight(square, *bitopt.mx_quantize(square, "e4m3"), 128, out=square),
           "dw overlaps dy")
    raises(lambda: bitopt.mx_quantize(x, "e4m3", codes=x.view(torch.uint8).view(-1)[:70 * 128].view(70, 128)), "overlaps x")
    raises(lambda: bitopt.mx_dequantize(q8[0][:16], q8[1][:16], 128, "e4m3",
                                        out=q8[0][:32].view(-1).view(torch.bfloat16).view(16, 128)), "out overlaps codes")
    raises(lambda: bitopt.mx_matmul(q[0][:1], q[1][:1], w[0][:8], w[1][:8], 128, out=w[0][:1, :16].view(torch.bfloat16)),
           "out overlaps b")
    y, saved = bitopt.swiglu_save8(x, x)
    raises(lambda: bitopt.swiglu_save8(x, x, saved=(saved[0], saved[1], saved[0], saved[3])), "overlaps up's codes")
    raises(lambda: bitopt.swiglu_save8(x[:-1], x[:-1], y=x[1:]), "y overlaps")
    g = torch.empty_like(x)
    raises(lambda: bitopt.swiglu_backward8(x, saved, dgate=g, dup=g), "dgate overlaps dup")
    raises(lambda: bitopt.swiglu_backward8(x, saved, dgate=x, dup=x), "dgate overlaps dup")
    assert torch.equal(y, bitopt.swiglu_save8(x, x)[0])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,cols", [(1, 7), (33, 205), (70, 512)])
def test_results_between_and_over_inputs(rows, cols, dtype):
    """Gate and up, and their gradients, as halves of one buffer; y over gate or up; dgate or dup
    over dy."""
    both = values(1, rows, 2 * cols, dtype)
    gate, up = both[:, :cols], both[:, cols:]
    dy = values(2, rows, cols, dtype)
    y, saved = bitopt.swiglu_save8(gate.contiguous(), up.contiguous())
    dgate, dup = bitopt.swiglu_backward8(dy, saved)
    grads = torch.empty_like(both)
    bitopt.swiglu_backward8(dy, saved, dgate=grads[:, :cols], dup=grads[:, cols:])
    assert torch.equal(grads, torch.cat((dgate, dup), 1))
    wide = torch.full((rows, 3 * cols), 9.0, dtype=DT[dtype], device="cuda")
    wide[:, :2 * cols] = both
    same = bitopt.swiglu_save8(wide[:, :cols], wide[:, cols:2 * cols], y=wide[:, 2 * cols:])
    assert torch.equal(same[0], y) and all(torch.equal(a, b) for a, b in zip(same[1], saved))
    for over in range(2):
        a, b = padded_rows(gate, 3, 1), padded_rows(up, 3, 1)
        same = bitopt.swiglu_save8(a, b, y=(a, b)[over])
        assert torch.equal(same[0], y) and all(torch.equal(u, v) for u, v in zip(same[1], saved))
        d, other = padded_rows(dy, 5, 1), torch.empty_like(dy)
        pair = (d, other) if over == 0 else (other, d)
        bitopt.swiglu_backward8(d, saved, dgate=pair[0], dup=pair[1])
        assert torch.equal(pair[0], dgate) and torch.equal(pair[1], dup)


class Handle:
    """A stream of another library: what the step and codec calls take too."""

    def __init__(self, stream):
        self.cuda_stream = stream.cuda_stream


@pytest.mark.parametrize("given", ["own", "default"])
def test_streams_of_other_libraries(monkeypatch, given):
    """Any object with a stream's handle: the work goes to that very stream."""
    x, gate = values(1, 70, 130, "bf16"), values(2, 70, 90, "bf16")
    w = bitopt.mx_quantize(values(3, 90, 130, "f32"))
    q = bitopt.mx_quantize(x, "e4m3")
    want = [bitopt.mx_linear(x, *w), bitopt.mx_linear_grad_input(gate, *w, 130), bitopt.mx_linear_grad_weight(gate, *q, 130),
            bitopt.mx_matmul(*q, *w, 130, "e4m3"), bitopt.mx_dequantize(*q, 130, "e4m3"), bitopt.swiglu_save8(gate, gate)[0]]
    torch.cuda.synchronize()
    own = torch.cuda.Stream() if given == "own" else torch.cuda.default_stream()
    handle, seen, real = Handle(own), [], bitopt.lib()

    class Library:
        def __getattr__(self, name):
            def call(*args):
                seen.append(args[-1])
                return getattr(real, name)(*args)
            return call if name.startswith(("bitopt_mx", "bitopt_swiglu")) else getattr(real, name)
    monkeypatch.setattr(bitopt, "lib", Library)
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):                      # neither the current stream nor the default one
        got = [bitopt.mx_linear(x, *w, stream=handle), bitopt.mx_linear_grad_input(gate, *w, 130, stream=handle),
               bitopt.mx_linear_grad_weight(gate, *q, 130, stream=handle),
               bitopt.mx_matmul(*q, *w, 130, "e4m3", stream=handle), bitopt.mx_dequantize(*q, 130, "e4m3", stream=handle),
               bitopt.swiglu_save8(gate, gate, stream=handle)[0]]
        codes = bitopt.mx_quantize(x, "e4m3", stream=handle)
        assert torch.cuda.current_stream() == other
    torch.cuda.synchronize()
    assert seen == [own.cuda_stream] * 7
    for a, b in zip(got + list(codes), want + list(q)):
        assert torch.equal(a, b)
    # the calls beside them take the same object
    monkeypatch.undo()
    flat, qmap = x.view(-1), bitopt.create_dynamic_map(True).cuda()
    want = bitopt.quantize_blockwise(flat, qmap)
    codes, absmax = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    torch.cuda.synchronize()
    bitopt.quantize_blockwise(flat, qmap, codes=codes, absmax=absmax, stream=handle)
    torch.cuda.synchronize()
    assert torch.equal(codes, want[0]) and torch.equal(absmax, want[1])


def test_results_have_no_history():
    """Arguments that require a gradient are taken, and their results require none."""
    master = torch.nn.Parameter(values(1, 90, 130, "f32"))
    x, dy = values(2, 5, 130, "bf16").requires_grad_(), values(3, 5, 90, "bf16")
    w, q = bitopt.mx_quantize(master), bitopt.mx_quantize(x, "e4m3")
    y = bitopt.mx_linear(x, *w)
    s, saved = bitopt.swiglu_save8(x, x)
    for t in (y, s, bitopt.mx_linear_grad_input(dy, *w, 130), bitopt.mx_linear_grad_weight(dy, *q, 130),
              *bitopt.swiglu_backward8(s, saved), bitopt.mx_dequantize(*w, 130)):
        assert not t.requires_grad and t.grad_fn is None

    class Linear(torch.autograd.Function):
        """The layer for automatic differentiation, made of the calls."""

        @staticmethod
        def forward(ctx, x, weight):
            ctx.w, ctx.x, ctx.k = bitopt.mx_quantize(weight), bitopt.mx_quantize(x, "e4m3"), x.shape[1]
            return bitopt.mx_linear(x, *ctx.w)

        @staticmethod
        def backward(ctx, dy):
            return (bitopt.mx_linear_grad_input(dy, *ctx.w, ctx.k), bitopt.mx_linear_grad_weight(dy, *ctx.x, ctx.k))

    got = Linear.apply(x, master)
    got.backward(dy)
    assert torch.equal(got, y) and torch.equal(x.grad, bitopt.mx_linear_grad_input(dy, *w, 130))
    assert torch.equal(master.grad, bitopt.mx_linear_grad_weight(dy, *q, 130))


@pytest.mark.parametrize("dtype", list(DT))
def test_gates_far_below_zero(dtype):
    """A sigmoid below 2^-126 counts as zero; down to there it is as exact as elsewhere."""
    big = 2.0**14 if dtype == "f16" else 2.0**100
    gate = torch.tensor([[-80.0, -86.0, -87.0, -87.5, -88.5, -95.0, -104.0, -1000.0]], device="cuda").to(DT[dtype])
    up = torch.full_like(gate, big)
    y, saved = bitopt.swiglu_save8(gate, up)
    exact = (gate.double() * torch.sigmoid(gate.double()) * big)[0]
    half = torch.finfo(DT[dtype]).eps / 2
    # the exponential's argument is off by |g| 2^-24, then a few roundings: (|g| + 8) 2^-23; and
    # half of fp16's smallest step
    limit = exact.abs() * ((gate.double()[0].abs() + 8) * 2.0**-23 + half) + (2.0**-25 if dtype == "f16" else 0)
    assert ((y[0].double() - exact).abs()[:3] <= limit[:3]).all()
    assert (y[0, 3:] == 0).all()
    dgate, dup = bitopt.swiglu_backward8(torch.ones_like(up), saved)    # dy up has to be finite
    codes = bitopt.mx_dequantize(saved[0], saved[1], 8, "e4m3")[0]
    assert (dgate[0, codes < -87.34] == 0).all() and (dup[0, codes < -87.34] == 0).all()

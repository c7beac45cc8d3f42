"""GPU: the embedding's gradient in wide tables whose tokens fill many windows: several columns of workgroups, joins by
groups of 256 lanes, and joins that go over the columns more than once.  Whole numbers, so every sum is exact in
any order, and rounded once into the result's type."""
import pytest
import torch

from bit_optimizers_block_amd import bitopt
from test_gpu_layer import tokens_of
from test_gpu_mx import DT

pytestmark = pytest.mark.gpu

# width 1025 and on: 256 lanes; above 2048: several workgroups of columns, the join's columns in turns
WIDE = [(9000, 300, 1024), (9000, 300, 1025), (9000, 300, 2048), (9000, 300, 2049), (3000, 5, 4099), (20000, 3, 4096),
        (17000, 70000, 1500)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    bitopt.lib()


@pytest.mark.parametrize("out", list(DT))
@pytest.mark.parametrize("kind", ["one", "often", "padded", "few"])
@pytest.mark.parametrize("count,vocab,width", WIDE)
def test_embedding_backward(count, vocab, width, kind, out):
    t = tokens_of(kind, count, vocab, count)
    tokens = torch.from_numpy(t).cuda()
    g = torch.Generator(device="cuda")
    g.manual_seed(width)
    # sums to 20000 * 50 < 2^24: exact in fp32; in fp16 below 65504
    dy = torch.randint(-50 if out != "f16" else -3, 51 if out != "f16" else 4, (count, width), device="cuda", generator=g)
    dy = dy.to(torch.bfloat16 if kind == "often" else torch.float32)
    want = torch.zeros(vocab, width, dtype=torch.float64, device="cuda")
    inside = (tokens >= 0) & (tokens < vocab)
    want.index_add_(0, tokens[inside], dy[inside].double())
    got = bitopt.embedding_backward(dy, tokens, vocab, dtype=DT[out])
    assert torch.equal(got, want.to(DT[out]))
    old = torch.full((vocab, width), 0.5, dtype=DT[out], device="cuda")
    bitopt.embedding_backward(dy, tokens, vocab, 2.0, out=old, accumulate=True)
    assert torch.equal(old, (2 * want + 0.5).to(DT[out]))


def test_columns_of_a_wide_table():
    """The window's length follows from count and width: slices of the columns give the same exact sums."""
    count, vocab, width = 8192, 50, 513
    tokens = torch.from_numpy(tokens_of("often", count, vocab)).cuda()
    dy = torch.randint(-50, 51, (count, width), device="cuda").float()
    whole = bitopt.embedding_backward(dy, tokens, vocab)
    assert torch.equal(whole[:, :512], bitopt.embedding_backward(dy[:, :512], tokens, vocab))
    assert torch.equal(whole[:, 512:], bitopt.embedding_backward(dy[:, 512:], tokens, vocab))

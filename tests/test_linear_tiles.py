"""gdn_linear where a CTA, or a pair of CTAs, takes several tiles one after the other: both
accumulators, their phases, and stages that go round from tile to tile."""
import pytest
import torch

from tests import layer_testlib as tl
from tests.test_linear import check

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops():
    from gated_deltanet_linear_02_gb300 import build, ops
    build.build()
    return ops


# Pairs of CTAs, 256 x 256 tiles: at least seven a pair; at least two, with an odd number of slices of K and
# ragged edges. Lone CTAs, 128 x 128 tiles of at most 128 rows with all of K: at least three a CTA.
SHAPES = [(4001, 9216, 2048), (2500, 5000, 328), (1, 60008, 264), (40, 60008, 264), (128, 60008, 200)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("out", [BF, F32])
def test_several_tiles(ops, M, N, K, out):
    g = tl.gen(M + N)
    x, w, b = tl.rnd(g, M, K), tl.rnd(g, N, K, scale=K ** -0.5), tl.rnd(g, N, dtype=F32)
    y = torch.full((M + 1, N), 7.0, dtype=out, device="cuda")
    check(ops, x, w, y[:M])
    r = tl.rnd(g, M, N, dtype=out)
    y[:M] = r
    check(ops, x, w, y[:M], bias=b, residual=y[:M], act="silu")
    assert (y[M] == 7).all()


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_the_same_bits_in_a_graph(ops, M, N, K):
    g = tl.gen(M + K)
    x, w, b, r = tl.rnd(g, M, K), tl.rnd(g, N, K, scale=K ** -0.5), tl.rnd(g, N, dtype=F32), tl.rnd(g, M, N)
    y, z = (torch.empty(M, N, dtype=BF, device="cuda") for _ in range(2))
    ops.linear(x, w, y, bias=b, residual=r, activation="gelu")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.linear(x, w, z, bias=b, residual=r, activation="gelu")
    for _ in range(3):
        z.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, z)
    assert ops.device_error() == ops.GDN_OK

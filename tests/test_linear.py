"""gdn_linear against the formula in 64 bits."""
import pytest
import torch

from tests import layer_testlib as tl

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops():
    from gated_deltanet_linear_02_gb300 import build, ops
    build.build()
    return ops


def check(ops, x, w, y, bias=None, residual=None, act="none"):
    """Runs the call; residual may be y (its values are kept for the formula)."""
    K = x.shape[1]
    r = residual.double() if residual is not None else None
    z = x.double() @ w.double().T
    mag = x.double().abs() @ w.double().abs().T
    if bias is not None:
        z, mag = z + bias.double(), mag + bias.double().abs()
    ref = tl.act64(z, act)
    if r is not None:
        ref = ref + r
    ops.linear(x, w, y, bias=bias, residual=residual, activation=act)
    assert ops.device_error() == ops.GDN_OK
    # the sum, an activation with a slope of at most 1.13, its own exp and division (below 2^-18), the residual's sum
    slack = 1.13 * (K / 16 + 8) * 2.0 ** -23 * mag + 2.0 ** -18 * z.abs().clamp(min=1) * (act != "none")
    slack = slack + 2.0 ** -23 * (0 if r is None else r.abs())
    assert tl.within(y, ref, slack)


# one row and few, both sides of a tile, several tiles; widths and depths that end inside a tile
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 7, 8, 9, 16, 17, 33, 64, 65, 128, 129, 300, 1025])
@pytest.mark.parametrize("N,K", [(8, 8), (72, 136), (264, 64), (1000, 2048), (2048, 4096)])
def test_sizes(ops, M, N, K):
    g = tl.gen(M * 7 + N + K)
    x, w = tl.rnd(g, M, K), tl.rnd(g, N, K, scale=K ** -0.5)
    y = torch.full((M + 1, N), 7.0, dtype=BF, device="cuda")
    check(ops, x, w, y[:M])
    assert (y[M] == 7).all()


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M", [1, 6, 40, 200, 2000])
def test_epilogues(ops, act, out, M):
    g = tl.gen(M)
    N, K = 520, 384
    x, w, b = tl.rnd(g, M, K), tl.rnd(g, N, K, scale=2 * K ** -0.5), tl.rnd(g, N, dtype=F32)
    y = torch.empty(M, N, dtype=out, device="cuda")
    check(ops, x, w, y, act=act)
    check(ops, x, w, y, bias=b, act=act)
    check(ops, x, w, y, residual=tl.rnd(g, M, N, dtype=out), act=act)
    check(ops, x, w, y, bias=b, residual=y, act=act)             # the stream in place


@pytest.mark.parametrize("M", [1, 4, 70, 513])
def test_strided_rows(ops, M):
    g = tl.gen(M)
    xs, ys, rs = tl.rnd(g, M, 400), torch.full((M, 360), 7.0, dtype=BF, device="cuda"), tl.rnd(g, M, 304)
    w = tl.rnd(g, 296, 264, scale=0.06)
    check(ops, xs[:, 64:328], w, ys[:, 16:312], residual=rs[:, 8:], act="silu")
    assert (ys[:, :16] == 7).all() and (ys[:, 312:] == 7).all()


@pytest.mark.parametrize("M", [3, 100])
def test_rows_stay_apart(ops, M):
    g = tl.gen(M)
    x, w = tl.rnd(g, M, 256), tl.rnd(g, 128, 256, scale=0.06)
    y0, y1 = torch.empty(M, 128, dtype=BF, device="cuda"), torch.empty(M, 128, dtype=BF, device="cuda")
    ops.linear(x, w, y0)
    x[1, 3] = float("nan")
    ops.linear(x, w, y1)
    assert y1[1].isnan().all()
    rest = torch.arange(M, device="cuda") != 1
    assert torch.equal(y0[rest], y1[rest])
    big = torch.tensor([-200.0, -90.0, 90.0, 200.0], device="cuda").repeat(32)   # activations where exp leaves fp32
    for act, want in (("silu", [0, 0, 90, 200]), ("sigmoid", [0, 0, 1, 1]), ("gelu", [0, 0, 90, 200])):
        ops.linear(torch.zeros_like(x), w, y0, bias=big, activation=act)
        assert (y0[:, :4].float().cpu() == torch.tensor(want).float()).all()


@pytest.mark.parametrize("M,N,K", [(1, 9216, 2048), (5, 2048, 4096), (96, 2048, 4096), (1300, 1032, 520)])
def test_same_bits_again_in_a_graph_and_on_another_stream(ops, M, N, K):
    g = tl.gen(9)
    x, w, r = tl.rnd(g, M, K), tl.rnd(g, N, K, scale=K ** -0.5), tl.rnd(g, M, N)
    y, z, s = (torch.empty(M, N, dtype=BF, device="cuda") for _ in range(3))
    ops.linear(x, w, y, residual=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ops.linear(x, w, s, residual=r, stream=side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.linear(x, w, z, residual=r)
    for _ in range(3):
        z.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, z)
    assert torch.equal(y, s)


def test_binding_refuses(ops):
    x, w, y = (torch.zeros(*s, dtype=BF, device="cuda") for s in ((4, 64), (32, 64), (4, 32)))
    for args, kw in (((x.float(), w, y), {}), ((x, w[:, :32], y), {}), ((x, w, y[:3]), {}), ((x, w, y), dict(activation="tanh")),
                     ((x, w, y), dict(residual=y.float())), ((x, w, y), dict(bias=y[0])), ((x.T, w, y), {}), ((x, w.T, y), {})):
        with pytest.raises((ValueError, TypeError)):
            ops.linear(*args, **kw)
    with pytest.raises(ops.GdnError):
        ops.linear(x, w, torch.zeros(4, 36, dtype=BF, device="cuda")[:, :32])        # rows 72 bytes apart
    ops.linear(x[:0], w, y[:0])

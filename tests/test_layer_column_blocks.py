"""Blocks of columns of one buffer as inputs and outputs of the operators around
the mixers: what shares no element is not refused."""
import pytest
import torch

from tests import layer_testlib as tl
from tests import test_layer_abi as abi

gpu = pytest.mark.gpu
D, BF, F32 = tl.D, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops():
    from gated_deltanet_linear_02_gb300 import build, ops
    build.build()
    return ops


@gpu
@pytest.mark.parametrize("M", [1, 3, 200])
def test_linear(ops, M):
    g = tl.gen(M)
    K, N = 264, 296
    buf, w = tl.rnd(g, M, K + 2 * N), tl.rnd(g, N, K, scale=0.06)
    for a, b, c in ((0, K, K + N), (2 * N, 0, N), (N, N + K, 0)):              # x, y, residual
        x, y, r = buf[:, a:a + K], buf[:, b:b + N], buf[:, c:c + N]
        want = torch.empty(M, N, dtype=BF, device="cuda")
        ops.linear(x.contiguous(), w, want, residual=r.contiguous())
        xk, rk = x.clone(), r.clone()
        ops.linear(x, w, y, residual=r)
        assert torch.equal(y, want) and torch.equal(x, xk) and torch.equal(r, rk)
    if M > 1:
        with pytest.raises(ops.GdnError):
            ops.linear(buf[:, :K], w, buf[:, K - 8:K - 8 + N])


@gpu
@pytest.mark.parametrize("M", [1, 3, 200])
@pytest.mark.parametrize("dt", [BF, F32])
def test_add_norm(ops, M, dt):
    g = tl.gen(M)
    buf = tl.rnd(g, M, 5 * D, dtype=dt)
    x, d, gate, xo, h = (buf[:, i * D:(i + 1) * D] for i in (3, 0, 4, 2, 1))
    p = ops.make_norm_params(1 + 0.1 * tl.rnd(g, D, dtype=F32))
    want = [torch.empty(M, D, dtype=dt, device="cuda") for _ in range(2)]
    ops.add_norm(p, x.contiguous(), d.contiguous(), *want, gate=gate.contiguous())
    ops.add_norm(p, x, d, xo, h, gate=gate)
    assert torch.equal(xo, want[0]) and torch.equal(h, want[1])


def test_blocks_that_share_columns_are_refused(ops):
    """Rows of 4,096 elements a buffer: an output that begins inside an input's columns, ends inside them, or
    wraps into the next row's. No call reaches the device."""
    D2, at = 2 * D, abi.at
    for o in (8, 2040, -8 + D2, D + 8):                            # in elements from delta's first one
        kw = dict(d=at(2), dr=D2, o=at(2) + 2 * o, orow=D2) if o != D + 8 else dict(d=at(2), dr=D2, h=at(2) + 2 * o, hr=D2)
        abi.refused(ops, abi.add_norm(ops, **kw), "overlaps")
        kw = dict(x=at(2) + 2 * o, xr=D2, h=at(2), hr=D2, o=0, d=0, dr=0)   # the input behind the output
        abi.refused(ops, abi.add_norm(ops, **kw), "overlaps")
    for y in (8, 248, 512 - 8, 512 - 56):
        abi.refused(ops, abi.linear(ops, xr=512, y=at(0) + 2 * y, yr=512), "overlaps")
    # other distances from row to row: by the address ranges
    abi.refused(ops, abi.linear(ops, xr=512, y=at(0) + 2 * 256, yr=1024), "overlaps")
    abi.refused(ops, abi.linear(ops, xr=512, y=at(0) + 2 * 256, yr=512, dt=ops.GDN_F32), "overlaps")


@gpu
def test_one_row_of_any_stride(ops):
    """A single row has no next one: its stride does not matter."""
    g = tl.gen(4)
    v, w = tl.rnd(g, D), tl.rnd(g, 64, D, scale=0.02)
    p = ops.make_norm_params(torch.ones(D, device="cuda"))
    want, got = (torch.empty(1, D, dtype=BF, device="cuda") for _ in range(2))
    ops.add_norm(p, v[None], None, None, want)
    ops.add_norm(p, v.expand(4, D)[:1], None, None, got)
    assert torch.equal(got, want)
    y, z = (torch.empty(1, 64, dtype=BF, device="cuda") for _ in range(2))
    ops.linear(v[None], w, y)
    ops.linear(v.expand(4, D)[:1], w, z)
    assert torch.equal(y, z)

"""The activations of gdn_linear far from zero, relative to their values."""
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


def through_bias(ops, v, act, dt, M):
    """act(v) as the call gives it: a product of zeros with v as its bias."""
    N = v.numel()
    x, w = torch.zeros(M, 8, dtype=BF, device="cuda"), torch.zeros(N, 8, dtype=BF, device="cuda")
    y = torch.empty(M, N, dtype=dt, device="cuda")
    ops.linear(x, w, y, bias=v, activation=act)
    assert ops.device_error() == ops.GDN_OK
    assert torch.equal(y[0].expand(M, N), y)
    return y[0]


@pytest.mark.parametrize("M", [1, 300])
@pytest.mark.parametrize("dt", [F32, BF])
def test_gelu(ops, M, dt):
    """v / 2 * erfc(-v / sqrt 2): the argument is off by at most 2^-23 of itself, which moves erfc
    by at most (v^2 + 1) of that; erfcf is good to 4 steps of 2^-23; a product; the output's rounding."""
    v = torch.linspace(-12, 12, 4096, device="cuda")
    y = through_bias(ops, v, "gelu", dt, M).double()
    ref = tl.act64(v.double(), "gelu")
    bound = (v.double() ** 2 + 6) * 2.0 ** -23 + tl.HALF[dt]
    assert ((y - ref).abs() <= bound * 1.01 * ref.abs()).all()


@pytest.mark.parametrize("M", [1, 300])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_silu_and_sigmoid_fp32(ops, M, act):
    """exp to 2^-23, a sum, a division, a product and the rounding at most 2^-24 each: below 2^-21."""
    v = torch.linspace(-87, 87, 4096, device="cuda")
    y = through_bias(ops, v, act, F32, M).double()
    ref = tl.act64(v.double(), act)
    assert ((y - ref).abs() <= 2.0 ** -21 * ref.abs()).all()
    # where exp leaves fp32's normal numbers: within one of its last steps of the value's scale
    v = torch.linspace(-120, -87, 512, device="cuda")
    y = through_bias(ops, v, act, F32, M).double()
    assert ((y - tl.act64(v.double(), act)).abs() <= 2.0 ** -21 * tl.act64(v.double(), act).abs() + v.abs().double() * 2.0 ** -148).all()


@pytest.mark.parametrize("M", [1, 300])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_silu_and_sigmoid_bf16(ops, M, act):
    """The output's rounding, and 2^-23 (4 + 2 |v|) of the value from the special functions; zero
    where the denominator passes 2^126."""
    v = torch.linspace(-87, 87, 4096, device="cuda")
    y = through_bias(ops, v, act, BF, M).double()
    ref = tl.act64(v.double(), act)
    assert ((y - ref).abs() <= (2.0 ** -8 + (4 + 2 * v.abs().double()) * 2.0 ** -23) * 1.01 * ref.abs()).all()
    y = through_bias(ops, torch.linspace(-200, -88.8, 256, device="cuda"), act, BF, M)
    assert (y.abs() < 2.0 ** -120).all()

"""gdn_moe: outputs that are not finite leave their neighbours alone."""
import pytest
import torch

from tests import layer_testlib as tl
from tests.test_moe import BOUND, make

pytestmark = pytest.mark.gpu
D, BF, F32 = tl.D, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops():
    from gated_deltanet_linear_02_gb300 import build, ops
    build.build()
    return ops


@pytest.mark.parametrize("M", [3, 40, 700])       # a pair's outputs in fp32, and in 16 bits scaled by blocks
@pytest.mark.parametrize("scale", [1e-6, 1.0, 1e6])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_one_output_dim_is_not_finite(ops, M, scale, bad):
    """A weight of `down` that is not finite makes one dim of its expert's tokens so; the 31
    dims beside it keep their values, of any magnitude."""
    g = tl.gen(M)
    W = tl.moe_weights(g, 8, 128)
    W["down"], W["sh_down"] = (W["down"].float() * scale).to(BF), (W["sh_down"].float() * scale).to(BF)
    x = tl.rnd(g, M, D)
    ids, w = tl.route64(x, W["router"], 2, True)
    hit = (ids == 3).any(-1)
    if M < 5:
        ids[0, 0], hit[0] = 3, True
    ref = tl.moe64(W, x, ids, w)
    W["down"][3, 700, 5] = bad
    out = torch.empty(M, D, device="cuda")
    ops.moe(make(ops, W, 2), x, out, ids=ids, weights=w.float())
    assert ops.device_error() == ops.GDN_OK
    assert hit.any() and not torch.isfinite(out[hit, 700]).any() and torch.isfinite(out[~hit, 700]).all()
    beside = [d for d in range(672, 704) if d != 700]
    assert torch.isfinite(out[:, beside]).all() and tl.relative(out[:, beside], ref[:, beside]) < BOUND[F32]
    rest = [d for d in range(D) if d != 700]
    assert tl.relative(out[:, rest], ref[:, rest]) < BOUND[F32]

"""gdn_moe after its router's wait gave up: no expert's output, no index that was
never written, a status that the host reads, and a context that works on."""
import pytest
import torch

from tests import layer_testlib as tl
from tests.test_moe import check, make

pytestmark = pytest.mark.gpu
D, BF, F32 = tl.D, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops():
    from gated_deltanet_linear_02_gb300 import build, ops
    build.build()
    return ops


@pytest.mark.parametrize("M", [5, 100, 300, 900])     # one cluster and several; outputs in fp32 and in 16 bits
@pytest.mark.parametrize("shared", [True, False])
def test_tokens_without_a_choice(ops, M, shared):
    g = tl.gen(M)
    W = tl.moe_weights(g, 16, 128, shared)
    p, x, r = make(ops, W, 4), tl.rnd(g, M, D), tl.rnd(g, M, D, dtype=F32)
    assert ops.device_error() == ops.GDN_OK
    torch.cuda.empty_cache()
    fill = torch.full((ops.moe_workspace_size(p, M),), 255, dtype=torch.uint8, device="cuda")     # what the call's scratch holds before
    del fill
    out = torch.full((M + 1, D), 7.0, device="cuda")
    ops.selftest_moe_lost_route(p, x, out[:M], residual=r)
    assert ops.device_error() == ops.GDN_ERR_TIMEOUT and ops.device_error() == ops.GDN_OK
    nobody, none = torch.full((M, 4), -1, dtype=torch.int32, device="cuda"), torch.zeros(M, 4, device="cuda")
    want = torch.empty(M, D, device="cuda")
    ops.moe(p, x, want, residual=r, ids=nobody, weights=none)
    assert torch.equal(out[:M], want) and (out[M] == 7).all()
    if not shared:
        assert torch.equal(want, r)
    check(ops, W, x, 4, F32, g=g)                                  # and the next call is whole


def test_refusals(ops):
    g = tl.gen(1)
    W = tl.moe_weights(g, 8, 128)
    x = tl.rnd(g, 4, D)
    with pytest.raises(ops.GdnError):
        ops.selftest_moe_lost_route(make(ops, W, 2), x, torch.empty_like(x))

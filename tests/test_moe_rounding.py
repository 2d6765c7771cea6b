"""What gdn_moe rounds between its products: the same tokens in one long call, whose pairs'
outputs are held in 16 bits scaled by blocks, and in short ones, where they stay in fp32."""
import pytest
import torch

from tests import layer_testlib as tl
from tests.test_moe import make

pytestmark = pytest.mark.gpu
D, F32 = tl.D, torch.float32


@pytest.fixture(scope="module")
def ops():
    from gated_deltanet_linear_02_gb300 import build, ops
    build.build()
    return ops


@pytest.mark.parametrize("shared", [True, False])
def test_blocks_of_the_long_form(ops, shared):
    """Each pair's output moves by at most 2^-11 of the largest of its block of 32, times its weight."""
    g = tl.gen(31)
    E, k, F, M = 8, 2, 128, 192
    W = tl.moe_weights(g, E, F, shared, sh_router=False)
    W["down"] = (W["down"].float() * torch.exp(tl.rnd(g, E, D, 1, dtype=F32))).to(torch.bfloat16)      # dims of many sizes
    x, p = tl.rnd(g, M, D), make(ops, W, k)
    ids, w = tl.route64(x, W["router"], k, True)
    w = w.float()
    assert M * k > 16 * E and 64 * k <= 16 * E
    long, short = torch.empty(M, D, device="cuda"), torch.empty(M, D, device="cuda")
    ops.moe(p, x, long, ids=ids, weights=w)
    for m in range(0, M, 64):
        ops.moe(p, x[m:m + 64], short[m:m + 64], ids=ids[m:m + 64].contiguous(), weights=w[m:m + 64].contiguous())
    assert ops.device_error() == ops.GDN_OK
    # the pairs' outputs one by one, in fp32 (a weight of 1 on one slot)
    slack = torch.zeros(M, D, dtype=torch.float64, device="cuda")
    none = make(ops, dict(W, sh_gate=None, sh_up=None, sh_down=None), 1)
    y = torch.empty(M, D, device="cuda")
    one = torch.ones(64, 1, device="cuda")

    def top(t):
        return t.double().abs().view(M, D // 32, 32).amax(-1, keepdim=True).expand(M, D // 32, 32).reshape(M, D)
    for j in range(k):
        for m in range(0, M, 64):
            ops.moe(none, x[m:m + 64], y[m:m + 64], ids=ids[m:m + 64, j:j + 1].contiguous(), weights=one)
        slack += w[:, j:j + 1].double() * top(y)
    if shared:
        for m in range(0, M, 64):
            ops.moe(p, x[m:m + 64], y[m:m + 64], ids=torch.full((64, k), -1, dtype=torch.int32, device="cuda"), weights=torch.ones(64, k, device="cuda"))
        slack += top(y)
    # beside it the fp32 sums of k + 1 terms, in both
    assert ((long.double() - short.double()).abs() <= (2.0 ** -11 + 4 * (k + 1) * 2.0 ** -24) * slack).all()
    assert not torch.equal(long, short)

"""The workspace of gdn_moe over its forms, without a GPU: one made for M tokens serves
every smaller call."""
import pytest

from tests import test_layer_abi as abi


@pytest.fixture(scope="module")
def ops():
    from gated_deltanet_linear_02_gb300 import build, ops
    build.build()
    return ops


@pytest.mark.parametrize("E,k,F,shared", [(256, 8, 512, True), (256, 8, 512, False), (256, 1, 128, True), (8, 2, 8192, True),
                                          (4, 2, 8192, False), (64, 8, 1024, True), (1, 1, 128, False), (16, 16, 2176, True)])
def test_never_shrinks(ops, E, k, F, shared):
    kw = dict(num_experts=E, top_k=k, ffn_dim=F, **({} if shared else dict(sh_gate=0, sh_up=0, sh_down=0, sh_router=0)))
    p = abi.params(ops, **kw)
    size = [ops.moe_workspace_size(Params(p), M) for M in range(0, 8300)]
    assert all(a <= b for a, b in zip(size, size[1:])) and size[8192] == size[8299]
    # the most that any call up to M asks for, and no more: a call of M with a byte less is refused
    # where its own form is the largest so far
    last = [m for m in (4, 16 * E // k) if m < 8192]
    for M in (1, *last):
        assert abi.moe(ops, p, M=M, n=size[M] - 1) == ops.GDN_ERR_WORKSPACE


class Params:
    """What the binding takes for parameters: their address."""
    def __init__(self, p):
        import ctypes
        self.keep, self._ref = p, ctypes.addressof(p)


@pytest.mark.gpu
def test_one_workspace_for_every_call(ops):
    import torch

    from tests import layer_testlib as tl
    from tests.test_moe import BOUND, make
    g = tl.gen(3)
    W = tl.moe_weights(g, 8, 128)
    p, x = make(ops, W, 2), tl.rnd(g, 70, tl.D)
    ws = torch.full((ops.moe_workspace_size(p, 70),), 255, dtype=torch.uint8, device="cuda")
    ids, w = tl.route64(x, W["router"], 2, True)
    for M in (70, 64, 65, 4, 5, 1):
        out = torch.empty(M, tl.D, device="cuda")
        ops.moe(p, x[:M], out, workspace=ws)
        assert ops.device_error() == ops.GDN_OK
        assert tl.relative(out, tl.moe64(W, x[:M], ids[:M], w[:M])) < BOUND[torch.float32]

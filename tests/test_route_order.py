"""The router's order where large terms cancel: the exact logits', whatever the
size of the terms that they are sums of."""
import pytest
import torch

from tests import layer_testlib as tl

pytestmark = pytest.mark.gpu
D, BF = tl.D, torch.bfloat16
E, K = 256, 8


@pytest.fixture(scope="module")
def ops():
    from gated_deltanet_linear_02_gb300 import build, ops
    build.build()
    return ops


def rows(g, M, amp, noise):
    """Rows of noise with two channels of +-amp, which every expert of `router` weighs alike."""
    x = tl.rnd(g, M, D, scale=noise)
    x[:, 5], x[:, 600] = amp, -amp
    return x


def weights(g):
    router = tl.rnd(g, E, D, scale=0.03)
    router[:, 5] = router[:, 600] = 0.25
    return router


CASES = [(300.0, 1.0), (7500.0, 1.0), (3e4, 1.0), (1e6, 1.0), (32.0, 0.005), (32.0, 1e-4), (3e4 * 2.0 ** 40, 2.0 ** 40),
         (3e4 * 2.0 ** -60, 2.0 ** -60)]


@pytest.mark.parametrize("M", [40, 3000])
@pytest.mark.parametrize("amp,noise", CASES)
@pytest.mark.parametrize("k", [1, 8, 16])
def test_many_tokens(ops, M, amp, noise, k):
    g = tl.gen(int(M + k))
    x, router = rows(g, M, amp, noise), weights(g)
    ids, w = torch.empty(M, k, dtype=torch.int32, device="cuda"), torch.empty(M, k, device="cuda")
    ops.moe_route(ops.make_moe_params(router, top_k=k), x, ids, w)
    assert ops.device_error() == ops.GDN_OK
    rid, _ = tl.route64(x, router, k, True)
    assert torch.equal(ids, rid)


@pytest.fixture(scope="module")
def tell(ops):
    """Experts whose outputs say who they are: expert e writes dims 8 e .. 8 e + 7 alone."""
    g = tl.gen(77)
    F = 128
    router, gate, up = weights(g), tl.rnd(g, E, F, D, scale=0.03), tl.rnd(g, E, F, D, scale=0.03)
    gate[:, :, [5, 600]] = up[:, :, [5, 600]] = 0
    down = torch.zeros(E, D, F, dtype=BF, device="cuda")
    for e in range(E):
        down[e, 8 * e:8 * e + 8] = tl.rnd(g, 8, F)
    return router, ops.make_moe_params(router, gate, up, down, top_k=K)


@pytest.mark.parametrize("M", [1, 4, 12])
@pytest.mark.parametrize("amp,noise", CASES[:6])
def test_the_layer_takes_the_same_experts(ops, tell, M, amp, noise):
    router, p = tell
    x = rows(tl.gen(M), 1200, amp, noise)
    out = torch.empty(1200, D, device="cuda")
    for m in range(0, 1200, M):
        ops.moe(p, x[m:m + M], out[m:m + M])
    assert ops.device_error() == ops.GDN_OK
    rid, _ = tl.route64(x, router, K, True)
    want = torch.zeros(1200, E, dtype=torch.bool, device="cuda").scatter_(1, rid.long(), True)
    assert torch.equal(out.view(1200, E, 8).ne(0).any(-1), want)


@pytest.mark.parametrize("M", [4, 130])
def test_rows_that_decide_nothing(ops, M):
    """Rows of zeros (a padded batch), of NaN and of infinities beside ordinary ones; router
    rows of zeros and of NaN."""
    g = tl.gen(9)
    x, router = tl.rnd(g, M, D), tl.rnd(g, E, D, scale=0.03)
    router[200:] = 0
    x[1] = 0
    x[2, 7] = float("inf")
    x[3] = float("nan")
    router[17, 3] = float("nan")
    ids, w = torch.empty(M, K, dtype=torch.int32, device="cuda"), torch.empty(M, K, device="cuda")
    ops.moe_route(ops.make_moe_params(router, top_k=K), x, ids, w)
    assert ops.device_error() == ops.GDN_OK
    rest = [i for i in range(M) if i not in (2, 3)]
    r = router.double()
    r[17] = 0
    logits = x[rest].double() @ r.T
    logits[:, 17] = -torch.inf
    rid = torch.sort(logits, dim=-1, descending=True, stable=True)[1][:, :K]
    assert torch.equal(ids[rest].long(), rid)
    assert ids[3].tolist() == list(range(K)) and w[[2, 3]].isnan().all()


@pytest.mark.parametrize("E", [24, 256])
@pytest.mark.parametrize("M", [3, 200])
def test_equal_sums_of_different_terms(ops, E, M):
    """Router rows that are permutations of one another, tokens whose elements are all the same:
    every logit is the same number, and the lowest indices are taken."""
    g = tl.gen(E)
    row = tl.rnd(g, D, scale=0.03)
    router = torch.stack([row[torch.randperm(D, generator=g, device="cuda")] for _ in range(E)])
    x = tl.rnd(g, M, 1).expand(M, D).contiguous()
    ids, w = torch.empty(M, K, dtype=torch.int32, device="cuda"), torch.empty(M, K, device="cuda")
    ops.moe_route(ops.make_moe_params(router, top_k=K), x, ids, w)
    assert ops.device_error() == ops.GDN_OK
    assert (ids == torch.arange(K, device="cuda")).all() and ((w - 1 / K).abs() <= 2.0 ** -24).all()

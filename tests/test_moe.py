"""gdn_moe_route and gdn_moe against the formulas in 64 bits."""
import pytest
import torch

from tests import layer_testlib as tl

pytestmark = pytest.mark.gpu
D, BF, F32 = tl.D, torch.bfloat16, torch.float32
# one rounding of the hidden activations (2^-8 at most, evenly spread), independent from
# one to the next: at most 2^-8 / sqrt(3) of the result as a norm; a bf16 output adds as much
BOUND = {F32: 2.0 ** -8 / 3 ** 0.5, BF: 2.0 ** -8 * (2 / 3) ** 0.5}


@pytest.fixture(scope="module")
def ops():
    from gated_deltanet_linear_02_gb300 import build, ops
    build.build()
    return ops


def make(ops, W, k, renorm=True):
    return ops.make_moe_params(W.get("router"), W["gate"], W["up"], W["down"], W.get("sh_gate"), W.get("sh_up"), W.get("sh_down"),
                               W.get("sh_router"), top_k=k, norm_topk=renorm)


def routed(ops, p, x):
    M = x.shape[0]
    ids = torch.full((M, p.top_k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((M, p.top_k), -7.0, device="cuda")
    ops.moe_route(p, x, ids, w)
    assert ops.device_error() == ops.GDN_OK
    return ids, w


# ---- the router

@pytest.mark.parametrize("M", [1, 2, 5, 31, 128, 129, 700, 2500])
@pytest.mark.parametrize("E,k,renorm", [(256, 8, True), (256, 16, False), (40, 6, False), (8, 1, True), (8, 8, True), (1, 1, True), (33, 2, False)])
def test_route(ops, M, E, k, renorm):
    g = tl.gen(M + E)
    x, router = tl.rnd(g, M, D), tl.rnd(g, E, D, scale=0.03)
    ids, w = routed(ops, ops.make_moe_params(router, top_k=k, norm_topk=renorm), x)
    rid, rw = tl.route64(x, router, k, renorm)
    assert torch.equal(ids, rid)
    # logits: sums of 16 times 16 products truncated (16 steps of 2^-23), 8 partial sums: below 2^-18 of the
    # root of the sum of their squares; a weight moves by at most twice that, and exp and division add 2^-22
    err = 2.0 ** -17 * float((x.double().norm(dim=1).max() * router.double().norm(dim=1).max()) / D ** 0.5)
    assert ((w.double() - rw).abs() <= rw * (err + 2.0 ** -21)).all()


def test_route_near_ties_and_ties(ops):
    """Rows of the router that differ in one last place, equal rows, and rows of zeros."""
    g = tl.gen(3)
    x, router = tl.rnd(g, 300, D), tl.rnd(g, 64, D, scale=0.03)
    for e in range(1, 40):                                         # neighbours that differ by one bf16 step in one place
        router[e] = router[0]
        router[e, 11 * e] *= 1 + 2.0 ** -7
    router[50:54] = router[49]
    x[7] = 0
    x[8] *= 2.0 ** -60
    x[9] *= 2.0 ** 40
    for k in (1, 5, 16):
        ids, w = routed(ops, ops.make_moe_params(router, top_k=k), x)
        rid, rw = tl.route64(x, router, k, True)
        assert torch.equal(ids, rid)
        assert ids[7].tolist() == list(range(k)) and (w[7] == 1 / k).all()


def test_route_large_terms_that_cancel(ops):
    """Channels far above the others whose contributions all experts share."""
    g = tl.gen(4)
    x, router = tl.rnd(g, 200, D), tl.rnd(g, 256, D, scale=0.03)
    x[:, 5], x[:, 600] = 300.0, -300.0
    router[:, 5] = router[:, 600] = 0.25
    ids, _ = routed(ops, ops.make_moe_params(router, top_k=8), x)
    rid, _ = tl.route64(x, router, 8, True)
    assert torch.equal(ids, rid)


def test_route_what_is_not_finite(ops):
    g = tl.gen(5)
    x, router = tl.rnd(g, 4, D), tl.rnd(g, 16, D, scale=0.03)
    clean, cw = routed(ops, ops.make_moe_params(router, top_k=3), x)
    x[1, 0] = float("nan")
    ids, w = routed(ops, ops.make_moe_params(router, top_k=3), x)
    assert ids[1].tolist() == [0, 1, 2] and w[1].isnan().all()
    rest = [0, 2, 3]
    assert torch.equal(ids[rest], clean[rest]) and torch.equal(w[rest], cw[rest])
    x[1, 0] = 1.0
    best = int(clean[0, 0])
    router[best, 4] = float("nan")
    ids, w = routed(ops, ops.make_moe_params(router, top_k=16), x)
    assert (ids[:, 15] == best).all() and (ids[:, :15] != best).all()


def test_route_strided_rows_and_padding(ops):
    g = tl.gen(6)
    wide, router = tl.rnd(g, 10, 2 * D), tl.rnd(g, 256, D, scale=0.03)
    p = ops.make_moe_params(router, top_k=8)
    ids, w = torch.full((12, 8), -7, dtype=torch.int32, device="cuda"), torch.full((12, 8), -7.0, device="cuda")
    ops.moe_route(p, wide[:, D:], ids[:10], w[:10])
    rid, _ = tl.route64(wide[:, D:], router, 8, True)
    assert torch.equal(ids[:10], rid) and (ids[10:] == -7).all() and (w[10:] == -7).all()


# ---- the whole layer

def check(ops, W, x, k, out_dt, residual=False, renorm=True, given=None, bound=None, g=None):
    p = make(ops, W, k, renorm)
    M = x.shape[0]
    r = tl.rnd(g, M, D, dtype=out_dt) if residual else None
    out = torch.full((M + 1, D), 7.0, dtype=out_dt, device="cuda")
    ws = torch.full((ops.moe_workspace_size(p, M),), 255, dtype=torch.uint8, device="cuda")     # whatever it held
    if given is None:
        ops.moe(p, x, out[:M], residual=r, workspace=ws)
        ids, w = tl.route64(x, W["router"], k, renorm)
    else:
        ids, w = given
        ops.moe(p, x, out[:M], residual=r, ids=ids, weights=w, workspace=ws)
    assert ops.device_error() == ops.GDN_OK
    assert (out[M] == 7).all()
    ref = tl.moe64(W, x, ids, w)
    if r is not None:
        ref = ref + r.double()
    assert tl.relative(out[:M], ref) < (bound or BOUND[out_dt])
    return out[:M]


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 16, 17, 33, 70, 257, 600, 1500])
@pytest.mark.parametrize("E,k,F,shared", [(64, 8, 512, True), (16, 2, 128, False), (8, 8, 384, True)])
@pytest.mark.parametrize("out", [BF, F32])
def test_sizes(ops, M, E, k, F, shared, out):
    g = tl.gen(M + E)
    W = tl.moe_weights(g, E, F, shared)
    check(ops, W, tl.rnd(g, M, D), k, out, residual=M % 2 == 0, renorm=M % 3 != 0, g=g)


@pytest.mark.parametrize("M", [1, 4, 24, 300])
def test_model_shape(ops, M):
    g = tl.gen(M)
    W = tl.moe_weights(g, 256, 512)
    check(ops, W, tl.rnd(g, M, D), 8, BF, residual=True, g=g)


@pytest.mark.parametrize("M", [1, 3, 40, 900])
def test_wide_experts_and_a_shared_one_without_gate(ops, M):
    g = tl.gen(M)
    W = tl.moe_weights(g, 4, 1280, True, sh_router=False)
    check(ops, W, tl.rnd(g, M, D), 2, F32, g=g)


@pytest.mark.parametrize("M", [4, 50, 700])
def test_given_routing(ops, M):
    """Ids that repeat, that are out of range, that all fall on one expert."""
    g = tl.gen(M)
    W = tl.moe_weights(g, 12, 256)
    x = tl.rnd(g, M, D)
    ids = torch.randint(-2, 14, (M, 4), generator=g, device="cuda", dtype=torch.int32)
    w = torch.randn(M, 4, generator=g, device="cuda")
    ids[0] = 5
    check(ops, W, x, 4, F32, given=(ids, w), g=g)
    check(ops, W, x, 4, F32, given=(torch.full_like(ids, 11), w), g=g)
    none = dict(W, sh_gate=None, sh_up=None, sh_down=None, sh_router=None)
    out = torch.full((M, D), 7.0, device="cuda")
    ops.moe(make(ops, none, 4), x, out, ids=torch.full_like(ids, 12), weights=w)       # nobody's token
    assert (out == 0).all()
    noroute = dict(W, router=None)
    check(ops, noroute, x, 4, F32, given=(ids, w), g=g)


@pytest.mark.parametrize("M", [1, 6, 40, 600])
def test_own_routing_is_the_router(ops, M):
    """Routing inside gives what a call with gdn_moe_route's answer gives."""
    g = tl.gen(M)
    W = tl.moe_weights(g, 64, 256)
    x, p = tl.rnd(g, M, D), make(ops, W, 8)
    a, b = torch.empty(M, D, device="cuda"), torch.empty(M, D, device="cuda")
    ops.moe(p, x, a)
    ids, w = routed(ops, p, x)
    ops.moe(p, x, b, ids=ids, weights=w)
    assert tl.relative(a, b.double()) < 1e-6


@pytest.mark.parametrize("M", [2, 4, 20])
@pytest.mark.parametrize("near", [3, 60])
def test_own_routing_near_ties(ops, M, near):
    """Router rows that differ in one last place: a few of them, and more than a warp has lanes."""
    g = tl.gen(M + near)
    W = tl.moe_weights(g, 64, 128)
    for e in range(1, near):
        W["router"][e] = W["router"][0]
        W["router"][e, 7 * e] *= 1 + 2.0 ** -7
    x = tl.rnd(g, M, D) + W["router"][0].float().mul(4).to(BF)      # those rows are the best of every token
    check(ops, W, x, 4, F32, g=g)


@pytest.mark.parametrize("M", [1, 9])
@pytest.mark.parametrize("E,k,F", [(64, 16, 128), (4, 2, 8192), (20, 5, 2048)])
def test_many_slots_and_wide_experts(ops, M, E, k, F):
    g = tl.gen(M + E)
    W = tl.moe_weights(g, E, F)
    check(ops, W, tl.rnd(g, M, D), k, BF, residual=True, g=g)
    check(ops, W, tl.rnd(g, 4, D), k, F32, g=g)


@pytest.mark.parametrize("M", [3, 8, 40, 600])
def test_rows_stay_apart(ops, M):
    g = tl.gen(M)
    W = tl.moe_weights(g, 8, 256)
    x, p = tl.rnd(g, M, D), make(ops, W, 2)
    a, b = torch.empty(M, D, device="cuda"), torch.empty(M, D, device="cuda")
    ops.moe(p, x, a)
    x[1, 9] = float("nan")
    x[2, 9] = float("inf")
    ops.moe(p, x, b)
    assert b[1].isnan().all() and not torch.isfinite(b[2]).all()
    rest = [i for i in range(M) if i not in (1, 2)]
    assert torch.equal(a[rest], b[rest])


def test_residual_in_place_strides_and_empty(ops):
    g = tl.gen(8)
    W = tl.moe_weights(g, 16, 128)
    p = make(ops, W, 4)
    for M in (2, 50):
        wide = tl.rnd(g, M, D + 64)
        x, r = wide[:, 64:], tl.rnd(g, M, D)
        want = torch.empty_like(r)
        ops.moe(p, x.contiguous(), want, residual=r)
        ops.moe(p, x, r, residual=r)
        assert torch.equal(r, want)
    ops.moe(p, x[:0], r[:0])


@pytest.mark.parametrize("scale", [1e-6, 1e6])
def test_outputs_of_any_magnitude(ops, scale):
    """The pairs' outputs of long calls are held in 16 bits with a scale of their own."""
    g = tl.gen(12)
    W = tl.moe_weights(g, 8, 128)
    W["down"], W["sh_down"] = (W["down"].float() * scale).to(BF), (W["sh_down"].float() * scale).to(BF)
    W["down"][3, 700] *= 2.0 ** 20                        # one dim far above the others
    x = tl.rnd(g, 700, D)
    out = check(ops, W, x, 2, F32, g=g)
    ids, w = tl.route64(x, W["router"], 2, True)
    ref = tl.moe64(W, x, ids, w)
    rest = [d for d in range(D) if d // 32 != 700 // 32]  # outside its block nothing is lost
    assert tl.relative(out[:, rest], ref[:, rest]) < BOUND[F32]


def test_more_tokens_than_a_window(ops):
    g = tl.gen(9)
    W = tl.moe_weights(g, 8, 128)
    M = 8192 + 333
    x, r = tl.rnd(g, M, D), tl.rnd(g, M, D)
    out = torch.empty(M, D, dtype=BF, device="cuda")
    ops.moe(make(ops, W, 2), x, out, residual=r)
    assert ops.device_error() == ops.GDN_OK
    ids, w = tl.route64(x, W["router"], 2, True)
    ref = tl.moe64(W, x, ids, w) + r.double()
    assert tl.relative(out, ref) < BOUND[BF]
    assert tl.relative(out[8192:], ref[8192:]) < BOUND[BF]


@pytest.mark.parametrize("M", [1, 7, 100, 1200])
def test_same_bits_again_in_a_graph_and_two_at_once(ops, M):
    g = tl.gen(10)
    W = tl.moe_weights(g, 32, 256)
    p, x = make(ops, W, 4), tl.rnd(g, M, D)
    y = torch.empty(M, D, dtype=BF, device="cuda")
    ws = ops.moe(p, x, y)
    z = torch.empty_like(y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.moe(p, x, z, workspace=ws)
    for _ in range(3):
        z.fill_(0)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, z)
    # two calls at once, each on its stream and workspace
    outs, streams = [torch.empty_like(y) for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        for o, s in zip(outs, streams):
            s.wait_stream(torch.cuda.current_stream())
            ops.moe(p, x, o, stream=s)
    torch.cuda.synchronize()
    assert ops.device_error() == ops.GDN_OK
    assert torch.equal(outs[0], y) and torch.equal(outs[1], y)


def test_binding_refuses(ops):
    g = tl.gen(11)
    W = tl.moe_weights(g, 8, 128)
    p, x = make(ops, W, 2), tl.rnd(g, 4, D)
    out = torch.empty_like(x)
    ids, w = routed(ops, p, x)
    for kw in (dict(ids=ids[:, :1], weights=w), dict(ids=ids.long(), weights=w), dict(residual=x.float()), dict(residual=x[:2]),
               dict(workspace=torch.empty(4096, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            ops.moe(p, x, out, **kw)
    with pytest.raises(ops.GdnError):
        ops.moe(p, x, out, ids=ids)
    with pytest.raises(ops.GdnError):
        ops.moe(p, x, out, workspace=torch.empty(512, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        ops.moe(p, x[:, :1024], out)
    with pytest.raises(ValueError):
        ops.make_moe_params(W["router"], W["gate"], W["up"], W["down"][:, :, :64])

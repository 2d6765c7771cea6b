"""The operators around the mixers without a GPU: sizes of workspaces and the
refusals of include/gdn.h. No call here reaches the device."""
import ctypes

import pytest

FAKE = 1 << 40          # 256-byte aligned, never dereferenced: every case fails a host check first
GAP = 1 << 36


def at(i):
    return FAKE + i * GAP


@pytest.fixture(scope="module")
def ops():
    from gated_deltanet_linear_02_gb300 import build, ops
    build.build()
    return ops


def refused(ops, st, word=""):
    assert st == ops.GDN_ERR_INVALID_ARG
    assert word in ops.last_error()


def add_norm(ops, **kw):
    a = dict(norm_w=at(0), post_w=0, rs=1.0, eps=1e-6, x=at(1), xr=2048, d=at(2), dr=2048, g=0, gr=0, o=at(3), orow=2048,
             h=at(4), hr=2048, M=4, sdt=ops.GDN_BF16, act=ops.GDN_BF16)
    a.update(kw)
    p = ops.gdn_norm_params(a["norm_w"], a["post_w"], a["rs"], a["eps"])
    return ops.lib().gdn_add_norm(ctypes.addressof(p), a["x"], a["xr"], a["d"], a["dr"], a["g"], a["gr"], a["o"], a["orow"],
                                  a["h"], a["hr"], a["M"], a["sdt"], a["act"], None)


def test_add_norm_refusals(ops):
    assert add_norm(ops, M=0) == ops.GDN_OK
    for kw in (dict(M=-1), dict(M=(1 << 24) + 1), dict(x=0), dict(x=at(1) + 4), dict(xr=2040), dict(xr=2052), dict(dr=4),
               dict(d=at(2) + 8), dict(d=0, g=at(5), gr=2048), dict(g=at(5), gr=8), dict(o=0, h=0), dict(norm_w=0),
               dict(norm_w=at(0) + 4), dict(post_w=at(6) + 4), dict(eps=-1.0), dict(eps=float("nan")), dict(sdt=7), dict(act=7),
               dict(o=at(2)), dict(h=at(1)), dict(h=at(3)), dict(o=at(1), orow=4096), dict(h=at(2), hr=4096),
               dict(o=at(1) + 16), dict(g=at(4), gr=2048), dict(g=at(3), gr=0)):
        refused(ops, add_norm(ops, **kw))
    assert ops.lib().gdn_add_norm(None, at(1), 2048, None, 0, None, 0, None, 0, at(4), 2048, 1, 1, 1, None) == ops.GDN_ERR_INVALID_ARG


def linear(ops, **kw):
    a = dict(x=at(0), xr=256, w=at(1), b=0, r=0, rr=0, y=at(2), yr=64, M=3, N=64, K=256, act=0, dt=ops.GDN_BF16)
    a.update(kw)
    return ops.lib().gdn_linear(a["x"], a["xr"], a["w"], a["b"], a["r"], a["rr"], a["y"], a["yr"], a["M"], a["N"], a["K"],
                                a["act"], a["dt"], None)


def test_linear_refusals(ops):
    assert linear(ops, M=0) == ops.GDN_OK
    for kw in (dict(M=-1), dict(M=(1 << 24) + 1), dict(N=0), dict(N=60), dict(N=(1 << 20) + 8), dict(K=0), dict(K=252, xr=252),
               dict(K=(1 << 20) + 8), dict(x=0), dict(w=0), dict(y=0), dict(x=at(0) + 2), dict(w=at(1) + 8), dict(b=at(3) + 4),
               dict(r=at(3) + 8, rr=64), dict(r=at(3), rr=56), dict(xr=248), dict(xr=260), dict(yr=56), dict(yr=68), dict(act=4),
               dict(act=-1), dict(dt=2), dict(y=at(0)), dict(y=at(1)), dict(y=at(3), b=at(3)), dict(r=at(2), rr=128),
               dict(r=at(2) + 16, rr=64)):
        refused(ops, linear(ops, **kw))
    refused(ops, linear(ops, dt=ops.GDN_F32, yr=66), "stride")


def params(ops, **kw):
    a = dict(router=at(0), gate=at(1), up=at(2), down=at(3), sh_gate=at(4), sh_up=at(5), sh_down=at(6), sh_router=at(7),
             num_experts=256, top_k=8, ffn_dim=512, norm_topk=1)
    a.update(kw)
    return ops.gdn_moe_params(*(a[n] for n, _ in ops.gdn_moe_params._fields_))


def moe(ops, p=None, **kw):
    a = dict(x=at(8), xr=2048, r=0, o=at(9), M=4, ids=0, w=0, ws=at(10), n=1 << 34, dt=ops.GDN_BF16)
    a.update(kw)
    p = p if p is not None else params(ops)
    return ops.lib().gdn_moe(ctypes.addressof(p), a["x"], a["xr"], a["r"], a["o"], a["M"], a["ids"], a["w"], a["ws"], a["n"],
                             a["dt"], None)


def test_moe_refusals(ops):
    assert moe(ops, M=0) == ops.GDN_OK
    for kw in (dict(M=-1), dict(M=(1 << 24) + 1), dict(x=0), dict(x=at(8) + 8), dict(xr=2040), dict(xr=2052), dict(o=0),
               dict(o=at(9) + 8), dict(r=at(11) + 8), dict(ids=at(12)), dict(w=at(12)), dict(ids=at(12) + 4, w=at(13)), dict(dt=2),
               dict(o=at(8)), dict(o=at(0)), dict(o=at(1)), dict(o=at(3) + 4096), dict(o=at(7)), dict(r=at(9) + 64),
               dict(ids=at(9), w=at(12)), dict(ws=at(8)), dict(ws=at(9)), dict(ws=at(2)), dict(r=at(10)),):
        refused(ops, moe(ops, **kw))
    for kw in (dict(num_experts=0), dict(num_experts=257), dict(top_k=0), dict(top_k=17), dict(num_experts=4, top_k=5),
               dict(ffn_dim=0), dict(ffn_dim=64), dict(ffn_dim=520), dict(ffn_dim=8320), dict(gate=0), dict(up=at(2) + 8),
               dict(down=0), dict(router=0), dict(sh_gate=0), dict(sh_up=0), dict(sh_down=0),
               dict(sh_gate=0, sh_up=0, sh_down=0), dict(sh_router=at(7) + 2)):
        refused(ops, moe(ops, params(ops, **kw)))
    for kw in (dict(ws=0), dict(ws=at(10) + 16), dict(n=100)):
        assert moe(ops, **kw) == ops.GDN_ERR_WORKSPACE
    assert "needed" in ops.last_error()


def test_moe_route_refusals(ops):
    def route(p=None, x=at(8), xr=2048, M=4, ids=at(9), w=at(10)):
        p = p if p is not None else params(ops)
        return ops.lib().gdn_moe_route(ctypes.addressof(p), x, xr, M, ids, w, None)
    assert route(M=0) == ops.GDN_OK
    for kw in (dict(M=-1), dict(x=0), dict(xr=8), dict(ids=0), dict(w=0), dict(ids=at(9) + 4), dict(w=at(9)), dict(ids=at(8)),
               dict(w=at(0)), dict(p=params(ops, router=0)), dict(p=params(ops, top_k=0)), dict(p=params(ops, num_experts=300))):
        refused(ops, route(**kw))


def test_moe_workspace_stops_growing(ops):
    def size(M, **kw):
        p = params(ops, **kw)
        return ops.lib().gdn_moe_workspace_size(ctypes.addressof(p), M)
    assert 0 < size(1) < size(64) < size(8192) == size(8193) == size(1 << 24)
    assert size(64, sh_gate=0) < size(64)
    assert size(-1) == 0 and size(64, ffn_dim=100) == 0 and size(64, top_k=0) == 0

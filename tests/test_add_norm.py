"""gdn_add_norm against the formula in 64 bits."""
import pytest
import torch

from tests import layer_testlib as tl

pytestmark = pytest.mark.gpu
D, EPS = tl.D, 1e-6
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops():
    from gated_deltanet_linear_02_gb300 import build, ops
    build.build()
    return ops


def ref(x, delta, gate, norm_w, post_w, rs, eps=EPS):
    """x_out, h and the sum of magnitudes that x_out's error is measured by."""
    x = x.double()
    mag = x.abs()
    if delta is not None:
        d = delta.double()
        if post_w is not None:
            d = tl.rms64(d, eps) * post_w.double()
        d = rs * (d if gate is None else d * gate.double())
        x, mag = x + d, mag + d.abs()
    inv = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    return x, None if norm_w is None else x * inv * norm_w.double(), mag, None if norm_w is None else mag * inv * norm_w.double().abs()


# A root of a mean of 2048 squares: 3 + 5 + 3 fp32 sums deep, a root and a division: below 2^-20 of it, twice with post_w.
SLACK = 2.0 ** -19


@pytest.mark.parametrize("sdt", [BF, F32])
@pytest.mark.parametrize("act", [BF, F32])
@pytest.mark.parametrize("M,post,gate", [(1, False, None), (1, True, "rows"), (2, True, None), (77, False, "one"), (300, True, "one")])
def test_matches_the_formula(ops, sdt, act, M, post, gate):
    g = tl.gen(M)
    x, d = tl.rnd(g, M, D, dtype=sdt), tl.rnd(g, M, D, scale=0.7, dtype=act)
    nw, pw = 1 + 0.1 * tl.rnd(g, D, dtype=F32), (1 + 0.1 * tl.rnd(g, D, dtype=F32) if post else None)
    gt = {None: None, "rows": tl.rnd(g, M, D, dtype=act), "one": tl.rnd(g, 1, D, dtype=act).expand(M, D)}[gate]
    xo, h = torch.empty(M, D, dtype=sdt, device="cuda"), torch.empty(M, D, dtype=act, device="cuda")
    ops.add_norm(ops.make_norm_params(nw, pw, 0.8, EPS), x, d, xo, h, gate=gt)
    rx, rh, mx, mh = ref(x, d, gt, nw, pw, torch.tensor(0.8, dtype=F32).item())
    assert tl.within(xo, rx, SLACK * mx) and tl.within(h, rh, SLACK * mh)


def test_parts_in_place_and_strides(ops):
    g = tl.gen(5)
    M = 19
    base, dl = tl.rnd(g, M, 2, D, dtype=F32), tl.rnd(g, M, 3 * D)
    x, d, h = base[:, 1], dl[:, D:2 * D], torch.empty(M, 2 * D, dtype=BF, device="cuda")[:, D:]
    nw = 1 + 0.1 * tl.rnd(g, D, dtype=F32)
    p = ops.make_norm_params(nw, None, 1.0, EPS)
    rx, rh, mx, mh = ref(x, d, None, nw, None, 1.0)
    keep = base[:, 0].clone()
    ops.add_norm(p, x, d, x, h)                                    # the stream in place
    assert tl.within(x, rx, SLACK * mx) and tl.within(h, rh, SLACK * mh) and torch.equal(base[:, 0], keep)
    only = torch.empty(M, D, dtype=BF, device="cuda")
    ops.add_norm(p, x, None, None, only)                           # a norm alone
    rx, rh, mx, mh = ref(x, None, None, nw, None, 1.0)
    assert tl.within(only, rh, SLACK * mh)
    dd = d.contiguous()
    rx, rh, mx, mh = ref(x, dd, None, nw, None, 1.0)
    xo = torch.empty(M, D, dtype=F32, device="cuda")
    ops.add_norm(p, x, dd, xo, dd)                                 # h over delta
    assert tl.within(xo, rx, SLACK * mx) and tl.within(dd, rh, SLACK * mh)
    xo2 = torch.empty_like(xo)
    ops.add_norm(ops.make_norm_params(None, None, 1.0, EPS), x, d, xo2, None)   # a sum alone
    rx, _, mx, _ = ref(x, d, None, None, None, 1.0)
    assert tl.within(xo2, rx, SLACK * mx)


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e18, 1e30])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_rows_of_any_magnitude(ops, scale, eps):
    g = tl.gen(6)
    x = tl.rnd(g, 3, D, dtype=F32) * scale
    nw = 1 + 0.1 * tl.rnd(g, D, dtype=F32)
    h = torch.empty(3, D, dtype=F32, device="cuda")
    ops.add_norm(ops.make_norm_params(nw, None, 1.0, eps), x, None, None, h)
    _, rh, _, mh = ref(x, None, None, nw, None, 1.0, torch.tensor(eps, dtype=F32).item())
    assert tl.within(h, rh, SLACK * mh)


def test_rows_stay_apart(ops):
    """Zeros, NaN and infinities stay in their row, rows past M are left as they are."""
    g = tl.gen(7)
    x = tl.rnd(g, 6, D)
    x[1], x[2, 5], x[3, 7] = 0, float("nan"), float("inf")
    nw = torch.ones(D, device="cuda")
    h = torch.full((8, D), 7.0, dtype=BF, device="cuda")
    ops.add_norm(ops.make_norm_params(nw, None, 1.0, EPS), x, None, None, h[:6])
    assert (h[6:] == 7).all() and (h[1] == 0).all() and h[2].isnan().all() and torch.isfinite(h[[0, 4, 5]]).all()
    assert h[3, 7].isnan() and (h[3, :7] == 0).all()
    ops.add_norm(ops.make_norm_params(nw, None, 1.0, 0.0), x[1:2], None, None, h[1:2])
    assert h[1].isnan().all()
    ops.add_norm(ops.make_norm_params(nw, None, 1.0, EPS), x[:0], None, None, h[:0])


def test_binding_refuses(ops):
    x = torch.zeros(2, D, dtype=BF, device="cuda")
    p = ops.make_norm_params(torch.ones(D, device="cuda"))
    for bad in (dict(delta=x.float()), dict(h=x[:1]), dict(x_out=x.float()), dict(gate=x[:, :8])):
        kw = dict(delta=x.clone(), x_out=None, h=torch.empty_like(x))
        kw.update(bad)
        with pytest.raises(ValueError):
            ops.add_norm(p, x, kw.pop("delta"), kw.pop("x_out"), kw.pop("h"), **kw)
    with pytest.raises(ValueError):
        ops.add_norm(p, x.cpu(), None, None, x)

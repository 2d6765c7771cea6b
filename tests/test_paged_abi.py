"""Host-side checks of the paged-cache entry points and the pins of their oracle,
without a GPU: every refusal comes before any CUDA work."""
import ctypes

import numpy as np
import pytest
import torch

FAKE, STEP = 0x10000000, 0x10000000           # aligned, far apart, never dereferenced


@pytest.fixture(scope="module")
def ops():
    from gated_deltanet_linear_02_gb300 import build, ops
    build.build()
    return ops


def parts(ops, **kw):
    cache = ops.gdn_kv_cache(FAKE, FAKE + STEP, 64, 16, ops.GDN_KV_BF16)
    batch = ops.gdn_paged_batch(FAKE + 2 * STEP, FAKE + 2 * STEP + 4096, None, 4, 4, 1, 8)
    params = ops.gdn_attn_params(FAKE + 3 * STEP, FAKE + 3 * STEP, FAKE + 3 * STEP, 128, 1e-6)
    for k, v in kw.items():
        for s in (cache, batch, params):
            if k in [f[0] for f in s._fields_]:
                setattr(s, k, v)
    return params, batch, cache


A, B_, C_, D_ = (FAKE + i * STEP for i in (4, 5, 6, 7))


def append(ops, p, b, c, k=A, kr=1024, kh=256, v=B_, q=None, qo=None, act=1, pos=None):
    return ops.lib().gdn_kv_append(ctypes.byref(p) if p else None, ctypes.byref(b) if b else None,
                                   ctypes.byref(c) if c else None, k, kr, kh, v, 1024, 256, q, 8192, 512, qo, pos, act, None)


def attend(ops, b, c, q=A, gate=B_, gr=8192, gh=512, out=C_, ws=D_, nbytes=1 << 40, od=1):
    return ops.lib().gdn_attn_paged(ctypes.byref(b), ctypes.byref(c), q, gate, gr, gh, out, ws, nbytes, od, None)


BAD = dict(page_size=[0, 8, 48, 256], num_pages=[0, -1, 1 << 30], B=[-1, 65536], M=[-1, 3, (1 << 24) + 1],
           max_pages=[0, -3, 1 << 29], max_q=[0, 2], format=[2, -1], page_table=[None, FAKE + 2], ctx_len=[None, FAKE + 1],
           cu_q=[FAKE + 3], k=[None, FAKE + 8], v=[None, FAKE + 8])


@pytest.mark.parametrize("field,value", [(f, v) for f, vs in BAD.items() for v in vs])
def test_bad_batches_and_caches_are_refused(ops, field, value):
    kw = {field: value}
    if field == "cu_q":
        kw["max_q"] = 4
    p, b, c = parts(ops, **kw)
    for st in (append(ops, p, b, c), attend(ops, b, c),
               ops.lib().gdn_kv_gather(ctypes.byref(b), ctypes.byref(c), A, B_, 1, None)):
        assert st == ops.GDN_ERR_INVALID_ARG, ops.last_error()
    size = ops.lib().gdn_attn_paged_workspace_size(ctypes.byref(b), ctypes.byref(c))
    assert (size == 0) == (field not in ("page_table", "ctx_len", "cu_q", "k", "v"))


def test_four_bit_cache_has_no_v(ops):
    p, b, c = parts(ops, format=ops.GDN_KV_Q4)
    assert append(ops, p, b, c) == ops.GDN_ERR_INVALID_ARG


def test_no_sequences_or_rows_is_a_no_op(ops):
    for kw in (dict(B=0, M=0), dict(B=0, M=5)):
        p, b, c = parts(ops, **kw)
        assert append(ops, p, b, c) == ops.GDN_OK and attend(ops, b, c) == ops.GDN_OK


@pytest.mark.parametrize("kw", [dict(k=None), dict(k=A + 8), dict(v=None), dict(kr=1020), dict(kh=252), dict(kh=128), dict(kr=-1024),
                                dict(q=C_), dict(qo=C_), dict(q=C_, qo=D_ + 8), dict(act=5), dict(pos=A + 2),
                                dict(k=FAKE), dict(v=FAKE + STEP), dict(q=C_, qo=A), dict(q=C_, qo=C_), dict(q=C_, qo=FAKE)])
def test_bad_append_arguments_are_refused(ops, kw):
    p, b, c = parts(ops)
    assert append(ops, p, b, c, **kw) == ops.GDN_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(norm_eps=-1.0), dict(norm_eps=float("nan")), dict(n_pos=0), dict(rope=FAKE + 4),
                                dict(q_norm_w=FAKE + 4), dict(k_norm_w=FAKE + 4)])
def test_bad_parameters_are_refused(ops, kw):
    p, b, c = parts(ops, **kw)
    assert append(ops, p, b, c) == ops.GDN_ERR_INVALID_ARG
    assert append(ops, None, b, c) == ops.GDN_ERR_INVALID_ARG
    st = ops.lib().gdn_attn_qk_norm_rope(ctypes.byref(p), A, 4096, 256, None, 0, 0, D_, 4, B_, None, 1, 1, None)
    assert st == ops.GDN_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,status", [(dict(q=None), 1), (dict(out=None), 1), (dict(out=C_ + 4), 1), (dict(gate=B_ + 8), 1),
                                       (dict(gr=8190), 1), (dict(gh=100), 1), (dict(od=7), 1), (dict(out=A), 1), (dict(out=B_), 1),
                                       (dict(out=FAKE), 1), (dict(ws=None), 3), (dict(ws=D_ + 4), 3), (dict(nbytes=8), 3)])
def test_bad_attention_arguments_are_refused(ops, kw, status):
    _, b, c = parts(ops)
    assert attend(ops, b, c, **kw) == status


@pytest.mark.parametrize("a", [(None, 4096, 256, None, D_, 4, B_, None, 1, 1), (A, 4090, 256, None, D_, 4, B_, None, 1, 1),
                               (A, 4096, 256, None, None, 4, B_, None, 1, 1), (A, 4096, 256, None, D_, -1, B_, None, 1, 1),
                               (A, 4096, 256, None, D_, 4, None, None, 1, 1), (A, 4096, 256, None, D_, 4, B_, C_, 1, 1),
                               (A, 4096, 256, C_, D_, 4, B_, None, 1, 1), (A, 8192, 512, None, D_, 4, A, None, 1, 1),
                               (A, 4096, 256, None, D_, 4, A, None, 0, 1), (A, 4096, 256, C_, D_, 4, B_, B_, 1, 1),
                               (A, 4096, 256, None, D_, 4, B_, None, 9, 1)])
def test_bad_norm_arguments_are_refused(ops, a):
    p, _, _ = parts(ops)
    q, qr, qh, k, pos, M, qo, ko, act, od = a
    st = ops.lib().gdn_attn_qk_norm_rope(ctypes.byref(p), q, qr, qh, k, 512, 256, pos, M, qo, ko, act, od, None)
    assert st == ops.GDN_ERR_INVALID_ARG


def test_binding_refuses_host_tensors(ops):
    t = torch.zeros(2, 16, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ops.attn_qk_norm_rope(ops.make_attn_params(), t, None, t)
    with pytest.raises(ValueError):
        ops.make_kv_cache(torch.zeros(4, 2, 16, 256, dtype=torch.bfloat16), torch.zeros(4, 2, 16, 256, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        ops.make_paged_batch(torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), 1)


# ---- pins of the oracle to facts from outside it

def test_oracle_bf16_rounding(orc):
    x = np.concatenate([np.random.default_rng(0).standard_normal(4000) * 10.0 ** np.random.default_rng(1).integers(-30, 30, 4000),
                        [0.0, 1.0 + 2 ** -8, 1.0 + 3 * 2 ** -8, -(1.0 + 2 ** -8), 2.0 ** -133, 3e38]])
    x = x.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(x).float().to(torch.bfloat16).double().numpy()
    np.testing.assert_array_equal(orc.bf16_of(x), want)


def test_oracle_norm_and_rotation(orc):
    r = np.random.default_rng(2)
    x = r.standard_normal((3, 5, 256))
    n = orc.norm_rope(x, np.ones(256), None, 0.0)
    np.testing.assert_allclose((n ** 2).mean(-1), 1.0, rtol=1e-12)
    # rotation: a quarter turn swaps the halves with one sign, dims past 64 stay, lengths are kept
    quarter = np.concatenate([np.zeros((3, 32)), np.ones((3, 32))], 1)
    y = orc.norm_rope(x, None, quarter)
    np.testing.assert_array_equal(y[..., :32], -x[..., 32:64])
    np.testing.assert_array_equal(y[..., 32:64], x[..., :32])
    np.testing.assert_array_equal(y[..., 64:], x[..., 64:])
    # the score of a rotated query and key depends on the difference of their positions only
    ang = np.arange(0, 20)[:, None] * 0.3 ** np.arange(32)[None]
    rows = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    q, k = r.standard_normal((1, 1, 256)), r.standard_normal((1, 1, 256))
    dot = lambda i, j: float((orc.norm_rope(q, None, rows[i:i + 1]) * orc.norm_rope(k, None, rows[j:j + 1])).sum())  # noqa: E731
    assert abs(dot(7, 2) - dot(15, 10)) < 1e-12 and abs(dot(7, 2) - dot(7, 3)) > 1e-6


def test_oracle_four_bits(orc):
    # 0..15 times a step are kept exactly; the ends are kept to the zero's and step's rounding; the error is half a step
    x = np.tile(np.arange(16.0) * 0.25 - 1.0, 16)
    c, s, z, v = orc.kv4(x)
    assert (s == 0.25).all() and (z == -1.0).all()
    np.testing.assert_array_equal(v, x)
    np.testing.assert_array_equal(c, np.tile(np.arange(16), 16).reshape(4, 64))
    x = np.random.default_rng(3).standard_normal((50, 256))
    c, s, z, v = orc.kv4(x)
    assert c.min() == 0 and c.max() == 15
    lim = np.repeat(s * 0.5 + 2 ** -8 * (np.abs(z) + 15 * s), 64, -1).reshape(50, 256)
    assert (np.abs(v - x) <= lim).all()
    assert np.isnan(orc.kv4(np.where(np.arange(256) == 70, np.inf, 1.0))[3][64:128]).all()
    assert (orc.kv4(np.full(256, 2.5))[3] == 2.5).all()


def test_oracle_causal_attention(orc):
    """One new token equals the decode oracle; a prompt equals its tokens one at
    a time; a token before the first position gives zeros."""
    r = np.random.default_rng(4)
    q, k, v, z = r.standard_normal((6, 16, 256)), r.standard_normal((2, 9, 256)), r.standard_normal((2, 9, 256)), r.standard_normal((6, 16, 256))
    got = orc.attn_causal(q, k, v, z, 3)
    for t in range(6):
        one = orc.attn_decode(q[t:t + 1], k[None], v[None], [4 + t], z[t:t + 1])[0]
        np.testing.assert_allclose(got[t], one, rtol=1e-12, atol=1e-14)
    early = orc.attn_causal(q, k, v, z, -2)
    assert not early[:2].any() and early[2].any()


def test_format_helpers_agree_with_the_header():
    from tests import paged_testlib as P
    codes = np.arange(256).reshape(4, 64) % 16
    b = P.row_bytes(codes)
    for g, c, i in ((0, 0, 0), (1, 3, 2), (3, 7, 3)):
        d = 8 * c + 2 * i
        assert b[16 * c + 4 * g + i] == codes[g, d] | (codes[g, d + 1] << 4)
    assert P.pack_records(np.zeros((2, 2, 32, 256))).shape == (2, 2, 4608)

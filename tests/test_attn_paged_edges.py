"""Paged attention at the edges of its formula: values that are not finite right
behind the append that writes them, scores of minus infinity, and weights that
underflow."""
import numpy as np
import pytest
import torch

from tests import append_testlib as A
from tests import paged_testlib as P

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ops():
    from gated_deltanet_linear_02_gb300 import build, ops
    build.build()
    return ops


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("new,ctx", [([20], [20]), ([5, 40], [300, 140])])
def test_attention_reads_what_the_append_before_it_wrote(ops, fmt, new, ctx):
    """The same rows appended in turn with and without infinities, each append followed
    by its attention with no wait between them: every output is that of its own rows."""
    rows = A.Rows(fmt, new, ctx, 16)
    plan, cache = rows.handles(ops)
    every = A.Rows(fmt, ctx, ctx, 16)                          # the contexts, finite
    fill = ops.make_paged_batch(plan._keep_alive[0], plan._keep_alive[1], every.M,
                                torch.tensor(every.cu, dtype=torch.int32, device=DEV), max(ctx))
    params = ops.make_attn_params()
    ops.kv_append(params, fill, cache, A.draw(1, every.M, 2, 256).to(DEV), A.draw(2, every.M, 2, 256).to(DEV))
    k, clean = A.draw(3, rows.M, 2, 256).to(DEV), A.draw(4, rows.M, 2, 256).to(DEV)
    dirty = clean.clone()
    hit = [int(rows.cu[i]) + n // 2 for i, n in enumerate(new)]
    for m in hit:
        dirty[m, 1, 70], dirty[m, 1, 130] = float("inf"), float("nan")
    q = A.draw(5, rows.M, 16, 256).to(DEV)
    ws = torch.empty(ops.attn_paged_workspace_size(plan, cache), dtype=torch.uint8, device=DEV)
    outs = [torch.empty(rows.M, 16, 256, device=DEV) for _ in range(8)]
    for i, out in enumerate(outs):
        ops.kv_append(params, plan, cache, k, dirty if i % 2 else clean)
        ops.attn_paged(plan, cache, q, out, None, ws)
    torch.cuda.synchronize()
    assert ops.device_error() == ops.GDN_OK
    assert torch.isfinite(outs[0]).all()
    see = np.zeros(rows.M, dtype=bool)
    for i, m in enumerate(hit):
        see[m:int(rows.cu[i + 1])] = True
    see = torch.from_numpy(see).to(DEV)
    dims = torch.zeros(256, dtype=torch.bool, device=DEV)
    if fmt == "bf16":
        dims[70] = dims[130] = True
    else:
        dims[64:192] = True                                    # their groups
    spoilt = see[:, None, None] & (torch.arange(16, device=DEV) >= 8)[None, :, None] & dims
    for i, out in enumerate(outs):
        if i % 2 == 0:
            assert torch.equal(out, outs[0])
        else:
            assert not torch.isfinite(out[spoilt]).any() and torch.isfinite(out[~spoilt]).all()
            if fmt == "bf16":                                  # finite rows enter as they are: the same bits
                assert torch.equal(out[~spoilt], outs[0][~spoilt])


def one_context(ops, fmt, L, new, k, v, q, page=64, repeat=1):
    """`new` last tokens of `repeat` sequences over one context of L rows k, v [L][2][256]: outputs [repeat * new][16][256]."""
    rows = A.Rows(fmt, [L], [L], page)
    plan, cache = rows.handles(ops)
    ops.kv_append(ops.make_attn_params(), plan, cache, k.to(DEV), v.to(DEV))
    table = plan._keep_alive[0].repeat(repeat, 1)
    batch = ops.make_paged_batch(table, torch.full((repeat,), L, dtype=torch.int32, device=DEV), new * repeat,
                                 torch.arange(0, new * repeat + 1, new, dtype=torch.int32, device=DEV), new)
    out = torch.full((new * repeat, 16, 256), 7.0, device=DEV)
    ops.attn_paged(batch, cache, q.to(DEV), out)
    torch.cuda.synchronize()
    assert ops.device_error() == ops.GDN_OK
    return out.cpu().double().numpy()


@pytest.mark.parametrize("L,new", [(40, 1), (40, 40), (300, 3), (300, 20), (20000, 1), (20000, 17)])
def test_scores_of_minus_infinity(ops, L, new):
    """Keys whose scores are all -infinity give NaN, as their softmax does (0 / 0), not
    the zeros of a token that sees nothing; beside finite scores they have no weight."""
    k, v, q = A.draw(11, L, 2, 256), A.draw(12, L, 2, 256), A.draw(13, new, 16, 256)
    q[..., 3] = q[..., 3].abs() + 0.5
    low = k.clone()
    low[:, 1, 3] = -float("inf")
    x = one_context(ops, "bf16", L, new, low, v, q)
    assert np.isnan(x[:, 8:]).all() and np.isfinite(x[:, :8]).all()
    some = k.clone()
    first = L - new + 1                                        # what the first token sees
    some[:first // 2, 1, 3] = -float("inf")
    some[first // 2 + 1::3, 1, 3] = -float("inf")
    x = one_context(ops, "bf16", L, new, some, v, q)
    kd, vd, qd = some.double().numpy(), v.double().numpy(), q.double().numpy()
    ref = np.zeros_like(x)
    for t in range(new):
        see = first + t
        for h in range(16):
            with np.errstate(invalid="ignore"):
                s = np.where(np.isinf(kd[:see, h // 8, 3]), -np.inf, np.nan_to_num(kd[:see, h // 8], neginf=0.0) @ qd[t, h] / 16)
            w = np.exp(s - s.max())
            ref[t, h] = (w / w.sum()) @ vd[:see, h // 8]
    # weights rounded to bf16: half a step of the spread and the mean, see paged_testlib
    assert (np.abs(x - ref) <= P.EPS / (1 - P.EPS) * 2 * np.abs(vd).max() + 1e-4 * np.abs(vd).max()).all()


@pytest.mark.parametrize("L,new", [(40, 1), (40, 3), (3000, 1), (3000, 3), (40000, 2)])
def test_scores_that_overflow_to_minus_infinity_over_4_bits(ops, L, new):
    """The same over 4-bit pages, whose keys are finite: scores past fp32 on the negative
    side are no zeros either."""
    k, v, q = A.draw(21, L, 2, 256), A.draw(22, L, 2, 256), A.draw(23, new, 16, 256).abs() + 0.5
    k[:, 1] = -3e38
    x = one_context(ops, "q4", L, new, k, v, q)
    assert np.isnan(x[:, 8:]).all() and np.isfinite(x[:, :8]).all()


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("L,new", [(700, 1), (700, 3), (700, 20), (30000, 1), (30000, 4)])
def test_a_value_that_is_not_finite_stays_when_its_weight_underflows(ops, fmt, L, new):
    """A value row with an infinity and a NaN early in the context, and a key far later
    whose score takes every other weight below fp32: the dims of the row (in 4 bits its
    groups) are not finite, the others are the late row's."""
    k, v, q = A.draw(31, L, 2, 256, scale=0.1), A.draw(32, L, 2, 256), A.draw(33, new, 16, 256)
    q[:] = q[:1, :1]
    v[5, 1, 70], v[5, 1, 200] = float("inf"), float("nan")
    late = L - new - 2
    k[late, 1] = 20 * q[0, 0]                                  # a score of about 300, the others near 0
    repeat = 152 if L == 700 else 8                            # whole contexts in a CTA; cut into pieces
    x = one_context(ops, fmt, L, new, k, v, q.repeat(repeat, 1, 1), repeat=repeat)
    dims = [70, 200] if fmt == "bf16" else list(range(64, 128)) + list(range(192, 256))
    clean = np.setdiff1d(np.arange(256), dims)
    assert not np.isfinite(x[:, 8:, dims]).any()
    assert np.isfinite(x[:, 8:, clean]).all() and np.isfinite(x[:, :8]).all()
    want = v[late, 1].double().numpy()
    step = 0.0 if fmt == "bf16" else (want.max() - want.min()) / 15
    assert (np.abs(x[:, 8:, clean] - want[clean]) <= P.EPS * np.abs(want).max() + step).all()


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("n", [1, 20])
def test_sequences_without_new_tokens_between(ops, fmt, n):
    """65,535 sequences, of which the first, one in the middle and the last have new tokens."""
    B, L, page = 65535, 200, 64
    per = -(-L // page)
    some = [0, 40000, B - 1]
    small = P.make_batch(70, fmt, [n] * 3, [L, 150, 64], page)
    table = torch.full((B, per), -1, dtype=torch.int32)
    ctx, new = torch.full((B,), 77, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    for i, s in enumerate(some):
        table[s, :small.table.shape[1]] = small.table[i]
        ctx[s], new[s] = small.ctx[i], n
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(new, 0)
    cache = ops.make_kv_cache(small.k.to(DEV), None if small.v is None else small.v.to(DEV))
    plan = ops.make_paged_batch(table.to(DEV), ctx.to(DEV), 3 * n, cu.to(DEV), n)
    out = torch.full((3 * n, 16, 256), 7.0, device=DEV)
    ops.attn_paged(plan, cache, small.q.to(DEV), out, small.gate.to(DEV))
    torch.cuda.synchronize()
    assert ops.device_error() == ops.GDN_OK
    P.compare(small, out, P.reference(small), f"{fmt} n {n}")
    kr, vr = (torch.empty(3 * n, 2, 256, device=DEV) for _ in range(2))
    ops.kv_gather(plan, cache, kr, vr)
    for i in range(3):
        k, v = (t[:, -n:].transpose(1, 0, 2) for t in small.kv[i])
        assert np.array_equal(kr[i * n:i * n + n].cpu().numpy(), k.astype(np.float32)) and np.array_equal(vr[i * n:i * n + n].cpu().numpy(), v.astype(np.float32))

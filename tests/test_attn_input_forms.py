"""Norms, rotation and appends on rows that take their kernels' rarer ways: groups
that differ within a row, and token counts on both sides of the choice between a
warp per row and warps that walk over stretches of tokens."""
import numpy as np
import pytest
import torch

from oracle import oracle
from tests import append_testlib as A
from tests import paged_testlib as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
WALK_Q4 = A.FEW_ROWS // 4 + 1     # tokens from which 4-bit appends walk


@pytest.fixture(scope="module")
def ops():
    from gated_deltanet_linear_02_gb300 import build, ops
    build.build()
    return ops


@pytest.mark.parametrize("M", [40, WALK_Q4])
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("how", ["keys", "weight", "rotation"])
def test_append_q4_groups_of_one_row_differ(ops, M, act, how):
    """Normed and rotated key rows with groups of zeros beside others (zeros in the
    keys or in the weight: a narrower head in 256 dims), and with one group all NaN
    (a position's rotation): a group that fp32 settles beside groups that it does not."""
    rows = A.Rows("q4", [M - 7, 7], [M - 7, 30], 32, pad_rows=2)
    kv = A.draw(71, rows.M, 4, 256, dtype=act)
    kw = 1 + A.draw(72, 256, dtype=torch.float32, scale=0.2)
    table = P.rope_table(M)
    k, v = kv[:, :2].clone(), kv[:, 2:]
    if how == "keys":
        for i, groups in enumerate([(1,), (2, 3), (0,), (1, 2, 3), (0, 1, 2, 3)]):
            for g in groups:
                k[i::7, :, 64 * g:64 * g + 64] = 0
    elif how == "weight":
        kw[128:] = 0
    else:
        table[3::5] = float("nan")
    params = ops.make_attn_params(None, kw.to(DEV), table.to(DEV))
    plan, cache = rows.handles(ops)
    d = k.to(DEV), v.to(DEV)
    ops.kv_append(params, plan, cache, *d)
    torch.cuda.synchronize()
    kk = oracle.norm_rope(k.double(), kw, table[np.maximum(rows.pos, 0)])
    A.check_q4(rows, cache._keep_alive[0], kk, v.double().numpy(), how)


def close(got, ref, label, sharp=2e-6):
    """fp32 arithmetic within `sharp` of the row's largest partner (mean of squares, root,
    two products, three roundings of the rotation: below 8e-7), half a step of the output.
    Below the normal numbers a rounding is off by half of the smallest step instead, 2^-150
    in fp32: the first product's counts w < 2 times and each of the first two |c| + |s| <=
    1.5 times, then come the rotation's two: (3 + 1.5 + 2) 2^-150 < 4 2^-149. In bf16 it is
    2^-134 at the end."""
    tol = sharp * np.abs(ref).max(-1, keepdims=True) * np.sqrt(2) + 4 * 2.0 ** -149
    if got.dtype == torch.bfloat16:
        tol = tol + np.maximum(P.EPS * (np.abs(ref) + tol), 2.0 ** -134)
    err = np.abs(got.cpu().double().numpy() - ref)
    assert (err <= tol).all(), f"{label}: {(err / tol).max():.2f} times the bound"


FAR = [1e-44, 1e-38, 1e-30, 1e-23, 3e-21, 1e-15, 1.0, 1e13, 1e14, 3e18, 1e25, 5e37]


@pytest.mark.parametrize("M", [len(FAR) * 4, len(FAR) * 305])
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("eps", [0.0, 1e-36, 1e-6])
def test_norms_of_rows_of_any_magnitude(ops, M, act, eps):
    """Rows whose squares leave fp32 on either side, for norms, appends in bf16 and the
    4-bit append, whose codes stay the definition's."""
    scale = torch.tensor(FAR).repeat(M // len(FAR))[:, None, None].double()
    big = lambda seed, heads: (A.draw(seed, M, heads, 256, dtype=torch.float32).double().clamp(-6, 6) * scale).to(act)  # noqa: E731
    q, k, v = big(81, 16), big(82, 2), A.draw(83, M, 2, 256, dtype=act)
    if eps == 0.0:                                     # no row of zeros, whose norm is 0 / 0
        tiny = 2.0 ** -133 if act == torch.bfloat16 else 2.0 ** -149
        q[..., 5], k[..., 5] = q[..., 5].clamp(min=tiny), k[..., 5].clamp(min=tiny)
    w, table = (1 + A.draw(84, 256, dtype=torch.float32, scale=0.2)).clamp(max=1.99), P.rope_table(M)
    pos = torch.arange(M, dtype=torch.int32)
    params = ops.make_attn_params(w.to(DEV), w.to(DEV), table.to(DEV), eps)
    qo, ko = torch.empty(M, 16, 256, device=DEV), torch.empty(M, 2, 256, device=DEV)
    ops.attn_qk_norm_rope(params, q.to(DEV), pos.to(DEV), qo, k.to(DEV), ko)
    kk = oracle.norm_rope(k.double(), w, table, eps)
    close(qo, oracle.norm_rope(q.double(), w, table, eps), "q")
    close(ko, kk, "k")
    for fmt in ("bf16", "q4"):
        rows = A.Rows(fmt, [M], [M], 64)
        plan, cache = rows.handles(ops)
        ops.kv_append(params, plan, cache, k.to(DEV), v.to(DEV))
        if fmt == "q4":
            A.check_q4(rows, cache._keep_alive[0], kk, v.double().numpy())
        else:
            close(cache._keep_alive[0].cpu()[rows.page_id, :, rows.off], kk, "cached k")


# ---- both sides of the choice between a warp per row and warps that walk over tokens

def sides(rows_per_token, limit=A.FEW_ROWS):
    return [limit // rows_per_token, limit // rows_per_token + 1]


@pytest.mark.parametrize("M", sides(18) + [4099])
@pytest.mark.parametrize("act,out", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                     (torch.float32, torch.bfloat16), (torch.float32, torch.float32)])
def test_norm_rope_of_many_tokens(ops, M, act, out):
    """Strided queries and keys, positions in any order, and padding among them, which
    is left as it is; queries alone, and keys without a weight."""
    n_pos = 3000
    joint, kv = A.draw(M, M, 16, 2, 256, dtype=act), A.draw(M + 1, M, 6, 256, dtype=act)
    q, k = joint[:, :, 0], kv[:, 1:3]
    qw, kw = 1 + A.draw(3, 256, dtype=torch.float32, scale=0.2), 1 + A.draw(4, 256, dtype=torch.float32, scale=0.2)
    table = P.rope_table(n_pos)
    pos = torch.randint(0, n_pos, (M,), generator=torch.Generator().manual_seed(M), dtype=torch.int32)
    pos[::97], pos[5::131] = -1, n_pos
    live = ((pos >= 0) & (pos < n_pos)).numpy()
    rows = table[pos.clamp(0, n_pos - 1).long()]
    d = joint.to(DEV)[:, :, 0], kv.to(DEV)[:, 1:3]
    for kweight in (kw, None):
        p = ops.make_attn_params(qw.to(DEV), None if kweight is None else kweight.to(DEV), table.to(DEV))
        qo, ko = (torch.full((M, heads, 256), 7.0, dtype=out, device=DEV) for heads in (16, 2))
        ops.attn_qk_norm_rope(p, d[0], pos.to(DEV), qo, d[1], ko)
        for got, want in ((qo, oracle.norm_rope(q.double(), qw, rows)), (ko, oracle.norm_rope(k.double(), kweight, rows))):
            close(got[live], want[live], "norm")
            assert (got[~live] == 7.0).all()
    alone = torch.full_like(qo, 7.0)
    ops.attn_qk_norm_rope(p, d[0], pos.to(DEV), alone)
    close(alone[live], oracle.norm_rope(q.double(), qw, rows)[live], "queries alone")


@pytest.mark.parametrize("M", sides(18) + [4099])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm_rope_of_many_tokens_in_place(ops, M, dtype):
    """Dense in place, with rows that leave fp32's squares (done apart) among the others,
    and a weight whose outputs would do so again."""
    q, k = A.draw(M, M, 16, 256, dtype=dtype), A.draw(M + 1, M, 2, 256, dtype=dtype)
    q[7::50, 3] *= 2.0 ** 70
    k[9::40] *= 2.0 ** 65
    w, table = 1 + A.draw(3, 256, dtype=torch.float32, scale=0.2), P.rope_table(M)
    for scale in (1.0, 2.0 ** -60):
        p = ops.make_attn_params((w * scale).to(DEV), (w * scale).to(DEV), table.to(DEV))
        x, y = q.to(DEV).clone(), k.to(DEV).clone()
        ops.attn_qk_norm_rope(p, x, torch.arange(M, dtype=torch.int32, device=DEV), x, y, y)
        close(x, oracle.norm_rope(q.double(), w * scale, table), "q in place")
        close(y, oracle.norm_rope(k.double(), w * scale, table), "k in place")


def ragged(M):
    """M packed rows: prompts, a sequence without tokens, single tokens, one whose context is
    shorter than its new tokens (the first ones have no position), then padding."""
    new = [M - 220, 0, 1, 150, 1, 60]
    return new, [M + 100, 40, 33, 90, 1, 800]


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("M,queries", [(m, True) for m in sides(20)] + [(m, False) for m in sides(4, A.FEW_ROWS_BF16)] + [(2500, True)])
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("own_positions", [False, True])
def test_append_bf16_of_many_tokens(ops, page, M, queries, act, own_positions):
    """Keys, values and queries of ragged sequences; a page id outside the cache, given
    positions outside the table: those rows are dropped, and nothing else changes."""
    new, ctx = ragged(M)
    rows = A.Rows("bf16", new, ctx, page, pad_rows=8, seed=M)
    rows.table[0, 1] = 1 << 29
    rows.page_id[(rows.seq == 0) & (rows.pos // page == 1)] = -1
    n_pos = max(ctx) + 1
    kw, table = 1 + A.draw(4, 256, dtype=torch.float32, scale=0.2), P.rope_table(n_pos)
    kv, q = A.draw(M, rows.M, 4, 256, dtype=act), A.draw(M + 1, rows.M, 16, 256, dtype=act)
    at = rows.pos.copy()
    given = None
    if own_positions:
        given = torch.randint(0, n_pos, (rows.M,), generator=torch.Generator().manual_seed(M), dtype=torch.int32)
        given[::61] = n_pos + 5
        at = given.numpy().astype(np.int64)
        rows.page_id[(at < 0) | (at >= n_pos)] = -1
        given = given.to(DEV)
    params = ops.make_attn_params((kw * 2).to(DEV), kw.to(DEV), table.to(DEV))
    plan, cache = rows.handles(ops)
    d, qo = kv.to(DEV), torch.full((rows.M, 16, 256), 7.0, dtype=torch.bfloat16, device=DEV)
    ops.kv_append(params, plan, cache, d[:, :2], d[:, 2:], q.to(DEV) if queries else None, qo if queries else None, given)
    s = rows.stored()
    turn = table[torch.from_numpy(np.clip(at, 0, n_pos - 1))]
    gk, gv = (t.cpu() for t in cache._keep_alive)
    close(gk[rows.page_id[s], :, rows.off[s]], oracle.norm_rope(kv[:, :2].double(), kw, turn)[s], "keys")
    assert torch.equal(gv[rows.page_id[s], :, rows.off[s]], kv[s, 2:].to(torch.bfloat16))
    for t in (gk, gv):
        t[rows.page_id[s], :, rows.off[s]] = 3.0
        assert (t == 3.0).all(), "a row that is no new token's changed"
    if queries:
        live = (rows.seq >= 0) & (at >= 0) & (at < n_pos)
        close(qo[live], oracle.norm_rope(q.double(), kw * 2, turn)[live], "queries")
        assert (qo[~live] == 7.0).all()


@pytest.mark.parametrize("M,queries", [(m, True) for m in sides(20)] + [(m, False) for m in sides(4)])
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
def test_append_q4_of_many_tokens(ops, M, queries, act):
    """The definition bit for bit, normed and rotated, over ragged sequences and padding;
    bf16 queries in place."""
    new, ctx = ragged(M)
    rows = A.Rows("q4", new, ctx, 32, pad_rows=8, seed=M)
    kw, table = 1 + A.draw(4, 256, dtype=torch.float32, scale=0.2), P.rope_table(max(ctx) + 1)
    kv, q = A.draw(M, rows.M, 4, 256, dtype=act), A.draw(M + 1, rows.M, 16, 256, dtype=act)
    params = ops.make_attn_params((kw * 2).to(DEV), kw.to(DEV), table.to(DEV))
    plan, cache = rows.handles(ops)
    d, x = kv.to(DEV), q.to(DEV).clone()
    qo = x if act == torch.bfloat16 else torch.zeros(rows.M, 16, 256, dtype=torch.bfloat16, device=DEV)
    ops.kv_append(params, plan, cache, d[:, :2], d[:, 2:], x if queries else None, qo if queries else None)
    turn = table[torch.from_numpy(np.clip(rows.pos, 0, max(ctx)))]
    A.check_q4(rows, cache._keep_alive[0], oracle.norm_rope(kv[:, :2].double(), kw, turn), kv[:, 2:].double().numpy())
    if queries:
        live = (rows.seq >= 0) & (rows.pos >= 0)
        close(qo[live], oracle.norm_rope(q.double(), kw * 2, turn)[live], "queries")
        assert torch.equal(qo[~live].cpu(), q[~live].to(torch.bfloat16) if act == torch.bfloat16 else torch.zeros_like(qo[~live].cpu()))


@pytest.mark.parametrize("M", [8, WALK_Q4])
def test_append_q4_rotated_keys_below_the_normal_numbers(ops, M):
    """A rotated group that is constant in fp32 and whose least value lies half a bf16 step
    and a little from 0: the little decides its zero."""
    rows = A.Rows("q4", [M], [M], 32)
    k, v = torch.zeros(M, 2, 256), A.draw(91, M, 2, 256, dtype=torch.float32)
    k[..., :64] = -2.0 ** -134
    k[1::2, :, :64] = 2.0 ** -134
    k[2::3, :, 64:128] = 2.0 ** -134                # not rotated: exact
    table = torch.cat([torch.ones(M, 32), torch.full((M, 32), 2.0 ** -17)], 1)
    plan, cache = rows.handles(ops)
    ops.kv_append(ops.make_attn_params(None, None, table.to(DEV)), plan, cache, k.to(DEV), v.to(DEV))
    A.check_q4(rows, cache._keep_alive[0], oracle.norm_rope(k.double(), None, table), v.double().numpy())

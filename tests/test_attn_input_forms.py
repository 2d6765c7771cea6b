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

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

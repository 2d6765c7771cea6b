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

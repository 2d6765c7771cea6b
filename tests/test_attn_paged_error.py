"""The paged attention's error as a norm (error_testlib), where the bounds of single
elements grow wider than the outputs: long contexts, and every kernel's own tests."""
import numpy as np
import pytest
import torch

from tests import append_testlib as A
from tests import error_testlib as E

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ops():
    from gated_deltanet_linear_02_gb300 import build, ops
    build.build()
    return ops


def shared_context(ops, fmt, L, page, k, v):
    """One context of L rows in pages of a cache, and the values that it holds (fp64 [2][L][256])."""
    per = -(-L // page)
    table = torch.randperm(per, generator=torch.Generator().manual_seed(L)).to(torch.int32).to(DEV)[None]
    cache = ops.make_kv_cache(*(torch.zeros(per, 2, page, 256, dtype=torch.bfloat16, device=DEV) for _ in range(2))) \
        if fmt == "bf16" else ops.make_kv_cache(torch.zeros(per, 2, page // 16, 4608, dtype=torch.uint8, device=DEV))
    one = ops.make_paged_batch(table, torch.tensor([L], dtype=torch.int32, device=DEV), L,
                               torch.tensor([0, L], dtype=torch.int32, device=DEV), L)
    ops.kv_append(ops.make_attn_params(), one, cache, k, v)
    kr, vr = (torch.empty(L, 2, 256, device=DEV) for _ in range(2))
    ops.kv_gather(one, cache, kr, vr)
    return table, cache, kr.double().transpose(0, 1), vr.double().transpose(0, 1)


@pytest.mark.parametrize("fmt,new", [("q4", 1), ("q4", 2), ("q4", 3), ("bf16", 1), ("bf16", 16)])
@pytest.mark.parametrize("L,how", [(4096, "random"), (16385, "random"), (65536, "random"), (65536, "half"), (65536, "even"), (65536, "one")])
def test_error_does_not_grow_with_the_context(ops, fmt, new, L, how):
    """152 sequences over one long context, so that one CTA goes through all of it: a
    sum over tens of thousands of positions keeps the error of a short one. 'half',
    'even' and 'one': the first eight, every second or the first of every 16 positions
    have nearly all the weight."""
    B, page = 152, 64
    q = A.draw(L + new, B * new, 16, 256).to(DEV)
    k, v = A.draw(L, L, 2, 256).to(DEV), A.draw(L + 1, L, 2, 256).to(DEV)
    if how != "random":
        q[:] = A.draw(77, 256).to(DEV)
        at = torch.arange(L, device=DEV) % 16
        k[(at >= 8) if how == "half" else (at % 2 == 1) if how == "even" else (at > 0)] = -0.5 * q[0, 0]   # scores near -8
    table, cache, kd, vd = shared_context(ops, fmt, L, page, k, v)
    plan = ops.make_paged_batch(table.repeat(B, 1), torch.full((B,), L, dtype=torch.int32, device=DEV), B * new,
                                torch.arange(0, (B + 1) * new, new, dtype=torch.int32, device=DEV) if new > 1 else None, new)
    out = torch.empty(B * new, 16, 256, device=DEV)
    ops.attn_paged(plan, cache, q, out)
    torch.cuda.synchronize()
    assert ops.device_error() == ops.GDN_OK
    got, ref = [], []
    for b in range(0, B, 38):                                   
        for m in {b * new, b * new + new - 1}:
            see = L - new + m % new + 1
            for h in range(2):
                w = torch.softmax(q[m, 8 * h:8 * h + 8].double() @ kd[h, :see].T / 16, -1)
                ref.append((w @ vd[h, :see]).cpu().numpy())
                got.append(out[m, 8 * h:8 * h + 8].cpu().double().numpy())
    err = E.relative(np.stack(got), np.stack(ref))
    print(f"{fmt} new {new} L {L} {how}: {err:.2e}")
    assert err <= E.bound(fmt == "q4", new, torch.float32), err

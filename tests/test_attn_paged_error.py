"""The paged attention's error as a norm (error_testlib), where the bounds of single
elements grow wider than the outputs: long contexts, and every kernel's own tests."""
import numpy as np
import pytest
import torch

from oracle import oracle
from tests import append_testlib as A
from tests import error_testlib as E
from tests import paged_testlib as P

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


def attend64(q, kd, vd, L, new, tokens):
    """The outputs of some packed rows, whose sequences have `new` tokens each at the end of one context."""
    ref = []
    for m in tokens:
        see = L - new + m % new + 1
        ref.append(torch.cat([torch.softmax(q[m, 8 * h:8 * h + 8].double() @ kd[h, :see].T / 16, -1) @ vd[h, :see]
                              for h in range(2)]))
    return torch.stack(ref).cpu().numpy()


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


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("new", [1, 2, 3, 16, 40])
@pytest.mark.parametrize("L", [20001, 70001])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_a_context_cut_into_pieces(ops, fmt, new, L, out_dtype):
    """One long context, whose items' pieces lie in many CTAs and are joined, every token."""
    q = A.draw(L + new, new, 16, 256).to(DEV)
    table, cache, kd, vd = shared_context(ops, fmt, L, 64, A.draw(L, L, 2, 256).to(DEV), A.draw(L + 1, L, 2, 256).to(DEV))
    plan = ops.make_paged_batch(table, torch.tensor([L], dtype=torch.int32, device=DEV), new,
                                torch.tensor([0, new], dtype=torch.int32, device=DEV), new)
    out = torch.empty(new, 16, 256, dtype=out_dtype, device=DEV)
    ops.attn_paged(plan, cache, q, out)
    torch.cuda.synchronize()
    assert ops.device_error() == ops.GDN_OK
    ref = attend64(q, kd, vd, L, new, range(new))
    for m in range(new):                                          # token by token: no item is wrong alone
        assert E.relative(out[m], ref[m]) <= E.bound(fmt == "q4", new, out_dtype)


def run(ops, b, out_dtype=torch.float32, one_token=False):
    plan, cache = P.handles(ops, b, one_token=one_token)
    out = torch.full((b.q.shape[0], 16, 256), 7.0, dtype=out_dtype, device=DEV)
    ops.attn_paged(plan, cache, b.q.to(DEV), out, b.gate.to(DEV))
    torch.cuda.synchronize()
    assert ops.device_error() == ops.GDN_OK
    return out


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("new,ctx", E.BATCHES)
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_batches_and_prompts(ops, fmt, new, ctx, out_dtype):
    b = P.make_batch(400, fmt, new, ctx, 32, pad_rows=2)
    out = run(ops, b, out_dtype, one_token=max(new) == 1)
    ref = P.reference(b)
    P.compare(b, out, ref, f"{fmt} new {new} ctx {ctx}")
    for i, n in enumerate(new):
        if n > 0 and ctx[i] >= 100:
            err = E.relative(out[int(b.cu[i]):int(b.cu[i]) + n], ref[i][0])
            assert err <= E.bound(fmt == "q4", max(new), out_dtype), (i, err)
    assert (out[-2:] == 7.0).all()


# ---- single tokens over 4-bit pages, whose kernel is its own

def single_bound(b, i):
    """E.bound, and what the scores may be off by: a group's 64 products are summed with 1,024 q in
    four instructions, each truncated to 2^-23 of the largest sum, 1,040 sum |q| at most. So a score
    is off by 4 * 4 * 2^-23 * 1,040 max sum |q| s / 16 and its weight by twice that, relative."""
    q = np.abs(b.q[i].double().numpy()).reshape(16, 4, 64).sum(-1).max()
    k = b.kv[i][0].reshape(2, -1, 4, 64)
    step = 1.01 * (k.max(-1) - k.min(-1)).max() / 15
    return E.bound(True, 1, torch.float32) + np.expm1(2 * 2.0 ** -23 * 1040 * q * step)


@pytest.mark.parametrize("sharp", [0.01, 3.0, 30.0])
@pytest.mark.parametrize("ctx", [[700, 150, 2, 1], [4097]])
def test_single_tokens_over_4_bits_sharp_and_flat_scores(ops, sharp, ctx):
    b = P.make_batch(501, "q4", [1] * len(ctx), ctx, 16, sharp=sharp)
    out = run(ops, b, one_token=True)
    ref = P.reference(b)
    for i in range(len(ctx)):
        assert E.relative(out[i], ref[i][0][0]) <= single_bound(b, i)


@pytest.mark.parametrize("scales", [(1e-7,), (1e-3,), (3e4, 1e5), (1e20,), (1.0, 1e6, 1e-4), (0.0, 1.0)])
@pytest.mark.parametrize("ctx", [[130, 700], [1300], [30]])
def test_single_tokens_over_4_bits_values_of_any_magnitude(ops, scales, ctx):
    b = P.make_batch(800, "q4", [1] * len(ctx), ctx, 32, pad_rows=1)
    for i, c in enumerate(ctx):
        k, v = b.kv[i]
        codes, steps, zeros, v = oracle.kv4((v * np.array(scales)[np.arange(c) // 150 % len(scales)][:, None]).astype(np.float32))
        for p in range(c):
            rec = b.k[int(b.table[i, p // 32]), :, p % 32 // 16].numpy()
            r = p % 16
            rec[:, 2048 + 128 * r:2176 + 128 * r] = P.row_bytes(codes[:, p])
            rec[:, 4352 + 16 * r:4368 + 16 * r] = P.bf16_bytes(np.stack([steps[:, p], zeros[:, p]], -1)).reshape(2, 16)
        b.kv[i] = (k, v)
    out, ref = run(ops, b, one_token=False), P.reference(b)
    P.compare(b, out, ref, f"scales {scales}")
    for i, c in enumerate(ctx):
        if ref[i][0].any() and c >= 100:
            assert E.relative(out[i], ref[i][0][0]) <= E.bound(True, 1, torch.float32)


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("new,ctx", [([1, 1, 1], [300, 17, 5000]), ([2, 1, 2], [40, 1, 300])])
def test_single_tokens_over_4_bits_values_that_are_not_finite(ops, page, new, ctx):
    """A NaN group in a value row: its dims are NaN for the tokens that see it. A NaN key in
    the last row: all of its head for the last token. Everything else as without them."""
    b = P.make_batch(510 + page, "q4", new, ctx, page, pad_rows=1)
    ref = P.reference(b)
    for i, n in enumerate(new):
        last = ctx[i] - 1
        pg, off = int(b.table[i, last // page]), last % page
        rec = b.k[pg, 1, off // 16].numpy()
        rec[4352 + 16 * (off % 16) + 4:4352 + 16 * (off % 16) + 8] = 0xFF     # the last row: group 1's step and zero
        b.k[pg, 0, off // 16].numpy()[4096 + 16 * (off % 16):4096 + 16 * (off % 16) + 4] = 0xFF
    got = run(ops, b).cpu().double().numpy()
    for i, n in enumerate(new):
        x, (r, tol) = got[int(b.cu[i]):int(b.cu[i]) + n], ref[i]
        assert np.isnan(x[n - 1, :8]).all() and np.isnan(x[n - 1, 8:, 64:128]).all()
        clean = np.ones_like(x, dtype=bool)
        clean[n - 1, :8] = clean[n - 1, 8:, 64:128] = False
        assert np.isfinite(x[clean]).all() and (np.abs(x - r)[clean] <= tol[clean]).all()

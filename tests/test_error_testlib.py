"""The error norm's bound finds the mistakes that matter, in the reference's own arithmetic."""
import numpy as np
import pytest
import torch

from oracle import oracle
from tests import error_testlib as E
from tests import paged_testlib as P


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("new,ctx", E.BATCHES)
def test_the_bound_tells_a_wrong_result_from_a_rounded_one(fmt, new, ctx):
    """Values and keys rounded to bf16, or the weights, stay inside; zeros, a
    half of the context left out, two tiles of values swapped and one tile's keys shifted by
    a row do not."""
    b = P.make_batch(400, fmt, new, ctx, 32)
    for i, n in enumerate(new):
        L = ctx[i]
        if n == 0 or L < 100:
            continue
        n0 = min(n, 24)                                # the last tokens, which see nearly all of it
        m = int(b.cu[i]) + n
        q, (k, v), first = b.q[m - n0:m].double().numpy(), b.kv[i], L - n0
        ref = oracle.attn_causal(q, k, v, None, first)
        limit = E.bound(fmt == "q4", max(new), torch.float32)
        assert E.relative(0 * ref, ref) > 100 * limit
        assert E.relative(oracle.attn_causal(q, k[:, L // 2:], v[:, L // 2:], None, first - L // 2), ref) > 20 * limit
        tile = np.arange(L)
        if L >= 256:
            tile[:256] = (tile[:256] + 128) % 256
            assert E.relative(oracle.attn_causal(q, k, v[:, tile], None, first), ref) > 20 * limit
        row = np.arange(L)
        row[:64] = np.roll(row[:64], 1)
        assert E.relative(oracle.attn_causal(q, k[:, row], v, None, first), ref) > 10 * limit
        if fmt == "q4" and max(new) > 2:
            assert E.relative(oracle.attn_causal(q, oracle.bf16_of(k), oracle.bf16_of(v), None, first), ref) <= limit
        else:                                          # weights rounded, their sum not
            scores = np.einsum("thd,hld->thl", q, k.repeat(8, 0)) / 16
            scores = np.where(np.arange(L) <= (first + np.arange(n0))[:, None, None], scores, -np.inf)
            w = np.exp(scores - scores.max(-1, keepdims=True))
            w = oracle.bf16_of(w) / w.sum(-1, keepdims=True)
            assert E.relative(np.einsum("thl,hld->thd", w, v.repeat(8, 0)), ref) <= limit

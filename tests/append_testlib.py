"""Helpers of the append tests that need many rows: batches without a reference
attention, and the 4-bit records of whole batches compared at once."""
from __future__ import annotations

import numpy as np
import torch

from oracle import oracle
from tests import paged_testlib as P

# rows (tokens x heads) above which the appends and norms walk over stretches of tokens
FEW_ROWS = 2 * 152 * 48
FEW_ROWS_BF16 = 2048              # keys and values alone into bf16 pages


def draw(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


class Rows:
    """Sequences with `new` tokens each on contexts `ctx`, in pages that hold a
    pattern; `seq`, `pos`, `page_id` and `off` of every packed row (padding: -1)."""

    def __init__(self, fmt, new, ctx, page, pad_rows=0, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.new, self.ctx, self.page, self.fmt = list(new), list(ctx), page, fmt
        per = max(1, -(-max(max(ctx), 1) // page))
        pages = len(new) * per + 2
        self.table = torch.randperm(pages, generator=g)[:len(new) * per].view(len(new), per).to(torch.int32)
        self.cu = np.concatenate([[0], np.cumsum(new)])
        self.M = int(self.cu[-1]) + pad_rows
        self.shape = (pages, 2, page, 256) if fmt == "bf16" else (pages, 2, page // 16, 4608)
        self.seq, self.pos = np.full(self.M, -1), np.full(self.M, -1)
        for i, n in enumerate(new):
            self.seq[self.cu[i]:self.cu[i + 1]] = i
            self.pos[self.cu[i]:self.cu[i + 1]] = np.arange(ctx[i] - n, ctx[i])
        ok = (self.seq >= 0) & (self.pos >= 0) & (self.pos // page < per)
        self.page_id = np.where(ok, self.table.numpy()[np.maximum(self.seq, 0), np.where(ok, self.pos // page, 0)], -1)
        self.off = self.pos % page

    def stored(self):
        """Packed rows that have a place in the cache."""
        return np.flatnonzero(self.page_id >= 0)

    def handles(self, ops, dev="cuda", one_token=False):
        if self.fmt == "bf16":
            cache = ops.make_kv_cache(*(torch.full(self.shape, 3.0, dtype=torch.bfloat16, device=dev) for _ in range(2)))
        else:
            cache = ops.make_kv_cache(torch.full(self.shape, 0xFF, dtype=torch.uint8, device=dev))
        plan = ops.make_paged_batch(self.table.to(dev), torch.tensor(self.ctx, dtype=torch.int32, device=dev), self.M,
                                    None if one_token else torch.tensor(self.cu, dtype=torch.int32, device=dev),
                                    1 if one_token else max(max(self.new), 1))
        return plan, cache


def check_q4(rows: Rows, records: torch.Tensor, k, v, label=""):
    """The records of the stored rows are the definition's for the fp64 keys and
    values k, v [M][2][256]: codes and steps bit for bit, zeros as values (a zero's
    sign is free); groups that hold a NaN or an infinity are NaN, with codes of 0. Nothing else changed."""
    at = rows.stored()
    rec = records.cpu().numpy()
    lines = rec[rows.page_id[at], :, rows.off[at] // 16]               # [n][2][4608]
    r = rows.off[at] % 16
    touched = np.zeros(rec.shape, dtype=bool)
    for code0, sz0, x in ((0, 4096, k), (2048, 4352, v)):
        c, s, z, val = oracle.kv4(np.asarray(x)[at])
        ci, si = (code0 + r * 128)[:, None] + np.arange(128), (sz0 + r * 16)[:, None] + np.arange(16)
        got_c = np.take_along_axis(lines, ci[:, None, :].repeat(2, 1), -1)
        got_s = np.ascontiguousarray(np.take_along_axis(lines, si[:, None, :].repeat(2, 1), -1))
        sz = torch.from_numpy(got_s).view(torch.bfloat16).double().numpy().reshape(len(at), 2, 4, 2)
        bad = np.isnan(val.reshape(len(at), 2, 4, 64)).any(-1)
        want = np.where(bad[..., None], 0.0, c)
        np.testing.assert_array_equal(got_c, P.row_bytes(want), err_msg=label + " codes")
        np.testing.assert_array_equal(sz[..., 0][~bad], s[~bad], err_msg=label + " steps")
        np.testing.assert_array_equal(sz[..., 1][~bad], z[~bad], err_msg=label + " zeros")
        assert np.isnan(sz[bad].sum(-1)).all(), label
        for h in range(2):
            touched[rows.page_id[at][:, None], h, (rows.off[at] // 16)[:, None], ci] = True
            touched[rows.page_id[at][:, None], h, (rows.off[at] // 16)[:, None], si] = True
    assert (rec[~touched] == 0xFF).all(), f"{label}: bytes of other rows changed"

"""Shared helpers of the paged-cache tests: seeded batches of sequences with
their caches in either format (packed here, independently of the library), the
fp64 reference, and the error bound of the attention."""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch

from oracle import oracle

HQ, HKV, D = 16, 2, 256
REC_BYTES = 4608


def rope_table(n_pos: int, base: float = 1e7) -> torch.Tensor:
    ang = torch.arange(n_pos, dtype=torch.float64)[:, None] * base ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def bf16_bytes(x: np.ndarray) -> np.ndarray:
    """fp64 values that are bf16 numbers -> their 2 bytes each."""
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).view(torch.uint8).numpy().reshape(*x.shape, 2)


def row_bytes(codes: np.ndarray) -> np.ndarray:
    """[..][4][64] codes -> [..][128] bytes in the format's order."""
    c = codes.astype(np.uint8).reshape(*codes.shape[:-2], 4, 8, 4, 2)
    b = c[..., 0] | (c[..., 1] << 4)                       # [.., g, c, b]
    return np.swapaxes(b, -3, -2).reshape(*codes.shape[:-2], 128)


def pack_records(kv: np.ndarray) -> np.ndarray:
    """Rows kv [2 (k, v)][..][R][256] -> records [..][R / 16][4608]."""
    parts, szs = [], []
    for t in kv:
        c, s, z, _ = oracle.kv4(t)
        lead = t.shape[:-2]
        parts.append(row_bytes(c).reshape(*lead, -1, 16 * 128))
        szs.append(bf16_bytes(np.stack([s, z], -1)).reshape(*lead, -1, 16 * 16))
    return np.concatenate([*parts, *szs], -1)


@dataclass
class Batch:
    q: torch.Tensor            # [M][16][256] bf16
    gate: torch.Tensor         # [M][16][256] bf16
    table: torch.Tensor        # [B][max_pages] int32
    ctx: torch.Tensor          # [B] int32
    cu: torch.Tensor           # [B+1] int32
    k: torch.Tensor            # caches
    v: torch.Tensor | None
    kv: list                   # per sequence (k, v) values [2][ctx][256] fp64
    new: list
    page: int


def make_batch(seed: int, fmt: str, new, ctx, page: int, pad_rows: int = 0, spare: int = 2, sharp: float = 1.0) -> Batch:
    """Sequences with `new` tokens on contexts `ctx` (a context may be shorter
    than its new tokens: the first ones then see nothing). Rows past a context
    and unused pages hold NaN."""
    g = torch.Generator().manual_seed(seed)
    B, M = len(ctx), sum(new) + pad_rows
    per = max(1, -(-max(max(ctx), 1) // page))
    pages = B * per + spare
    table = torch.randperm(pages, generator=g)[:B * per].view(B, per).to(torch.int32)
    k = torch.full((pages, HKV, page, D), float("nan"))
    v = torch.full((pages, HKV, page, D), float("nan"))
    kv = []
    for b in range(B):
        L = max(ctx[b], 0)
        kb = (torch.randn(HKV, L, D, generator=g) * sharp).to(torch.bfloat16).float()
        vb = torch.randn(HKV, L, D, generator=g).to(torch.bfloat16).float()
        kv.append((kb.double().numpy(), vb.double().numpy()))
        for p in range(-(-L // page)):
            n = min(page, L - p * page)
            k[table[b, p], :, :n] = kb[:, p * page:p * page + n]
            v[table[b, p], :, :n] = vb[:, p * page:p * page + n]
    if fmt == "bf16":
        kc, vc = k.to(torch.bfloat16), v.to(torch.bfloat16)
    else:
        rec = pack_records(np.stack([k.double().numpy(), v.double().numpy()]))
        kc, vc = torch.from_numpy(np.ascontiguousarray(rec)), None
        kv = [tuple(oracle.kv4(t)[3] if t.size else t for t in both) for both in kv]
    q = torch.randn(M, HQ, D, generator=g).to(torch.bfloat16)
    gate = torch.randn(M, HQ, D, generator=g).to(torch.bfloat16)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return Batch(q, gate, table, torch.tensor(ctx, dtype=torch.int32), torch.tensor(cu, dtype=torch.int32), kc, vc, kv,
                 list(new), page)


def handles(ops, b: Batch, dev="cuda", one_token=False):
    """The batch's tensors on the device, and its library handles."""
    t = lambda x: None if x is None else x.to(dev)  # noqa: E731
    cache = ops.make_kv_cache(t(b.k), t(b.v))
    plan = ops.make_paged_batch(t(b.table), t(b.ctx), b.q.shape[0], None if one_token else t(b.cu), max(max(b.new), 1))
    return plan, cache


def reference(b: Batch, seqs=None, gate=True):
    """{sequence: (fp64 output [n][16][256], bound without the output rounding)}."""
    out = {}
    for i in range(len(b.new)) if seqs is None else seqs:
        m0, n = int(b.cu[i]), b.new[i]
        k, v = b.kv[i]
        q = b.q[m0:m0 + n].double().numpy()
        z = b.gate[m0:m0 + n].double().numpy() if gate else None
        first = int(b.ctx[i]) - n
        ref = oracle.attn_causal(q, k, v, None, first)
        sig = 1.0 / (1.0 + np.exp(-z)) if gate else 1.0
        out[i] = (ref * sig, _bound(b, q, k, v, ref, first) * sig)
    return out


EPS = 2.0 ** -8            # half a step of bf16, relative


def _bound(b: Batch, q, k, v, o, first):
    """Error bound of the ungated outputs o, per element.

    bf16 cache: the softmax weights enter the value product rounded to bf16
    (relative 2^-8), normalised by the sum of either the rounded or the exact
    weights: |o' - o| <= 2^-8 / (1 - 2^-8) * (max_p |v_p - o| + |o|).
    4-bit cache, one token: the weights times the step of each group are rounded
    instead, and multiply v - z >= 0, at most the group's range: the same factor
    times the largest range among the visible rows. More tokens: the cached
    values enter rounded to bf16: |v| 2^-8 directly, and the scores move by at
    most ds = 2^-8 sum_d |q_d k_d| / 16, the weights by a factor exp(+-2 ds) after
    normalisation.
    Everywhere 1e-4 max |v| for fp32 sums and exponentials."""
    n, L = q.shape[0], k.shape[1]
    tol = np.zeros_like(o)
    if L == 0:
        return tol
    f = EPS / (1 - EPS)
    last = np.minimum(first + np.arange(n), L - 1)
    some = last >= 0
    at = np.maximum(last, 0)
    four = b.v is None
    for g in range(HKV):
        mx, mn = np.maximum.accumulate(v[g], 0)[at], np.minimum.accumulate(v[g], 0)[at]
        top = np.maximum(np.abs(mx), np.abs(mn))
        if four:
            grp = v[g].reshape(L, 4, 64)
            rng = np.repeat(np.maximum.accumulate(grp.max(-1) - grp.min(-1), 0)[at], 64, -1)
        for h in range(8 * g, 8 * g + 8):
            spread = np.maximum(mx - o[:, h], o[:, h] - mn)
            t = f * (spread + np.abs(o[:, h])) + 1e-4 * top.max(-1, keepdims=True)
            if four:
                t += f * 1.07 * rng                     # (hi - lo) / 15 rounded up: codes reach 15 s <= 1.004 (hi - lo) + |z - lo|
                if max(b.new) > 1:
                    ds = EPS * (np.abs(q[:, h]) @ np.abs(k[g]).T / 16.0).max(1)
                    t += (np.expm1(2 * ds)[:, None]) * spread + f * top
            tol[:, h] = t
    tol[~some] = 0.0
    return tol


def compare(b: Batch, out: torch.Tensor, ref: dict, label=""):
    got = out.detach().cpu().double().numpy()
    worst = 0.0
    for i, (r, tol) in ref.items():
        m0, n = int(b.cu[i]), b.new[i]
        x = got[m0:m0 + n]
        if out.dtype == torch.bfloat16:
            tol = tol + EPS * (np.abs(r) + tol)
        assert np.isfinite(x).all(), f"{label}: sequence {i}: non-finite output"
        err = np.abs(x - r)
        if err.size:
            worst = max(worst, float((err / np.maximum(tol, 1e-30)).max()))
            assert (err <= tol).all(), (f"{label}: sequence {i}: {int((err > tol).sum())} elements outside the bound, "
                                        f"worst {(err / np.maximum(tol, 1e-30)).max():.2f} times")
    print(f"{label}: worst element at {worst:.2f} of its bound")

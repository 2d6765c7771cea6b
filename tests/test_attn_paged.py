"""Causal attention over the paged cache against the fp64 oracle, every element
against the bound that paged_testlib derives."""
import numpy as np
import pytest
import torch

from oracle import oracle
from tests import paged_testlib as P

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def ops():
    from gated_deltanet_linear_02_gb300 import build, ops
    build.build()
    return ops


def run(ops, b, out_dtype=torch.bfloat16, one_token=False, gate=True, fill=7.0):
    plan, cache = P.handles(ops, b, one_token=one_token)
    out = torch.full((b.q.shape[0], 16, 256), fill, dtype=out_dtype, device=DEV)
    ops.attn_paged(plan, cache, b.q.to(DEV), out, b.gate.to(DEV) if gate else None)
    torch.cuda.synchronize()
    assert ops.device_error() == ops.GDN_OK
    return out


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("ctx", [[1], [2, 15, 16, 17, 31, 33], [127, 128, 129, 0, 300, 64], [1025, 5, 513]])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_one_token(ops, fmt, page, ctx, out_dtype):
    b = P.make_batch(100 + page, fmt, [1] * len(ctx), ctx, page, pad_rows=2)
    out = run(ops, b, out_dtype, one_token=True)
    P.compare(b, out, P.reference(b), f"{fmt} page {page} ctx {ctx}")
    assert (out[-2:] == 7.0).all(), "padding rows changed"
    for i, c in enumerate(ctx):
        if c == 0:
            assert not out[i].any()


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("new,ctx", [([2], [2]), ([3, 0, 8, 1], [40, 9, 8, 129]), ([8, 5], [3, 260]),
                                     ([15, 16, 17], [100, 16, 333]), ([33], [33]), ([130, 1], [200, 700])])
def test_several_tokens(ops, fmt, page, new, ctx):
    """Draft tokens and prompts; contexts shorter than their new tokens (the
    first ones see nothing and give zeros), sequences without tokens, padding."""
    b = P.make_batch(200 + page, fmt, new, ctx, page, pad_rows=3)
    out = run(ops, b)
    P.compare(b, out, P.reference(b), f"{fmt} page {page} new {new} ctx {ctx}")
    assert (out[-3:] == 7.0).all(), "padding rows changed"
    for i, n in enumerate(new):
        for t in range(max(0, n - ctx[i])):
            assert not out[int(b.cu[i]) + t].any()


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("new,ctx", [([257], [1300]), ([513, 64], [513, 900])])
def test_prompts(ops, fmt, new, ctx):
    b = P.make_batch(300, fmt, new, ctx, 32)
    P.compare(b, run(ops, b, torch.float32), P.reference(b), f"{fmt} new {new} ctx {ctx}")


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_sharp_scores(ops, fmt):
    """Scores of +-100 and more: a few weights carry the sum, the running maximum
    moves often, and weights below 2^-126 vanish."""
    b = P.make_batch(301, fmt, [1, 4, 30], [700, 300, 150], 16, sharp=30.0)
    out = run(ops, b, torch.float32)
    for i in range(3):
        m0, n = int(b.cu[i]), b.new[i]
        k, v = b.kv[i]
        # the scores' own fp32 (and, with several tokens in 4 bits, bf16) rounding moves the weights here:
        # outputs stay inside the hull of the values and near the oracle where one weight dominates
        x = out[m0:m0 + n].cpu().double().numpy() * (1 + np.exp(-b.gate[m0:m0 + n].double().numpy()))
        ref = oracle.attn_causal(b.q[m0:m0 + n], k, v, None, int(b.ctx[i]) - n)
        assert np.isfinite(x).all()
        for h in range(16):
            hi, lo = v[h // 8].max(0), v[h // 8].min(0)
            slack = 0.02 * (hi - lo)
            assert (x[:, h] <= hi + slack).all() and (x[:, h] >= lo - slack).all()
        if fmt == "bf16" or max(b.new) == 1:
            assert np.abs(x - ref).max() < 0.05 * np.abs(ref).max()


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_no_gate_and_strided_gate(ops, fmt):
    b = P.make_batch(310, fmt, [1, 1, 1], [70, 8, 200], 16)
    P.compare(b, run(ops, b, gate=False), P.reference(b, gate=False), "no gate")
    joint = torch.zeros(3, 16, 2, 256, dtype=torch.bfloat16, device=DEV)
    joint[:, :, 1] = b.gate.to(DEV)
    plan, cache = P.handles(ops, b)
    outs = []
    for gate in (b.gate.to(DEV), joint[:, :, 1]):
        out = torch.empty(3, 16, 256, device=DEV)
        ops.attn_paged(plan, cache, b.q.to(DEV), out, gate)
        outs.append(out)
    assert torch.equal(*outs)


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("new", [1, 3])
def test_long_context_few_rows(ops, fmt, new):
    """One sequence of 70,001 positions (many CTAs share one row), and a batch
    whose second sequence is short."""
    n, L, page = new, 70001, 64
    g = torch.Generator(device=DEV).manual_seed(9)
    per = -(-L // page)
    table = torch.randperm(2 * per, generator=g, device=DEV).view(2, per).to(torch.int32)
    kv = [torch.randn(2 * per, 2, page, 256, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]
    ctx = [L, 100]
    b = P.Batch(torch.randn(2 * n, 16, 256, generator=g, device=DEV).to(torch.bfloat16).cpu(),
                torch.randn(2 * n, 16, 256, generator=g, device=DEV).to(torch.bfloat16).cpu(), table.cpu(),
                torch.tensor(ctx, dtype=torch.int32), torch.tensor([0, n, 2 * n], dtype=torch.int32), None, None, [], [n, n], page)
    if fmt == "bf16":
        b.k, b.v = kv
    else:
        b.k = torch.zeros(2 * per, 2, page // 16, 4608, dtype=torch.uint8, device=DEV)
        all_rows = ops.make_paged_batch(table, torch.tensor([per * page] * 2, dtype=torch.int32, device=DEV), 2 * per * page,
                                        torch.tensor([0, per * page, 2 * per * page], dtype=torch.int32, device=DEV), per * page)
        flat = [t[table.long()].transpose(2, 3).reshape(-1, 2, 256) for t in kv]
        ops.kv_append(ops.make_attn_params(), all_rows, ops.make_kv_cache(b.k), *flat)
    for i in range(2):
        rows = [t[table[i].long()].transpose(0, 1).reshape(2, -1, 256)[:, :ctx[i]].cpu().double().numpy() for t in kv]
        b.kv.append(tuple(oracle.kv4(t)[3] for t in rows) if fmt == "q4" else tuple(rows))
    P.compare(b, run(ops, b, torch.float32, one_token=n == 1), P.reference(b), f"{fmt} L={L} new={new}")


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_many_short_sequences(ops, fmt):
    ctx = [(i * 37) % 90 for i in range(700)]
    b = P.make_batch(320, fmt, [1] * 700, ctx, 16)
    P.compare(b, run(ops, b, one_token=True), P.reference(b, seqs=range(0, 700, 23)), "700 sequences")
    out = run(ops, b, one_token=False)
    P.compare(b, out, P.reference(b, seqs=range(0, 700, 23)), "700 sequences, packed")


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_pages_past_four_gib(ops, fmt):
    """Pages whose byte offsets pass 32 bits, the last page among them."""
    page = 128
    pages = (10 << 30) // (2 * page * 512) if fmt == "bf16" else (6 << 30) // (2 * page // 16 * 4608)
    b = P.make_batch(330, fmt, [1, 5], [300, 140], page)
    far = torch.tensor([pages - 1, pages // 2, pages - 7, 11, pages - 2, pages * 3 // 4], dtype=torch.int32)[:b.table.numel()]
    shape = (pages, 2, page, 256) if fmt == "bf16" else (pages, 2, page // 16, 4608)
    caches = []
    for t in (b.k, b.v):
        if t is None:
            caches.append(None)
            continue
        big = torch.empty(shape, dtype=t.dtype, device=DEV)
        for at, p in zip(far.tolist(), b.table.flatten().tolist()):
            big[at] = t[p].to(DEV)
        caches.append(big)
    b.table = far.view(b.table.shape)
    b.k, b.v = caches
    P.compare(b, run(ops, b), P.reference(b), f"{fmt} {pages} pages")


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("new", [1, 20])
def test_bad_pages_and_lengths_stay_inside(ops, fmt, new):
    """Page ids outside the cache read as zeros; contexts past the table read
    what the table holds; negative ones nothing. The other sequences are right."""
    b = P.make_batch(340, fmt, [new] * 4, [60, 100, 50, 77], 16)
    b.table[1, 2] = 1 << 30
    b.table[1, 4] = -1
    b.ctx[2] = -3
    for i, p in ((1, 2), (1, 4)):
        for t in b.kv[1]:
            t[:, p * 16:p * 16 + 16] = 0
    ref = P.reference(b, seqs=[0, 1, 3])
    out = run(ops, b)
    P.compare(b, out, ref, "bad pages")
    m0 = int(b.cu[2])
    assert not out[m0:m0 + new].any()


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("new", [1, 3, 40])
def test_context_past_the_table(ops, fmt, new):
    """ctx_len beyond max_pages * page_size: the positions that exist are read."""
    b = P.make_batch(350, fmt, [new], [64], 16)
    plan, cache = P.handles(ops, b)
    b.ctx[0] = 64 + new + 5                                     # every new token sees all 64 rows
    k, v = b.kv[0]
    out = run(ops, b, torch.float32)
    q, z = b.q.double().numpy(), b.gate.double().numpy()
    ref = oracle.attn_causal(q, k, v, None, 64)
    sig = 1 / (1 + np.exp(-z))
    P.compare(b, out, {0: (ref * sig, P._bound(b, q, k, v, ref, 64) * sig)}, "past the table")


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("new", [1, 6, 70])
def test_deterministic_shared_pages_streams_and_graphs(ops, fmt, new):
    """The same bits from an eager call, another stream, and replays of two
    captured graphs that share a workspace; two sequences that share pages."""
    b = P.make_batch(360, fmt, [new, new], [400, 400], 32)
    b.table[1] = b.table[0]                                     # the whole context shared
    b.kv[1] = b.kv[0]
    plan, cache = P.handles(ops, b)
    q, gate = b.q.to(DEV), b.gate.to(DEV)
    ws = torch.empty(max(16, ops.attn_paged_workspace_size(plan, cache)), dtype=torch.uint8, device=DEV)
    outs = [torch.zeros(2 * new, 16, 256, device=DEV) for _ in range(4)]
    ops.attn_paged(plan, cache, q, outs[0], gate, ws)
    P.compare(b, outs[0], P.reference(b), "shared pages")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ops.attn_paged(plan, cache, q, outs[1], gate, ws)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for out in outs[2:]:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            ops.attn_paged(plan, cache, q, out, gate, ws)
        graphs.append(gr)
    ws.fill_(0xFF)                                              # workspace contents need no initialisation
    for gr in graphs * 2:
        gr.replay()
    torch.cuda.synchronize()
    assert ops.device_error() == ops.GDN_OK
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
    # a captured step reads the lengths of the day: shorten a context in place and replay
    plan._keep_alive[1][0] = 250
    graphs[0].replay()
    b.ctx[0] = 250
    b.kv[0] = tuple(t[:, :250] for t in b.kv[0])
    P.compare(b, outs[2], P.reference(b), "replayed with another length")


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("new,ctx", [([2, 16], [300, 16]), ([3, 20], [1000, 131]), ([16, 5, 130], [135, 260, 700])])
def test_values_that_are_not_finite_stay_with_the_tokens_that_see_them(ops, fmt, page, new, ctx):
    """Infinities and NaN in the value row of a new token, and NaN in the key row
    of the last one: tokens before it give what they give without, the others
    infinities and NaN in those dims alone (all dims for the key)."""
    b = P.make_batch(700 + page, fmt, new, ctx, page, pad_rows=1)
    ref = P.reference(b)
    at, dims = {}, {}
    for i, n in enumerate(new):
        j = n // 2
        pos = ctx[i] - n + j
        pg, off = int(b.table[i, pos // page]), pos % page
        if fmt == "bf16":
            b.v[pg, 1, off, 5], b.v[pg, 1, off, 77], b.v[pg, 1, off, 255] = float("inf"), -float("inf"), float("nan")
            dims[i] = [5, 77, 255]
        else:
            rec = b.k[pg, 1, off // 16].numpy()
            rec[4352 + 16 * (off % 16) + 4:4352 + 16 * (off % 16) + 8] = 0xFF     # group 1's step and zero: NaN
            dims[i] = list(range(64, 128))
        at[i] = j
        last = ctx[i] - 1
        pg, off = int(b.table[i, last // page]), last % page
        if fmt == "bf16":
            b.k[pg, 0, off, 9] = float("nan")
        else:
            b.k[pg, 0, off // 16].numpy()[4096 + 16 * (off % 16):4096 + 16 * (off % 16) + 4] = 0xFF
    for dtype in (torch.float32, torch.bfloat16):
        got = run(ops, b, dtype).cpu().double().numpy()
        for i, n in enumerate(new):
            x, (r, tol) = got[int(b.cu[i]):int(b.cu[i]) + n], ref[i]
            if dtype == torch.bfloat16:
                tol = tol + P.EPS * (np.abs(r) + tol)
            clean = np.ones_like(x, dtype=bool)
            clean[n - 1, :8] = False                       # the last token sees the NaN key
            assert np.isnan(x[n - 1, :8]).all()
            hit = np.ix_(range(at[i], n), range(8, 16), dims[i])
            clean[hit] = False
            if fmt == "bf16":
                assert (x[at[i]:, 8:, 5] == np.inf).all() and (x[at[i]:, 8:, 77] == -np.inf).all()
                assert np.isnan(x[at[i]:, 8:, 255]).all()
            else:
                assert np.isnan(x[hit]).all()
            assert np.isfinite(x[clean]).all() and (np.abs(x - r)[clean] <= tol[clean]).all()


@pytest.mark.parametrize("scales", [(1e-7,), (1e-3,), (3e4, 1e5), (1e20,), (1.0, 1e6, 1e-4), (0.0, 1.0)])
@pytest.mark.parametrize("new,ctx", [([3, 17], [130, 700]), ([70], [1300])])
def test_values_of_any_magnitude(ops, scales, new, ctx):
    """4-bit values beyond fp16's range, far below it, and both in one context, by
    turns of 150 positions: within the bound wherever they lie."""
    b = P.make_batch(800, "q4", new, ctx, 32, pad_rows=1)
    for i, c in enumerate(ctx):
        k, v = b.kv[i]
        at = np.array(scales)[np.arange(c) // 150 % len(scales)]
        codes, steps, zeros, v = oracle.kv4((v * at[:, None]).astype(np.float32))
        for p in range(c):
            rec = b.k[int(b.table[i, p // 32]), :, p % 32 // 16].numpy()
            r = p % 16
            rec[:, 2048 + 128 * r:2176 + 128 * r] = P.row_bytes(codes[:, p])
            rec[:, 4352 + 16 * r:4368 + 16 * r] = P.bf16_bytes(np.stack([steps[:, p], zeros[:, p]], -1)).reshape(2, 16)
        b.kv[i] = (k, v)
    P.compare(b, run(ops, b, torch.float32), P.reference(b), f"scales {scales} new {new}")


@pytest.mark.parametrize("raw", [False, True])
def test_another_stream_allocates_its_own_workspace(ops, raw):
    """Without a workspace the call takes one from its own stream's memory: the
    current stream's blocks may still be in use there."""
    b = P.make_batch(900, "bf16", [20], [300], 16)
    ref = run(ops, b)
    side = torch.cuda.Stream()
    plan, cache = P.handles(ops, b)
    q, gate, out = b.q.to(DEV), b.gate.to(DEV), torch.empty(20, 16, 256, dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    for _ in range(20):
        busy = torch.full((1 << 22,), 1.0, device=DEV).mul_(2.0)   # its block is free for the current stream alone
        del busy
        ops.attn_paged(plan, cache, q, out, gate, stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert ops.device_error() == ops.GDN_OK and torch.equal(out, ref)


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_a_conversation(ops, fmt):
    """The operators together as a layer uses them: a prompt appended and
    attended, a second chunk on top, then single tokens and a few draft tokens;
    each step against the oracle over the whole history."""
    steps, page, B = [37, 20, 1, 1, 4, 1], 16, 2
    r = lambda seed, *s: torch.randn(*s, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)  # noqa: E731
    total = sum(steps)
    table = torch.randperm(2 * B * 5)[:B * 5].view(B, 5).to(torch.int32).to(DEV)
    cache = ops.make_kv_cache(*(torch.full((2 * B * 5, 2, page, 256), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))) \
        if fmt == "bf16" else ops.make_kv_cache(torch.full((2 * B * 5, 2, 1, 4608), 255, dtype=torch.uint8, device=DEV))
    qw, kw = 1 + 0.1 * r(1, 256).float(), 1 + 0.1 * r(2, 256).float()
    rope = P.rope_table(total)
    params = ops.make_attn_params(qw.to(DEV), kw.to(DEV), rope.to(DEV))
    hist = [[np.zeros((2, 0, 256)), np.zeros((2, 0, 256))] for _ in range(B)]
    pos = 0
    for s, n in enumerate(steps):
        news = [n, n] if n == 1 else [n, n - 1]
        lens = [pos + n, max(pos + n - 1, 0)] if n > 1 else [pos + 1, hist[1][0].shape[1] + 1]
        news[1] = lens[1] - hist[1][0].shape[1]
        M = sum(news)
        joint, kv = r(10 + s, M, 16, 2, 256), r(50 + s, M, 4, 256)
        cu = torch.tensor([0, news[0], M], dtype=torch.int32)
        plan = ops.make_paged_batch(table, torch.tensor(lens, dtype=torch.int32, device=DEV), M,
                                    None if max(news) == 1 and M == B else cu.to(DEV), max(news))
        d, dk = joint.to(DEV), kv.to(DEV)
        q, out = (torch.empty(M, 16, 256, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        ops.kv_append(params, plan, cache, dk[:, :2], dk[:, 2:], d[:, :, 0], q)
        ops.attn_paged(plan, cache, q, out, d[:, :, 1])
        torch.cuda.synchronize()
        assert ops.device_error() == ops.GDN_OK
        b = P.Batch(q.cpu(), joint[:, :, 1], table.cpu(), torch.tensor(lens, dtype=torch.int32), cu, cache._keep_alive[0],
                    cache._keep_alive[1], [], news, page)
        for i in range(B):
            sl = slice(int(cu[i]), int(cu[i + 1]))
            at = torch.arange(lens[i] - news[i], lens[i])
            kk = oracle.norm_rope(kv[sl, :2].double(), kw, rope[at]).transpose(1, 0, 2)
            vv = kv[sl, 2:].double().numpy().transpose(1, 0, 2)
            kk, vv = (oracle.kv4(kk)[3], oracle.kv4(vv)[3]) if fmt == "q4" else (oracle.bf16_of(kk), vv)
            hist[i] = [np.concatenate([hist[i][0], kk], 1), np.concatenate([hist[i][1], vv], 1)]
        b.kv = [tuple(h) for h in hist]
        # a key's bf16 rounding can fall the other way on the GPU (fp32 before it): one step of bf16 on a
        # few elements moves a score by at most 2^-7 |q k| / 16, far inside the weights' own rounding
        P.compare(b, out, P.reference(b), f"{fmt} step {s}")
        pos += n


def test_matches_contiguous_decode(ops):
    """The same context as a contiguous cache through gdn_attn_decode: both
    kernels within their bounds of each other."""
    L, page = 384, 128
    b = P.make_batch(370, "bf16", [1, 1], [L, L], page)
    out = run(ops, b, torch.float32, one_token=True)
    k, v = (torch.stack([t[b.table[i].long()].transpose(0, 1).reshape(2, L, 256) for i in range(2)]).contiguous().to(DEV) for t in (b.k, b.v))
    ref = torch.empty_like(out)
    ops.attn_decode(b.q.to(DEV), k, v, b.ctx.to(DEV), b.gate.to(DEV), ref)
    bounds = P.reference(b)
    tol = np.concatenate([bounds[i][1] for i in range(2)])
    assert (np.abs((out - ref).cpu().double().numpy()) <= 2 * tol).all()

"""Per-head norms with rotation, and the paged cache's writes and reads, against
the fp64 oracle.

Norm and rotation: the fp32 arithmetic is within 2e-6 of the row's largest
partner (mean of squares, rsqrt, two products, the rotation's three roundings:
below 7e-7 in all), plus half a step of the output type. 4-bit rows are compared
bit for bit: their definition is exact."""
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


def draw(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


def close(got, ref, dtype, label):
    """`ref` fp64 [.., 256]; the row's largest magnitude scales the fp32 error."""
    tol = 2e-6 * np.abs(ref).max(-1, keepdims=True) * np.sqrt(2)
    if dtype == torch.bfloat16:
        tol = tol + P.EPS * (np.abs(ref) + tol)
    err = np.abs(got.cpu().double().numpy() - ref)
    assert (err <= tol).all(), f"{label}: {(err / tol).max():.2f} times the bound"


@pytest.mark.parametrize("M", [1, 2, 7, 33, 300])
@pytest.mark.parametrize("act,out", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                     (torch.float32, torch.bfloat16), (torch.float32, torch.float32)])
def test_norm_rope(ops, M, act, out):
    joint = draw(M, M, 16, 2, 256, dtype=act).to(DEV)
    q, k = joint[:, :, 0], draw(M + 1, M, 6, 256, dtype=act).to(DEV)[:, 1:3]
    qw, kw = 1 + draw(3, 256, dtype=torch.float32, scale=0.2), 1 + draw(4, 256, dtype=torch.float32, scale=0.2)
    table = P.rope_table(5000)
    pos = torch.randint(0, 5000, (M,), generator=torch.Generator().manual_seed(M), dtype=torch.int32)
    p = ops.make_attn_params(qw.to(DEV), kw.to(DEV), table.to(DEV), 1e-6)
    qo, ko = torch.empty(M, 16, 256, dtype=out, device=DEV), torch.empty(M, 2, 256, dtype=out, device=DEV)
    ops.attn_qk_norm_rope(p, q, pos.to(DEV), qo, k, ko)
    rows = table[pos.long()]
    close(qo, oracle.norm_rope(q.cpu().double(), qw, rows), out, "q")
    close(ko, oracle.norm_rope(k.cpu().double(), kw, rows), out, "k")
    # queries alone give the same bits
    q2 = torch.empty_like(qo)
    ops.attn_qk_norm_rope(p, q, pos.to(DEV), q2)
    assert torch.equal(q2, qo)


@pytest.mark.parametrize("norm,rot", [(True, False), (False, True), (False, False)])
def test_norm_rope_parts_left_out(ops, norm, rot):
    M = 9
    q, k, w = draw(1, M, 16, 256), draw(2, M, 2, 256), 1 + draw(3, 256, dtype=torch.float32, scale=0.2)
    table, pos = P.rope_table(64), torch.arange(M, dtype=torch.int32) * 7
    p = ops.make_attn_params(w.to(DEV) if norm else None, None, table.to(DEV) if rot else None)
    qo, ko = torch.empty(M, 16, 256, device=DEV), torch.empty(M, 2, 256, device=DEV)
    ops.attn_qk_norm_rope(p, q.to(DEV), pos.to(DEV) if rot else None, qo, k.to(DEV), ko)
    rows = table[pos.long()] if rot else None
    close(qo, oracle.norm_rope(q.double(), w if norm else None, rows), torch.float32, "q")
    close(ko, oracle.norm_rope(k.double(), None, rows), torch.float32, "k")


def test_norm_rope_in_place_padding_zeros_and_far_positions(ops):
    # dense in place; positions outside the table are padding; a zero row stays zero
    M, n_pos = 6, 1 << 18
    q = draw(5, M, 16, 256)
    q[2] = 0
    w, table = 1 + draw(3, 256, dtype=torch.float32, scale=0.2), P.rope_table(n_pos)
    pos = torch.tensor([0, -1, 3, n_pos, n_pos - 1, 77777], dtype=torch.int32)
    p = ops.make_attn_params(w.to(DEV), None, table.to(DEV))
    x = q.to(DEV).clone()
    ops.attn_qk_norm_rope(p, x, pos.to(DEV), x)
    got = x.cpu()
    assert torch.equal(got[1], q[1]) and torch.equal(got[3], q[3]) and not got[2].any()
    live = [0, 4, 5]
    close(x[live], oracle.norm_rope(q[live].double(), w, table[pos[live].long()]), torch.bfloat16, "in place")


def test_empty_calls(ops):
    p = ops.make_attn_params()
    e = torch.empty(0, 16, 256, dtype=torch.bfloat16, device=DEV)
    ops.attn_qk_norm_rope(p, e, None, e.clone())


# ---- the paged cache

def setup(ops, seed, fmt, new, ctx, page, act=torch.bfloat16, pad_rows=0, norm=True, rot=True, scale=1.0):
    b = P.make_batch(seed, fmt, new, ctx, page, pad_rows)
    M = b.q.shape[0]
    kv = draw(seed + 1, M, 4, 256, dtype=act, scale=scale)
    kw = 1 + draw(seed + 2, 256, dtype=torch.float32, scale=0.2)
    table = P.rope_table(max(max(ctx), 1) + 1)
    params = ops.make_attn_params(kw.to(DEV), kw.to(DEV) if norm else None, table.to(DEV) if rot else None)
    return b, kv[:, :2], kv[:, 2:], kw if norm else None, table if rot else None, params


def expected(b, k, v, kw, table, fmt):
    """The cache's bytes after the append, and the rows' values, by token."""
    kc, vc = b.k.clone(), None if b.v is None else b.v.clone()
    rows = {}
    for i, n in enumerate(b.new):
        for t in range(n):
            m, pos = int(b.cu[i]) + t, int(b.ctx[i]) - n + t
            if pos < 0 or pos // b.page >= b.table.shape[1]:
                continue
            kk = oracle.norm_rope(k[m:m + 1].double(), kw, None if table is None else table[pos:pos + 1])[0]
            rows[m] = (kk, v[m].double().numpy(), int(b.table[i, pos // b.page]), pos % b.page)
    return kc, vc, rows


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("new,ctx", [([1], [1]), ([1, 1, 1], [5, 16, 17]), ([3, 0, 20, 1], [3, 9, 150, 129]),
                                     ([40, 7], [30, 300]), ([1] * 70, list(range(1, 71)))])
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
def test_append_bf16(ops, page, new, ctx, act):
    b, k, v, kw, table, params = setup(ops, 10, "bf16", new, ctx, page, act, pad_rows=3)
    plan, cache = P.handles(ops, b)
    q, qo = draw(77, b.q.shape[0], 16, 256, dtype=act).to(DEV), torch.full((b.q.shape[0], 16, 256), 7.0, dtype=torch.bfloat16, device=DEV)
    ops.kv_append(params, plan, cache, k.to(DEV), v.to(DEV), q, qo)
    kc, vc, rows = expected(b, k, v, kw, table, "bf16")
    gk, gv = (t.cpu() for t in cache._keep_alive)
    seen = torch.zeros(kc.shape[0], kc.shape[2], dtype=torch.bool)
    for m, (kk, vv, p, off) in rows.items():
        close(gk[p, :, off], kk, torch.bfloat16, f"key {m}")
        assert torch.equal(gv[p, :, off], v[m].to(torch.bfloat16)), f"value {m}"
        seen[p, off] = True
    keep = ~seen[:, None, :, None].expand_as(kc)
    same = lambda x, y: torch.equal(x[keep].view(torch.int16), y[keep].view(torch.int16))  # noqa: E731
    assert same(gk, kc) and same(gv, vc), "a row that is no new token's changed"
    # the queries of the same launch; padding rows and tokens without a position are left alone
    w2 = params._keep_alive[0].cpu()
    for m in range(b.q.shape[0]):
        if m >= int(b.cu[-1]):
            assert (qo[m] == 7.0).all()
        elif m in rows:
            i = int(np.searchsorted(b.cu.numpy()[1:], m, side="right"))
            pos = int(b.ctx[i]) - (int(b.cu[i + 1]) - m)
            close(qo[m:m + 1], oracle.norm_rope(q[m:m + 1].cpu().double(), w2, table[pos:pos + 1]), torch.bfloat16, "q")


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("new,ctx", [([1], [1]), ([1, 1, 1], [5, 16, 17]), ([3, 0, 20, 1], [3, 9, 150, 129]), ([600], [700])])
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("norm,rot", [(True, True), (False, False)])
def test_append_q4_is_the_definition_bit_for_bit(ops, page, new, ctx, act, norm, rot):
    b, k, v, kw, table, params = setup(ops, 20, "q4", new, ctx, page, act, norm=norm, rot=rot)
    plan, cache = P.handles(ops, b)
    ops.kv_append(params, plan, cache, k.to(DEV), v.to(DEV))
    want, _, rows = expected(b, k, v, kw, table, "q4")
    want = want.numpy().copy()
    for m, (kk, vv, p, off) in rows.items():
        for at, sz, x in ((0, 4096, kk), (2048, 4352, vv)):
            c, s, z, _ = oracle.kv4(x)
            r = off % 16
            want[p, :, off // 16, at + r * 128:at + r * 128 + 128] = P.row_bytes(c)
            want[p, :, off // 16, sz + r * 16:sz + r * 16 + 16] = P.bf16_bytes(np.stack([s, z], -1)).reshape(2, 16)
    got = cache._keep_alive[0].cpu().numpy()
    bad = np.argwhere(got != want)
    assert not len(bad), f"{len(bad)} bytes differ, first at {bad[:3].tolist()}"


@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
def test_append_q4_scaled_rotation_and_offset_rows(ops, act):
    """Rotation tables with factors above 1, and rows whose offset is far larger than
    their range: the definition bit for bit, over rows enough to meet borders between
    codes, steps and zeros."""
    M = 1500
    b, k, v, kw, table, _ = setup(ops, 50, "q4", [M], [M], 32, act)
    table = table * 3.0
    v[::3] = (v[::3].float() * 0.01 + 37.0).to(act)
    k[::5] = (k[::5].float() * 0.003 - 1.0).to(act)
    plan, cache = P.handles(ops, b)
    ops.kv_append(ops.make_attn_params(None, kw.to(DEV), table.to(DEV)), plan, cache, k.to(DEV), v.to(DEV))
    kk = oracle.norm_rope(k.double(), kw, table[:M])
    kr, vr = (torch.empty(M, 2, 256, device=DEV) for _ in range(2))
    ops.kv_gather(plan, cache, kr, vr)
    got = cache._keep_alive[0].cpu().numpy()
    pos = np.arange(M)
    rec = got[b.table.numpy()[0][pos // 32], :, pos % 32 // 16]               # [M][2][4608]
    for at, sz, x in ((0, 4096, kk), (2048, 4352, v.double().numpy())):
        c, st, z, _ = oracle.kv4(x)
        rows = rec.reshape(M, 2, -1)
        codes = np.stack([rows[m, :, at + m % 16 * 128:at + m % 16 * 128 + 128] for m in pos])
        steps = np.stack([rows[m, :, sz + m % 16 * 16:sz + m % 16 * 16 + 16] for m in pos])
        np.testing.assert_array_equal(steps, P.bf16_bytes(np.stack([st, z], -1)).reshape(M, 2, 16))
        np.testing.assert_array_equal(codes, P.row_bytes(c))


@pytest.mark.parametrize("where", ["weight", "rotation", "huge"])
def test_append_q4_parameters_that_are_not_finite(ops, where):
    """NaN in a weight or in the rotation of one position, or a weight that
    overflows: the groups that hold it read NaN, the others as ever."""
    M = 40
    b, k, v, kw, table, _ = setup(ops, 60, "q4", [M], [M], 16)
    kw, table = kw.clone(), table.clone()
    if where == "weight":
        kw[70] = float("nan")
    elif where == "huge":
        kw[70] = float("inf")
    else:
        table[7, 3] = float("nan")
    plan, cache = P.handles(ops, b)
    ops.kv_append(ops.make_attn_params(None, kw.to(DEV), table.to(DEV)), plan, cache, k.to(DEV), v.to(DEV))
    kr, vr = (torch.empty(M, 2, 256, device=DEV) for _ in range(2))
    ops.kv_gather(plan, cache, kr, vr)
    for got, x in ((kr, oracle.norm_rope(k.double(), kw, table[:M])), (vr, v.double())):
        np.testing.assert_array_equal(got.cpu().numpy(), oracle.kv4(x)[3].astype(np.float32))


def test_append_q4_corner_rows(ops):
    """Constant groups, zeros, exact ties, infinities and NaN, subnormals, huge
    ranges: bit for bit, except that groups that hold a non-finite value read NaN."""
    M = 12
    v = draw(31, M, 2, 256, dtype=torch.float32)
    v[0] = 0
    v[1] = 1.5
    v[2] = (torch.arange(256) % 31).float() / 2                 # ties: zero 0, step 1 (bf16(15 / 15)), halves
    v[3, :, 7] = float("inf")
    v[4, :, 200] = float("nan")
    v[5] *= 1e-39
    v[6] *= 3e37
    v[7, :, 64:] = -3.25
    v[8] = torch.where(torch.arange(256) % 2 == 0, 3e38, -3e38)
    v[9, :, :64] = (torch.arange(64) % 16).float() * 2 ** -9 + 100
    v[10] = v[10].to(torch.bfloat16).float()
    k = v.flip(0).contiguous()
    b = P.make_batch(32, "q4", [M], [M], 16)
    plan, cache = P.handles(ops, b)
    ops.kv_append(ops.make_attn_params(), plan, cache, k.to(DEV), v.to(DEV))
    kr, vr = (torch.empty(M, 2, 256, device=DEV) for _ in range(2))
    ops.kv_gather(plan, cache, kr, vr)
    for got, x in ((kr, k), (vr, v)):
        want = oracle.kv4(x.double())[3].astype(np.float32)
        np.testing.assert_array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_gather_reads_whole_contexts(ops, fmt, out):
    ctx = [33, 1, 0, 130]
    b = P.make_batch(40, fmt, ctx, ctx, 32, pad_rows=2)
    plan, cache = P.handles(ops, b)
    M = b.q.shape[0]
    kr, vr = (torch.full((M, 2, 256), 7.0, dtype=out, device=DEV) for _ in range(2))
    ops.kv_gather(plan, cache, kr, vr)
    k2 = torch.full_like(kr, 7.0)
    ops.kv_gather(plan, cache, k2, None)
    assert torch.equal(k2, kr)
    for i, n in enumerate(ctx):
        m0 = int(b.cu[i])
        for got, ref in ((kr, b.kv[i][0]), (vr, b.kv[i][1])):
            want = torch.from_numpy(np.ascontiguousarray(ref.transpose(1, 0, 2))).float().to(out)
            assert torch.equal(got[m0:m0 + n].cpu(), want)
    assert (kr[-2:] == 7.0).all() and (vr[-2:] == 7.0).all()


@pytest.mark.parametrize("fmt", ["bf16", "q4"])
def test_positions_pages_and_contexts_out_of_range_touch_nothing(ops, fmt):
    """A page id outside the cache, a context past the table, a negative context
    and a rotation row outside the table: those tokens are dropped, the others
    are stored, and nothing else changes."""
    b = P.make_batch(50, fmt, [1, 1, 1, 1, 2], [20, 20, 40, 0, 18], 16)
    b.table[0, 1] = 10 ** 6
    b.table[1, 1] = -5
    b.ctx[2] = 16 * b.table.shape[1] + 1                        # one past the table
    b.ctx[3] = -7
    plan, cache = P.handles(ops, b)
    before = [t.clone() for t in cache._keep_alive if t is not None]
    kv = draw(51, 6, 4, 256).to(DEV)
    pos = torch.tensor([1, 1, 1, 1, 99, 2], dtype=torch.int32, device=DEV)
    params = ops.make_attn_params(None, None, P.rope_table(8).to(DEV))
    ops.kv_append(params, plan, cache, kv[:, :2], kv[:, 2:], positions=pos)
    torch.cuda.synchronize()
    p, off = int(b.table[4, 1]), 17 % 16                       # only token 5, position 17 of sequence 4
    for was, now in zip(before, [t for t in cache._keep_alive if t is not None]):
        w, n = was.view(torch.uint8).flatten(2).clone(), now.view(torch.uint8).flatten(2)
        assert not torch.equal(w[p], n[p])
        w[p] = n[p]
        assert torch.equal(w, n)
    kr, vr = (torch.full((6, 2, 256), 7.0, device=DEV) for _ in range(2))
    ops.kv_gather(plan, cache, kr, vr)
    assert not kr[:4].any() and not vr[:4].any() and vr[5].any()
    assert off == 1


def test_append_other_stream_and_graph(ops):
    b, k, v, kw, table, params = setup(ops, 60, "q4", [5, 3], [20, 90], 32)
    k, v = k.to(DEV), v.to(DEV)
    plan, cache = P.handles(ops, b)
    ops.kv_append(params, plan, cache, k, v)
    want = cache._keep_alive[0].clone()
    plan2, cache2 = P.handles(ops, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ops.kv_append(params, plan2, cache2, k, v)
    side.synchronize()
    assert torch.equal(cache2._keep_alive[0], want)
    plan3, cache3 = P.handles(ops, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.kv_append(params, plan3, cache3, k, v)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(cache3._keep_alive[0], want)

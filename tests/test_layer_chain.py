"""The operators together as a full-attention layer uses them: residual + norm,
joint projection, norms + rotation + paged append, paged attention, output
projection onto the residual stream, norm, mixture of experts onto the stream;
a prompt, then decode steps, eager and captured."""
import math

import pytest
import torch

from tests import layer_testlib as tl
from tests import paged_testlib as pl

pytestmark = pytest.mark.gpu
D, BF, F32, EPS = tl.D, torch.bfloat16, torch.float32, 1e-6
HQ, HKV, HD = 16, 2, 256
PAGE, PER = 16, 6
# bf16 roundings along one layer: normed input, projection, rotated q and k, attention weights and
# output, stream, normed input, hidden activations, output: ten of at most 2^-8 / sqrt(3) each as a
# norm, added up as if they were not independent
BOUND = 10 * 2.0 ** -8 / 3 ** 0.5


@pytest.fixture(scope="module")
def ops():
    from gated_deltanet_linear_02_gb300 import build, ops
    build.build()
    return ops


class Layer:
    def __init__(self, ops, E=32, k=4, F=256):
        g = tl.gen(21)
        self.ops, self.k = ops, k
        self.n1, self.n2, self.qn, self.kn = (1 + 0.1 * tl.rnd(g, n, dtype=F32) for n in (D, D, HD, HD))
        self.wqkv = tl.rnd(g, 2 * HQ * HD + 2 * HKV * HD, D, scale=D ** -0.5)
        self.wo = tl.rnd(g, D, HQ * HD, scale=(HQ * HD) ** -0.5)
        self.W = tl.moe_weights(g, E, F)
        self.rope = pl.rope_table(PAGE * PER).cuda()
        self.kc, self.vc = (torch.full((2 * PER, HKV, PAGE, HD), float("nan"), dtype=BF, device="cuda") for _ in range(2))
        self.table = torch.randperm(2 * PER, generator=torch.Generator().manual_seed(3)).view(2, PER).int().cuda()
        self.norm1, self.norm2 = ops.make_norm_params(self.n1, norm_eps=EPS), ops.make_norm_params(self.n2, norm_eps=EPS)
        self.attn = ops.make_attn_params(self.qn, self.kn, self.rope, EPS)
        self.cache = ops.make_kv_cache(self.kc, self.vc)
        W = self.W
        self.moe = ops.make_moe_params(W["router"], W["gate"], W["up"], W["down"], W["sh_gate"], W["sh_up"], W["sh_down"],
                                       W["sh_router"], top_k=k)

    def buffers(self, M):
        e = lambda *s, dt=BF: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
        return dict(h=e(M, D), qkv=e(M, self.wqkv.shape[0]), q=e(M, HQ, HD), o=e(M, HQ, HD), h2=e(M, D))

    def run(self, x, plan, b, ws):
        """One layer on the residual stream x [M][2048] bf16, in place."""
        ops, M = self.ops, x.shape[0]
        ops.add_norm(self.norm1, x, None, None, b["h"])
        ops.linear(b["h"], self.wqkv, b["qkv"])
        joint = b["qkv"][:, :2 * HQ * HD].view(M, HQ, 2, HD)
        kv = b["qkv"][:, 2 * HQ * HD:].view(M, 2 * HKV, HD)
        ops.kv_append(self.attn, plan, self.cache, kv[:, :HKV], kv[:, HKV:], joint[:, :, 0], b["q"])
        ops.attn_paged(plan, self.cache, b["q"], b["o"], joint[:, :, 1], ws[0])
        ops.linear(b["o"].view(M, HQ * HD), self.wo, x, residual=x)
        ops.add_norm(self.norm2, x, None, None, b["h2"])
        ops.moe(self.moe, b["h2"], x, residual=x, workspace=ws[1])

    def workspaces(self, plan, M):
        n = self.ops.attn_paged_workspace_size(plan, self.cache), self.ops.moe_workspace_size(self.moe, M)
        return [torch.full((k,), 255, dtype=torch.uint8, device="cuda") for k in n]

    def reference(self, x, news, K, V, ids, w):
        """The layer in 64 bits: x [M][2048], per sequence the keys and values so far
        (extended here); the experts are the ones the library chose."""
        x = x.double()
        y = tl.rms64(x, EPS) * self.n1.double() @ self.wqkv.double().T
        q, gate = y[:, :2 * HQ * HD].view(-1, HQ, 2, HD).unbind(2)
        k, v = y[:, 2 * HQ * HD:].view(-1, 2, HKV, HD).unbind(1)
        out, m = [], 0
        for s, n in enumerate(news):
            at = K[s].shape[0] + torch.arange(n, device="cuda")
            rot = self.rope.double()[at]

            def turn(t, nw):
                t = tl.rms64(t, EPS) * nw.double()
                c, sn = rot[:, None, :32], rot[:, None, 32:]
                return torch.cat([t[..., :32] * c - t[..., 32:64] * sn, t[..., 32:64] * c + t[..., :32] * sn, t[..., 64:]], -1)
            qs = turn(q[m:m + n], self.qn)
            K[s] = torch.cat([K[s], turn(k[m:m + n], self.kn)])
            V[s] = torch.cat([V[s], v[m:m + n]])
            kk, vv = K[s].repeat_interleave(8, 1), V[s].repeat_interleave(8, 1)
            sc = torch.einsum("nhd,lhd->hnl", qs, kk) / 16
            sc = sc.masked_fill(torch.arange(kk.shape[0], device="cuda") > at[None, :, None], -math.inf)
            out.append(torch.einsum("hnl,lhd->nhd", torch.softmax(sc, -1), vv) * torch.sigmoid(gate[m:m + n]))
            m += n
        x = x + torch.cat(out).reshape(-1, HQ * HD) @ self.wo.double().T
        return x + tl.moe64(self.W, tl.rms64(x, EPS) * self.n2.double(), ids, w)


def plan_of(ops, L, news, ctx):
    cu = torch.tensor([0, news[0], sum(news)], dtype=torch.int32, device="cuda")
    one = max(news) == 1
    return ops.make_paged_batch(L.table, ctx, sum(news), None if one else cu, max(news))


def test_prompt_then_decode(ops):
    L = Layer(ops)
    g = tl.gen(22)
    ctx = torch.zeros(2, dtype=torch.int32, device="cuda")
    K, V = [torch.zeros(0, HKV, HD, dtype=torch.float64, device="cuda") for _ in range(2)], \
        [torch.zeros(0, HKV, HD, dtype=torch.float64, device="cuda") for _ in range(2)]
    for news in ([37, 70], [1, 1], [3, 2], [1, 1]):
        M = sum(news)
        x = tl.rnd(g, M, D)
        x0 = x.clone()
        ctx += torch.tensor(news, dtype=torch.int32, device="cuda")
        plan = plan_of(ops, L, news, ctx)
        b, ws = L.buffers(M), L.workspaces(plan, M)
        L.run(x, plan, b, ws)
        ids, w = torch.empty(M, L.k, dtype=torch.int32, device="cuda"), torch.empty(M, L.k, device="cuda")
        ops.moe_route(L.moe, b["h2"], ids, w)
        assert ops.device_error() == ops.GDN_OK
        ref = L.reference(x0, news, K, V, ids, w)
        assert tl.relative(x, ref) < BOUND
    # the last step again, captured: the same rows are written, so the same bits come out
    graph = torch.cuda.CUDAGraph()
    y = x0.clone()
    with torch.cuda.graph(graph):
        L.run(y, plan, b, ws)
    for _ in range(2):
        y.copy_(x0)
        for t in ws:
            t.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(x, y)
    assert ops.device_error() == ops.GDN_OK

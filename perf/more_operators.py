"""Workloads of what stands around the token mixers in a hybrid layer, with plain forms.

The operators carry a layer of the model from the mixer's output to the next
layer's input (width 2048, mixture of experts with a shared expert):

- ``add_norm``  adds a block's output to the residual stream (optionally normed,
                gated and scaled on the way) and gives the next block's normed input;
- ``linear``    a matrix product with bias, activation and residual in its epilogue;
- ``route``     the router: the chosen experts of each token and their weights;
- ``moe``       the whole mixture-of-experts layer: router, the experts' gated
                products, the shared expert with its own gate, and the residual.

``own`` selects the library's calls; otherwise ``run`` computes the same thing
in elementary torch operations. ``exact`` is the definition in 64 bits.
"""
import math

import torch

own = False

D = 2048                          # width of the residual stream
EPS = 1e-6


def listed():
    def c(name, **kw):
        return dict(name=name, **kw)
    return [
        # one new token of one conversation between two blocks: nothing but latency
        c("add_norm_one_token", op="add_norm", rows=1, stream="bf16", post=False, gate="none"),
        # a prompt with a norm after the block, gates per token and a 32-bit residual stream
        c("add_norm_prompt_4096", op="add_norm", rows=4096, stream="fp32", post=True, gate="rows"),
        # one token through the joint query, gate, key and value projection of a full-attention layer
        c("linear_one_token", op="linear", rows=1, n=9216, k=2048, act="none", bias=False, residual=False, out="bf16"),
        # a decode batch through an output projection, with the residual stream
        c("linear_decode_96", op="linear", rows=96, n=2048, k=4096, act="none", bias=False, residual=True, out="bf16"),
        # a ragged prompt through a wide projection with bias and activation
        c("linear_prompt_4001", op="linear", rows=4001, n=9216, k=2048, act="silu", bias=True, residual=False, out="bf16"),
        # the router alone, for a decode batch and for a prompt
        c("route_decode_256", op="route", rows=256, experts=256, topk=8, renorm=True),
        c("route_prompt_4096", op="route", rows=4096, experts=256, topk=8, renorm=True),
        # the whole layer for one token, for draft tokens of one conversation, for
        # small and large decode batches, and for a prompt
        c("moe_one_token", op="moe", rows=1, experts=256, topk=8, ffn=512, shared=True, renorm=True, residual=True),
        c("moe_four_tokens", op="moe", rows=4, experts=256, topk=8, ffn=512, shared=True, renorm=True, residual=True),
        c("moe_decode_24", op="moe", rows=24, experts=256, topk=8, ffn=512, shared=True, renorm=True, residual=True),
        c("moe_decode_256", op="moe", rows=256, experts=256, topk=8, ffn=512, shared=True, renorm=True, residual=True),
        c("moe_prompt_4096", op="moe", rows=4096, experts=256, topk=8, ffn=512, shared=True, renorm=True, residual=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    kind = rng.choice(["add_norm", "linear", "linear", "linear", "route", "moe", "moe", "moe"])
    if kind == "add_norm":
        return dict(op=kind, rows=_log_int(rng, 1, 4096), stream=rng.choice(["bf16", "fp32"]), post=rng.random() < 0.5,
                    gate=rng.choice(["none", "rows", "shared"]))
    if kind == "linear":
        return dict(op=kind, rows=_log_int(rng, 1, 4096), n=8 * _log_int(rng, 8, 1152), k=8 * _log_int(rng, 16, 512),
                    act=rng.choice(["none", "silu", "gelu", "sigmoid"]), bias=rng.random() < 0.5, residual=rng.random() < 0.5,
                    out="bf16")
    experts = rng.choice([8, 40, 64, 128, 256])
    topk = min(rng.choice([1, 2, 4, 6, 8]), experts)
    if kind == "route":
        return dict(op=kind, rows=_log_int(rng, 1, 4096), experts=experts, topk=topk, renorm=rng.random() < 0.7)
    ffn = rng.choice([128, 256, 384, 512, 1024]) if experts < 256 else rng.choice([128, 256, 512])
    rows = _log_int(rng, 1, min(4096, (4096 * 9 * 512) // ((topk + 1) * ffn)))
    return dict(op=kind, rows=rows, experts=experts, topk=topk, ffn=ffn, shared=rng.random() < 0.7, renorm=rng.random() < 0.7,
                residual=rng.random() < 0.7)


def work(case):
    M = case["rows"]
    if case["op"] == "add_norm":
        s = 4 if case["stream"] == "fp32" else 2
        gates = {"none": 0, "rows": M * D * 2, "shared": D * 2}[case["gate"]]
        return {"bytes": M * D * (2 * s + 2 + 2) + gates + D * 4 * (2 if case["post"] else 1), "flops": M * D * 8}
    if case["op"] == "linear":
        n, k = case["n"], case["k"]
        o = 4 if case["out"] == "fp32" else 2
        return {"bytes": (M * k + n * k) * 2 + M * n * o * (2 if case["residual"] else 1) + (n * 4 if case["bias"] else 0), "flops": 2 * M * n * k}
    E, k = case["experts"], case["topk"]
    route = {"bytes": (M + E) * D * 2, "flops": 2 * M * E * D}
    if case["op"] == "route":
        return {"bytes": route["bytes"] + M * k * 8, "flops": route["flops"]}
    F = case["ffn"]
    used = E * (1 - (1 - k / E) ** M) + (1 if case["shared"] else 0)       # experts that some token takes, for even routing
    return {"bytes": int(route["bytes"] + used * 3 * F * D * 2 + M * D * 2 * (2 if case["residual"] else 1)),
            "flops": route["flops"] + 6 * M * (k + (1 if case["shared"] else 0)) * F * D}


def prepare(case, seed):
    dev, bf = "cuda", torch.bfloat16
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    rn = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    rb = lambda s, *n: torch.randn(*n, generator=g, device=dev, dtype=bf).mul_(s)  # noqa: E731
    S = {"case": dict(case)}
    M, op = case["rows"], case["op"]
    if op == "add_norm":
        dt = torch.float32 if case["stream"] == "fp32" else bf
        S["x"], S["delta"] = rn(M, D).to(dt), rb(0.7, M, D)
        S["norm_w"], S["post_w"] = 1 + 0.1 * rn(D), (1 + 0.1 * rn(D) if case["post"] else None)
        S["gate"] = {"none": lambda: None, "rows": lambda: rb(0.5, M, D), "shared": lambda: rb(0.5, 1, D).expand(M, D)}[case["gate"]]()
        S["x_out"], S["h"] = torch.empty(M, D, dtype=dt, device=dev), torch.empty(M, D, dtype=bf, device=dev)
    elif op == "linear":
        n, k = case["n"], case["k"]
        dt = torch.float32 if case["out"] == "fp32" else bf
        S["x"], S["w"] = rb(1.0, M, k), rb(1 / math.sqrt(k), n, k)
        S["bias"] = 0.5 * rn(n) if case["bias"] else None
        S["residual"] = rn(M, n).to(dt) if case["residual"] else None
        S["y"] = torch.empty(M, n, dtype=dt, device=dev)
    else:
        E, k = case["experts"], case["topk"]
        # normed rows with a direction in common: some experts are taken more often than others
        S["x"] = (0.95 * rn(M, D) + 0.3 * rn(1, D)).to(bf)
        S["router"] = rb(0.03, E, D)
        if op == "route":
            S["ids"] = torch.empty(M, k, dtype=torch.int32, device=dev)
            S["weights"] = torch.empty(M, k, device=dev)
        else:
            F = case["ffn"]
            S["gate"], S["up"], S["down"] = rb(0.03, E, F, D), rb(0.03, E, F, D), rb(0.06, E, D, F)
            for n, s, shape in (("sh_gate", 0.03, (F, D)), ("sh_up", 0.03, (F, D)), ("sh_down", 0.06, (D, F)), ("sh_router", 0.03, (D,))):
                S[n] = rb(s, *shape) if case["shared"] else None
            S["residual"] = rb(1.0, M, D) if case["residual"] else None
            S["out"] = torch.empty(M, D, dtype=bf, device=dev)
    if own:
        from gated_deltanet_linear_02_gb300 import ops
        S["ops"] = ops
        if op == "add_norm":
            S["params"] = ops.make_norm_params(S["norm_w"], S["post_w"], res_scale=0.8, norm_eps=EPS)
        elif op == "route":
            S["params"] = ops.make_moe_params(S["router"], top_k=case["topk"], norm_topk=case["renorm"])
        elif op == "moe":
            S["params"] = ops.make_moe_params(S["router"], S["gate"], S["up"], S["down"], S["sh_gate"], S["sh_up"], S["sh_down"],
                                              S["sh_router"], top_k=case["topk"], norm_topk=case["renorm"])
            S["ws"] = torch.empty(ops.moe_workspace_size(S["params"], M), dtype=torch.uint8, device=dev)
    return S


# ---- one pass

def run(S):
    case = S["case"]
    op = case["op"]
    if own:
        ops = S["ops"]
        if op == "add_norm":
            ops.add_norm(S["params"], S["x"], S["delta"], S["x_out"], S["h"], gate=S["gate"])
            return S["x_out"], S["h"]
        if op == "linear":
            ops.linear(S["x"], S["w"], S["y"], bias=S["bias"], residual=S["residual"], activation=case["act"])
            return S["y"]
        if op == "route":
            ops.moe_route(S["params"], S["x"], S["ids"], S["weights"])
            return S["ids"], S["weights"]
        ops.moe(S["params"], S["x"], S["out"], residual=S["residual"], workspace=S["ws"])
        return S["out"]
    if op == "add_norm":
        d = S["delta"].float()
        if S["post_w"] is not None:
            d = _rms(d) * S["post_w"]
        if S["gate"] is not None:
            d = d * S["gate"].float()
        s = S["x"].float() + 0.8 * d
        return s.to(S["x"].dtype), (_rms(s) * S["norm_w"]).to(torch.bfloat16)
    if op == "linear":
        y = torch.matmul(S["x"].float(), S["w"].float().T)
        if S["bias"] is not None:
            y += S["bias"]
        y = _act(y, case["act"])
        if S["residual"] is not None:
            y = y + S["residual"].float()
        return y.to(S["y"].dtype)
    ids, w = _route(S["x"], S["router"], case)
    if op == "route":
        return ids.int(), w.float()
    return _moe(S, case, ids, w.float())


def _rms(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _act(y, name):
    if name == "silu":
        return y * torch.sigmoid(y)
    if name == "gelu":
        return 0.5 * y * (1 + torch.erf(y / math.sqrt(2)))
    return torch.sigmoid(y) if name == "sigmoid" else y


def _route(x, router, case):
    """The chosen experts, best first (ties: the lowest), and their weights. The
    logits in 64 bits: the choice is between neighbours."""
    logits = torch.matmul(x.double(), router.double().T)
    top, ids = (t[:, : case["topk"]] for t in torch.sort(logits, dim=-1, descending=True, stable=True))
    e = torch.exp(top - top[:, :1])
    whole = e if case["renorm"] else torch.exp(logits - top[:, :1])
    return ids, e / whole.sum(-1, keepdim=True)


def _moe(S, case, ids, w):
    M, k, E, F = case["rows"], case["topk"], case["experts"], case["ffn"]
    x = S["x"].float()
    pair = ids.reshape(-1)
    if M * k <= E:                        # few tokens: each pair's weights
        xp = x.repeat_interleave(k, 0)[:, :, None]
        a, b = (torch.matmul(S[n][pair].float(), xp) for n in ("gate", "up"))
        y = torch.matmul(S["down"][pair].float(), a * torch.sigmoid(a) * b)[:, :, 0]
    else:                                 # rows sorted by expert, padded to the fullest one
        order = torch.argsort(pair, stable=True)
        count = torch.bincount(pair, minlength=E)
        rank = torch.empty_like(pair)
        rank[order] = torch.arange(M * k, device=x.device) - (torch.cumsum(count, 0) - count)[pair[order]]
        rows = torch.zeros(E, int(count.max()), dtype=torch.long, device=x.device)
        rows[pair, rank] = torch.arange(M * k, device=x.device) // k
        xe = x[rows]
        a, b = (torch.matmul(xe, S[n].float().transpose(1, 2)) for n in ("gate", "up"))
        y = torch.matmul(a * torch.sigmoid(a) * b, S["down"].float().transpose(1, 2))[pair, rank]
    out = (y.view(M, k, D) * w[:, :, None]).sum(1)
    if case["shared"]:
        a, b = torch.matmul(x, S["sh_gate"].float().T), torch.matmul(x, S["sh_up"].float().T)
        y = torch.matmul(a * torch.sigmoid(a) * b, S["sh_down"].float().T)
        out = out + torch.sigmoid(torch.matmul(x, S["sh_router"].float()))[:, None] * y
    if case["residual"]:
        out = out + S["residual"].float()
    return out.to(torch.bfloat16)


# ---- the definition in 64 bits, expert by expert

def exact(case, seed):
    S = prepare(case, seed)
    op = case["op"]
    if op == "add_norm":
        d = S["delta"].double()
        if case["post"]:
            d = d / ((d * d).sum(-1, keepdim=True) / D + EPS).sqrt() * S["post_w"].double()
        if S["gate"] is not None:
            d = d * S["gate"].double()
        s = S["x"].double() + 0.8 * d
        return s, s / ((s * s).sum(-1, keepdim=True) / D + EPS).sqrt() * S["norm_w"].double()
    x = S["x"].double()
    if op == "linear":
        y = torch.einsum("mk,nk->mn", x, S["w"].double())
        y = y + S["bias"].double() if case["bias"] else y
        y = {"none": lambda: y, "silu": lambda: y / (1 + torch.exp(-y)), "sigmoid": lambda: 1 / (1 + torch.exp(-y)),
             "gelu": lambda: y * 0.5 * torch.erfc(-y / 2 ** 0.5)}[case["act"]]()
        return y + S["residual"].double() if case["residual"] else y
    p = torch.softmax(torch.einsum("md,ed->me", x, S["router"].double()), -1)
    left, ids, w = p.clone(), [], []
    for _ in range(case["topk"]):                          # the best that is left
        best = left.amax(-1, keepdim=True)
        at = (left == best).int().argmax(-1, keepdim=True)
        ids.append(at)
        w.append(best)
        left.scatter_(1, at, -1.0)
    ids, w = torch.cat(ids, 1), torch.cat(w, 1)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    if op == "route":
        return ids.int(), w
    out = S["residual"].double() if case["residual"] else torch.zeros_like(x)
    for e in range(case["experts"]):
        tok, slot = (ids == e).nonzero(as_tuple=True)
        if tok.numel():
            a, b = x[tok] @ S["gate"][e].double().T, x[tok] @ S["up"][e].double().T
            out.index_add_(0, tok, (a / (1 + torch.exp(-a)) * b) @ S["down"][e].double().T * w[tok, slot][:, None])
    if case["shared"]:
        a, b = x @ S["sh_gate"].double().T, x @ S["sh_up"].double().T
        g = 1 / (1 + torch.exp(-(x @ S["sh_router"].double())))
        out = out + g[:, None] * ((a / (1 + torch.exp(-a)) * b) @ S["sh_down"].double().T)
    return out

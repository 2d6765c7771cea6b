"""What the tests of the operators around the mixers share: inputs, plain forms
in 64 bits, and how far an output may be from them.

Roundings: a number rounded to nearest in type t is off by at most HALF[t] of
its value. Sums: fp32 sums over n terms in a tree of depth d are off by at most
about d 2^-24 of the sum of magnitudes; the tensor core adds 16 products at a
time and truncates, so at most one step of 2^-23 of that sum per 16 of K."""
from __future__ import annotations

import math

import torch

D = 2048
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def rnd(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device=g.device) * scale).to(dtype)


def rms64(x, eps):
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt()


def act64(v, name):
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return 0.5 * v * torch.special.erfc(-v / math.sqrt(2))
    return torch.sigmoid(v) if name == "sigmoid" else v


def route64(x, router, k, renorm):
    logits = x.double() @ router.double().T
    top, ids = (t[:, :k] for t in torch.sort(logits, dim=-1, descending=True, stable=True))
    e = torch.exp(top - top[:, :1])
    return ids.int(), e / (e if renorm else torch.exp(logits - top[:, :1])).sum(-1, keepdim=True)


def moe64(W, x, ids, w):
    """The sum over the given experts and the shared one, without the residual.
    W: dict of weights; ids outside [0, E) contribute nothing."""
    x = x.double()
    out = torch.zeros(x.shape[0], D, dtype=torch.float64, device=x.device)

    def expert(rows, g, u, d):
        a = rows @ g.double().T
        return (a * torch.sigmoid(a) * (rows @ u.double().T)) @ d.double().T
    for e in range(W["gate"].shape[0]):
        tok, slot = (ids == e).nonzero(as_tuple=True)
        if tok.numel():
            out.index_add_(0, tok, expert(x[tok], W["gate"][e], W["up"][e], W["down"][e]) * w.double()[tok, slot][:, None])
    if W.get("sh_gate") is not None:
        y = expert(x, W["sh_gate"], W["sh_up"], W["sh_down"])
        out += y if W.get("sh_router") is None else torch.sigmoid(x @ W["sh_router"].double())[:, None] * y
    return out


def moe_weights(g, E, F, shared=True, sh_router=True):
    W = dict(router=rnd(g, E, D, scale=0.03), gate=rnd(g, E, F, D, scale=0.03), up=rnd(g, E, F, D, scale=0.03),
             down=rnd(g, E, D, F, scale=0.06))
    if shared:
        W.update(sh_gate=rnd(g, F, D, scale=0.03), sh_up=rnd(g, F, D, scale=0.03), sh_down=rnd(g, D, F, scale=0.06))
        if sh_router:
            W["sh_router"] = rnd(g, D, scale=0.03)
    return W


def relative(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


def within(got, ref, slack):
    """|got - ref| <= the output's own rounding + slack, element by element."""
    err = (got.double() - ref).abs()
    return bool((err <= HALF[got.dtype] * (ref.abs() + slack) + slack).all())

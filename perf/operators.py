"""Workloads of the full-attention layers' cache operators, with plain forms.

The operators are the ones a hybrid model's full-attention layers need around
their key/value cache (16 query heads, 2 KV heads, head dim 256, rotation over
the first 64 dims):

- ``norm``    per-head RMSNorm of queries and keys with the position rotation;
- ``append``  keys (normed and rotated on the way) and values into a paged
              cache, bf16 or 4-bit;
- ``attend``  attention of new tokens (one per sequence, a few draft tokens, or
              a prompt) over the paged cache, bf16 or 4-bit, with the sigmoid
              output gate;
- ``step``    the three of them as one decode step uses them.

``own`` selects the library's calls; otherwise ``run`` computes the same thing
in elementary torch operations. ``exact`` is the definition in 64 bits.

The 4-bit cache: a (token, KV head) row of 256 values is 4 groups of 64, each
with lo = min, hi = max, zero z = bf16(lo), step s = bf16((hi - lo) / 15),
codes c = clamp(round((x - z) / s), 0, 15) and value z + s c. Pages are records
of 16 rows: key codes (16 x 128 bytes), value codes, key steps and zeros
(16 x 4 x 2 bf16), value steps and zeros. Within a row's 128 bytes, byte
16 c + 4 g + b holds dims 64 g + 8 c + 2 b (low nibble) and + 1 (high nibble).
"""
import math

import torch

own = False

HQ, HKV, D, ROT = 16, 2, 256, 64
GROUP, NG = 64, 4
REC = 16                          # rows per 4-bit record
REC_BYTES = REC * (128 + 128 + 16 + 16)
EPS = 1e-6
BASE = 10000000.0                 # rotation base
GOLD = 0.6180339887498949


def listed():
    def c(name, **kw):
        return dict(name=name, **kw)
    return [
        # one new token of one conversation: nothing but latency
        c("norm_one_token", op="norm", tokens=1, far=32768),
        # a 4096-token prompt through the norms and rotation
        c("norm_prompt_4096", op="norm", tokens=4096, far=4096),
        # a decode batch's keys and values into the bf16 cache
        c("append_bf16_decode_256", op="append", fmt="bf16", batch=256, new=1, context=1000, page=64),
        # ragged prompts written into the bf16 cache, pages of 16
        c("append_bf16_prompts", op="append", fmt="bf16", batch=3, new=1801, context=2500, page=16),
        # a decode batch into the 4-bit cache, rows read back
        c("append_q4_decode_64", op="append", fmt="q4", batch=64, new=1, context=777, page=32),
        # a prompt into the 4-bit cache, rows read back
        c("append_q4_prompt_4096", op="append", fmt="q4", batch=1, new=4096, context=4096, page=64),
        # one long conversation, one new token
        c("attend_bf16_one_long", op="attend", fmt="bf16", batch=1, new=1, context=32768, page=64),
        # a decode batch over ragged contexts of up to 4096
        c("attend_bf16_decode_256", op="attend", fmt="bf16", batch=256, new=1, context=4096, page=64),
        # a whole 4096-token prompt
        c("attend_bf16_prompt_4096", op="attend", fmt="bf16", batch=1, new=4096, context=4096, page=64),
        # the same decode batch over the 4-bit cache
        c("attend_q4_decode_256", op="attend", fmt="q4", batch=256, new=1, context=4096, page=64),
        # prompt chunks of ragged lengths on top of longer 4-bit contexts
        c("attend_q4_chunks", op="attend", fmt="q4", batch=3, new=517, context=6001, page=32),
        # a decode step of 16 sequences on the 4-bit cache: norms, append,
        # attention, and the new rows read back
        c("step_q4_decode_16", op="step", fmt="q4", batch=16, new=1, context=2049, page=16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    kind = rng.choice(["norm", "append", "append", "attend", "attend", "attend", "step"])
    if kind == "norm":
        return dict(op="norm", tokens=_log_int(rng, 1, 4096), far=_log_int(rng, 1, 65536))
    fmt, page = rng.choice(["bf16", "q4"]), rng.choice([16, 32, 64, 128])
    if kind == "append":
        batch = _log_int(rng, 1, 256)
        new = 1 if rng.random() < 0.4 else _log_int(rng, 2, max(2, 4096 // batch))
        context = new + _log_int(rng, 1, max(1, min(4096, 200000 // batch - new)))
        return dict(op="append", fmt=fmt, batch=batch, new=new, context=context, page=page)
    if kind == "step":
        batch = _log_int(rng, 1, 128)
        return dict(op="step", fmt=fmt, batch=batch, new=1, context=_log_int(rng, 1, min(16384, 262144 // batch)), page=page)
    form = rng.choice(["one", "few", "prompt"])
    if form == "one":
        batch = _log_int(rng, 1, 256)
        return dict(op="attend", fmt=fmt, batch=batch, new=1, context=_log_int(rng, 1, min(65536, (1 << 20) // batch)), page=page)
    if form == "few":
        batch = _log_int(rng, 1, 64)
        new = rng.randint(2, 8)
        return dict(op="attend", fmt=fmt, batch=batch, new=new, context=new + _log_int(rng, 1, min(32768, (1 << 18) // batch)), page=page)
    new = _log_int(rng, 9, 2048)
    context = new + _log_int(rng, 1, min(16384, (1 << 22) // new))
    batch = _log_int(rng, 1, max(1, min(8, (1 << 23) // (new * context))))
    return dict(op="attend", fmt=fmt, batch=batch, new=new, context=context, page=page)


def _lengths(case):
    """(new tokens, context with them) of each sequence: the first has the
    case's sizes, the others spread down to half of them."""
    news, ctxs = [], []
    for i in range(case["batch"]):
        f = (i * GOLD) % 1.0
        n = max(1, case["new"] - int(f * case["new"] / 2))
        news.append(n)
        ctxs.append(max(n, case["context"] - int(f * case["context"] / 2)))
    return news, ctxs


def work(case):
    tok_qk = (HQ + HKV) * D * 2
    if case["op"] == "norm":
        M = case["tokens"]
        return {"bytes": M * (2 * tok_qk + 256 + 4) + 2048, "flops": M * (HQ + HKV) * D * 6}
    news, ctxs = _lengths(case)
    M, total = sum(news), sum(ctxs)
    row = HKV * 2 * (D * 2 if case["fmt"] == "bf16" else 144)      # one cached token
    table = total // case["page"] * 4 + case["batch"] * 8
    append = M * (HKV * 2 * D * 2 + row + 256) + table
    if case["op"] == "append":
        back = M * (row + HKV * 2 * D * 2) if case["fmt"] == "q4" else 0
        return {"bytes": append + back, "flops": M * HKV * D * 12}
    seen = sum(n * c - n * (n - 1) // 2 for n, c in zip(news, ctxs))
    attend = {"bytes": M * 3 * HQ * D * 2 + total * row + table, "flops": 4 * seen * HQ * D}
    if case["op"] == "attend":
        return attend
    back = M * (row + HKV * 2 * D * 2) if case["fmt"] == "q4" else 0
    return {"bytes": attend["bytes"] + append + back + M * 2 * HQ * D * 2, "flops": attend["flops"] + M * (HQ + 2 * HKV) * D * 8}


# ---- inputs

def _pack4(x, pages, page):
    """fp32 [pages][2][page][256] -> (codes u8 [pages][2][page][128] in the
    record's byte order, steps and zeros bf16 [pages][2][page][4][2])."""
    v = x.view(pages, HKV, page, NG, GROUP)
    lo, hi = v.amin(-1), v.amax(-1)
    z = lo.to(torch.bfloat16)
    s = ((hi - lo) / 15).to(torch.bfloat16)
    c = ((v - z.float()[..., None]) / s.float()[..., None]).round_().clamp_(0, 15).to(torch.uint8)
    c = c.view(pages, HKV, page, NG, 8, 4, 2)
    b = c[..., 0] | (c[..., 1] << 4)                                # [.., g, chunk, byte]
    return b.transpose(3, 4).reshape(pages, HKV, page, 128), torch.stack([s, z], -1)


def _records(kc, ksz, vc, vsz):
    """The parts of _pack4 for keys and values as 16-row records."""
    pages, page = kc.shape[0], kc.shape[2]
    r = lambda t: t.contiguous().view(torch.uint8).reshape(pages, HKV, page // REC, -1)  # noqa: E731
    return torch.cat([r(kc), r(vc), r(ksz), r(vsz)], -1).contiguous()


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    rn = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    bf = torch.bfloat16
    S = {"case": dict(case)}
    op = case["op"]
    if op == "norm":
        M, far = case["tokens"], case["far"]
        n_pos = far
        S["positions"] = torch.randint(0, far, (M,), generator=g, device=dev, dtype=torch.int32) if M < far \
            else torch.arange(M, device=dev, dtype=torch.int32) % far
    else:
        news, ctxs = _lengths(case)
        B, M, page = case["batch"], sum(news), case["page"]
        per = -(-max(ctxs) // page)
        pages = B * per + 3
        S["page_table"] = torch.randperm(pages, generator=g, device=dev)[:B * per].view(B, per).to(torch.int32)
        S["ctx_len"] = torch.tensor(ctxs, dtype=torch.int32, device=dev)
        cu = [0]
        for n in news:
            cu.append(cu[-1] + n)
        S["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        n_pos = max(ctxs)
    S["M"] = M
    # the input projections' output: queries and gates joint per head, keys and values beside them
    joint = rn(M, HQ, 2, D).to(bf)
    S["q"], S["gate"] = joint[:, :, 0], joint[:, :, 1]
    kv = rn(M, 2 * HKV, D).to(bf)
    S["k"], S["v"] = kv[:, :HKV], kv[:, HKV:]
    if op != "attend":
        S["q_norm"], S["k_norm"] = 1 + 0.1 * rn(D), 1 + 0.1 * rn(D)
        inv = BASE ** (-torch.arange(0, ROT, 2, dtype=torch.float64, device=dev) / ROT)
        ang = torch.arange(n_pos, dtype=torch.float64, device=dev)[:, None] * inv
        S["rope"] = torch.cat([ang.cos(), ang.sin()], 1).float()
    if op in ("attend", "step"):
        S["qn"] = rn(M, HQ, D).to(bf)            # normed and rotated queries (a step overwrites them)
        S["out"] = torch.empty(M, HQ, D, dtype=bf, device=dev)
    else:
        S["qn"] = torch.empty(M, HQ, D, dtype=bf, device=dev)
    if op == "norm":
        S["kn"] = torch.empty(M, HKV, D, dtype=bf, device=dev)
    else:
        if case["fmt"] == "bf16":
            S["kc"], S["vc"] = rn(pages, HKV, page, D).to(bf), rn(pages, HKV, page, D).to(bf)
        else:
            kp = _pack4(rn(pages, HKV, page, D), pages, page)
            vp = _pack4(rn(pages, HKV, page, D), pages, page)
            S["cache4"] = _records(*kp, *vp)
        if op in ("append", "step") and case["fmt"] == "q4":
            S["kr"], S["vr"] = (torch.empty(M, HKV, D, dtype=bf, device=dev) for _ in range(2))
    if own:
        from gated_deltanet_linear_02_gb300 import ops
        S["ops"] = ops
        if op != "attend":
            S["params"] = ops.make_attn_params(S["q_norm"], S["k_norm"], S["rope"], EPS)
        if op != "norm":
            S["cache"] = ops.make_kv_cache(S["kc"], S["vc"]) if case["fmt"] == "bf16" else ops.make_kv_cache(S["cache4"])
            S["plan"] = ops.make_paged_batch(S["page_table"], S["ctx_len"], S["M"], None if max(news) == 1 else S["cu"], max(news))
        if op in ("attend", "step"):
            S["ws"] = torch.empty(ops.attn_paged_workspace_size(S["plan"], S["cache"]), dtype=torch.uint8, device=dev)
    return S


# ---- one pass

def run(S):
    case = S["case"]
    op = case["op"]
    if own:
        ops = S["ops"]
        if op == "norm":
            ops.attn_qk_norm_rope(S["params"], S["q"], S["positions"], S["qn"], S["k"], S["kn"])
            return S["qn"], S["kn"]
        if op == "append":
            if case["fmt"] == "bf16":
                ops.kv_append(S["params"], S["plan"], S["cache"], S["k"], S["v"], S["q"], S["qn"])
                return S["kc"], S["vc"], S["qn"]
            ops.kv_append(S["params"], S["plan"], S["cache"], S["k"], S["v"])
            ops.kv_gather(S["plan"], S["cache"], S["kr"], S["vr"])
            return S["kr"], S["vr"]
        if op == "step":
            ops.kv_append(S["params"], S["plan"], S["cache"], S["k"], S["v"], S["q"], S["qn"])
        ops.attn_paged(S["plan"], S["cache"], S["qn"], S["out"], S["gate"], S["ws"])
        if op == "attend":
            return S["out"]
        if case["fmt"] == "bf16":
            return S["out"], S["kc"], S["vc"]
        ops.kv_gather(S["plan"], S["cache"], S["kr"], S["vr"])
        return S["out"], S["kr"], S["vr"]
    if op == "norm":
        at = S["rope"][S["positions"].long()]
        return tuple(_norm_rope(x.float(), w, at).to(torch.bfloat16) for x, w in ((S["q"], S["q_norm"]), (S["k"], S["k_norm"])))
    seq, pos = _places(S)
    if op == "append":
        wide = case["fmt"] == "q4"                       # codes are decided next to borders: 64 bits
        at = S["rope"][pos]
        k = _norm_rope(S["k"].double(), S["k_norm"].double(), at.double()) if wide else _norm_rope(S["k"].float(), S["k_norm"], at)
        if wide:
            kq, vq = _quantise(k), _quantise(S["v"].double())
            _store4(S, seq, pos, kq, vq)
            return _held(kq), _held(vq)
        _store16(S, seq, pos, k, S["v"])
        return S["kc"], S["vc"], _norm_rope(S["q"].float(), S["q_norm"], at).to(torch.bfloat16)
    q = S["qn"].float()
    if op == "step":
        at = S["rope"][pos]
        q = _norm_rope(S["q"].float(), S["q_norm"], at).to(torch.bfloat16).float()
        if case["fmt"] == "q4":
            kq, vq = _quantise(_norm_rope(S["k"].double(), S["k_norm"].double(), at.double())), _quantise(S["v"].double())
            _store4(S, seq, pos, kq, vq)
            return _attend(S, q, seq, pos), _held(kq), _held(vq)
        _store16(S, seq, pos, _norm_rope(S["k"].float(), S["k_norm"], at), S["v"])
        return _attend(S, q, seq, pos), S["kc"], S["vc"]
    return _attend(S, q, seq, pos)


def _places(S):
    """Sequence and position of each new token."""
    t = torch.arange(S["M"], device=S["cu"].device)
    cu = S["cu"].long()
    seq = torch.searchsorted(cu[1:], t, right=True)
    return seq, S["ctx_len"].long()[seq] - (cu[seq + 1] - t)


def _norm_rope(x, w, at):
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    c, s = at[:, None, :ROT // 2], at[:, None, ROT // 2:]
    a, b = y[..., :ROT // 2], y[..., ROT // 2:ROT]
    return torch.cat([a * c - b * s, b * c + a * s, y[..., ROT:]], -1)


def _quantise(x):
    """Codes, steps and zeros (64 bits) of [M][2][256]."""
    v = x.unflatten(-1, (NG, GROUP))
    lo, hi = v.amin(-1), v.amax(-1)
    z = lo.to(torch.bfloat16).double()
    s = ((hi - lo) / 15).to(torch.bfloat16).double()
    c = ((v - z[..., None]) / s[..., None]).round().clamp(0, 15)
    return torch.where(s[..., None] > 0, c, torch.zeros_like(c)), s, z


def _held(q):
    """The values that 4-bit rows stand for."""
    c, s, z = q
    return (c * s[..., None] + z[..., None]).flatten(-2).to(torch.bfloat16)


def _store16(S, seq, pos, k, v):
    page = S["case"]["page"]
    p = S["page_table"].long()[seq, pos // page]
    S["kc"][p, :, pos % page] = k.to(torch.bfloat16)
    S["vc"][p, :, pos % page] = v


def _store4(S, seq, pos, kq, vq):
    page = S["case"]["page"]
    p, off = S["page_table"].long()[seq, pos // page], pos % page
    rec = S["cache4"]
    M = seq.numel()
    col = 0
    parts = []
    for c, _, _ in (kq, vq):
        n = c.to(torch.uint8).view(M, HKV, NG, 8, 4, 2)
        parts.append((n[..., 0] | (n[..., 1] << 4)).transpose(2, 3).reshape(M, HKV, 128))
    for _, s, z in (kq, vq):
        parts.append(torch.stack([s, z], -1).to(torch.bfloat16).view(M, HKV, 2 * NG).view(torch.uint8))
    for b in parts:                                   # four parts of a record
        w = b.shape[-1]
        at = col + (off % REC)[:, None] * w + torch.arange(w, device=off.device)
        rec[p[:, None, None], torch.arange(HKV, device=off.device)[None, :, None], (off // REC)[:, None, None], at[:, None, :]] = b
        col += REC * w


def _cached(S):
    """Keys and values of each sequence in order, fp32 [B][2][L][256]."""
    page, table = S["case"]["page"], S["page_table"].long()
    B, per = table.shape
    if S["case"]["fmt"] == "bf16":
        pick = lambda t: t[table].permute(0, 2, 1, 3, 4).reshape(B, HKV, per * page, D).float()  # noqa: E731
        return pick(S["kc"]), pick(S["vc"])
    rec = S["cache4"][table].permute(0, 2, 1, 3, 4).reshape(B, HKV, per * page // REC, REC_BYTES)
    half = REC * 128

    def values(codes, sz):
        b = codes.reshape(B, HKV, per * page, 8, NG, 4).transpose(3, 4)
        c = torch.stack([b & 15, b >> 4], -1).reshape(B, HKV, per * page, NG, GROUP).float()
        sz = sz.contiguous().view(torch.bfloat16).reshape(B, HKV, per * page, NG, 2).float()
        return (c * sz[..., :1] + sz[..., 1:]).flatten(-2)
    return values(rec[..., :half], rec[..., 2 * half:2 * half + 256]), values(rec[..., half:2 * half], rec[..., 2 * half + 256:])


def _attend(S, q, seq, pos):
    K, V = _cached(S)
    B, L = K.shape[0], K.shape[2]
    cu = S["cu"].long()
    n = max(_lengths(S["case"])[0])
    t = torch.arange(n, device=q.device)
    tok = torch.minimum(cu[:-1, None] + t, cu[1:, None] - 1)             # [B][n], the last one repeated
    qb = q[tok].unflatten(2, (HKV, HQ // HKV)).permute(0, 2, 1, 3, 4).reshape(B, HKV, n * (HQ // HKV), D)
    s = torch.matmul(qb, K.transpose(-1, -2)).div_(math.sqrt(D)).view(B, HKV, n, HQ // HKV, L)
    hide = torch.arange(L, device=q.device) > pos[tok][:, None, :, None, None]
    s.masked_fill_(hide, -math.inf)
    s.sub_(s.amax(-1, keepdim=True)).exp_()
    s.div_(s.sum(-1, keepdim=True))
    o = torch.matmul(s.view(B, HKV, n * (HQ // HKV), L), V).view(B, HKV, n, HQ // HKV, D).permute(0, 2, 1, 3, 4).reshape(B, n, HQ, D)
    o = o[seq, torch.arange(S["M"], device=q.device) - cu[seq]]
    return (o * torch.sigmoid(S["gate"].float())).to(torch.bfloat16)


# ---- the definition in 64 bits, token by token and sequence by sequence

def _turn64(x, w, rows):
    x = x.double()
    r = (x.pow(2).sum(-1) / D + EPS).pow(-0.5)
    y = x * r[..., None] * w.double()
    h = ROT // 2
    z = torch.complex(y[..., :h], y[..., h:ROT]) * torch.complex(rows[:, :h].double(), rows[:, h:].double())[:, None]
    return torch.cat([z.real, z.imag, y[..., ROT:]], -1)


def _four_bits64(x):
    out = torch.empty_like(x)
    for g in range(NG):
        v = x[..., g * GROUP:(g + 1) * GROUP]
        lo = v.min(-1, keepdim=True).values
        hi = v.max(-1, keepdim=True).values
        z, s = lo.bfloat16().double(), ((hi - lo) / 15.0).bfloat16().double()
        out[..., g * GROUP:(g + 1) * GROUP] = z + s * torch.clamp(torch.round((v - z) / s), 0, 15)
    return out


def exact(case, seed):
    S = prepare(case, seed)
    if case["op"] == "norm":
        rows = S["rope"][S["positions"].long()]
        return _turn64(S["q"], S["q_norm"], rows), _turn64(S["k"], S["k_norm"], rows)
    news, ctxs = _lengths(case)
    page, dev = case["page"], S["cu"].device
    where = [torch.arange(c - n, c, device=dev) for n, c in zip(news, ctxs)]
    pos = torch.cat(where)
    k = v = q = None
    if case["op"] != "attend":
        rows = S["rope"][pos]
        k, v, q = _turn64(S["k"], S["k_norm"], rows), S["v"].double(), _turn64(S["q"], S["q_norm"], rows)
    if case["op"] == "append":
        if case["fmt"] == "q4":
            return _four_bits64(k), _four_bits64(v)
        kc, vc, m = S["kc"].double(), S["vc"].double(), 0
        for b, at in enumerate(where):
            p = S["page_table"][b].long()[at // page]
            kc[p, :, at % page], vc[p, :, at % page] = k[m:m + len(at)], v[m:m + len(at)]
            m += len(at)
        return kc, vc, q
    out, m, ks, vs = [], 0, [], []
    if case["op"] == "step" and case["fmt"] == "bf16":
        kc, vc = S["kc"].double(), S["vc"].double()
    for b, at in enumerate(where):
        n, L = len(at), ctxs[b]
        p = S["page_table"][b].long()[: -(-L // page)]
        if case["fmt"] == "bf16":
            K, Vv = (t[p].transpose(0, 1).flatten(1, 2)[:, :L].double() for t in (S["kc"], S["vc"]))
        else:
            K, Vv = (t[:, :L] for t in _read64(S["cache4"][p]))
        qq = S["qn"][m:m + n].double()
        if case["op"] == "step":
            K, Vv = K.clone(), Vv.clone()
            kb, vb = k[m:m + n].transpose(0, 1), v[m:m + n].transpose(0, 1)
            if case["fmt"] == "q4":
                kb, vb = _four_bits64(kb), _four_bits64(vb)
                ks.append(kb.transpose(0, 1))
                vs.append(vb.transpose(0, 1))
            else:
                kc[p[at // page], :, at % page], vc[p[at // page], :, at % page] = kb.transpose(0, 1), vb.transpose(0, 1)
            K[:, at], Vv[:, at] = kb, vb
            qq = q[m:m + n]
        o = torch.empty(n, HQ, D, dtype=torch.float64, device=dev)
        see = torch.arange(L, device=dev) <= at[:, None]
        for h in range(HQ):
            w = torch.softmax((qq[:, h] @ K[h // 8].T / 16.0).masked_fill(~see, -math.inf), -1)
            o[:, h] = w @ Vv[h // 8]
        out.append(o / (1 + torch.exp(-S["gate"][m:m + n].double())))
        m += n
    if case["op"] == "attend":
        return torch.cat(out)
    return (torch.cat(out), kc, vc) if case["fmt"] == "bf16" else (torch.cat(out), torch.cat(ks), torch.cat(vs))


def _read64(rec):
    """Records [pages][2][page / 16][bytes] -> keys, values [2][rows][256]."""
    rec = rec.transpose(0, 1).flatten(1, 2)
    got = []
    for at, sz in ((0, 4096), (2048, 4352)):
        b = rec[..., at:at + 2048].reshape(HKV, -1, 8, NG, 4).long()
        f = rec[..., sz:sz + 256].contiguous().view(torch.bfloat16).reshape(HKV, -1, NG, 2).double()
        v = torch.empty(*b.shape, 2, dtype=torch.float64, device=rec.device)
        v[..., 0], v[..., 1] = b % 16, b // 16
        v = v.transpose(2, 3).flatten(3)
        got.append((f[..., 1:] + f[..., :1] * v).flatten(2))
    return got

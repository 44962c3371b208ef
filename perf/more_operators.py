"""The operators of an 8-bit decoder step around the 4-bit linears, as measurable cases.

Four operators, each in its plain form (elementary torch operations in 32 bits,
rounded once at the end) and as the calls a program makes of the library:

  norm    ``ops.add_rmsnorm_q8``: the residual's addition and the RMS norm, with the
          Q8 rows and scales that the W4A8 linears read
  store   ``ops.qk_norm_rope_kv8``: head norms, rotation, and the store of keys and
          values into a paged cache held in 8 bits, with one power-of-two scale for
          each 16 tokens of a head (``ops.dequantize_kv8`` reads it back)
  attn    ``ops.attention_kv8``: causal attention over that cache, whole or through a
          sliding window beside a few first tokens that stay visible
  logp    ``ops.token_logprobs``: log probabilities of given tokens, the entropy and
          the top alternatives of each row of logits

A case is a dict of plain values; ``op`` names the operator.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 16        # tokens of a head that share one scale
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the norm before the projections of one decoded token, where only latency counts
        dict(name="norm_t1_h2048", op="norm", T=1, H=2048, x="bf16", r="bf16"),
        # drafted tokens; f32 rows as the linears give them, an odd width
        dict(name="norm_t13_h5121", op="norm", T=13, H=5121, x="f32", r="bf16"),
        # a prompt of 4096 tokens in a wide model
        dict(name="norm_t4096_h8192", op="norm", T=4096, H=8192, x="bf16", r="bf16"),
        # one decoded token for each of 128 young requests: most blocks hold tokens already
        dict(name="store_b128_t1", op="store", B=128, new=1, ctx=60, Hq=32, Hkv=8, D=128, R=128, page=32, inter=False,
             inp="f32", out="bf16", norm=True, heads_first=True),
        # two prompts, 4096 tokens between them
        dict(name="store_b2_t2730", op="store", B=2, new=2730, ctx=777, Hq=32, Hkv=8, D=128, R=128, page=64, inter=False,
             inp="bf16", out="bf16", norm=True, heads_first=False),
        # one token of one request: latency alone
        dict(name="attn_b1_t1_1k", op="attn", B=1, new=1, ctx=1000, Hq=16, Hkv=4, D=64, page=16, dtype="bf16", window=0,
             sinks=0, heads_first=True),
        # a full decode batch over long contexts, the keys and values read once
        dict(name="attn_b64_t1_16k", op="attn", B=64, new=1, ctx=16384, Hq=32, Hkv=8, D=128, page=32, dtype="bf16",
             window=0, sinks=0, heads_first=True),
        # four drafted tokens each, a window of 4096 beside four first tokens over long contexts; seven query heads a key head
        dict(name="attn_b16_t4_w4096", op="attn", B=16, new=4, ctx=30001, Hq=28, Hkv=4, D=128, page=64, dtype="f16",
             window=4096, sinks=4, heads_first=False),
        # two pieces of long prompts behind what the cache has of them
        dict(name="attn_b2_t2048_6k", op="attn", B=2, new=2048, ctx=6000, Hq=32, Hkv=8, D=128, page=64, dtype="bf16",
             window=0, sinks=0, heads_first=True),
        # one sampled token with the alternatives shown beside it
        dict(name="logp_t1_v32000", op="logp", T=1, V=32000, x="f32", top=5),
        # drafted tokens of a batch, an odd vocabulary
        dict(name="logp_t32_v100003", op="logp", T=32, V=100003, x="f32", top=20),
        # the log probabilities of a prompt
        dict(name="logp_t2048_v131072", op="logp", T=2048, V=131072, x="bf16", top=20),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["norm", "store", "attn", "attn", "logp"])
    if op == "norm":
        return dict(op=op, T=_log(rng, 1, 4096), H=_log(rng, 100, 16384), x=rng.choice(["f32", "bf16", "f16"]),
                    r=rng.choice(["f32", "bf16", "f16"]))
    if op == "logp":
        return dict(op=op, T=_log(rng, 1, 2048), V=_log(rng, 1000, 262144), x=rng.choice(["f32", "bf16", "f16"]),
                    top=rng.choice([0, 1, 5, 20, 32]))
    Hkv = rng.randint(1, 8)
    heads = dict(Hq=Hkv * rng.choice([1, 2, 4, 5, 8]), Hkv=Hkv, page=rng.choice([16, 32, 64, 128]),
                 heads_first=rng.random() < 0.5)
    B = _log(rng, 1, 128)
    if op == "store":
        D = rng.choice([64, 80, 96, 128, 256])
        return dict(op=op, B=B, new=_log(rng, 1, 2730), ctx=_log(rng, 1, 4096), D=D, R=rng.choice([D, D // 32 * 16]),
                    inter=rng.random() < 0.4, inp=rng.choice(["f32", "bf16", "f16"]), out=rng.choice(["bf16", "f16"]),
                    norm=rng.random() < 0.7, **heads)
    window = rng.choice([0, 0, _log(rng, 1, 8192)])
    return dict(op=op, B=B, new=_log(rng, 1, 2048), ctx=_log(rng, 1, 32768), D=rng.choice([64, 80, 128]),
                dtype=rng.choice(["bf16", "f16"]), window=window, sinks=rng.choice([0, 1, 4, 100]) if window else 0, **heads)


def _cost(case):
    w = work(case)
    return w["bytes"] + w["flops"] / 250


def draw(rng):
    top = {}
    for c in listed():
        top[c["op"]] = max(top.get(c["op"], 0.0), _cost(c))
    while True:
        c = _draw(rng)
        if c["op"] == "attn" and c["B"] * (c["ctx"] + c["new"]) * c["Hkv"] * c["D"] > 64 * 16400 * 8 * 128:
            continue    # a cache beyond the largest listed one
        if c["op"] == "attn" and c["B"] * c["new"] * (c["ctx"] + c["new"]) * c["Hq"] > 2 * 2048 * 8192 * 32:
            continue    # scores of the plain form beyond the largest listed ones
        if _cost(c) <= top[c["op"]]:
            return c


def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi], the largest always hi."""
    return [hi - (hi - lo) * i // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _lengths(case):
    """Lengths in the cache and of the new tokens (their order is shuffled by the seed)."""
    return _spread(case["ctx"] // 2, case["ctx"], case["B"]), _spread((case["new"] + 1) // 2, case["new"], case["B"])


def _pairs(c, n, window, sinks):
    """(query, key) pairs that the mask leaves, and keys that some query sees, of one request."""
    p = np.arange(c, c + n, dtype=np.int64)
    lo = np.maximum(p - window + 1, 0) if window else np.zeros_like(p)
    first = np.minimum(lo, sinks)
    return int((p - lo + 1 + first).sum()), int(c + n - lo[0] + min(sinks, lo[0]))


def work(case):
    op = case["op"]
    if op == "norm":
        n = case["T"] * case["H"]
        return {"bytes": n * (BYTES[case["x"]] + 2 * BYTES[case["r"]] + 1) + 4 * case["H"] + 4 * case["T"], "flops": 8 * n}
    if op == "logp":
        n = case["T"] * case["V"]
        return {"bytes": n * BYTES[case["x"]] + case["T"] * (12 + 8 * case["top"]), "flops": 5 * n}
    ctx, new = _lengths(case)
    T, D = sum(new), case["D"]
    if op == "store":
        kv = T * case["Hkv"] * D * 2
        blocks = sum(-(-(c + n) // BLOCK) - c // BLOCK for c, n in zip(ctx, new))
        held = sum(-(-(c + n) // case["page"]) * case["page"] for c, n in zip(ctx, new)) * case["Hkv"] * D * 2
        # the rows; queries and codes written; scale bytes read and written; positions and angles; the cache's values
        return {"bytes": T * (case["Hq"] + 2 * case["Hkv"]) * D * BYTES[case["inp"]] + T * case["Hq"] * D * 2 + kv
                + blocks * case["Hkv"] * 4 + T * (4 + 4 * case["R"]) + 3 * held,
                "flops": T * (case["Hq"] + case["Hkv"]) * D * 7 + 3 * kv + held}
    both = [_pairs(c, n, case["window"], case["sinks"]) for c, n in zip(ctx, new)]
    keys = sum(k for _, k in both)
    return {"bytes": keys * case["Hkv"] * (2 * D + 2 / BLOCK) + T * case["Hq"] * D * 4,
            "flops": 4 * sum(p for p, _ in both) * case["Hq"] * D}


# ---------------------------------------------------------------- inputs

def _requests(case, seed):
    """Lengths, offsets and a block table, as a scheduler keeps them on the GPU."""
    g = np.random.default_rng(seed)
    ctx, new = _lengths(case)
    order = g.permutation(case["B"])
    ctx, new = np.array(ctx, np.int32)[order], np.array(new, np.int32)[order]
    page = case["page"]
    width = -(-(case["ctx"] + case["new"]) // page)
    need = -(-(ctx + new) // page)
    pages = int(need.sum()) + 3
    ids = g.permutation(pages).astype(np.int32)
    col = np.arange(width)
    at = np.cumsum(need) - need
    table = np.where(col < need[:, None], ids[np.minimum(at[:, None] + col, pages - 1)], -1).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    pos = np.concatenate([np.arange(c, c + n) for c, n in zip(ctx, new)]).astype(np.int32)
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    return dict(case=case, pages=pages, tokens=int(new.sum()), ctx=cuda(ctx), cu=cuda(cu), table=cuda(table),
                positions=cuda(pos))


def _cache(case, pages, gen):
    """Codes of a key or value cache, seen as [page, token, head, value], and their scale bytes."""
    t, H, D = case["page"], case["Hkv"], case["D"]
    shape = (pages, H, t, D) if case["heads_first"] else (pages, t, H, D)
    codes = torch.empty(shape, dtype=torch.int8, device="cuda")
    for part in codes.split(max(1, (1 << 28) // (H * t * D))):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda", dtype=torch.bfloat16).mul_(32).round_().clamp_(-127, 127))
    scales = torch.randint(121, 124, (pages, H, t // BLOCK), generator=gen, device="cuda", dtype=torch.uint8)
    return (codes.transpose(1, 2) if case["heads_first"] else codes), scales


def prepare(case, seed):
    op = case["op"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    randn = lambda *s, dtype=torch.float32: torch.randn(s, generator=gen, device="cuda", dtype=dtype)  # noqa: E731
    if op == "norm":
        return dict(case=case, x=randn(case["T"], case["H"]).to(DTYPES[case["x"]]),
                    r=(2 * randn(case["T"], case["H"])).to(DTYPES[case["r"]]), w=1 + 0.1 * randn(case["H"]))
    if op == "logp":
        T, V = case["T"], case["V"]
        x = randn(T, V, dtype=DTYPES[case["x"]]).mul_(2.0)
        # most tokens are likely ones: their logit stands out
        ids = torch.randint(0, V, (T,), generator=gen, device="cuda")
        lift = torch.rand((T, 1), generator=gen, device="cuda") * 14
        x.scatter_add_(1, ids[:, None], lift.to(x.dtype))
        return dict(case=case, x=x, ids=ids.to(torch.int32))
    s = _requests(case, seed)
    s["k"], s["k_scale"] = _cache(case, s["pages"], gen)
    s["v"], s["v_scale"] = _cache(case, s["pages"], gen)
    if op == "attn":
        s["q"] = (1.5 * randn(s["tokens"], case["Hq"], case["D"])).to(DTYPES[case["dtype"]])
        return s
    D, R = case["D"], case["R"]
    top = case["ctx"] + case["new"]
    inv = 10000.0 ** (-np.arange(R // 2, dtype=np.float64) / max(1, R // 2))
    ang = np.arange(top, dtype=np.float64)[:, None] * inv
    s["cos_sin"] = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
    s["qkv"] = randn(s["tokens"], (case["Hq"] + 2 * case["Hkv"]) * D).to(DTYPES[case["inp"]])
    s["wq"], s["wk"] = (1 + 0.1 * randn(D), 1 + 0.1 * randn(D)) if case["norm"] else (None, None)
    return s


# ---------------------------------------------------------------- plain forms

def _norm_plain(s):
    h = (s["x"].float() + s["r"].float()).to(s["r"].dtype)
    hf = h.float()
    y = hf * torch.rsqrt(hf.square().mean(-1, keepdim=True) + EPS) * s["w"]
    sx = y.abs().amax(-1) / 127
    q = torch.round(y / torch.where(sx > 0, sx, 1.0)[:, None]).clamp(-127, 127)
    return dict(values=(q * sx[:, None]).to(torch.bfloat16), scales=sx, residual=h)


def _places(s):
    """Of each token: its page, its place there, and the block of 16 tokens (of all pages) that it lies in."""
    page = s["case"]["page"]
    t = torch.arange(s["tokens"], device="cuda")
    cu = s["cu"].long()
    b = torch.searchsorted(cu[1:], t, right=True)
    pos = s["ctx"].long()[b] + t - cu[b]
    pid, off = s["table"].long()[b, pos // page], pos % page
    return b, pos, pid, off, pid * (page // BLOCK) + off // BLOCK


def _exponent(top):
    """The least e >= -127 with top <= 127 * 2^e."""
    m, e = torch.frexp(top)
    return torch.where(top > 0, e - 7 + (m > 127 / 128).to(e.dtype), -127).clamp(min=-127).long()


def _append_plain(codes, scales, x, s):
    """x [tokens, Hkv, D] f32 into codes [page, token, head, value] and scales [page, head, block], both in place."""
    P, page, H, D = codes.shape
    b, pos, pid, off, blk = _places(s)
    n = page // BLOCK
    byte = scales.transpose(1, 2).reshape(P * n, H).long()
    # tokens of a block that stay: those of the request before its new ones
    kept = torch.zeros(P * n, dtype=torch.long, device="cuda")
    kept.scatter_reduce_(0, blk, torch.minimum(s["ctx"].long()[b] - pos // BLOCK * BLOCK, torch.tensor(BLOCK, device="cuda")).clamp(min=0),
                         "amax")
    top = torch.zeros((P * n, H), device="cuda")
    top.scatter_reduce_(0, blk[:, None].expand(-1, H), x.abs().amax(-1), "amax")
    touched = torch.zeros(P * n, dtype=torch.bool, device="cuda")
    touched[blk] = True
    e = _exponent(top)
    e = torch.where((kept > 0)[:, None], torch.maximum(e, byte - 127), e)
    e = torch.where(touched[:, None], e, byte - 127)
    # the kept tokens' codes under the new scale
    at = torch.nonzero(touched & (kept > 0))[:, 0]
    tok = torch.arange(BLOCK, device="cuda")
    p, o = (at // n)[:, None].expand(-1, BLOCK), (at % n * BLOCK)[:, None] + tok
    old = codes[p, o].float()                                           # [blocks, 16, H, D]
    new = torch.round(torch.ldexp(old, (byte[at] - 127 - e[at])[:, None, :, None]))
    keep = (tok < kept[at][:, None])[..., None, None]
    codes[p, o] = torch.where(keep, new, old).to(torch.int8)
    codes[pid, off] = torch.round(torch.ldexp(x, -e[blk][..., None])).clamp(-127, 127).to(torch.int8)
    scales.copy_((e + 127).view(P, n, H).transpose(1, 2))


def _values(codes, scales):
    """What codes and scale bytes stand for, [page, token, head, value] in f32."""
    e = (scales.int() - 127).transpose(1, 2).repeat_interleave(BLOCK, 1)
    return torch.ldexp(codes.float(), e[..., None])


def _store_plain(s):
    case = s["case"]
    T, Hq, Hkv, D, R = s["tokens"], case["Hq"], case["Hkv"], case["D"], case["R"]
    x = s["qkv"].float().view(T, Hq + 2 * Hkv, D)
    cs = s["cos_sin"][s["positions"].long()][:, None]
    cos, sin = cs[..., : R // 2], cs[..., R // 2:]

    def head(h, w):
        if w is not None:
            h = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * w
        r = h[..., :R]
        if case["inter"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r[..., : R // 2], r[..., R // 2:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([r, h[..., R:]], -1)

    q = head(x[:, :Hq], s["wq"]).to(DTYPES[case["out"]])
    _append_plain(s["k"], s["k_scale"], head(x[:, Hq: Hq + Hkv], s["wk"]), s)
    _append_plain(s["v"], s["v_scale"], x[:, Hq + Hkv:], s)
    return dict(q=q, k=_values(s["k"], s["k_scale"]).to(torch.bfloat16), v=_values(s["v"], s["v_scale"]).to(torch.bfloat16))


def _attn_plain(s):
    case = s["case"]
    B, Hq, Hkv, D, page = (case[k] for k in ("B", "Hq", "Hkv", "D", "page"))
    G, T, L = Hq // Hkv, case["new"], case["ctx"] + case["new"]
    ctx, cu, q = s["ctx"].long(), s["cu"].long(), s["q"]
    n = cu[1:] - cu[:-1]
    key = torch.arange(L, device=q.device)
    real = key < (ctx + n)[:, None]
    pid = s["table"].long()[:, key // page].clamp(min=0)                  # [B, L]

    def gather(codes, scales):
        e = scales.transpose(1, 2)[pid, (key % page // BLOCK).expand(B, L)].int() - 127   # [B, L, Hkv]
        return torch.ldexp(codes[pid, key % page].float(), e[..., None])

    i = torch.arange(T, device=q.device)
    row = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)                   # [B, T]
    qf = q.float()[row].view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    score = (qf @ gather(s["k"], s["k_scale"]).permute(0, 2, 3, 1)).view(B, Hkv, T, G, L)
    score *= 1 / math.sqrt(D)
    p = ctx[:, None] + i                                                  # [B, T] positions
    see = (key <= p[..., None]) & real[:, None, :]
    if case["window"]:
        see &= (p[..., None] - key < case["window"]) | (key < case["sinks"])
    score.masked_fill_(~see[:, None, :, None, :], -math.inf)
    score -= score.amax(-1, keepdim=True).clamp(min=-1e30)
    score.exp_()
    z = score.sum(-1, keepdim=True)
    score /= torch.where(z > 0, z, 1.0)
    v = torch.where(real[..., None, None], gather(s["v"], s["v_scale"]), 0.0)
    o = (score.view(B, Hkv, T * G, L) @ v.permute(0, 2, 1, 3)).view(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4)
    live = i < n[:, None]
    out = torch.empty_like(q)
    out[row[live]] = o.reshape(B, T, Hq, D)[live].to(q.dtype)
    return dict(out=out)


def _logp_plain(s):
    x, V, top = s["x"].float(), s["case"]["V"], s["case"]["top"]
    m = x.amax(-1, keepdim=True)
    d = x - m
    p = d.exp()
    z = p.sum(-1, keepdim=True)
    logz = z.log()
    entropy = logz[:, 0] - (p * d).sum(-1) / z[:, 0]
    del p
    logp = d.gather(1, s["ids"].long()[:, None])[:, 0] - logz[:, 0]
    # the order of (value, lowest index): whole numbers that sort like the floats, the index below them
    bits = (x + 0.0).view(torch.int32).long()
    keys = torch.where(bits >= 0, bits, -2 ** 31 - bits) * 2 ** 32 + (V - 1 - torch.arange(V, device=x.device))
    ids = V - 1 - torch.topk(keys, top, dim=-1, sorted=True)[0] % 2 ** 32
    return dict(logp=logp, entropy=entropy, top_ids=ids.int(), top_logp=d.gather(1, ids) - logz)


# ---------------------------------------------------------------- the library's calls

def _run_own(s):
    from w4a16_int4_quantized_gb300 import ops
    case = s["case"]
    op = case["op"]
    if op == "norm":
        q, sx, h, _ = ops.add_rmsnorm_q8(s["x"], s["r"], s["w"], eps=EPS)
        values = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
        return dict(values=torch.mul(q, sx[:, None], out=values), scales=sx, residual=h)
    if op == "logp":
        logp, entropy, ids, top = ops.token_logprobs(s["x"], s["ids"], top=case["top"])
        return dict(logp=logp, entropy=entropy, top_ids=ids, top_logp=top)
    cache = ops.Kv8Cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if op == "store":
        q = ops.qk_norm_rope_kv8(s["qkv"], case["Hq"], s["wq"], s["wk"], s["positions"], s["cos_sin"], s["table"],
                                 s["ctx"], s["cu"], cache, eps=EPS, interleaved=case["inter"],
                                 out_dtype=DTYPES[case["out"]])
        k, v = ops.dequantize_kv8(cache, torch.bfloat16)
        return dict(q=q, k=k, v=v)
    return dict(out=ops.attention_kv8(s["q"], cache, s["table"], s["ctx"], s["cu"], scale=1.0 / math.sqrt(case["D"]),
                                      max_len=case["ctx"] + case["new"], max_new=case["new"], window=case["window"],
                                      sinks=case["sinks"]))


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm_plain, "store": _store_plain, "attn": _attn_plain, "logp": _logp_plain}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _norm_exact, "store": _store_exact, "attn": _attn_exact, "logp": _logp_exact}[case["op"]](s)


def _norm_exact(s):
    h = (s["x"].double() + s["r"].double()).to(s["r"].dtype)
    d = h.double()
    y = d / torch.sqrt((d * d).sum(-1, keepdim=True) / d.shape[1] + EPS) * s["w"].double()
    sx = torch.linalg.vector_norm(y, ord=math.inf, dim=-1, keepdim=True) / 127.0
    return dict(values=torch.round(y / sx.clamp(min=1e-300)) * sx, scales=sx[:, 0], residual=h.double())


def _store_exact(s):
    case = s["case"]
    T, Hq, Hkv, D, R, page = s["tokens"], case["Hq"], case["Hkv"], case["D"], case["R"], case["page"]
    x = s["qkv"].double().view(T, -1, D)
    h = x[:, : Hq + Hkv]
    if case["norm"]:
        w = torch.cat([s["wq"].double().expand(Hq, D), s["wk"].double().expand(Hkv, D)])
        h = h / torch.sqrt((h * h).sum(-1, keepdim=True) / D + EPS) * w
    at = s["cos_sin"].double()[s["positions"].long()]
    turn = torch.complex(at[:, : R // 2], at[:, R // 2:])[:, None]
    if case["inter"]:
        z = torch.view_as_complex(h[..., :R].reshape(T, Hq + Hkv, R // 2, 2).contiguous()) * turn
        rot = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(h[..., : R // 2].contiguous(), h[..., R // 2: R].contiguous()) * turn
        rot = torch.cat([z.real, z.imag], -1)
    h = torch.cat([rot, h[..., R:]], -1)
    cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
    out = {}
    for name, new in (("k", h[:, Hq:]), ("v", x[:, Hq + Hkv:])):
        codes = s[name].double()
        unit = torch.exp2(s[name + "_scale"].double() - 127.0)            # [page, head, block]
        for b, c in enumerate(ctx):
            n = cu[b + 1] - cu[b]
            # the request's blocks from the first that changes on, padded with what lies around the new tokens
            c0 = c // BLOCK * BLOCK
            pos = torch.arange(c0, -(-(c + n) // BLOCK) * BLOCK, device="cuda")
            pid, off = s["table"][b].long()[pos // page], pos % page
            raw = codes[pid, off].view(-1, BLOCK, Hkv, D)
            u = unit[pid, :, off // BLOCK].view(-1, BLOCK, Hkv)[:, 0]     # [blocks, head]
            vals = torch.zeros((pos.numel(), Hkv, D), dtype=torch.float64, device="cuda")
            vals[c - c0: c - c0 + n] = new[cu[b]: cu[b + 1]]
            peak = vals.view(-1, BLOCK, Hkv, D).abs().amax((1, 3))
            # 2^e: at least peak / 127, and not less than the unit of a block with kept tokens
            e = torch.ceil(torch.log2(torch.where(peak > 0, peak, 1.0) / 127.0))
            grown = torch.where(peak > 0, torch.exp2(e.clamp(min=-127.0)), 2.0 ** -127)
            if c > c0:
                grown[0] = torch.maximum(grown[0], u[0])
            k = torch.round(vals.view(-1, BLOCK, Hkv, D) / grown[:, None, :, None])
            if c > c0:
                k[0, : c - c0] = torch.round(raw[0, : c - c0] * (u[0] / grown[0])[:, None])
            end = c + n - c0 - (k.shape[0] - 1) * BLOCK                   # tokens of the last block
            k[-1, end:] = raw[-1, end:]
            codes[pid, off] = k.view(-1, Hkv, D)
            unit[pid, :, off // BLOCK] = grown[:, None].expand(-1, BLOCK, -1).reshape(-1, Hkv)
        out[name] = codes * unit.repeat_interleave(BLOCK, 2).transpose(1, 2)[..., None]
    return dict(q=h[:, :Hq], k=out["k"], v=out["v"])


def _attn_exact(s):
    case = s["case"]
    Hq, Hkv, D, page, window, sinks = (case[k] for k in ("Hq", "Hkv", "D", "page", "window", "sinks"))
    G = Hq // Hkv
    cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b, c in enumerate(ctx):
        n = cu[b + 1] - cu[b]
        blocks = s["table"][b, : -(-(c + n) // page)].long()
        j = torch.arange(c + n, device="cuda")
        back = (c + torch.arange(n, device="cuda"))[:, None] - j          # how far a key lies behind a query
        see = back >= 0
        if window:
            see &= (back < window) | (j < sinks)
        for h in range(Hkv):
            k, v = (s[x][blocks, :, h].reshape(-1, BLOCK, D).double()
                    * torch.pow(2.0, s[x + "_scale"][blocks, h].double() - 127).view(-1, 1, 1) for x in ("k", "v"))
            k, v = k.reshape(-1, D)[: c + n], v.reshape(-1, D)[: c + n]
            for g in range(h * G, h * G + G):
                sc = s["q"][cu[b]: cu[b + 1], g].double() @ k.T * D ** -0.5
                out[cu[b]: cu[b + 1], g] = torch.softmax(torch.where(see, sc, -math.inf), -1) @ v
    return dict(out=out)


def _logp_exact(s):
    top = s["case"]["top"]
    parts = []
    for x, ids in zip(s["x"].split(64), s["ids"].long().split(64)):
        order = torch.sort(x.float(), dim=-1, descending=True, stable=True)[1][:, :top]
        lp = torch.log_softmax(x.double(), -1)
        parts.append((lp.gather(1, ids[:, None])[:, 0], -(lp.exp() * lp).sum(-1), order.int(), lp.gather(1, order)))
    logp, entropy, ids, vals = (torch.cat(p) for p in zip(*parts))
    return dict(logp=logp, entropy=entropy, top_ids=ids, top_logp=vals)


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(k)) for k in range(6)]:
        print(c, work(c))

"""The operators of the decoder step around the 4-bit linears, as measurable cases.

Five operators, each in its plain form (elementary torch operations in 32 bits,
rounded once at the end) and as the calls a program makes of the library:

  plan    ``ops.draft_plan``: block tables, slots, positions and ancestor masks
          of the drafted tokens of a batch of requests, from their lengths
  rope    ``ops.qk_norm_rope``: the norm of each query and key head, the rotation
          by position, and the store of keys and values into a paged cache
  attn    ``ops.tree_attention``: attention of drafted token trees over that cache
  quant   ``ops.quantize_mxfp4`` / ``ops.dequantize_mxfp4``: microscaled 4-bit
          floating point (e2m1 values, one power-of-two scale for 32)
  linear  ``ops.linear_mxfp4`` (bf16 activations) and ``ops.quantize_mxfp4`` +
          ``ops.linear_mxfp4_a4`` (both sides in 4 bits) on such weights

A case is a dict of plain values; ``op`` names the operator.
"""
import math
import random

import numpy as np
import torch

own = False

BLOCK = 32        # values that share one scale
MAX_DRAFT = 128   # drafted tokens of one request
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one request, one token: the plan of an undrafted decode step, where only latency counts
        dict(name="plan_b1_t1", op="plan", B=1, new=1, ctx=1000, page=16, tree=False),
        # a full serving batch of drafted trees
        dict(name="plan_b256_t64", op="plan", B=256, new=64, ctx=8192, page=16, tree=True),
        # eight tokens of a small decode step, f32 as the linears give it
        dict(name="rope_t8_d64_f32", op="rope", T=8, Hq=16, Hkv=4, D=64, R=64, page=16, inter=False,
             inp="f32", out="bf16", heads_first=True),
        # a prompt of 4096 tokens; grouped heads, partly rotated
        dict(name="rope_t4096_d128", op="rope", T=4096, Hq=32, Hkv=8, D=128, R=128, page=32, inter=False,
             inp="bf16", out="bf16", heads_first=False),
        # one token of one request: an undrafted decode step
        dict(name="attn_b1_t1_1k", op="attn", B=1, new=1, Hq=16, Hkv=4, D=64, ctx=1000, page=16, dtype="bf16",
             heads_first=True),
        # a ragged batch of small trees: seven query heads to a key head, an odd context
        dict(name="attn_b8_t24_4k", op="attn", B=8, new=24, Hq=28, Hkv=4, D=128, ctx=4097, page=16, dtype="f16",
             heads_first=False),
        # a large batch of wide trees over long contexts
        dict(name="attn_b32_t64_8k", op="attn", B=32, new=64, Hq=32, Hkv=8, D=128, ctx=8192, page=32, dtype="bf16",
             heads_first=True),
        # the activations of a small ragged batch, odd length
        dict(name="quant_m7_k2047", op="quant", R=7, K=2047, inp="bf16"),
        # a weight matrix at load time (gate and up projections)
        dict(name="quant_n13312_k2048", op="quant", R=13312, K=2048, inp="f32"),
        # a decode step's square projection, one token
        dict(name="linear_m1_n2048", op="linear", M=1, N=2048, K=2048, a4=False, out="f32"),
        # drafted tokens of one request through gate and up
        dict(name="linear_m13_n13312", op="linear", M=13, N=13312, K=2048, a4=False, out="bf16"),
        # a prompt through gate and up, activations in 4 bits too
        dict(name="linear_a4_m2048_n13312", op="linear", M=2048, N=13312, K=2048, a4=True, out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw(rng):
    op = rng.choice(["plan", "rope", "attn", "attn", "quant", "linear", "linear"])
    if op == "plan":
        return dict(op=op, B=_log(rng, 1, 256), new=_log(rng, 1, MAX_DRAFT), ctx=_log(rng, 1, 8192),
                    page=rng.choice([16, 32, 64]), tree=rng.random() < 0.7)
    if op == "rope":
        D = rng.choice([32, 64, 80, 96, 128, 256])
        Hkv = rng.randint(1, 8)
        return dict(op=op, T=_log(rng, 1, 4096), Hq=Hkv * rng.choice([1, 2, 4, 7]), Hkv=Hkv, D=D,
                    R=rng.choice([D, D // 32 * 16]), page=rng.choice([16, 32, 64]), inter=rng.random() < 0.4,
                    inp=rng.choice(["f32", "bf16", "f16"]), out=rng.choice(["bf16", "f16"]),
                    heads_first=rng.random() < 0.5)
    if op == "attn":
        Hkv = rng.randint(1, 8)
        return dict(op=op, B=_log(rng, 1, 32), new=_log(rng, 1, MAX_DRAFT), Hq=Hkv * rng.choice([1, 2, 4, 5, 8]),
                    Hkv=Hkv, D=rng.choice([64, 80, 128]), ctx=_log(rng, 1, 8192), page=rng.choice([16, 32, 64]),
                    dtype=rng.choice(["bf16", "f16"]), heads_first=rng.random() < 0.5)
    if op == "quant":
        return dict(op=op, R=_log(rng, 1, 13312), K=_log(rng, 31, 4096), inp=rng.choice(["f32", "bf16", "f16"]))
    a4 = rng.random() < 0.5
    return dict(op=op, M=_log(rng, 17, 2048) if a4 else _log(rng, 1, 16), N=_log(rng, 100, 13312),
                K=32 * _log(rng, 4, 128), a4=a4, out="bf16" if a4 else rng.choice(["f32", "bf16"]))


def draw(rng):
    top = {}
    for c in listed():
        w = work(c)
        top[c["op"]] = max(top.get(c["op"], 0.0), w["bytes"] + w["flops"] / 250)
    while True:
        c = _draw(rng)
        w = work(c)
        if w["bytes"] + w["flops"] / 250 <= top[c["op"]]:
            return c


def _spread(lo, hi, n):
    """n whole numbers spread evenly over [lo, hi], the largest always hi."""
    return [hi - (hi - lo) * i // max(1, n - 1) if n > 1 else hi for i in range(n)]


def _lengths(case):
    """Context and drafted lengths of the batch (their order is shuffled by the seed)."""
    ctx = _spread(case["ctx"] // 2, case["ctx"], case["B"])
    new = _spread((case["new"] + 1) // 2, case["new"], case["B"])
    return ctx, new


def work(case):
    op = case["op"]
    if op == "plan":
        ctx, new = _lengths(case)
        tok = sum(new)
        pages = sum(-(-(c + n) // case["page"]) - -(-c // case["page"]) for c, n in zip(ctx, new))
        # lengths, parents, the free pages taken; table entries, offsets, slots, positions, masks
        return {"bytes": 8 * case["B"] + 4 * tok + 8 * pages + 4 * (case["B"] + 1) + tok * (8 + 4 + 16) + 4,
                "flops": 0}
    if op == "rope":
        n = case["T"] * (case["Hq"] + 2 * case["Hkv"]) * case["D"]
        el = {"f32": 4, "bf16": 2, "f16": 2}
        rot = case["T"] * (case["Hq"] + case["Hkv"])
        return {"bytes": n * (el[case["inp"]] + el[case["out"]]) + case["T"] * (4 * case["R"] + 12) + 8 * case["D"],
                "flops": rot * (4 * case["D"] + 3 * case["R"])}
    if op == "attn":
        ctx, new = _lengths(case)
        kv = sum(c + n for c, n in zip(ctx, new)) * case["Hkv"] * case["D"] * 4
        qo = sum(new) * case["Hq"] * case["D"] * 4
        fl = sum(4 * n * (c + n) for c, n in zip(ctx, new)) * case["Hq"] * case["D"]
        return {"bytes": kv + qo + sum(new) * 16, "flops": fl}
    nb = -(-case["K"] // BLOCK)
    if op == "quant":
        # the input; codes and scales written and read back; the values they stand for, in bf16
        el = {"f32": 4, "bf16": 2, "f16": 2}[case["inp"]]
        return {"bytes": case["R"] * (case["K"] * (el + 2) + 2 * nb * 17), "flops": 0}
    y = {"f32": 4, "bf16": 2}[case["out"]]
    return {"bytes": case["N"] * nb * 17 + case["M"] * case["K"] * 2 + case["M"] * case["N"] * y,
            "flops": 2 * case["M"] * case["N"] * case["K"]}


# ---------------------------------------------------------------- inputs

def _trees(new, tree, g):
    """Parents of each request's drafted tokens: an earlier token of the request, or -1 for a root."""
    parents = []
    for n in new:
        i = np.arange(n)
        # each token hangs on one of the few tokens before it: branches of a beam; a chain without `tree`
        p = i - 1 - (np.floor(g.random(n) * 6).astype(np.int64) if tree else 0)
        parents.append(np.maximum(p, -1))
    return np.concatenate(parents).astype(np.int32)


def _requests(case, seed, tree=True):
    """Lengths, parents and a half-filled block table, as a scheduler keeps them on the GPU."""
    g = np.random.default_rng(seed)
    ctx, new = _lengths(case)
    order = g.permutation(case["B"])
    ctx, new = np.array(ctx, np.int32)[order], np.array(new, np.int32)[order]
    page = case["page"]
    width = -(-(case["ctx"] + case["new"]) // page)
    have, need = -(-ctx // page), -(-(ctx + new) // page)
    pages = int(need.sum()) + 7
    ids = g.permutation(pages).astype(np.int32)
    table = np.full((case["B"], width), -1, np.int32)
    at = 0
    for b in range(case["B"]):
        table[b, : have[b]] = ids[at: at + have[b]]
        at += have[b]
    cuda = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    return dict(case=case, pages=pages, tokens=int(new.sum()), ctx=cuda(ctx), new=cuda(new),
                parents=cuda(_trees(new, tree, g)), free=cuda(ids[at:].copy()), table=cuda(table))


def _cache(case, pages, gen, dtype):
    """Key or value cache, seen as [page, token, head, value], in either order of tokens and heads."""
    P, t, H, D = pages, case["page"], case["Hkv"], case["D"]
    if case["heads_first"]:
        return torch.randn((P, H, t, D), generator=gen, device="cuda", dtype=dtype).transpose(1, 2)
    return torch.randn((P, t, H, D), generator=gen, device="cuda", dtype=dtype)


def prepare(case, seed):
    op = case["op"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    randn = lambda *s, dtype=torch.float32: torch.randn(s, generator=gen, device="cuda", dtype=dtype)  # noqa: E731
    if op == "plan":
        return _requests(case, seed, case["tree"])
    if op == "rope":
        T, D, R = case["T"], case["D"], case["R"]
        dt, do = DTYPES[case["inp"]], DTYPES[case["out"]]
        g = np.random.default_rng(seed)
        pages = -(-T // case["page"]) + 3
        slots = np.sort(g.permutation(pages * case["page"])[:T]).astype(np.int64)
        top = T + 512
        pos = np.arange(T, dtype=np.int32) + int(g.integers(0, 512))
        inv = 10000.0 ** (-np.arange(R // 2, dtype=np.float64) / max(1, R // 2))
        ang = np.arange(top, dtype=np.float64)[:, None] * inv
        cos_sin = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
        return dict(case=case, qkv=randn(T, (case["Hq"] + 2 * case["Hkv"]) * D).to(dt),
                    wq=1 + 0.1 * randn(D), wk=1 + 0.1 * randn(D), cos_sin=torch.from_numpy(cos_sin).cuda(),
                    positions=torch.from_numpy(pos).cuda(), slots=torch.from_numpy(slots).cuda(),
                    k=_cache(case, pages, gen, do), v=_cache(case, pages, gen, do))
    if op == "attn":
        s = _requests(case, seed)
        plan = _plan_plain(s)
        dt = DTYPES[case["dtype"]]
        s.update(cu=plan["cu"], mask=plan["mask"], table=plan["table"],
                 q=(1.5 * randn(s["tokens"], case["Hq"], case["D"])).to(dt),
                 k=_cache(case, s["pages"], gen, dt), v=_cache(case, s["pages"], gen, dt))
        return s
    if op == "quant":
        return dict(case=case, x=(0.02 * randn(case["R"], case["K"])).to(DTYPES[case["inp"]]))
    w, sw = _pack(*_quantize_plain(0.02 * randn(case["N"], case["K"])))
    return dict(case=case, x=randn(case["M"], case["K"]).to(torch.bfloat16), w=w, sw=sw)


# ---------------------------------------------------------------- plain forms

def _plan_plain(s):
    case, page = s["case"], s["case"]["page"]
    ctx, table, free, cap = s["ctx"].long(), s["table"], s["free"], s["parents"].numel()
    n = s["new"].long().clamp(0, MAX_DRAFT)
    B, width = table.shape
    cu = torch.cat([n.new_zeros(1), n.cumsum(0)])
    have = (ctx + page - 1) // page
    need = torch.minimum((ctx + n + page - 1) // page, torch.tensor(width, device=ctx.device))
    take = (need - have).clamp(min=0)
    first = take.cumsum(0) - take
    col = torch.arange(width, device=ctx.device)
    at = first[:, None] + col - have[:, None]
    page_id = torch.where(at < free.numel(), free[at.clamp(0, free.numel() - 1)], -1)
    table = torch.where((col >= have[:, None]) & (col < need[:, None]), page_id, table)
    # the tokens, in the requests' order
    t = torch.arange(cap, device=ctx.device)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=B - 1)
    i = t - cu[b]
    live = t < cu[-1]
    p = ctx[b] + i
    block = p // page
    pid = table[b, block.clamp(max=width - 1)].long()
    slots = torch.where(live & (block < width) & (pid >= 0), pid * page + p % page, -1)
    # ancestors: the closure of the parent relation, by squaring
    T = MAX_DRAFT
    par = s["parents"].long()
    par = torch.where((par >= 0) & (par < i), par, -1)
    reach = torch.zeros((B, T, T), device=ctx.device)
    reach[b[live], i[live], i[live]] = 1
    edge = live & (par >= 0)
    reach[b[edge], i[edge], par[edge]] = 1
    for _ in range(7):
        reach = (reach @ reach).clamp(max=1)
    rows = reach[b, i.clamp(0, T - 1)] * live[:, None]
    bit = torch.ones(32, dtype=torch.int64, device=ctx.device) << torch.arange(32, device=ctx.device)
    words = (rows.view(cap, 4, 32).long() * bit).sum(-1)
    mask = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
    positions = torch.where(live, ctx[b] + rows.sum(1).long() - 1, 0)
    return dict(cu=cu.int(), table=table, slots=slots, positions=positions.int(), mask=mask,
                taken=take.sum().int().view(1))


def _rope_plain(s):
    case = s["case"]
    T, Hq, Hkv, D, R = (case[k] for k in ("T", "Hq", "Hkv", "D", "R"))
    x = s["qkv"].float().view(T, Hq + 2 * Hkv, D)
    cs = s["cos_sin"][s["positions"].long()][:, None]
    cos, sin = cs[..., : R // 2], cs[..., R // 2:]

    def head(h, w):
        h = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * w
        r = h[..., :R]
        if case["inter"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r[..., : R // 2], r[..., R // 2:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([r, h[..., R:]], -1)

    out = DTYPES[case["out"]]
    q = head(x[:, :Hq], s["wq"]).to(out)
    k, v = head(x[:, Hq: Hq + Hkv], s["wk"]).to(out), x[:, Hq + Hkv:].to(out)
    page, off = s["slots"] // case["page"], s["slots"] % case["page"]
    s["k"][page, off] = k
    s["v"][page, off] = v
    return dict(q=q, k=s["k"], v=s["v"])


def _attn_plain(s):
    case = s["case"]
    B, Hq, Hkv, D, page = (case[k] for k in ("B", "Hq", "Hkv", "D", "page"))
    G, T, L = Hq // Hkv, case["new"], case["ctx"] + case["new"]
    ctx, cu, q = s["ctx"].long(), s["cu"].long(), s["q"]
    n = cu[1:] - cu[:-1]
    key = torch.arange(L, device=q.device)
    real = key < (ctx + n)[:, None]
    pid = s["table"].long()[:, key // page].clamp(min=0)
    k = s["k"][pid, key % page].float()                                   # [B, L, Hkv, D]
    v = torch.where(real[..., None, None], s["v"][pid, key % page].float(), 0.0)
    i = torch.arange(T, device=q.device)
    row = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)                   # [B, T]
    qf = q.float()[row].view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    score = (qf @ k.permute(0, 2, 3, 1)).view(B, Hkv, T, G, L) / math.sqrt(D)
    j = key - ctx[:, None]                                                # drafted index of each key
    jc = j.clamp(0, MAX_DRAFT - 1)
    word = s["mask"].long()[row[:, :, None], (jc // 32)[:, None, :]]
    see = torch.where(j[:, None, :] < 0, True, (word >> (jc % 32)[:, None, :]) & 1 != 0) & real[:, None, :]
    score = score.masked_fill(~see[:, None, :, None, :], -math.inf)
    m = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(score - m)
    del score
    z = p.sum(-1, keepdim=True)
    p = (p / torch.where(z > 0, z, 1.0)).view(B, Hkv, T * G, L)
    o = (p @ v.permute(0, 2, 1, 3)).view(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    live = i < n[:, None]
    out = torch.empty_like(q)
    out[row[live]] = o[live].to(q.dtype)
    return dict(out=out)


def _quantize_plain(x):
    """Values on the e2m1 grid [R, nb, 32] and the biased exponent of each block's scale [R, nb]."""
    x = x.float()
    R, K = x.shape
    nb = -(-K // BLOCK)
    x = torch.nn.functional.pad(x, (0, nb * BLOCK - K)).view(R, nb, BLOCK)
    top = x.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top)[1].long() - 1 - 2, -127).clamp(min=-127)
    v = torch.ldexp(x, -e[..., None])
    a = v.abs().clamp(max=6.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    a = torch.round(a / step) * step                                      # ties to even
    return torch.copysign(a, v), (e + 127).to(torch.uint8)


def _pack(v, e):
    """Codes [R, nb * 16] (low nibble first) and scale bytes [R, nb]."""
    mag = (v.abs().unsqueeze(-1) > torch.tensor(E2M1, device=v.device)[:-1] + 1e-3).sum(-1)
    code = mag + 8 * torch.signbit(v)
    code = code.view(v.shape[0], -1, 2)
    return (code[..., 0] + 16 * code[..., 1]).to(torch.uint8).contiguous(), e.contiguous()


def _values(codes, e):
    """The f32 values that packed codes and scale bytes stand for, [R, nb * 32]."""
    grid = torch.tensor(E2M1 + tuple(-g for g in E2M1), device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], -1).long()
    v = grid[c].view(codes.shape[0], -1, BLOCK)
    return torch.ldexp(v, e.long()[..., None] - 127).view(codes.shape[0], -1)


def _quant_plain(s):
    v, e = _quantize_plain(s["x"])
    values = torch.ldexp(v, e.long()[..., None] - 127).view(v.shape[0], -1)[:, : s["case"]["K"]]
    return dict(values=values.to(torch.bfloat16), scales=e)


def _linear_plain(s):
    case, x = s["case"], s["x"].float()
    if case["a4"]:
        v, e = _quantize_plain(x)
        x = torch.ldexp(v, e.long()[..., None] - 127).view(x.shape[0], -1)[:, : case["K"]]
    return (x @ _values(s["w"], s["sw"])[:, : case["K"]].T).to(DTYPES[case["out"]])


# ---------------------------------------------------------------- the library's calls

def _run_own(s):
    from w4a16_int4_quantized_gb300 import ops
    case = s["case"]
    op = case["op"]
    if op == "plan":
        cu, slots, positions, mask, taken = ops.draft_plan(s["ctx"], s["new"], s["parents"], s["free"], s["table"],
                                                           case["page"])
        return dict(cu=cu, table=s["table"], slots=slots, positions=positions, mask=mask, taken=taken)
    if op == "rope":
        q = ops.qk_norm_rope(s["qkv"], case["Hq"], s["wq"], s["wk"], s["positions"], s["cos_sin"], s["slots"],
                             s["k"], s["v"], eps=1e-6, interleaved=case["inter"])
        return dict(q=q, k=s["k"], v=s["v"])
    if op == "attn":
        return dict(out=ops.tree_attention(s["q"], s["k"], s["v"], s["table"], s["ctx"], s["cu"], s["mask"],
                                           scale=1.0 / math.sqrt(case["D"]), max_len=case["ctx"] + case["new"],
                                           max_new=case["new"]))
    if op == "quant":
        codes, scales = ops.quantize_mxfp4(s["x"])
        return dict(values=ops.dequantize_mxfp4(codes, scales, case["K"], torch.bfloat16), scales=scales)
    if case["a4"]:
        xq, sx = ops.quantize_mxfp4(s["x"])
        return ops.linear_mxfp4_a4(xq, sx, s["w"], s["sw"], case["K"], out_dtype=DTYPES[case["out"]])
    return ops.linear_mxfp4(s["x"], s["w"], s["sw"], out_dtype=DTYPES[case["out"]])


def run(state):
    if own:
        return _run_own(state)
    return {"plan": _plan_plain, "rope": _rope_plain, "attn": _attn_plain, "quant": _quant_plain,
            "linear": _linear_plain}[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _plan_exact, "rope": _rope_exact, "attn": _attn_exact, "quant": _quant_exact,
            "linear": _linear_exact}[case["op"]](s)


def _plan_exact(s):
    page = s["case"]["page"]
    ctx, new, par, free = (s[k].cpu().tolist() for k in ("ctx", "new", "parents", "free"))
    table = s["table"].cpu().numpy().copy()
    cu, slots, pos, masks, taken = [0], [], [], [], 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        for blk in range(-(-c // page), min(-(-(c + n) // page), table.shape[1])):
            table[b, blk] = free[taken] if taken < len(free) else -1
            taken += 1
        rows = []
        for i in range(n):
            p = par[cu[-1] + i]
            rows.append((1 << i) | (rows[p] if 0 <= p < i else 0))
            blk, off = divmod(c + i, page)
            pid = int(table[b, blk]) if blk < table.shape[1] else -1
            slots.append(pid * page + off if pid >= 0 else -1)
            pos.append(c + bin(rows[i]).count("1") - 1)
        masks += rows
        cu.append(cu[-1] + n)
    words = np.array([[(r >> (32 * w)) & 0xFFFFFFFF for w in range(4)] for r in masks], np.uint32).view(np.int32)
    return dict(cu=np.array(cu, np.int32), table=table, slots=np.array(slots, np.int64),
                positions=np.array(pos, np.int32), mask=words, taken=np.array([taken], np.int32))


def _rope_exact(s):
    case = s["case"]
    T, Hq, Hkv, D, R = (case[k] for k in ("T", "Hq", "Hkv", "D", "R"))
    x = s["qkv"].double().view(T, -1, D)
    w = torch.cat([s["wq"].double().expand(Hq, D), s["wk"].double().expand(Hkv, D)])
    h = x[:, : Hq + Hkv]
    h = h / torch.sqrt((h * h).sum(-1, keepdim=True) / D + 1e-6) * w
    at = s["cos_sin"].double()[s["positions"].long()]
    turn = torch.complex(at[:, : R // 2], at[:, R // 2:])[:, None]
    if case["inter"]:
        z = torch.view_as_complex(h[..., :R].reshape(T, Hq + Hkv, R // 2, 2).contiguous()) * turn
        rot = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(h[..., : R // 2].contiguous(), h[..., R // 2: R].contiguous()) * turn
        rot = torch.cat([z.real, z.imag], -1)
    h = torch.cat([rot, h[..., R:]], -1)
    k, v = s["k"].double(), s["v"].double()
    k[s["slots"] // case["page"], s["slots"] % case["page"]] = h[:, Hq:]
    v[s["slots"] // case["page"], s["slots"] % case["page"]] = x[:, Hq + Hkv:]
    return dict(q=h[:, :Hq], k=k, v=v)


def _attn_exact(s):
    case = s["case"]
    Hq, Hkv, D, page = (case[k] for k in ("Hq", "Hkv", "D", "page"))
    G = Hq // Hkv
    cu, ctx = s["cu"].tolist(), s["ctx"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    bits = (s["mask"].long()[:, :, None] >> torch.arange(32, device="cuda")) & 1
    bits = bits.view(-1, MAX_DRAFT).bool()
    for b, c in enumerate(ctx):
        n = cu[b + 1] - cu[b]
        if n == 0:
            continue
        blocks = s["table"][b, : -(-(c + n) // page)].long()
        see = torch.ones((n, c + n), dtype=torch.bool, device="cuda")
        see[:, c:] = bits[cu[b]: cu[b + 1], :n]
        for h in range(Hkv):
            k = s["k"][blocks, :, h].reshape(-1, D)[: c + n].double()
            v = s["v"][blocks, :, h].reshape(-1, D)[: c + n].double()
            q = s["q"][cu[b]: cu[b + 1], h * G: (h + 1) * G].double()
            sc = torch.einsum("tgd,ld->tgl", q, k) * D ** -0.5
            sc = torch.where(see[:, None], sc, -math.inf)
            out[cu[b]: cu[b + 1], h * G: (h + 1) * G] = torch.softmax(sc, -1) @ v
    return dict(out=out)


def _quantize_exact(x):
    """The nearest e2m1 value (ties to the even code) under the scale 2^(floor(log2 max) - 2), in 64 bits."""
    R, K = x.shape
    nb = -(-K // BLOCK)
    pad = torch.zeros((R, nb * BLOCK), dtype=torch.float64, device=x.device)
    pad[:, :K] = x.double()
    pad = pad.view(R, nb, BLOCK)
    top = pad.abs().amax(-1)
    e = torch.floor(torch.log2(torch.where(top > 0, top, 1.0)))
    e = torch.where(top > 0, e - 2, -127.0).clamp(min=-127.0)
    a = pad.abs() / torch.exp2(e)[..., None]
    # the bounds between neighbours; a value on a bound goes to the neighbour whose code is even
    lo = torch.tensor([0.25, 1.25, 2.5, 5.0], dtype=torch.float64, device=x.device)
    hi = torch.tensor([0.75, 1.75, 3.5], dtype=torch.float64, device=x.device)
    idx = (a[..., None] > lo).sum(-1) + (a[..., None] >= hi).sum(-1)
    v = torch.tensor(E2M1, dtype=torch.float64, device=x.device)[idx]
    return torch.copysign(v, pad) * torch.exp2(e)[..., None], (e + 127).to(torch.uint8)


def _quant_exact(s):
    v, e = _quantize_exact(s["x"])
    return dict(values=v.view(v.shape[0], -1)[:, : s["case"]["K"]].contiguous(), scales=e)


def _linear_exact(s):
    case = s["case"]
    w = s["w"].long()
    code = torch.stack([w % 16, w // 16], -1).flatten(1)
    val = torch.tensor(E2M1, dtype=torch.float64, device="cuda")[code % 8] * (1.0 - 2.0 * (code // 8))
    val = val * torch.exp2(s["sw"].double() - 127.0).repeat_interleave(BLOCK, 1)
    x = s["x"].double()
    if case["a4"]:
        x = _quantize_exact(x)[0].view(x.shape[0], -1)
    return x[:, : case["K"]] @ val[:, : case["K"]].T


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(k)) for k in range(6)]:
        print(c, work(c))

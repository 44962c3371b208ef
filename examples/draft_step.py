"""One decode step of drafted tokens through the attention half of a decoder layer.

A batch of requests, each with a context in a paged cache and a small tree of
drafted tokens, goes through the calls of one layer as a serving loop makes them:

  draft_plan      pages, cache slots, positions and ancestor masks of the step
  linear_mxfp4    the q/k/v projection on MXFP4 weights (bf16 activations)
  qk_norm_rope    head norms and rotation; keys and values into the cache
  tree_attention  the drafted tokens over their contexts and ancestors
  linear_mxfp4    the output projection

The plan is made once for a step and serves all of its layers; the workspace is
kept from layer to layer.  Sizes are those of the microdecoder body: 1024 wide,
16 heads of 64.  Run it on the GPU:  python examples/draft_step.py
"""
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

WIDTH, HEADS, HEAD_DIM, PAGE = 1024, 16, 64, 16


class Layer:
    """Weights in MXFP4 and the norm weights of one layer."""

    def __init__(self, ops, gen):
        randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.w_qkv, self.s_qkv = ops.quantize_mxfp4(0.02 * randn(3 * WIDTH, WIDTH))
        self.w_o, self.s_o = ops.quantize_mxfp4(0.02 * randn(WIDTH, WIDTH))
        self.q_norm, self.k_norm = 1 + 0.1 * randn(HEAD_DIM), 1 + 0.1 * randn(HEAD_DIM)


def angles(top):
    inv = 10000.0 ** (-torch.arange(HEAD_DIM // 2, device="cuda", dtype=torch.float64) / (HEAD_DIM // 2))
    a = torch.arange(top, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def attention_half(ops, layer, x, plan, table, ctx, cos_sin, k_cache, v_cache, max_len, max_new, workspace):
    """x bf16 [tokens, WIDTH] -> the layer's attention output, f32 [tokens, WIDTH]."""
    cu, slots, positions, mask, _ = plan
    qkv = ops.linear_mxfp4(x, layer.w_qkv, layer.s_qkv)
    q = ops.qk_norm_rope(qkv, HEADS, layer.q_norm, layer.k_norm, positions, cos_sin, slots, k_cache, v_cache)
    o = ops.tree_attention(q, k_cache, v_cache, table, ctx, cu, mask, scale=1 / math.sqrt(HEAD_DIM), max_len=max_len,
                           max_new=max_new, workspace=workspace)
    return ops.linear_mxfp4(o.view(-1, WIDTH), layer.w_o, layer.s_o)


def run(contexts=(37, 180, 5), parents=((-1, 0, 0, 1, 1, 2), (-1,), (-1, -1, 0, 1, 3)), seed=0):
    """The step, and the same step on dense f32 weights with plain torch; returns both."""
    from w4a16_int4_quantized_gb300 import ops
    gen = torch.Generator(device="cuda").manual_seed(seed)
    layer = Layer(ops, gen)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    B, new = len(contexts), [len(p) for p in parents]
    max_len, max_new, T = max(c + n for c, n in zip(contexts, new)), max(new), sum(new)

    # the cache: pages of the contexts are there, the step takes more from the free ones
    have = [-(-c // PAGE) for c in contexts]
    pages = sum(have) + 2 * B
    table = torch.full((B, -(-max_len // PAGE)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(have):
        table[b, :n] = torch.arange(at, at + n, device="cuda")
        at += n
    free = torch.arange(at, pages, dtype=torch.int32, device="cuda")
    k_cache, v_cache = (torch.randn((pages, PAGE, HEADS, HEAD_DIM), generator=gen, device="cuda").bfloat16()
                        for _ in range(2))
    ctx, cos_sin = i32(contexts), angles(max_len)

    plan = ops.draft_plan(ctx, i32(new), i32([p for tree in parents for p in tree]), free, table, PAGE)
    workspace = torch.empty(ops.tree_attention_workspace_bytes(B, HEADS, HEADS, HEAD_DIM, max_len, max_new),
                            dtype=torch.uint8, device="cuda")
    x = torch.randn((T, WIDTH), generator=gen, device="cuda").bfloat16()
    y = attention_half(ops, layer, x, plan, table, ctx, cos_sin, k_cache, v_cache, max_len, max_new, workspace)
    return y, plain(ops, layer, x, contexts, parents, plan, table, cos_sin, k_cache, v_cache)


def plain(ops, layer, x, contexts, parents, plan, table, cos_sin, k_cache, v_cache):
    """The same outputs, token by token; contexts are read from the cache, drafted tokens computed here."""
    w_qkv = ops.dequantize_mxfp4(layer.w_qkv, layer.s_qkv, WIDTH)
    w_o = ops.dequantize_mxfp4(layer.w_o, layer.s_o, WIDTH)
    qkv = (x.float() @ w_qkv.T).view(-1, 3, HEADS, HEAD_DIM)

    def turn(h, w, pos):
        h = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * w
        a, b = h.chunk(2, -1)
        c, s = cos_sin[pos].chunk(2, -1)
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    out, t0 = [], 0
    for b, (c, tree) in enumerate(zip(contexts, parents)):
        at = torch.arange(c, device="cuda")
        pid = table[b].long()[at // PAGE]
        keys, values = [k_cache[pid, at % PAGE].float()], [v_cache[pid, at % PAGE].float()]
        paths = []
        for i, p in enumerate(tree):
            paths.append((paths[p] if p >= 0 else []) + [i])
            pos = c + len(paths[i]) - 1
            keys.append(turn(qkv[t0 + i, 1], layer.k_norm, pos)[None])
            values.append(qkv[t0 + i, 2][None])
        k, v = torch.cat(keys), torch.cat(values)
        for i, path in enumerate(paths):
            see = torch.cat([at, c + torch.tensor(path, device="cuda")])
            q = turn(qkv[t0 + i, 0], layer.q_norm, c + len(path) - 1)
            p = torch.softmax(torch.einsum("hd,lhd->hl", q, k[see]) / math.sqrt(HEAD_DIM), -1)
            out.append(torch.einsum("hl,lhd->hd", p, v[see]).reshape(WIDTH))
        t0 += len(tree)
    return torch.stack(out) @ w_o.T


if __name__ == "__main__":
    from w4a16_int4_quantized_gb300 import build
    build.build()
    got, want = run()
    err = ((got - want).norm() / want.norm()).item()
    print(f"{got.shape[0]} drafted tokens of 3 requests: relative difference to the plain step {err:.2e}")

"""A decoder layer's attention half and an answer's log probabilities, with 8-bit rows and an 8-bit cache.

A batch of requests, each with a context in a paged cache that is held in 8 bits, takes some
new tokens (one of a plain decode step, a few drafted ones, a piece of a prompt) through the calls
that a serving loop on the W4A8 linears makes:

  add_rmsnorm_q8      the residual's addition and the norm, with the Q8 rows that the linears read
  linear_q4           the q/k/v projection (packed 4-bit weights)
  qk_norm_rope_kv8    head norms and rotation; keys and values into the cache, 16 tokens a scale
  attention_kv8       the new tokens over their contexts, through a window beside the first tokens
  linear_q4_f32       the output projection
  add_rmsnorm_q8, linear_q4   the last norm and the logits
  token_logprobs      log probabilities of the tokens that follow, the entropy and alternatives

Sizes are those of the microdecoder body: 1024 wide, 16 heads of 64.  Run it on the
GPU:  python examples/decode8_step.py
"""
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

WIDTH, HEADS, KV_HEADS, HEAD_DIM, PAGE, VOCAB = 1024, 16, 4, 64, 32, 2048


class Layer:
    """4-bit weights with their channel scales, and the norm weights."""

    def __init__(self, ops, gen):
        randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.qkv = ops.quantize_matrix_q4(0.02 * randn((HEADS + 2 * KV_HEADS) * HEAD_DIM, WIDTH))
        self.o = ops.quantize_matrix_q4(0.02 * randn(WIDTH, HEADS * HEAD_DIM))
        self.head = ops.quantize_matrix_q4(0.05 * randn(VOCAB, WIDTH))
        self.norm, self.last_norm = 1 + 0.1 * randn(WIDTH), 1 + 0.1 * randn(WIDTH)
        self.q_norm, self.k_norm = 1 + 0.1 * randn(HEAD_DIM), 1 + 0.1 * randn(HEAD_DIM)


def angles(top):
    inv = 10000.0 ** (-torch.arange(HEAD_DIM // 2, device="cuda", dtype=torch.float64) / (HEAD_DIM // 2))
    a = torch.arange(top, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def step(ops, layer, x, residual, batch, cache, window, sinks, top):
    """x f32 [tokens, WIDTH], residual bf16 -> (logp, entropy, top_ids, top_logp) of the batch's next tokens."""
    table, ctx, cu, positions, cos_sin, max_len, max_new, nexts = batch
    q8, sx, h, _ = ops.add_rmsnorm_q8(x, residual, layer.norm)
    qkv = ops.linear_q4(q8, sx, *layer.qkv)
    q = ops.qk_norm_rope_kv8(qkv, HEADS, layer.q_norm, layer.k_norm, positions, cos_sin, table, ctx, cu, cache)
    o = ops.attention_kv8(q, cache, table, ctx, cu, scale=1 / math.sqrt(HEAD_DIM), max_len=max_len, max_new=max_new,
                          window=window, sinks=sinks)
    y, _, _ = ops.linear_q4_f32(o.view(-1, HEADS * HEAD_DIM).float(), *layer.o)
    q8, sx, _, _ = ops.add_rmsnorm_q8(y, h, layer.last_norm)
    return ops.token_logprobs(ops.linear_q4(q8, sx, *layer.head), nexts, top=top)


def make(ops, contexts, new, seed):
    """A layer, a batch and its cache, half filled."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    layer = Layer(ops, gen)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    need = [-(-(c + n) // PAGE) for c, n in zip(contexts, new)]
    max_len, T = max(c + n for c, n in zip(contexts, new)), sum(new)
    table = torch.full((len(contexts), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n, device="cuda")
        at += n
    cache = ops.Kv8Cache.empty(at, PAGE, KV_HEADS, HEAD_DIM)
    for codes, scales in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        codes.copy_((32 * torch.randn(codes.shape, generator=gen, device="cuda")).round().clamp(-127, 127))
        scales.fill_(127 - 5)
    batch = (table, i32(contexts), i32([sum(new[:i]) for i in range(len(new) + 1)]),
             i32([c + i for c, n in zip(contexts, new) for i in range(n)]), angles(max_len), max_len, max(new),
             torch.randint(0, VOCAB, (T,), generator=gen, device="cuda").to(torch.int32))
    x = torch.randn((T, WIDTH), generator=gen, device="cuda")
    residual = torch.randn((T, WIDTH), generator=gen, device="cuda").bfloat16()
    return layer, batch, cache, x, residual


def plain(ops, layer, batch, cache, x, residual, window, sinks):
    """The log probabilities of all tokens [tokens, VOCAB] from the same step on dense weights in 32 bits, without the
    8-bit rows and keys and values (but for those that the cache held before)."""
    table, ctx, cu, positions, cos_sin, _, _, _ = batch
    dense = lambda w: ((torch.stack([w[0] & 15, w[0] >> 4], -1).flatten(1).float() - 8) * w[1][:, None])  # noqa: E731
    norm = lambda h, w: h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * w  # noqa: E731
    held = ops.dequantize_kv8(cache, torch.float32)
    h = (x + residual.float()).bfloat16().float()
    qkv = (norm(h, layer.norm) @ dense(layer.qkv).T).view(-1, HEADS + 2 * KV_HEADS, HEAD_DIM)

    def turn(a, w):
        a = norm(a, w)
        c, s = cos_sin[positions.long()][:, None].chunk(2, -1)
        u, v = a.chunk(2, -1)
        return torch.cat([u * c - v * s, v * c + u * s], -1)

    q, k, v = turn(qkv[:, :HEADS], layer.q_norm), turn(qkv[:, HEADS: HEADS + KV_HEADS], layer.k_norm), qkv[:, HEADS + KV_HEADS:]
    out = []
    for b, c in enumerate(ctx.tolist()):
        t0, t1 = int(cu[b]), int(cu[b + 1])
        at = torch.arange(c, device="cuda")
        pid = table[b].long()[at // PAGE]
        keys, values = (torch.cat([m[pid, at % PAGE], n[t0:t1]]).repeat_interleave(HEADS // KV_HEADS, 1)
                        for m, n in zip(held, (k, v)))
        j = torch.arange(c + t1 - t0, device="cuda")
        back = j[c:, None] - j
        see = (back >= 0) & ((back < window) | (j < sinks) if window else True)
        p = torch.einsum("thd,lhd->htl", q[t0:t1], keys) / math.sqrt(HEAD_DIM)
        p = torch.softmax(p.masked_fill(~see, -math.inf), -1)
        out.append(torch.einsum("htl,lhd->thd", p, values).reshape(t1 - t0, -1))
    h = (torch.cat(out) @ dense(layer.o).T + h).bfloat16().float()
    return torch.log_softmax(norm(h, layer.last_norm) @ dense(layer.head).T, -1)


def run(contexts=(37, 500, 5), new=(3, 1, 20), window=64, sinks=4, top=5, seed=0):
    """The step and the plain log probabilities; returns (its four results, the tokens asked for, all plain ones)."""
    from w4a16_int4_quantized_gb300 import ops
    layer, batch, cache, x, residual = make(ops, contexts, new, seed)
    want = plain(ops, layer, batch, cache, x, residual, window, sinks)
    return step(ops, layer, x, residual, batch, cache, window, sinks, top), batch[-1], want


if __name__ == "__main__":
    from w4a16_int4_quantized_gb300 import build
    build.build()
    (logp, entropy, ids, _), nexts, want = run()
    off = (logp - want.gather(1, nexts.long()[:, None])[:, 0]).abs().max().item()
    print(f"{logp.numel()} tokens of 3 requests: log probabilities within {off:.3f} of the plain step in 32 bits, "
          f"mean entropy {entropy.mean().item():.2f}")

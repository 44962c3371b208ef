"""Plain forms of the 8-bit cache in 64 bits, request by request, for the tests."""
import torch

BLOCK = 16


def values(codes, scales):
    """[page, token, head, value] in 64 bits."""
    unit = torch.exp2(scales.double() - 127.0)
    unit = torch.where(scales == 255, float("nan"), unit)
    return codes.double() * unit.transpose(1, 2).repeat_interleave(BLOCK, 1)[..., None]


def rows_of(cache_values, table_row, n, page):
    """Tokens 0 .. n - 1 of a request, [n, head, value]; NaN rows for pages outside."""
    P = cache_values.shape[0]
    j = torch.arange(n, device=cache_values.device)
    if n == 0:
        return cache_values.new_zeros((0, *cache_values.shape[2:])), j.bool()
    block, table_row = j // page, table_row.to(j.device)
    pid = torch.where(block < table_row.numel(), table_row.long()[block.clamp(max=table_row.numel() - 1)], -1)
    ok = (pid >= 0) & (pid < P)
    return cache_values[pid.clamp(0, P - 1), j % page], ok


def scale_byte(top):
    """The least 2^(s - 127) whose 127-fold is not below top (64 bits)."""
    m, e = torch.frexp(top)
    s = torch.where(top > 0, e - 7 + (m > 127 / 128).to(e.dtype), torch.tensor(-127, device=top.device, dtype=e.dtype))
    return (s.clamp(min=-127) + 127).long()


def append(codes, scales, new, table_row, ctx, n, page):
    """new [n, head, value] behind ctx tokens of a request, in place (codes as float64, scales as int64)."""
    for first in range(ctx // BLOCK * BLOCK if n else ctx, ctx + n, BLOCK):
        blk = first // page
        if blk >= table_row.numel() or not 0 <= int(table_row[blk]) < codes.shape[0]:
            continue
        p, off = int(table_row[blk]), first % page
        lo, hi = max(first, ctx), min(first + BLOCK, ctx + n)
        x = new[lo - ctx: hi - ctx].double()
        kept = lo - first
        top = x.abs().amax((0, 2))
        s = torch.where(x.isfinite().all(2).all(0), scale_byte(top.nan_to_num(0.0, 0.0)), 255)
        old = scales[p, :, off // BLOCK].clone()
        if kept:
            s = torch.maximum(s, old)
            held = codes[p, off: off + kept]
            shrunk = torch.round(held * torch.exp2((old - s).double())[None, :, None])
            codes[p, off: off + kept] = torch.where((s == 255)[None, :, None] & (old != 255)[None, :, None], 0.0,
                                                    torch.where((s == old)[None, :, None], held, shrunk))
        c = torch.round(x / torch.exp2(s.double() - 127.0)[None, :, None])
        codes[p, off + kept: off + kept + hi - lo] = torch.where((s == 255)[None, :, None], 0.0, c)
        scales[p, :, off // BLOCK] = s


def attention(q, kv, vv, table, ctx, cu, scale, page, window=0, sinks=0, max_new=1 << 30):
    """(out, bound of |v| and of sum |q k| scale per row) in 64 bits; rows of no token stay NaN."""
    T, Hq, D = q.shape
    H = kv.shape[2]
    G = Hq // H
    out = torch.full((T, Hq, D), float("nan"), dtype=torch.float64, device=q.device)
    vmax = torch.zeros((T, Hq), dtype=torch.float64, device=q.device)
    smax = torch.zeros((T, Hq), dtype=torch.float64, device=q.device)
    for b in range(table.shape[0]):
        c, t0, n = int(ctx[b]), int(cu[b]), int(cu[b + 1]) - int(cu[b])
        if n == 0:
            continue
        k, ok = rows_of(kv, table[b], c + n, page)
        v, _ = rows_of(vv, table[b], c + n, page)
        j = torch.arange(c + n, device=q.device)
        back = (c + torch.arange(n, device=q.device))[:, None] - j
        see = (back >= 0) & ok
        if window:
            see &= (back < window) | (j < sinks)
        m = min(n, max_new)
        for h in range(Hq):
            qh, kh, vh = q[t0: t0 + m, h].double(), k[:, h // G], v[:, h // G]
            sc = torch.where(see[:m], qh @ kh.T * scale, -float("inf"))
            top = sc.amax(-1, keepdim=True)
            p = torch.exp(sc - torch.where(top == -float("inf"), 0.0, top))
            z = p.sum(-1, keepdim=True)
            vz = torch.where(see[:m].any(0)[:, None], vh, 0.0)
            o = torch.where(see[:m, :, None], p[..., None] * vz, 0.0).sum(1) if m * (c + n) * D < 1 << 24 else p @ vz
            out[t0: t0 + m, h] = torch.where(z > 0, o / torch.where(z > 0, z, 1.0), torch.where(z.isnan(), z, 0.0))
            vmax[t0: t0 + m, h] = torch.where(see[:m], vh.abs().amax(-1), 0.0).amax(-1)
            smax[t0: t0 + m, h] = torch.where(see[:m], qh.abs() @ kh.abs().T * scale, 0.0).amax(-1)
    return out, vmax, smax
